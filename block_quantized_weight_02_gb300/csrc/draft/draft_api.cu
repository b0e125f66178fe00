// The C entry points of a drafting step: argument checks and launches.
#include <cmath>

#include "../kv8/kv8_checks.h"
#include "draft.cuh"

using namespace cq;
using namespace cq::kv8;
using namespace cq::draft;

namespace {

cq_status check_rope(const char* who, const cq_rope_spec* r, int64_t D, const int32_t* pos, Rope* out) {
    if (!r || !r->freq) return fail(CQ_ERR_NULL, "%s: null pointer (frequencies)", who);
    if (r->rot < 16 || r->rot % 16 || r->rot > D)
        return fail(CQ_ERR_SHAPE, "%s: rot must be a multiple of 16, at least 16 and at most D (rot=%lld D=%lld)", who, (long long)r->rot, (long long)D);
    if (r->layout != CQ_ROPE_HALF && r->layout != CQ_ROPE_PAIRS) return fail(CQ_ERR_ARG, "%s: unknown layout %d", who, r->layout);
    if (!std::isfinite(r->mag)) return fail(CQ_ERR_ARG, "%s: mag must be finite", who);
    if (!aligned(r->freq, 4) || !aligned(pos, 4)) return fail(CQ_ERR_ALIGN, "%s: freq and pos must be 4-byte aligned", who);
    *out = Rope{r->freq, pos, (int)r->rot / 2, r->mag};
    return CQ_OK;
}

cq_status check_mask(const char* who, const uint32_t* mask, int64_t ldm, int64_t max_q) {
    if (!aligned(mask, 4)) return fail(CQ_ERR_ALIGN, "%s: mask must be 4-byte aligned", who);
    if (ldm < 1 || ldm > INT32_MAX || ldm < (max_q + 31) / 32)
        return fail(CQ_ERR_SHAPE, "%s: mask rows must hold max_q bits (ldm=%lld max_q=%lld)", who, (long long)ldm, (long long)max_q);
    return CQ_OK;
}

}  // namespace

extern "C" {

cq_status cq_rope(const void* X, int xt, int64_t T, int64_t H, int64_t D, int64_t ldx, const cq_rope_spec* rope,
                  const int32_t* pos, void* Y, int yt, int64_t ldy, void* stream) {
    const char* who = "cq_rope";
    clear_last_error();
    if (!X || !Y || !pos) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    cq_status st;
    Rope r;
    if ((st = check_type(who, xt, true)) || (st = check_type(who, yt, true))) return st;
    if (H < 1 || D < 16 || D % 16 || D > 1024 || H > INT32_MAX / D)
        return fail(CQ_ERR_SHAPE, "%s: need H>=1, D a multiple of 16 up to 1024, H*D<2^31 (H=%lld D=%lld)", who, (long long)H, (long long)D);
    if ((st = check_T(who, T, H)) || (st = check_rope(who, rope, D, pos, &r)) || (st = check_rows(who, "X", X, ldx, H * D, xt)) ||
        (st = check_rows(who, "Y", Y, ldy, H * D, yt)))
        return st;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(X), y0 = reinterpret_cast<uintptr_t>(Y);
    const uintptr_t x1 = x0 + ((T - 1) * ldx + H * D) * size_of(xt), y1 = y0 + ((T - 1) * ldy + H * D) * size_of(yt);
    // (rows between one another's: the columns of a pitch that both have)
    const bool apart = ldx * size_of(xt) == ldy * size_of(yt) && xt == yt && [&] {
        const uintptr_t pitch = ldx * size_of(xt), width = H * D * size_of(xt), d = x0 < y0 ? y0 - x0 : x0 - y0;
        return d % pitch >= width && pitch - d % pitch >= width;
    }();
    if (x0 < y1 && y0 < x1 && !(x0 == y0 && xt == yt && ldx == ldy) && !apart)
        return fail(CQ_ERR_ARG, "%s: Y must be X (of its type and pitch) or not overlap it", who);
    if ((st = check_device())) return st;
    return launched(launch_rope(X, xt, (int)T, (int)H, (int)D, ldx, r, rope->layout, Y, yt, ldy, static_cast<cudaStream_t>(stream)),
                    "rotary positions");
}

cq_status cq_rope_freqs(int64_t rot, double base, int kind, double factor, double low, double high, double trained,
                        float* freq, float* mag) {
    const char* who = "cq_rope_freqs";
    clear_last_error();
    if (!freq || !mag) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    if (rot < 16 || rot % 16 || rot > 1024) return fail(CQ_ERR_SHAPE, "%s: rot must be a multiple of 16 up to 1024 (got %lld)", who, (long long)rot);
    if (kind < CQ_ROPE_PLAIN || kind > CQ_ROPE_BANDS) return fail(CQ_ERR_ARG, "%s: unknown kind %d", who, kind);
    if (!(base > 1.0) || !std::isfinite(base)) return fail(CQ_ERR_ARG, "%s: base must be finite and above 1", who);
    if (kind != CQ_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return fail(CQ_ERR_ARG, "%s: factor must be finite and at least 1", who);
    if (kind >= CQ_ROPE_RAMP && (!(low > 0.0) || !(high > low) || !(trained > 0.0) || !std::isfinite(high) || !std::isfinite(trained)))
        return fail(CQ_ERR_ARG, "%s: need 0 < low < high and trained > 0", who);
    constexpr double PI = 3.14159265358979323846;
    if (kind == CQ_ROPE_BASE) base *= std::pow(factor, (double)rot / (double)(rot - 2));
    // the pair that turns n times within the trained context
    auto pair_of = [&](double n) { return rot * std::log(trained / (2.0 * PI * n)) / (2.0 * std::log(base)); };
    const double by = kind == CQ_ROPE_PLAIN || kind == CQ_ROPE_BASE ? 1.0 : factor;
    double from = 0.0, to = 0.0;
    if (kind == CQ_ROPE_RAMP) {
        from = std::fmax(std::floor(pair_of(high)), 0.0);
        to = std::fmin(std::ceil(pair_of(low)), (double)(rot - 1));
        if (!(to - from >= 0.001)) to = from + 0.001;
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / (double)rot);
        double kept = 1.0;                               // share that is not divided
        if (kind == CQ_ROPE_LINEAR) kept = 0.0;
        if (kind == CQ_ROPE_RAMP) kept = 1.0 - std::fmin(std::fmax(((double)i - from) / (to - from), 0.0), 1.0);
        if (kind == CQ_ROPE_BANDS) kept = std::fmin(std::fmax((trained * f / (2.0 * PI) - low) / (high - low), 0.0), 1.0);
        freq[i] = (float)(f * kept + f / by * (1.0 - kept));
    }
    *mag = kind == CQ_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return CQ_OK;
}

cq_status cq_kv8_write_rope(const cq_kv8_cache* cache, const void* K, const void* V, int xt, int64_t T, int64_t ldk,
                            int64_t ldv, const int32_t* q_start, const int32_t* lens, const cq_rope_spec* rope,
                            const int32_t* pos, void* stream) {
    const char* who = "cq_kv8_write_rope";
    clear_last_error();
    if (!lens) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    if (!cache) return fail(CQ_ERR_NULL, "%s: null pointer (cache)", who);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Cache c;
    Rope r;
    int* err = nullptr;
    cq_status st = check_rope(who, rope, cache->D, pos, &r);
    if (!st) st = check_store(who, cache, &c, K, V, xt, T, ldk, ldv, q_start, lens, s, &err);
    if (st) return st;
    const Batch b = {q_start, lens, nullptr, (int)T, err};
    return launched(launch_write_rope(c, b, (int)cache->D, K, V, xt, ldk, ldv, r, rope->layout, s), "cache write");
}

cq_status cq_attn_kv8_tree(const void* Q, int xt, int64_t T, int64_t Hq, int64_t ldq, const cq_kv8_cache* cache,
                           const int32_t* q_start, const int32_t* lens, int64_t max_q, float scale, const uint32_t* mask,
                           int64_t ldm, void* O, int yt, int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream) {
    const char* who = "cq_attn_kv8_tree";
    clear_last_error();
    if (!mask) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnArgs a;
    cq_status st = check_mask(who, mask, ldm, std::min(max_q, T));
    // (every row of a sequence sees its tokens up to the last, but for what the mask hides)
    if (!st) st = attn_args(who, Q, xt, T, Hq, ldq, cache, q_start, lens, max_q, scale, 0, 0, O, yt, ldo, lse, ws, ws_bytes, s, &a);
    if (st) return st;
    a.mask = mask;
    a.ldm = ldm;
    a.stall = (int)options().test_stall.exchange(0);
    return launched(launch_attn_tree(a, s), "attention");
}

cq_status cq_verify(const void* P, int pt, int64_t T, int64_t V, int64_t ldp, const void* Q, int64_t ldq,
                    const int32_t* tokens, const uint32_t* mask, int64_t ldm, const int32_t* q_start, int64_t B,
                    int64_t max_q, const float* u, const float* u_last, int32_t* out, int32_t* path, int64_t ldo,
                    int32_t* count, void* stream) {
    const char* who = "cq_verify";
    clear_last_error();
    if (!P || !tokens || !q_start || !u || !u_last || !out || !path || !count) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    cq_status st;
    if ((st = check_type(who, pt, true))) return st;
    if (V < 1 || V >= 1 << 30) return fail(CQ_ERR_SHAPE, "%s: need 1<=V<2^30 (V=%lld)", who, (long long)V);
    if ((st = check_T(who, T, 1)) || (st = check_rows(who, "P", P, ldp, V, pt)) || (Q && (st = check_rows(who, "Q", Q, ldq, V, pt)))) return st;
    if (B < 1 || B > 65536 || max_q < 1 || max_q > 1024 || ldo < max_q || ldo > INT32_MAX)
        return fail(CQ_ERR_SHAPE, "%s: need 1<=B<=65536, 1<=max_q<=1024, ldo>=max_q (B=%lld max_q=%lld ldo=%lld)", who, (long long)B,
                    (long long)max_q, (long long)ldo);
    if (mask && (st = check_mask(who, mask, ldm, max_q))) return st;
    for (const void* p : {(const void*)tokens, (const void*)q_start, (const void*)u, (const void*)u_last, (const void*)out,
                          (const void*)path, (const void*)count})
        if (!aligned(p, 4)) return fail(CQ_ERR_ALIGN, "%s: index and number arrays must be 4-byte aligned", who);
    if ((st = check_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int* err = stream_error_word(s);
    if (!err) return CQ_ERR_CUDA;
    const VerifyArgs a = {P, Q, ldp, ldq, tokens, mask, ldm, q_start, u, u_last, out, path, count, ldo, pt, (int)T, (int)V, (int)B,
                          (int)max_q, err};
    return launched(launch_verify(a, s), "check of drafted tokens");
}

}  // extern "C"

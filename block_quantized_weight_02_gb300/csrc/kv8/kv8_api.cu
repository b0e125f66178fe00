// The C entry points of the 8-bit key/value cache: argument checks and launches.
#include <cmath>

#include "kv8.cuh"

namespace cq {
namespace kv8 {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

cq_status check_device() {
    int dev = 0, major = 0, minor = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 3)
        return fail(CQ_ERR_ARCH, "device %d is sm_%d%d, this library is built for sm_103a", dev, major, minor);
    return CQ_OK;
}

cq_status check_cache(const char* who, const cq_kv8_cache* c, Cache* out) {
    if (!c || !c->Kq || !c->Vq || !c->Ks || !c->Vs || !c->table) return fail(CQ_ERR_NULL, "%s: null pointer (cache)", who);
    if (c->D != 64 && c->D != 128) return fail(CQ_ERR_SHAPE, "%s: D must be 64 or 128 (got %lld)", who, (long long)c->D);
    if (c->pages < 1 || c->Hkv < 1 || c->Hkv > 1024 || c->page < BLK || c->page % BLK || c->pages > INT32_MAX ||
        c->page > INT32_MAX || c->page > INT32_MAX / c->Hkv || c->pages > INT32_MAX / (c->page * c->Hkv))
        return fail(CQ_ERR_SHAPE, "%s: need pages>=1, 1<=Hkv<=1024, page%%32==0, pages*Hkv*page<2^31 (pages=%lld Hkv=%lld page=%lld)",
                    who, (long long)c->pages, (long long)c->Hkv, (long long)c->page);
    if (c->B < 1 || c->B > 65536 || c->ldt < 1 || c->ldt > INT32_MAX)
        return fail(CQ_ERR_SHAPE, "%s: need 1<=B<=65536, ldt>=1 (B=%lld ldt=%lld)", who, (long long)c->B, (long long)c->ldt);
    if (!aligned(c->Kq, 16) || !aligned(c->Vq, 16) || !aligned(c->Ks, 16) || !aligned(c->Vs, 16) || !aligned(c->table, 4))
        return fail(CQ_ERR_ALIGN, "%s: cache pointers must be 16-byte aligned (table: 4)", who);
    *out = Cache{{c->Kq, c->Vq}, {c->Ks, c->Vs}, c->table, c->ldt, (int)c->pages, (int)c->Hkv, (int)c->page, (int)c->B};
    return CQ_OK;
}

int64_t size_of(int t) { return t == CQ_F32 ? 4 : 2; }

cq_status check_type(const char* who, int t, bool f32) {
    if (t != CQ_F16 && t != CQ_BF16 && !(f32 && t == CQ_F32))
        return fail(CQ_ERR_DTYPE, "%s: the type must be fp16%s bf16%s (got %d)", who, f32 ? "," : " or", f32 ? " or f32" : "", t);
    return CQ_OK;
}

// rows of `width` elements at a pitch of `ld`
cq_status check_rows(const char* who, const char* what, const void* p, int64_t ld, int64_t width, int t) {
    if (ld < width || ld > (1LL << 31) || ld * size_of(t) % 16)
        return fail(CQ_ERR_SHAPE, "%s: the pitch of %s must be at least %lld elements and a multiple of 16 bytes (got %lld)", who,
                    what, (long long)width, (long long)ld);
    if (!aligned(p, 16)) return fail(CQ_ERR_ALIGN, "%s: %s must be 16-byte aligned", who, what);
    return CQ_OK;
}

cq_status check_T(const char* who, int64_t T, int64_t heads) {
    if (T < 1 || T > INT32_MAX / heads) return fail(CQ_ERR_SHAPE, "%s: need T>=1, T*heads<2^31 (T=%lld)", who, (long long)T);
    return CQ_OK;
}

// K and V rows of write and read; *err receives the stream's error word.
cq_status check_store(const char* who, const cq_kv8_cache* cache, Cache* c, const void* K, const void* V, int t, int64_t T,
                      int64_t ldk, int64_t ldv, const int32_t* start, const int32_t* other, cudaStream_t s, int** err) {
    cq_status st;
    if (!K || !V || !start) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    if ((st = check_cache(who, cache, c)) || (st = check_type(who, t, true)) || (st = check_T(who, T, cache->Hkv)) ||
        (st = check_rows(who, "K", K, ldk, cache->Hkv * cache->D, t)) ||
        (st = check_rows(who, "V", V, ldv, cache->Hkv * cache->D, t)))
        return st;
    if ((T / BLK + 2 * cache->B) * cache->Hkv * 2 > INT32_MAX) return fail(CQ_ERR_SHAPE, "%s: too many blocks for one call", who);
    if (!aligned(start, 4) || !aligned(other, 4)) return fail(CQ_ERR_ALIGN, "%s: index arrays must be 4-byte aligned", who);
    if ((st = check_device())) return st;
    *err = stream_error_word(s);
    return *err ? CQ_OK : CQ_ERR_CUDA;
}

cq_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? CQ_OK : cuda_fail(e, what); }

}  // namespace
}  // namespace kv8
}  // namespace cq

using namespace cq;
using namespace cq::kv8;

extern "C" {

cq_status cq_kv8_write(const cq_kv8_cache* cache, const void* K, const void* V, int xt, int64_t T, int64_t ldk,
                       int64_t ldv, const int32_t* q_start, const int32_t* lens, void* stream) {
    clear_last_error();
    if (!lens) return fail(CQ_ERR_NULL, "cq_kv8_write: null pointer");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Cache c;
    int* err = nullptr;
    cq_status st = check_store("cq_kv8_write", cache, &c, K, V, xt, T, ldk, ldv, q_start, lens, s, &err);
    if (st) return st;
    const Batch b = {q_start, lens, nullptr, (int)T, err};
    return launched(launch_write(c, b, (int)cache->D, K, V, xt, ldk, ldv, s), "cache write");
}

cq_status cq_kv8_read(const cq_kv8_cache* cache, const int32_t* first, const int32_t* out_start, void* K, void* V,
                      int yt, int64_t T, int64_t ldk, int64_t ldv, void* stream) {
    clear_last_error();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Cache c;
    int* err = nullptr;
    cq_status st = check_store("cq_kv8_read", cache, &c, K, V, yt, T, ldk, ldv, out_start, first, s, &err);
    if (st) return st;
    const Batch b = {out_start, nullptr, first, (int)T, err};
    return launched(launch_read(c, b, (int)cache->D, K, V, yt, ldk, ldv, s), "cache read-back");
}

size_t cq_attn_kv8_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    if (T < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || D < 1 || B < 1 || max_q < 1) return 0;
    return attn_workspace_upto(T, Hq, Hkv, D, B, max_q);
}

cq_status cq_attn_kv8(const void* Q, int xt, int64_t T, int64_t Hq, int64_t ldq, const cq_kv8_cache* cache,
                      const int32_t* q_start, const int32_t* lens, int64_t max_q, float scale, int causal,
                      int64_t window, void* O, int yt, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
    const char* who = "cq_attn_kv8";
    clear_last_error();
    if (!Q || !O || !q_start || !lens || !ws) return fail(CQ_ERR_NULL, "%s: null pointer", who);
    cq_status st;
    Cache c;
    if ((st = check_cache(who, cache, &c)) || (st = check_type(who, xt, false)) || (st = check_type(who, yt, true))) return st;
    if (Hq < 1 || Hq % cache->Hkv || Hq / cache->Hkv > 64)
        return fail(CQ_ERR_SHAPE, "%s: Hq must be a multiple of Hkv, at most 64 times it (Hq=%lld Hkv=%lld)", who, (long long)Hq,
                    (long long)cache->Hkv);
    if ((st = check_T(who, T, Hq)) || (st = check_rows(who, "Q", Q, ldq, Hq * cache->D, xt)) ||
        (st = check_rows(who, "O", O, ldo, Hq * cache->D, yt)))
        return st;
    if (max_q < 1) return fail(CQ_ERR_SHAPE, "%s: max_q must be at least 1", who);
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(CQ_ERR_ARG, "%s: scale must be finite and positive", who);
    if (window < 0 || (causal != 0 && causal != 1) || (!causal && window))
        return fail(CQ_ERR_ARG, "%s: causal must be 0 or 1, window >= 0 and only with causal", who);
    if (!aligned(q_start, 4) || !aligned(lens, 4) || !aligned(lse, 4)) return fail(CQ_ERR_ALIGN, "%s: index arrays and lse must be 4-byte aligned", who);
    max_q = std::min(max_q, T);
    window = std::min<int64_t>(window, INT32_MAX);   // the same tokens (positions are 31-bit), and no overflow of p - window
    const size_t need = attn_workspace(T, Hq, cache->Hkv, cache->D, cache->B, max_q);
    if (!aligned(ws, 256) || ws_bytes < need) return fail(CQ_ERR_WORKSPACE, "%s: workspace needs %zu bytes, 256-aligned", who, need);
    if ((st = check_device())) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int* err = stream_error_word(s);
    if (!err) return CQ_ERR_CUDA;
    const Batch b = {q_start, lens, nullptr, (int)T, err};
    const AttnArgs a = {c, b, Q, O, lse, ldq, ldo, xt, yt, (int)Hq, (int)cache->D, (int)max_q, causal, window, scale, ws,
                        (int)options().test_stall.exchange(0)};
    return launched(launch_attn(a, s), "attention");
}

}  // extern "C"

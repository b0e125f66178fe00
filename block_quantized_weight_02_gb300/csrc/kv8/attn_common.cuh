// What the attention kernels share: queries to fp16, codes to fp16, outputs.
#pragma once
#include "kv8.cuh"

namespace cq {
namespace kv8 {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// A wait for an mbarrier's phase that ends after limit_ns or once *stop is set (false then).  Short code: the kernels
// have many waits, and their loops have to stay in the instruction cache.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit_ns, const volatile int* stop) {
    uint64_t t0 = 0;
    for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
        if (i & 63u) continue;
        const uint64_t t = global_timer_ns();
        if (i == 0) t0 = t;
        if (*stop || t - t0 > limit_ns) return false;
    }
    return true;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Exponent lv of a value block's scale: a power of two of at least 2^-64 (less, if no token was ever written: codes are 0
// then), or NaN (whose scores are NaN).
__device__ __forceinline__ int value_exp(float s) { return s == s ? max((int)(__float_as_uint(s) >> 23) - 127, -64) : -64; }

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Two codes (bytes of w ^ 0x80808080 picked by sel) -> fp16 exactly: with 0x64 as the high byte
// u = code + 128 reads as 1024 + u, and minus 1152 is the code.
__device__ __forceinline__ uint32_t codes_f16(uint32_t u, uint32_t sel) {
    return sub_f16x2(prmt(u, 0x64646464u, sel), 0x64806480u);
}

// bf16 queries reach fp16 behind a power of two per row that puts the row's largest
// magnitude in [2^13, 2^14): exact for values within 2^27 of it.  Returns the shift.
__device__ __forceinline__ int guard_of(float amax) {
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;
    return amax == 0.f || e == 128 ? 0 : min(max(13 - e, -114), 126);
}

__device__ __forceinline__ void store_out(void* p, int64_t i, int t, float v) {
    if (t == CQ_F32) static_cast<float*>(p)[i] = v;
    else if (t == CQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
// Four neighbouring outputs (i a multiple of four).
__device__ __forceinline__ void store_out4(void* p, int64_t i, int t, float a, float b, float c, float d) {
    if (t == CQ_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
    } else if (t == CQ_F16) {
        *reinterpret_cast<uint2*>(static_cast<__half*>(p) + i) = make_uint2(pack_f16(a, b), pack_f16(c, d));
    } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
    }
}

// The tokens [lo, hi) that row i of a sequence with n rows and L tokens sees.
__device__ __forceinline__ int row_hi(int i, int n, int L, int causal) { return causal ? max(L - n + i + 1, 0) : L; }
__device__ __forceinline__ int row_lo(int i, int n, int L, int64_t window) {
    return window ? (int)max((int64_t)0, (int64_t)(L - n + i) - window + 1) : 0;
}

// The softmax's maximum is not taken over the scores s (log2 units) but over z = s + lv, the log2 of what a token's weight
// times its value block's scale comes to: m = max z, p = 2^(z - m) multiplies the codes, and the normaliser takes
// 2^(s - m) = p 2^-lv.  So the fp16 weights are fine where the result is large, whatever the scales of the blocks are, and a
// block that a row does not see, or sees under scores that leave it no weight, does not enter.  It costs nothing: lv is the
// addend of the multiplication that makes s.
//
// In f32 p is 0 below 2^-126, where p 2^-lv may still count if lv is far below that of the maximum (zeros beside values of
// 2^30 and more).  A block whose exponent is more than APART below the largest so far, which is always more than the weights
// need, gets its part of the normaliser from exponentials of its own.
constexpr int APART = 80;
// A normaliser may be large where the factor 2^d that lowers it is too small for f32: it is lowered by the root, twice.
__device__ __forceinline__ float root_of(float d) { return ex2(0.5f * d); }

// What a sum against the maximum m0 counts against m.
__device__ __forceinline__ float since(float m0, float m) { return m0 == -INFINITY ? 1.f : ex2(m0 - m); }

// An unfinished result: O before the division, the maximum (of z) and the normaliser of each row.
template <int D, int R>
struct PartOf {
    float m[R], l[R];
    float o[R][D];
    __device__ __forceinline__ const float4* quad(int r, int d) const { return reinterpret_cast<const float4*>(&o[r][d]); }
};
// What ends a row.  Its normaliser is 0 if it sees no token (O = 0, lse = -inf), and if it sees only scores of -inf, whose
// softmax is 0 / 0: that one's normaliser becomes NaN.  Rows see a token from `first_seeing` on: of n rows behind fewer
// tokens the first stand before token 0.
__device__ __forceinline__ int first_seeing(const AttnArgs& a, int n, int L) {
    return a.causal ? max(n - L, 0) * (a.Hq / a.c.Hkv) : L > 0 ? 0 : INT32_MAX;
}
__device__ __forceinline__ float row_sum(float l, int f, int first) {
    return l == 0.f && f >= first ? __uint_as_float(0x7FC00000u) : l;
}
__device__ __forceinline__ float inv_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

// Joins the partials part(0) .. part(cnt - 1) of KV head h's row f (a (token, head) pair of the sequence whose first
// tensor row is q0; rows from `first` on see a token), row r of the partials, NQ x 4 channels from d on: into `out`
// (nullable), else the output.  AT partials are read at a time; FAR ones come from other CTAs.
template <bool FAR, class T>
__device__ __forceinline__ T part_ld(const T* p) { return FAR ? __ldcg(p) : *p; }
template <bool FAR, int D, int NQ, int AT, class P, class F>
__device__ __forceinline__ void join(const AttnArgs& a, int q0, int first, int h, int f, int r, int d, int cnt, F part, P* out) {
    float m = -INFINITY, l = 0.f;
    float4 o[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < cnt; j0 += AT) {
        float pm[AT], pl[AT];
        float4 v[AT][NQ];
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            pm[j] = -INFINITY;
            pl[j] = 0.f;
#pragma unroll
            for (int q = 0; q < NQ; ++q) v[j][q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j0 + j < cnt) {
                const P* p = part(j0 + j);
                pm[j] = part_ld<FAR>(&p->m[r]);
                pl[j] = part_ld<FAR>(&p->l[r]);
#pragma unroll
                for (int q = 0; q < NQ; ++q) v[j][q] = part_ld<FAR>(p->quad(r, d + 4 * q));
            }
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < AT; ++j) top = fmaxf(top, pm[j]);
        const float kr = m == -INFINITY ? 0.f : root_of(m - top), keep = kr * kr;
        l = l * kr * kr;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            o[q].x *= keep;
            o[q].y *= keep;
            o[q].z *= keep;
            o[q].w *= keep;
        }
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            if (pm[j] == -INFINITY && pl[j] == 0.f) continue;    // saw nothing
            const float wr = pm[j] == -INFINITY ? 1.f : root_of(pm[j] - top), w = wr * wr;   // -inf with a sum: NaN scores
            l = fmaf(pl[j] * wr, wr, l);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                o[q].x = fmaf(v[j][q].x, w, o[q].x);
                o[q].y = fmaf(v[j][q].y, w, o[q].y);
                o[q].z = fmaf(v[j][q].z, w, o[q].z);
                o[q].w = fmaf(v[j][q].w, w, o[q].w);
            }
        }
        m = top;
    }
    if (out) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) *const_cast<float4*>(out->quad(r, d + 4 * q)) = o[q];
        if (d == 0) {
            out->m[r] = m;
            out->l[r] = l;
        }
    } else {
        const int G = a.Hq / a.c.Hkv, row = q0 + f / G, head = h * G + f % G;
        const int64_t at = row * a.ldo + (int64_t)head * D + d;
        l = row_sum(l, f, first);
        const float inv = inv_sum(l);
#pragma unroll
        for (int q = 0; q < NQ; ++q) store_out4(a.O, at + 4 * q, a.yt, o[q].x * inv, o[q].y * inv, o[q].z * inv, o[q].w * inv);
        if (a.lse && d == 0) a.lse[(int64_t)row * a.Hq + head] = lse_of(m, l);
    }
}

}  // namespace kv8
}  // namespace cq

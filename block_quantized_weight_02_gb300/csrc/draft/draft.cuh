// Shared declarations of a drafting step: rotary positions and the launchers of
// its translation units.
#pragma once
#include "../../../include/cq_draft.h"
#include "../kv8/kv8.cuh"

namespace cq {
namespace draft {

struct Rope {
    const float* freq;
    const int32_t* pos;    // nullable where a row's place is known
    int half;              // rot / 2
    float mag;
};

cudaError_t launch_rope(const void* X, int xt, int T, int H, int D, int64_t ldx, const Rope& rope, int layout, void* Y, int yt,
                        int64_t ldy, cudaStream_t s);
cudaError_t launch_write_rope(const kv8::Cache& c, const kv8::Batch& b, int D, const void* K, const void* V, int xt, int64_t ldk,
                              int64_t ldv, const Rope& rope, int layout, cudaStream_t s);

struct VerifyArgs {
    const void *P, *Q;
    int64_t ldp, ldq;
    const int32_t* tokens;
    const uint32_t* mask;
    int64_t ldm;
    const int32_t* q_start;
    const float *u, *u_last;
    int32_t *out, *path, *count;
    int64_t ldo;
    int pt, T, V, B, max_q;
    int* err;
};
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);

#ifdef __CUDACC__

// ---- angles ----------------------------------------------------------------------------------------------------------
// A frequency of f radians a position is f / 2 pi turns, kept modulo 1 as a 64-bit fraction; a position times that
// fraction, modulo 2^64, is the angle, whatever the position's size and sign.  f is m 2^e with a 24-bit m, so m times a
// 128-bit 1 / 2 pi, shifted, is the fraction to 2^-64, and the angle is exact to 2^-33 of a turn for 31-bit positions.
// (In f32 the product p f alone would be 0.06 radians off at position 2^20.)
struct Turn {
    uint64_t f;
    bool bad;              // f is not finite, or too large
};
__device__ __forceinline__ Turn turn_of(float freq) {
    constexpr uint64_t HI = 0x28be60db9391054aull, LO = 0x7f09d5f47d4d3770ull;   // 2^128 / 2 pi
    const uint32_t u = __float_as_uint(freq);
    const int e = (int)(u >> 23 & 255) - 150;            // f = m 2^e (subnormal ones: 0)
    const uint64_t m = e == -150 ? 0 : (u & 0x7FFFFFu) | 0x800000u;
    const uint64_t mid = m * HI, carry = __umul64hi(m, LO);
    const uint64_t p1 = mid + carry, p2 = __umul64hi(m, HI) + (p1 < mid);
    const int r = max(-e, 8);                            // the fraction is (p2 p1) >> r
    uint64_t f = r < 64 ? p1 >> r | p2 << (64 - r) : r < 128 ? p2 >> (r - 64) : 0;
    return {u >> 31 ? 0 - f : f, e > -8};
}

// Cosine and sine of t / 2^64 turns, in f32 with an error of little more than the last rounding: the angle is taken to the nearest quarter,
// x in [-pi/4, pi/4] in two floats, and the series of sin x - x and cos x - 1 + x^2 / 2 (next terms below 2^-33) correct
// leading parts that are exact.
__device__ __forceinline__ void cos_sin(uint64_t t, float& c, float& s) {
    constexpr float K = 0x1.921fb6p-30f, K2 = -0x1.777a5cp-55f, KL = 0x1.921fb6p-56f;   // 2 pi / 2^32, and / 2^58
    const uint32_t top = (uint32_t)(t >> 32), low = (uint32_t)t, q = (top + (1u << 29)) >> 30;
    const uint32_t r = top - (q << 30);                  // 30 bits and a sign; the upper 24 first, then the rest and `low`
    const float rh = (float)(int)(r & ~63u), rl = (float)((r & 63u) << 26 | low >> 6);
    const float x = __fmul_rn(rh, K), xl = fmaf(rl, KL, fmaf(rh, K2, fmaf(rh, K, -x)));
    const float z = __fmul_rn(x, x), zl = fmaf(2.f * x, xl, fmaf(x, x, -z));
    float p = fmaf(z, -1.f / 39916800.f, 1.f / 362880.f);
    p = fmaf(z, p, -1.f / 5040.f);
    p = fmaf(z, p, 1.f / 120.f);
    p = fmaf(z, p, -1.f / 6.f);
    const float sn = x + fmaf(x * z, p, xl);
    p = fmaf(z, 1.f / 479001600.f, -1.f / 3628800.f);
    p = fmaf(z, p, 1.f / 40320.f);
    p = fmaf(z, p, -1.f / 720.f);
    p = fmaf(z, p, 1.f / 24.f);
    const float h = fmaf(-0.5f, z, 1.f), lost = fmaf(-0.5f, z, 1.f - h);
    const float cs = h + fmaf(z * z, p, fmaf(-0.5f, zl, lost));
    const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
    c = __uint_as_float(__float_as_uint(a) ^ ((q + 1) & 2) << 30);
    s = __uint_as_float(__float_as_uint(b) ^ (q & 2) << 30);
}
// Of a pair at position p, times mag (NaN: a frequency that is no number).
__device__ __forceinline__ float mag_of(const Turn& f, float mag) { return f.bad ? __uint_as_float(0x7FC00000u) : mag; }
__device__ __forceinline__ void cos_sin_at(const Turn& f, int p, float mag, float& c, float& s) {
    cos_sin(f.f * (uint64_t)(int64_t)p, c, s);
    c *= mag;
    s *= mag;
}

// A pair turned: each product is rounded, then their sum, as the same steps in f32 anywhere else would.
__device__ __forceinline__ float turn_first(float a, float b, float c, float s) { return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)); }
__device__ __forceinline__ float turn_second(float a, float b, float c, float s) { return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)); }
// Two pairs at once: a and b become what turn_first and turn_second give.
__device__ __forceinline__ void turn2(uint64_t& a, uint64_t& b, uint64_t c, uint64_t s) {
    const uint64_t p = sub2(mul2(a, c), mul2(b, s)), q = add2(mul2(b, c), mul2(a, s));
    a = p;
    b = q;
}

#endif  // __CUDACC__

}  // namespace draft
}  // namespace cq

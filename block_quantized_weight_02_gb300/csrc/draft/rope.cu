// Rotary positions of rows of heads, and the cache's write with rotated keys.
//
// Both are one pass over the data and bound by HBM: a (token, pair) angle costs about 80 instructions, so each
// block of threads makes a table of its tokens' cosines and sines in shared memory once, while its rows are on their way,
// and every head takes its factors from there.
//
// Measured: 16384 tokens of 32 heads of 128 channels in bf16 46 us, 5.8 TB/s; 3001 tokens of 24 heads, 48 of 96 channels in
// pairs, f32 to bf16, 9.6 us.  Four prompts of 20001 to 32768 tokens, 8 heads of 128 channels, written from bf16 108 us, 5.7 TB/s
// (109 without rotation); one token each of 96 sequences 7.0 us, latency.
#include "../kv8/store_common.cuh"
#include "draft.cuh"

namespace cq {
namespace draft {
namespace {

using kv8::In;

// ---- rows ------------------------------------------------------------------------------------------------------------
// A unit is 8 neighbouring channels of a head, together with their partners 8 channels rot/2 on in the half layout:
// everything is moved 16 bytes at a time, and in place too, as a thread reads its units before it writes them.
constexpr int THREADS = 256;
template <class X, int LAYOUT>
constexpr int EACH = sizeof(X) == 4 && LAYOUT == CQ_ROPE_HALF ? 2 : 4;   // units that a thread has under way

template <class X>
struct Eight {                                           // 8 channels as they lie in memory
    uint4 v[sizeof(X) / 2];
    __device__ __forceinline__ void load(const X* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (sizeof(X) == 2) {
            In<X>::get(v[0], f);
        } else {
            float a[4], b[4];
            In<X>::get(v[0], a);
            In<X>::get(v[1], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
        }
    }
};
template <class Y>
__device__ __forceinline__ void store8(Y* p, const float (&f)[8]) {
    if constexpr (sizeof(Y) == 2) {
        *reinterpret_cast<uint4*>(p) = In<Y>::put(f);
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

struct Rows {
    const void* x;
    void* y;
    int64_t ldx, ldy;
    int T, H, D, per;      // per: tokens of a block of threads
};

template <class X, class Y, int LAYOUT>
__global__ void __launch_bounds__(THREADS) k_rope(const Rows a, const Rope rope) {
    constexpr bool HALVES = LAYOUT == CQ_ROPE_HALF;
    constexpr int E = EACH<X, LAYOUT>;
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ float4 table4[];
    float* cs = reinterpret_cast<float*>(table4);        // [per][half] cosines, then sines
    float* sn = cs + a.per * rope.half;
    const int64_t t0 = (int64_t)blockIdx.x * a.per;
    const int n = (int)min((int64_t)a.per, a.T - t0);
    const int turned = HALVES ? rope.half / 8 : rope.half / 4;                     // units of a head with pairs
    const int units = turned + (a.D - 2 * rope.half) / 8, all = units * a.H * n;
    const X* x = static_cast<const X*>(a.x) + t0 * a.ldx;
    Y* y = static_cast<Y*>(a.y) + t0 * a.ldy;
    for (int i0 = 0; i0 < all; i0 += THREADS * E) {
        Eight<X> f[E], g[HALVES ? E : 1];
        int tok[E], unit[E], ch[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = i0 + e * THREADS + threadIdx.x, h = i / units, u = i - h * units, t = h / a.H;
            // (the half layout's channels past the rotated ones follow both halves)
            tok[e] = t;
            unit[e] = i < all ? u : -1;
            ch[e] = (h - t * a.H) * a.D + (HALVES && u >= turned ? 8 * u + rope.half : 8 * u);
            if (i < all) {
                f[e].load(x + t * a.ldx + ch[e]);
                if (HALVES && u < turned) g[HALVES ? e : 0].load(x + t * a.ldx + ch[e] + rope.half);
            }
        }
        if (i0 == 0) {                                   // the table, while the first rows are on their way
            for (int i = threadIdx.x; i < n * rope.half; i += THREADS) {
                const int t = i / rope.half, k = i - t * rope.half;
                const Turn w = turn_of(__ldcg(rope.freq + k));
                cos_sin_at(w, __ldcg(rope.pos + t0 + t), mag_of(w, rope.mag), cs[i], sn[i]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (unit[e] < 0) continue;
            float lo[8], hi[8];
            f[e].get(lo);
            Y* to = y + tok[e] * a.ldy + ch[e];
            if (unit[e] < turned) {
                constexpr int N = HALVES ? 8 : 4;        // pairs of a unit
                if (HALVES) g[HALVES ? e : 0].get(hi);
                const int k = tok[e] * rope.half + N * unit[e];
#pragma unroll
                for (int j = 0; j < N; j += 4) {
                    const float4 p = *reinterpret_cast<const float4*>(cs + k + j), q = *reinterpret_cast<const float4*>(sn + k + j);
                    const float c[4] = {p.x, p.y, p.z, p.w}, s[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& a0 = HALVES ? lo[j + i] : lo[2 * i];
                        float& b0 = HALVES ? hi[j + i] : lo[2 * i + 1];
                        const float a1 = turn_first(a0, b0, c[i], s[i]), b1 = turn_second(a0, b0, c[i], s[i]);
                        a0 = a1;
                        b0 = b1;
                    }
                }
                if (HALVES) store8(to + rope.half, hi);
            }
            store8(to, lo);
        }
    }
}

template <class X, class Y>
cudaError_t rope_as(Rows a, const Rope& rope, int layout, cudaStream_t s) {
    // tokens of a block of threads: enough units for all threads, a table of at most 32 KB
    const int units = (rope.half / (layout == CQ_ROPE_HALF ? 8 : 4) + (a.D - 2 * rope.half) / 8) * a.H;
    a.per = std::max(1, std::min({THREADS * (layout == CQ_ROPE_HALF ? EACH<X, CQ_ROPE_HALF> : EACH<X, CQ_ROPE_PAIRS>) / units, 4096 / rope.half, a.T}));
    const size_t smem = (size_t)a.per * rope.half * 8;
    const dim3 grid((a.T + a.per - 1) / a.per);
    if (layout == CQ_ROPE_HALF) return kv8::launch_pdl(k_rope<X, Y, CQ_ROPE_HALF>, grid, dim3(THREADS), smem, s, a, rope);
    return kv8::launch_pdl(k_rope<X, Y, CQ_ROPE_PAIRS>, grid, dim3(THREADS), smem, s, a, rope);
}
template <class X>
cudaError_t rope_from(const Rows& a, int yt, const Rope& rope, int layout, cudaStream_t s) {
    if (yt == CQ_F16) return rope_as<X, __half>(a, rope, layout, s);
    if (yt == CQ_BF16) return rope_as<X, __nv_bfloat16>(a, rope, layout, s);
    return rope_as<X, float>(a, rope, layout, s);
}

// ---- keys and values to the cache -----------------------------------------------------------------------------------
// A block of threads has one block of 32 tokens, and some or all of its heads: its table serves them all.  Two warps
// have one head's keys or values, 16 tokens each, and exchange their largest magnitudes; a lane has 8 channels of a token,
// in the half layout four and their partners, so that the turned values stay in registers between the magnitudes and the
// codes (with a whole block to a warp they took 226, and turning twice instead cost more than the warps gained).
// The next head's rows are on their way meanwhile (16-bit rows, or 64 channels).  W warps: 8, two heads at a time; 4 where
// there is one head, so that an SM has more blocks.

// Four channels, as they lie in memory.
template <class X>
struct Four {
    uint32_t v[sizeof(X)];
    __device__ __forceinline__ void load(const X* p, bool in) {
        if constexpr (sizeof(X) == 2) {
            const uint2 u = in ? __ldcs(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
            v[0] = u.x, v[1] = u.y;
        } else {
            const uint4 u = in ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(X) == 4) return __uint_as_float(v[i]);
        else if constexpr (std::is_same<X, __half>::value) return __half2float(__ushort_as_half((unsigned short)(v[i / 2] >> 16 * (i & 1))));
        else return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
};

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <class X, int D, int LAYOUT, int W>
struct Writer {
    static constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 16 / RPI;     // lanes a row, rows a step, steps
    static constexpr bool AHEAD = sizeof(X) * D <= 256;  // two heads' rows at once fit the registers
    const kv8::Cache& c;
    const kv8::Item& it;
    const float4 *cs4, *sn4;                             // rows of D / 2 cosines and sines
    uint32_t (*tops)[W];
    int half;                                            // rot / 2

    // The block's rows out of `src` (row it.lo's), FULL: all 32.
    template <bool FULL>
    __device__ __forceinline__ void run(const X* src, int64_t ld, int head, int step, const Rope& rope, float freq, int k, int wide) {
        using namespace kv8;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = warp >> 1 & 1;
        const int row0 = 16 * (warp & 1) + lane / LPR, unit = lane % LPR;
        const int turned = half / 4;                     // units of a row with pairs
        const bool turns = !kv && unit < turned;
        const int ch = LAYOUT == CQ_ROPE_PAIRS ? 8 * unit : unit < turned ? 4 * unit : 8 * unit;
        const int ch2 = LAYOUT == CQ_ROPE_HALF && unit < turned ? ch + half : ch + 4;
        auto in = [&](int i) { return FULL || (row0 + i * RPI >= it.lo && row0 + i * RPI < it.hi); };
        const X* from = src + (row0 - it.lo) * ld + ch;
        Four<X> u[IT][2];
        auto load = [&](int head) {
            const X* p = from + head * D;
#pragma unroll
            for (int i = 0; i < IT; ++i, p += RPI * ld) {
                u[i][0].load(p, in(i));
                u[i][1].load(p + (ch2 - ch), in(i));
            }
        };
        if (head < c.Hkv) load(head);
        table(rope, freq, k, wide);
        __syncthreads();
        float* sp = (kv ? c.s[1] : c.s[0]) + it.block;
        int8_t* dst = (kv ? c.q[1] : c.q[0]) + it.block * (BLK * D) + row0 * D + ch;
        const int blocks = c.page / BLK;                 // from a head's blocks to the next one's
        for (int n = 0; head < c.Hkv; head += step, n ^= 1) {
            uint64_t f[IT][4];                           // a row's channels in pairs: ch .., ch2 ..
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) f[i][j] = pair(u[i][j / 2].get(2 * (j & 1)), u[i][j / 2].get(2 * (j & 1) + 1));
            if (AHEAD && head + step < c.Hkv) load(head + step);
            float* sph = sp + (int64_t)head * blocks;
            int8_t* to = dst + (int64_t)head * blocks * (BLK * D);
            const float s0 = !FULL && it.lo > 0 ? *sph : 0.f;
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (turns && in(i)) {
                    const float4 p = cs4[(row0 + i * RPI) * (D / 8) + unit], q = sn4[(row0 + i * RPI) * (D / 8) + unit];
                    if (LAYOUT == CQ_ROPE_HALF) {
                        turn2(f[i][0], f[i][2], pair(p.x, p.y), pair(q.x, q.y));
                        turn2(f[i][1], f[i][3], pair(p.z, p.w), pair(q.z, q.w));
                    } else {                             // (a, b) (a, b) of two pairs at a time
                        const float c4[4] = {p.x, p.y, p.z, p.w}, s4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 v = unpair(f[i][j]);
                            f[i][j] = pair(turn_first(v.x, v.y, c4[j], s4[j]), turn_second(v.x, v.y, c4[j], s4[j]));
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = unpair(f[i][j]);
                    top = max_abs(top, v.x, v.y);
                }
            }
            const uint32_t m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            if (lane == 0) tops[n][warp] = m0;
            named_bar_sync(1 + (warp >> 1), 64);         // (both have the old scale, too)
            const uint32_t m = max(m0, tops[n][warp ^ 1]);
            const bool bad = m >= 0x7F800000u || s0 != s0;
            const float s1 = bad ? __uint_as_float(0x7FC00000u) : fmaxf(s0, pow2(scale_exp(__uint_as_float(m))));
            const float inv = bad ? 0.f : 1.0f / s1;     // exact: a power of two
            if (!FULL && it.lo > 0 && s1 > s0) {         // the kept codes move to the larger scale
                const float ratio = s0 * inv;
                for (int i = 0; i < IT && row0 + i * RPI < it.lo; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t* p = reinterpret_cast<uint32_t*>(to + i * RPI * D + (e ? ch2 - ch : 0));
                        const uint32_t w = *p;
                        *p = pack4(code_of(byte_f(w, 0), ratio), code_of(byte_f(w, 1), ratio), code_of(byte_f(w, 2), ratio),
                                   code_of(byte_f(w, 3), ratio));
                    }
            }
            if (bad) {                                   // (a spoilt block's codes are 0)
#pragma unroll
                for (int i = 0; i < IT; ++i) f[i][0] = f[i][1] = f[i][2] = f[i][3] = 0;
            }
            const uint64_t by = pair(inv, inv), one = pair(12582912.0f, 12582912.0f);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (!in(i)) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e) {            // the codes are the sums' low bytes, as in code_of
                    const uint64_t a = fma2(f[i][2 * e], by, one), b = fma2(f[i][2 * e + 1], by, one);
                    *reinterpret_cast<uint32_t*>(to + i * RPI * D + (e ? ch2 - ch : 0)) =
                        pack4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
                }
            }
            if (lane == 0 && !(warp & 1)) *sph = s1;
            if (!AHEAD && head + step < c.Hkv) load(head + step);
        }
    }

    // Cosines and sines of the block's rows; a thread keeps to one pair (k of `wide`, a power of two).
    __device__ __forceinline__ void table(const Rope& rope, float freq, int k, int wide) const {
        float* cs = reinterpret_cast<float*>(const_cast<float4*>(cs4));
        float* sn = reinterpret_cast<float*>(const_cast<float4*>(sn4));
        constexpr int PASSES = D / (2 * W);              // of 32 W / wide rows, at most
        const int step = W * 32 / wide, r0 = it.lo + threadIdx.x / wide;
        int p[PASSES];
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int at = r0 - it.lo + i * step;
            p[i] = rope.pos && at < it.hi - it.lo ? __ldcg(rope.pos + it.row0 + at) : it.tok0 + at;
        }
        const Turn f = turn_of(freq);
        const float mag = mag_of(f, rope.mag);
        if (k < half)
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r0 + i * step;
                if (r < it.hi) cos_sin_at(f, p[i], mag, cs[r * (D / 2) + k], sn[r * (D / 2) + k]);
            }
    }
};

template <class X, int D, int LAYOUT, int W>
__global__ void __launch_bounds__(W * 32, (sizeof(X) * D == 128 ? 3 : 2) * 8 / W) k_write_rope(const kv8::Cache c, const kv8::Batch b, const X* K, const X* V,
                                                              int64_t ldk, int64_t ldv, const Rope rope, int groups) {
    __shared__ float4 cs4[kv8::BLK * D / 8], sn4[kv8::BLK * D / 8];
    __shared__ uint32_t tops[2][W];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, kv = warp >> 1 & 1;
    int wide = 8;
    while (wide < rope.half) wide *= 2;
    const int k = threadIdx.x & (wide - 1);
    const float freq = k < rope.half ? __ldcg(rope.freq + k) : 0.f;
    const kv8::Item it = kv8::find_item<true>(c, b, blockIdx.x / groups, kv, 0);
    if (!it.ok) return;                                  // (the same for the whole block of threads)
    Writer<X, D, LAYOUT, W> w = {c, it, cs4, sn4, tops, rope.half};
    const int64_t ld = kv ? ldv : ldk;
    const X* src = (kv ? V : K) + it.row0 * ld;
    const int head = (int)(blockIdx.x % groups) * (W / 4) + (warp >> 2), step = W / 4 * groups;
    if (it.hi - it.lo == kv8::BLK) w.template run<true>(src, ld, head, step, rope, freq, k, wide);
    else w.template run<false>(src, ld, head, step, rope, freq, k, wide);
}

template <class X, int D>
cudaError_t write_as(const kv8::Cache& c, const kv8::Batch& b, const void* K, const void* V, int64_t ldk, int64_t ldv, const Rope& rope,
                     int layout, cudaStream_t s) {
    const X *k = static_cast<const X*>(K), *v = static_cast<const X*>(V);
    // Blocks of threads of a block of tokens: one makes the table once, but goes through its heads two at a time; so more
    // while the grid has at most three an SM (two run at a time, and half of them may find no tokens).  Over 252 shapes (1 to 300
    // sequences with 1, 6 or 40 tokens, 2, 8 and 16 heads, both widths, bf16 and f32) three are 1.5 % behind the best of 1, 2, 3, 4 and 6 an
    // SM on average, two 4.7 %, four 2.1 %: one token each of 96 sequences 7.0 us (four: 8.7), 64 sequences 6.8 (two: 6.2, four:
    // 6.9, one: 8.2), 160 with 16 heads of 64 channels 11.9, as with four (six: 8.9).
    const int64_t slots = kv8::store_slots(c, b);
    const int groups = (int)std::max<int64_t>(1, std::min<int64_t>((c.Hkv + 1) / 2, 3LL * num_sms() / slots));
    const dim3 grid((unsigned)(slots * groups));
    auto run = [&](auto kernel, int warps) { return kv8::launch_pdl(kernel, grid, dim3(warps * 32), 0, s, c, b, k, v, ldk, ldv, rope, groups); };
    if (layout == CQ_ROPE_HALF) return c.Hkv == 1 ? run(k_write_rope<X, D, CQ_ROPE_HALF, 4>, 4) : run(k_write_rope<X, D, CQ_ROPE_HALF, 8>, 8);
    return c.Hkv == 1 ? run(k_write_rope<X, D, CQ_ROPE_PAIRS, 4>, 4) : run(k_write_rope<X, D, CQ_ROPE_PAIRS, 8>, 8);
}
template <class X>
cudaError_t write_from(const kv8::Cache& c, const kv8::Batch& b, int D, const void* K, const void* V, int64_t ldk, int64_t ldv,
                       const Rope& rope, int layout, cudaStream_t s) {
    return D == 128 ? write_as<X, 128>(c, b, K, V, ldk, ldv, rope, layout, s) : write_as<X, 64>(c, b, K, V, ldk, ldv, rope, layout, s);
}

}  // namespace

cudaError_t launch_rope(const void* X, int xt, int T, int H, int D, int64_t ldx, const Rope& rope, int layout, void* Y, int yt,
                        int64_t ldy, cudaStream_t s) {
    const Rows a = {X, Y, ldx, ldy, T, H, D, 0};
    if (xt == CQ_F16) return rope_from<__half>(a, yt, rope, layout, s);
    if (xt == CQ_BF16) return rope_from<__nv_bfloat16>(a, yt, rope, layout, s);
    return rope_from<float>(a, yt, rope, layout, s);
}
cudaError_t launch_write_rope(const kv8::Cache& c, const kv8::Batch& b, int D, const void* K, const void* V, int xt, int64_t ldk,
                              int64_t ldv, const Rope& rope, int layout, cudaStream_t s) {
    if (xt == CQ_F16) return write_from<__half>(c, b, D, K, V, ldk, ldv, rope, layout, s);
    if (xt == CQ_BF16) return write_from<__nv_bfloat16>(c, b, D, K, V, ldk, ldv, rope, layout, s);
    return write_from<float>(c, b, D, K, V, ldk, ldv, rope, layout, s);
}

}  // namespace draft
}  // namespace cq

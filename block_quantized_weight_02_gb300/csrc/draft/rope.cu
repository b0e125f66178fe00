// Rotary positions of rows of heads, and the cache's write with rotated keys.
//
// Both are one pass over the data and bound by HBM: a (token, pair) angle costs about 80 instructions, so each
// block of threads makes a table of its tokens' cosines and sines in shared memory once, while its rows are on their way,
// and every head takes its factors from there.
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
template <class X>
constexpr int EACH = sizeof(X) == 2 ? 4 : 2;             // units that a thread has under way

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
    constexpr int E = EACH<X>;
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
                cos_sin_at(turn_of(__ldcg(rope.freq + k)), __ldcg(rope.pos + t0 + t), rope.mag, cs[i], sn[i]);
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
    a.per = std::max(1, std::min({THREADS * EACH<X> / units, 4096 / rope.half, a.T}));
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
// One warp has one block of 32 tokens of one head, as in the write without rotation; the warps of a block of
// threads have up to four heads of the keys and of the values of one block of tokens, and make its table together while
// their rows are on the way.
constexpr int HEADS = 4;

template <class X, int D, int LAYOUT>
__global__ void __launch_bounds__(2 * HEADS * 32) k_write_rope(const kv8::Cache c, const kv8::Batch b, const X* K, const X* V,
                                                               int64_t ldk, int64_t ldv, const Rope rope, int groups) {
    using namespace kv8;
    pdl_launch_dependents();
    pdl_wait();
    constexpr int N = In<X>::N, LPR = D / N, RPI = 32 / LPR, IT = BLK / RPI;   // lanes a row, rows a step
    __shared__ float4 cs4[BLK * D / 8], sn4[BLK * D / 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = (int)(blockIdx.x % groups) * HEADS + (warp >> 1);
    const Item it = find_item<true>(c, b, blockIdx.x / groups, warp & 1, head);
    if (!it.ok) return;                                  // (the same for the whole block of threads)
    const bool mine = head < c.Hkv;
    const int sub = lane / LPR, col = (lane % LPR) * N;
    const int64_t ld = it.kv ? ldv : ldk;
    const X* src = (it.kv ? V : K) + it.row0 * ld + (int64_t)head * D + col;
    uint4 u[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub;
        u[i] = make_uint4(0, 0, 0, 0);
        if (mine && r >= it.lo && r < it.hi) u[i] = __ldcs(reinterpret_cast<const uint4*>(src + (r - it.lo) * ld));
    }
    float* cs = reinterpret_cast<float*>(cs4);
    float* sn = reinterpret_cast<float*>(sn4);
    // Factors in chunks of four pairs, rows of D / 8 chunks.  Half layout, 16-bit rows: a lane takes two neighbouring
    // chunks; the even ones lie ahead of the odd ones, so that lanes read neighbouring chunks.
    auto chunk = [&](int k) { return LAYOUT == CQ_ROPE_HALF && N == 8 ? (k >> 1) + (k & 1) * (D / 16) : k; };
    for (int i = it.lo * rope.half + threadIdx.x; i < it.hi * rope.half; i += blockDim.x) {
        const int r = i / rope.half, k = i - r * rope.half, at = r * (D / 2) + 4 * chunk(k >> 2) + (k & 3);
        const int p = rope.pos ? __ldcg(rope.pos + it.row0 + (r - it.lo)) : it.tok0 + (r - it.lo);
        cos_sin_at(turn_of(__ldcg(rope.freq + k)), p, rope.mag, cs[at], sn[at]);
    }
    __syncthreads();
    if (!mine) return;
    // A key's channels are turned where they are needed, for the block's largest magnitude and again for the codes: kept in
    // between, in f32, they would take twice the registers of the rows and leave half the warps.
    const int h = rope.half;
    const bool first = col < h, turns = !it.kv && col < 2 * h;
    const int from = !turns ? lane : first ? lane + h / N : lane - h / N;    // half layout: the lane with the partners
    const int at = LAYOUT == CQ_ROPE_HALF ? (first ? col : col - h) / 4 : col / 2;
    store_block<D, N>(c, it, [&](int i, float (&f)[N]) {
        In<X>::get(u[i], f);
        if (it.kv) return;                               // (the same for the whole warp)
        const int r = i * RPI + sub;
        const bool turn = turns && r >= it.lo && r < it.hi;
        if constexpr (LAYOUT == CQ_ROPE_HALF) {
            uint4 w;
            w.x = __shfl_sync(0xffffffffu, u[i].x, from);
            w.y = __shfl_sync(0xffffffffu, u[i].y, from);
            w.z = __shfl_sync(0xffffffffu, u[i].z, from);
            w.w = __shfl_sync(0xffffffffu, u[i].w, from);
            if (!turn) return;
            float g[N];
            In<X>::get(w, g);
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const float4 p = cs4[r * (D / 8) + chunk(at + j / 4)], q = sn4[r * (D / 8) + chunk(at + j / 4)];
                const float c4[4] = {p.x, p.y, p.z, p.w}, s4[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[j + e] = first ? turn_first(f[j + e], g[j + e], c4[e], s4[e]) : turn_second(g[j + e], f[j + e], c4[e], s4[e]);
            }
        } else {
            if (!turn) return;
            float c4[N / 2], s4[N / 2];
            if constexpr (N == 8) {
                const float4 p = *reinterpret_cast<const float4*>(cs + r * (D / 2) + at), q = *reinterpret_cast<const float4*>(sn + r * (D / 2) + at);
                c4[0] = p.x, c4[1] = p.y, c4[2] = p.z, c4[3] = p.w;
                s4[0] = q.x, s4[1] = q.y, s4[2] = q.z, s4[3] = q.w;
            } else {
                const float2 p = *reinterpret_cast<const float2*>(cs + r * (D / 2) + at), q = *reinterpret_cast<const float2*>(sn + r * (D / 2) + at);
                c4[0] = p.x, c4[1] = p.y;
                s4[0] = q.x, s4[1] = q.y;
            }
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float a0 = f[2 * j], b0 = f[2 * j + 1];
                f[2 * j] = turn_first(a0, b0, c4[j], s4[j]);
                f[2 * j + 1] = turn_second(a0, b0, c4[j], s4[j]);
            }
        }
    });
}

template <class X, int D>
cudaError_t write_as(const kv8::Cache& c, const kv8::Batch& b, const void* K, const void* V, int64_t ldk, int64_t ldv, const Rope& rope,
                     int layout, cudaStream_t s) {
    const X *k = static_cast<const X*>(K), *v = static_cast<const X*>(V);
    const int groups = (c.Hkv + HEADS - 1) / HEADS;
    const dim3 grid((unsigned)(kv8::store_slots(c, b) * groups)), block(2 * std::min(c.Hkv, HEADS) * 32);
    if (layout == CQ_ROPE_HALF) return kv8::launch_pdl(k_write_rope<X, D, CQ_ROPE_HALF>, grid, block, 0, s, c, b, k, v, ldk, ldv, rope, groups);
    return kv8::launch_pdl(k_write_rope<X, D, CQ_ROPE_PAIRS>, grid, block, 0, s, c, b, k, v, ldk, ldv, rope, groups);
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

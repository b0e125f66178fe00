// Attention over the 8-bit cache for few query rows per sequence (single tokens,
// short guesses): at most 16 rows of one KV head, a row being a (token, head of the
// group) pair.
//
// Bound by HBM: the cache is read once.  The work is the list of all visible blocks
// (32 tokens of one KV head, keys and values: 8 KB at D = 128), ordered by sequence,
// head and token, cut into equal contiguous shares, one per warp of the grid: ragged
// lengths balance themselves, and a share crosses from one head or sequence to the
// next without any barrier.  Each warp owns a ring of blocks that TMA fills ahead of it
// across those borders.
//
// One block: S = Q K^T as m16n8k16 products (rows x tokens), the running maximum and
// sum in f32 registers, then O += P V with the score fragments as the first operand,
// so nothing of the softmax leaves registers.  The codes become fp16 in registers,
// exactly.  The operands' inner order is free as long as both sides agree: a lane takes 4
// neighbouring codes of its token as one k16 step's part (keys), and 16 neighbouring
// channels of its tokens as the 16 output tiles (values), so every shared-memory load is
// 16 bytes, without bank conflicts under the copies' swizzle.
//
// A key block's scale multiplies the scores in f32.  A value block's scale 2^lv joins the
// exponent, w = 2^(s - m + 15 + lv - ref) with ref the largest lv so far, so the weights
// fill fp16's range (11 bits down to 2^-29 of the largest weight) whatever the scales are;
// the normaliser takes w 2^(ref - lv).
//
// Shares that do not hold a whole (sequence, head) leave (O, m, l) partials; the CTA's own
// are joined after a barrier, those across CTAs by a second small kernel, always in share
// order, so results do not depend on timing.
#include "attn_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int NW = 8;                 // warps per CTA
constexpr int ROWS = 16;
constexpr int MAX_CTAS = 256;         // workspace bound
constexpr int P_EXP = 15;             // weights carry 2^15

struct Maps {
    CUtensorMap t[2];                 // keys, values: {D, pages * Hkv * page}, box {D, 32}
};

// Workspace: per-warp partials [MAX_CTAS * NW][2], per-CTA partials [MAX_CTAS][2], then each CTA's two segments.
template <int D>
struct Part {
    float o[ROWS][D];
    float m[ROWS], l[ROWS];
};
template <int D>
struct Space {
    Part<D> warp[MAX_CTAS * NW][2];
    Part<D> cta[MAX_CTAS][2];
    int seg[MAX_CTAS][2];             // segment of cta[i][0] (began earlier) and cta[i][1] (began here, goes on), or -1
};

template <int D>
struct Ring {
    static constexpr int ST = D == 128 ? 3 : 6;           // blocks in the ring of a warp: 192 KB a CTA
    static constexpr int TILE = BLK * D;                  // bytes of a block's keys or values
    static constexpr int BYTES = NW * ST * 2 * TILE;
};

struct Seq {
    int b, q0, n, L, first, units;    // blocks first .. first + units - 1 (L = 0: one unit without a block)
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
    Seq s;
    s.b = b;
    s.q0 = __ldg(a.b.q_start + b);
    s.n = __ldg(a.b.q_start + b + 1) - s.q0;
    s.L = __ldg(a.b.lens + b);
    s.first = row_lo(0, s.n, s.L, a.window) / BLK;
    s.units = s.n == 0 ? 0 : max(1, (s.L + BLK - 1) / BLK - s.first);
    return s;
}

// Position in the list of blocks.
struct Cursor {
    Seq s;
    int h, i;                          // head, block of the segment
    __device__ __forceinline__ void next(const AttnArgs& a) {
        if (++i < s.units) return;
        i = 0;
        if (++h < a.c.Hkv) return;
        h = 0;
        do s = seq_of(a, min(s.b + 1, a.c.B - 1)); while (s.units == 0 && s.b < a.c.B - 1);
    }
};

__device__ __forceinline__ uint4 lds128(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
    return v;
}

// The 16 x D result of a warp: lane (g, t) holds rows g and g + 8, channels t * D/4 ...
template <int D>
struct Acc {
    static constexpr int DL = D / 4;   // channels of a lane
    float o[D / 8][4];                 // output tile nn: rows g, g, g + 8, g + 8; channels t DL + nn, t DL + DL/2 + nn
    float m[2], l[2];
    __device__ __forceinline__ float ch(int row, int i) const {   // channel t DL + i of row g + 8 row
        return o[i % (DL / 2)][2 * row + i / (DL / 2)];
    }
};

template <int D>
__device__ __forceinline__ void write_part(Part<D>* p, const Acc<D>& c, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = g + 8 * k;
        if (r >= rows) continue;
        float4* o = reinterpret_cast<float4*>(&p->o[r][t * Acc<D>::DL]);
#pragma unroll
        for (int i = 0; i < Acc<D>::DL / 4; ++i)
            o[i] = make_float4(c.ch(k, 4 * i), c.ch(k, 4 * i + 1), c.ch(k, 4 * i + 2), c.ch(k, 4 * i + 3));
        if (t == 0) {
            p->m[r] = c.m[k];
            p->l[r] = c.l[k];
        }
    }
}

__device__ __forceinline__ float inv_sum(float l) { return l == 0.f ? 0.f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
}

template <int D>
__device__ __forceinline__ void write_out(const AttnArgs& a, const Acc<D>& c, const Seq& s, int h) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = a.Hq / a.c.Hkv;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = g + 8 * k;
        if (r >= s.n * G) continue;
        const int row = s.q0 + r / G, head = h * G + r % G;
        const float f = inv_sum(c.l[k]);
        const int64_t at = row * a.ldo + (int64_t)head * D + t * Acc<D>::DL;
#pragma unroll
        for (int i = 0; i < Acc<D>::DL / 4; ++i)
            store_out4(a.O, at + 4 * i, a.yt, c.ch(k, 4 * i) * f, c.ch(k, 4 * i + 1) * f, c.ch(k, 4 * i + 2) * f,
                       c.ch(k, 4 * i + 3) * f);
        if (a.lse && t == 0) a.lse[(int64_t)row * a.Hq + head] = lse_of(c.m[k], c.l[k]);
    }
}

// Joins partials part(0) .. part(cnt - 1) of one segment: into `out` (nullable), else the output rows.
// All threads of the CTA.
template <int D, class F>
__device__ __forceinline__ void join(const AttnArgs& a, const Seq& s, int h, int cnt, F part, Part<D>* out) {
    const int G = a.Hq / a.c.Hkv, rows = s.n * G;
    for (int k = threadIdx.x; k < rows * (D / 4); k += NW * 32) {
        const int r = k / (D / 4), d = k % (D / 4) * 4;
        float m = -INFINITY;
        for (int j = 0; j < cnt; ++j) m = fmaxf(m, __ldcg(&part(j)->m[r]));
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < cnt; ++j) {
            const Part<D>* p = part(j);
            const float pm = __ldcg(&p->m[r]), w = pm == -INFINITY ? 0.f : ex2(pm - m);
            const float pl = __ldcg(&p->l[r]);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(&p->o[r][d]));
            if (pm == -INFINITY && pl == 0.f) continue;    // saw nothing
            l += pl * w;
            o.x += v.x * w;
            o.y += v.y * w;
            o.z += v.z * w;
            o.w += v.w * w;
        }
        if (out) {
            *reinterpret_cast<float4*>(&out->o[r][d]) = o;
            if (d == 0) {
                out->m[r] = m;
                out->l[r] = l;
            }
        } else {
            const int row = s.q0 + r / G, head = h * G + r % G;
            const float f = inv_sum(l);
            store_out4(a.O, row * a.ldo + (int64_t)head * D + d, a.yt, o.x * f, o.y * f, o.z * f, o.w * f);
            if (a.lse && d == 0) a.lse[(int64_t)row * a.Hq + head] = lse_of(m, l);
        }
    }
}

// PT: fp16 terms that carry a weight (one for 16-bit outputs, two for f32).
template <int D, int PT>
__global__ void __launch_bounds__(NW * 32, 1) k_attn_decode(const __grid_constant__ Maps maps, const AttnArgs a,
                                                            uint64_t wait_ns) {
    using R = Ring<D>;
    constexpr int KS = D / 16;           // k16 steps of a score
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[NW][R::ST];
    __shared__ float2 scales[NW][R::ST]; // the staged blocks' key scale and value scale
    __shared__ int64_t pre[NW * 32 + 1]; // units before each thread's sequences
    __shared__ int64_t wsum[NW];
    __shared__ int wseg[NW][2];          // segment of each warp's two partials, or -1
    __shared__ int stop;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring0 = ((smem_u32(raw) + 1023u) & ~1023u) + warp * (R::ST * 2 * R::TILE);
    Space<D>* sp = static_cast<Space<D>*>(a.ws);
    if (lane == 0)
        for (int i = 0; i < R::ST; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    if (threadIdx.x == 0) stop = 0;
    fence_mbar_init();
    pdl_launch_dependents();
    pdl_wait();

    // ---- the list of blocks: units per sequence, summed in order; every entry is checked
    const int per = (a.c.B + NW * 32 - 1) / (NW * 32);     // sequences of a thread
    int64_t mine = 0;
    bool bad = false;
    for (int b = threadIdx.x * per; b < min((int)(threadIdx.x + 1) * per, a.c.B); ++b) {
        const int qs = __ldg(a.b.q_start + b), qe = __ldg(a.b.q_start + b + 1), L = __ldg(a.b.lens + b);
        if (!rows_ok(qs, qe, a.b.T, a.max_q) || L < 0 || L > a.c.ldt * a.c.page) bad = true;
        else mine += (int64_t)seq_of(a, b).units * a.c.Hkv;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            set_err(a.b.err, DEV_INDEX);
            sp->seg[blockIdx.x][0] = sp->seg[blockIdx.x][1] = -1;
        }
        return;
    }
    int64_t inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int i = 0; i < NW; ++i) {
        if (i < warp) before += wsum[i];
        total += wsum[i];
    }
    pre[threadIdx.x] = before + inc - mine;
    if (threadIdx.x == 0) pre[NW * 32] = total;
    __syncthreads();
    // Shares: of the CTAs, at least NW units each while there are few; of its warps.
    const int64_t ctas = min((int64_t)gridDim.x, (total + NW - 1) / NW);
    const bool busy = blockIdx.x < ctas;
    const int64_t c0 = busy ? total * blockIdx.x / ctas : 0, c1 = busy ? total * (blockIdx.x + 1) / ctas : 0;
    const int64_t u0 = c0 + (c1 - c0) * warp / NW, u1 = c0 + (c1 - c0) * (warp + 1) / NW;

    auto seek = [&](int64_t u, Cursor& c) {      // u < total
        int lo = 0, hi = NW * 32;                // pre[lo] <= u < pre[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pre[mid] <= u) lo = mid; else hi = mid;
        }
        int64_t at = u - pre[lo];
        int b = lo * per;
        while (true) {
            c.s = seq_of(a, b);
            const int64_t all = (int64_t)c.s.units * a.c.Hkv;
            if (at < all) break;
            at -= all;
            ++b;
        }
        c.h = (int)(at / c.s.units);
        c.i = (int)(at % c.s.units);
    };

    if (lane < 2) wseg[warp][lane] = -1;
    if (u0 < u1) {
        Cursor cons, prod;
        seek(u0, cons);
        prod = cons;
        int64_t pu = u0;                         // next unit to load
        int pstage = 0;
        // 32 blocks' pages and scales at a time, one per lane
        int have = 0, used = 0, row = 0;
        float2 sc = make_float2(0.f, 0.f);

        auto produce = [&]() {
            if (pu >= u1) return;
            if (prod.s.L > 0) {
                if (used == have) {
                    have = (int)min((int64_t)min(32, prod.s.units - prod.i), u1 - pu);
                    used = 0;
                    if (lane < have) {
                        const int tok = (prod.s.first + prod.i + lane) * BLK;
                        int pid = __ldg(a.c.table + prod.s.b * a.c.ldt + tok / a.c.page);
                        if (pid < 0 || pid >= a.c.pages) {   // read some page instead: the result is void
                            set_err(a.b.err, DEV_INDEX);
                            pid = 0;
                        }
                        row = (pid * a.c.Hkv + prod.h) * a.c.page + tok % a.c.page;
                        sc = make_float2(__ldg(a.c.s[0] + row / BLK), __ldg(a.c.s[1] + row / BLK));
                    }
                }
                const int r = __shfl_sync(0xffffffffu, row, used);
                if (lane == used) scales[warp][pstage] = sc;
                __syncwarp();                     // lane 0's arrival publishes it
                if (lane == 0) {
                    const uint32_t bar = smem_u32(&bars[warp][pstage]), dst = ring0 + pstage * 2 * R::TILE;
                    mbar_arrive_expect_tx(bar, 2 * R::TILE);
                    tma_load_2d(dst, &maps.t[0], bar, 0, r);
                    tma_load_2d(dst + R::TILE, &maps.t[1], bar, 0, r);
                }
                ++used;
                pstage = pstage + 1 == R::ST ? 0 : pstage + 1;
            }
            ++pu;
            if (pu < u1) {
                const int h = prod.h, b = prod.s.b;
                prod.next(a);
                if (prod.h != h || prod.s.b != b) have = used = 0;
            }
        };
        for (int i = 0; i < R::ST; ++i) produce();

        const int G = a.Hq / a.c.Hkv;
        int stage = 0, parity = 0;
        int64_t u = u0;
        bool alive = true;
        while (u < u1 && alive) {
            // ---- a segment: one head of one sequence
            const Seq s = cons.s;
            const int h = cons.h, from = cons.i;
            const int until = (int)min((int64_t)s.units, from + (u1 - u));
            uint32_t q[KS][4];
            float qf[2];                          // score to log2 units, without the block's scale
            int rlo[2], rhi[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = g + 8 * k;
                const bool in = r < s.n * G;
                const int i = r / G, head = h * G + r % G;
                rhi[k] = in ? row_hi(i, s.n, s.L, a.causal) : 0;
                rlo[k] = in ? row_lo(i, s.n, s.L, a.window) : 0;
                uint4 w[KS / 2];
                const char* src = static_cast<const char*>(a.Q) + 2 * ((s.q0 + i) * a.ldq + (int64_t)head * D + t * (D / 4));
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) w[j] = in ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
                float f = 1.f;
                uint32_t v[KS * 2];
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) {
                    v[4 * j] = w[j].x;
                    v[4 * j + 1] = w[j].y;
                    v[4 * j + 2] = w[j].z;
                    v[4 * j + 3] = w[j].w;
                }
                if (a.xt == CQ_BF16) {
                    uint32_t mx = 0;
#pragma unroll
                    for (int j = 0; j < KS * 2; ++j) mx = max(mx, max((v[j] << 16) & 0x7FFFFFFFu, v[j] & 0x7FFF0000u));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const int sh = guard_of(__uint_as_float(mx));
                    f = pow2i(-sh);
                    const float up = pow2i(sh);
#pragma unroll
                    for (int j = 0; j < KS * 2; ++j)
                        v[j] = pack_f16(__uint_as_float(v[j] << 16) * up, __uint_as_float(v[j] & 0xFFFF0000u) * up);
                }
                qf[k] = a.scale * LOG2E * f;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    q[j][k] = v[2 * j];
                    q[j][2 + k] = v[2 * j + 1];
                }
            }
            // blocks in [free_lo, free_hi) tokens need no mask
            const int free_hi = row_hi(0, s.n, s.L, a.causal), free_lo = row_lo(s.n - 1, s.n, s.L, a.window);
            Acc<D> acc;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) acc.o[i][0] = acc.o[i][1] = acc.o[i][2] = acc.o[i][3] = 0.f;
            acc.m[0] = acc.m[1] = -INFINITY;
            acc.l[0] = acc.l[1] = 0.f;
            int ref = -64;                        // largest value-scale exponent so far

            for (int i = from; i < until && s.L > 0; ++i) {
                const uint32_t bar = smem_u32(&bars[warp][stage]);
                if (!mbar_wait_spin(bar, parity, wait_ns, &stop)) {
                    alive = false;
                    break;
                }
                const uint32_t kt = ring0 + stage * 2 * R::TILE, vt = kt + R::TILE;
                const float2 bs = scales[warp][stage];
                const int tok0 = (s.first + i) * BLK;
                float x[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const int r = 8 * nt + g;
                    uint32_t w[KS];
                    if constexpr (D == 128) {
                        const uint4 p = lds128(kt + r * 128 + (((2 * t) ^ (r & 7)) << 4));
                        const uint4 p2 = lds128(kt + r * 128 + (((2 * t + 1) ^ (r & 7)) << 4));
                        w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w;
                        w[4] = p2.x, w[5] = p2.y, w[6] = p2.z, w[7] = p2.w;
                    } else {
                        const uint4 p = lds128(kt + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
                        w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w;
                    }
                    x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        const uint32_t v = w[j] ^ 0x80808080u;
                        mma_16816_f16(x[nt], q[j], codes_f16(v, 0x4140u), codes_f16(v, 0x4342u));
                    }
                }
                // scores in log2 units; a value scale of NaN spoils them like a key scale of NaN
                const float ks = bs.y == bs.y ? bs.x : bs.y;
                const float f0 = qf[0] * ks, f1 = qf[1] * ks;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    x[nt][0] *= f0;
                    x[nt][1] *= f0;
                    x[nt][2] *= f1;
                    x[nt][3] *= f1;
                }
                if (tok0 < free_lo || tok0 + BLK > free_hi) {
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tok = tok0 + 8 * nt + 2 * t + (e & 1);
                            if (tok < rlo[e >> 1] || tok >= rhi[e >> 1]) x[nt][e] = -INFINITY;
                        }
                }
                float mx0 = acc.m[0], mx1 = acc.m[1];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    mx0 = fmaxf(mx0, fmaxf(x[nt][0], x[nt][1]));
                    mx1 = fmaxf(mx1, fmaxf(x[nt][2], x[nt][3]));
                }
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
                const int lv0 = bs.y == bs.y ? exp_of(bs.y) : ref;
                if (__any_sync(0xffffffffu, mx0 > acc.m[0] || mx1 > acc.m[1]) || lv0 > ref) {
                    const int nref = max(ref, lv0);
                    const float a0 = mx0 > acc.m[0] ? ex2(acc.m[0] - mx0) : 1.f;
                    const float a1 = mx1 > acc.m[1] ? ex2(acc.m[1] - mx1) : 1.f;
                    const float rf = pow2i(max(ref - nref, -126));
                    ref = nref;
                    acc.m[0] = mx0;
                    acc.m[1] = mx1;
                    acc.l[0] *= a0;
                    acc.l[1] *= a1;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        acc.o[n][0] *= a0 * rf;
                        acc.o[n][1] *= a0 * rf;
                        acc.o[n][2] *= a1 * rf;
                        acc.o[n][3] *= a1 * rf;
                    }
                }
                const int lv = max(lv0, ref - 64);
                const float s0 = (float)(P_EXP + lv - ref) - (acc.m[0] == -INFINITY ? 0.f : acc.m[0]);
                const float s1 = (float)(P_EXP + lv - ref) - (acc.m[1] == -INFINITY ? 0.f : acc.m[1]);
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    x[nt][0] = ex2(x[nt][0] + s0);
                    x[nt][1] = ex2(x[nt][1] + s0);
                    x[nt][2] = ex2(x[nt][2] + s1);
                    x[nt][3] = ex2(x[nt][3] + s1);
                    sum0 += x[nt][0] + x[nt][1];
                    sum1 += x[nt][2] + x[nt][3];
                }
                const float back = pow2i(ref - lv - P_EXP);
                acc.l[0] = fmaf(sum0, back, acc.l[0]);
                acc.l[1] = fmaf(sum1, back, acc.l[1]);
                uint32_t p[2][4], p2[2][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float lo = x[2 * kk + (e >> 1)][2 * (e & 1)], hi = x[2 * kk + (e >> 1)][2 * (e & 1) + 1];
                        p[kk][e] = pack_f16(lo, hi);
                        if (PT == 2) {
                            const float2 r = unpack_f16(p[kk][e]);
                            p2[kk][e] = pack_f16(lo - r.x, hi - r.y);
                        }
                    }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    // tokens 16 kk + 2 t, + 1, + 8, + 9: D/8 neighbouring channels each
                    constexpr int W = D / 32;
                    uint32_t v[4][W];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int r = 16 * kk + 2 * t + (e & 1) + 8 * (e >> 1);
                        if constexpr (D == 128) {
                            const uint4 y = lds128(vt + r * 128 + ((g ^ (r & 7)) << 4));
                            v[e][0] = y.x, v[e][1] = y.y, v[e][2] = y.z, v[e][3] = y.w;
                        } else {
                            const uint2 y = lds64(vt + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
                            v[e][0] = y.x, v[e][1] = y.y;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e][j] ^= 0x80808080u;
                        const uint32_t a01 = prmt(v[0][j], v[1][j], 0x5140u), a23 = prmt(v[0][j], v[1][j], 0x7362u);
                        const uint32_t b01 = prmt(v[2][j], v[3][j], 0x5140u), b23 = prmt(v[2][j], v[3][j], 0x7362u);
                        const uint32_t b[4][2] = {{codes_f16(a01, 0x4140u), codes_f16(b01, 0x4140u)},
                                                  {codes_f16(a01, 0x4342u), codes_f16(b01, 0x4342u)},
                                                  {codes_f16(a23, 0x4140u), codes_f16(b23, 0x4140u)},
                                                  {codes_f16(a23, 0x4342u), codes_f16(b23, 0x4342u)}};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            mma_16816_f16(acc.o[4 * j + e], p[kk], b[e][0], b[e][1]);
                            if (PT == 2) mma_16816_f16(acc.o[4 * j + e], p2[kk], b[e][0], b[e][1]);
                        }
                    }
                }
                __syncwarp();                     // the stage is free
                stage = stage + 1 == R::ST ? 0 : stage + 1;
                parity ^= stage == 0;
                produce();
            }
            if (s.L == 0) produce();
            if (!alive) break;
            // ---- the segment's end, or the share's
            u += until - from;
            const float un = pow2i(ref - P_EXP);
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.o[n][e] *= un;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                acc.l[k] += __shfl_xor_sync(0xffffffffu, acc.l[k], 1);
                acc.l[k] += __shfl_xor_sync(0xffffffffu, acc.l[k], 2);
            }
            if (from == 0 && until == s.units) {
                write_out<D>(a, acc, s, h);
            } else {
                const int slot = from == 0 ? 1 : 0;   // began here and goes on, or began earlier
                write_part<D>(&sp->warp[blockIdx.x * NW + warp][slot], acc, s.n * G);
                if (lane == 0) wseg[warp][slot] = s.b * a.c.Hkv + h;
            }
            cons.i = until - 1;
            if (u < u1) cons.next(a);
        }
        if (!alive) {
            // a copy did not come in time: tell the CTA, wait (with the limit) for what is still on its way
            if (lane == 0) {
                atomicExch(&stop, 1);
                set_err(a.b.err, DEV_TIMEOUT);
            }
            const volatile int never = 0;
            for (int i = 0; i < R::ST; ++i) {
                mbar_wait(smem_u32(&bars[warp][stage]), parity, wait_ns, &never);
                stage = stage + 1 == R::ST ? 0 : stage + 1;
                parity ^= stage == 0;
            }
        }
    }
    __syncthreads();
    // ---- the CTA's partials, in order: runs of one segment are joined
    if (threadIdx.x == 0) sp->seg[blockIdx.x][0] = sp->seg[blockIdx.x][1] = -1;
    if (stop || !busy) return;
    for (int i = 0; i < 2 * NW;) {
        const int seg = wseg[i >> 1][i & 1];
        if (seg < 0) {
            ++i;
            continue;
        }
        int e = i, cnt = 0;
        for (; e < 2 * NW && (wseg[e >> 1][e & 1] == seg || wseg[e >> 1][e & 1] < 0); ++e) cnt += wseg[e >> 1][e & 1] == seg;
        const Seq s = seq_of(a, seg / a.c.Hkv);
        const int h = seg % a.c.Hkv;
        // the segment's first unit is here iff its first partial began its segment
        const bool begins = (i & 1) == 1;
        bool ends = true;                 // its last unit is here iff the next unit of the CTA is another segment's
        if (e == 2 * NW && c1 < total) {
            Cursor c;
            seek(c1, c);
            ends = c.i == 0;
        }
        auto part = [&](int j) {
            for (int k = i; k < e; ++k)
                if (wseg[k >> 1][k & 1] == seg && j-- == 0) return (const Part<D>*)&sp->warp[blockIdx.x * NW + (k >> 1)][k & 1];
            return (const Part<D>*)nullptr;
        };
        Part<D>* out = begins && ends ? nullptr : &sp->cta[blockIdx.x][begins ? 1 : 0];
        join<D>(a, s, h, cnt, part, out);
        if (out && threadIdx.x == 0) sp->seg[blockIdx.x][begins ? 1 : 0] = seg;
        i = e;
    }
}

// Joins the segments that lie across CTAs: CTA i takes the one that began in share i.
template <int D>
__global__ void __launch_bounds__(NW * 32) k_attn_join(const AttnArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const Space<D>* sp = static_cast<const Space<D>*>(a.ws);
    const int i = blockIdx.x, seg = __ldcg(&sp->seg[i][1]);
    if (seg < 0) return;
    int cnt = 1;
    while (i + cnt < (int)gridDim.x && __ldcg(&sp->seg[i + cnt][0]) == seg) ++cnt;
    const Seq s = seq_of(a, seg / a.c.Hkv);
    join<D>(a, s, seg % a.c.Hkv, cnt, [&](int j) { return j == 0 ? &sp->cta[i][1] : &sp->cta[i + j][0]; }, nullptr);
}

template <int D, int PT>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    Maps maps;
    const uint64_t dims[2] = {(uint64_t)D, (uint64_t)a.c.pages * a.c.Hkv * a.c.page}, strides[1] = {(uint64_t)D};
    const uint32_t box[2] = {(uint32_t)D, (uint32_t)BLK};
    for (int i = 0; i < 2; ++i)
        if (!encode_tiled(&maps.t[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.c.q[i], dims, strides, box,
                          D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    constexpr size_t smem = Ring<D>::BYTES + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, PT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)std::min(num_sms(), MAX_CTAS);
    e = launch_pdl(k_attn_decode<D, PT>, dim3(ctas), dim3(NW * 32), smem, s, maps, a, (uint64_t)options().wait_ns.load());
    if (e != cudaSuccess) return e;
    return launch_pdl(k_attn_join<D>, dim3(ctas), dim3(NW * 32), 0, s, a);
}

}  // namespace

bool decode_serves(int64_t rows) { return rows <= ROWS; }
size_t decode_workspace(int64_t D) { return D == 128 ? sizeof(Space<128>) : sizeof(Space<64>); }

cudaError_t launch_decode(const AttnArgs& a, cudaStream_t s) {
    if (a.D == 128) return a.yt == CQ_F32 ? run<128, 2>(a, s) : run<128, 1>(a, s);
    return a.yt == CQ_F32 ? run<64, 2>(a, s) : run<64, 1>(a, s);
}

}  // namespace kv8
}  // namespace cq

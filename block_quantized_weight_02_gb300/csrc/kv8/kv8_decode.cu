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
// One block: S^T = K Q^T as m16n8k16 products (tokens x rows), the running maximum and
// sum in f32 registers, then O^T += V^T P^T; an 8 x 8 transpose in registers turns the
// score fragments into the second operand.  With the rows as the narrow side a group of
// up to 8 rows takes half the products that rows x tokens would (they pad rows to 16).
// For f32 outputs a weight goes in two fp16 terms.
//
// Measured, calls in a chain: 4 rows of 8 heads of 128 channels, 32 sequences of 1000 to 32767 tokens, 178 us, 6.1 TB/s
// (the shares are equal, but a third of the SMs draw 10 % less from memory and end last).  16 rows over 3 x 110000 tokens,
// 4 heads: 86 us with f16 outputs, 3.9 TB/s, 106 with f32, bound by instructions (conversions, products, exponentials).
// One row of 16 heads of 64 channels behind a window of 1024 tokens, 48 sequences: 38 us, 2.4 TB/s (35 out of a graph), of
// which the list and the first load take 6 and the joins 8.  8 rows of 4 heads of one sequence of 777 tokens: 14 us of
// latency.
// The codes become fp16 in registers, exactly.  The operands' inner order is free as long
// as both sides agree: a lane takes 4 neighbouring codes of its token as one k16 step's
// part (keys), and D/8 neighbouring channels of its tokens as the output tiles (values),
// so every shared-memory load is 16 bytes (values at D = 64: 8), without bank conflicts
// under the copies' swizzle.
//
// A key block's scale multiplies the scores in f32.  A value block's scale 2^lv joins the
// exponent, w = 2^(s + lv - m + 15) with m the row's largest s + lv, so the weights fill
// fp16's range (11 bits down to 2^-29 of the largest) whatever the scales are; the
// normaliser takes w 2^-lv.
//
// Shares that do not hold a whole (sequence, head) leave (O, m, l) partials; the CTA's own
// are joined after a barrier, those across CTAs by a second small kernel, always in share
// order, so results do not depend on timing.
#include "attn_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int ROWS = 16;
constexpr int MAX_CTAS = 160;         // workspace bound: a full GB300 has no more SMs
constexpr int MAX_NW = 12;
constexpr int P_EXP = 15;             // weights carry 2^15
// One-term weights' products add up in the tensor cores, which truncate (up to 3e-9 of the sum a token): after so many blocks
// of a segment the accumulators go to a sum in the workspace, 5e-5 at most.  Sequences without room for more take the kernel
// without (WIN false): a 1024-token window over 48 sequences 38.4 us against 39.5.
constexpr int WINDOW = 512;

struct Maps {
    CUtensorMap t[2];                 // keys, values: {D, pages * Hkv * page}, box {D, 32}
};

template <int D>
using Part = PartOf<D, ROWS>;
// Workspace: partials of segments that end inside a warp's share, sums, partials of the CTAs, the CTAs' two segments.
template <int D>
struct Space {
    Part<D> warp[MAX_CTAS * MAX_NW];
    Part<D> sum[MAX_CTAS * MAX_NW];   // of a warp's earlier windows
    Part<D> cta[MAX_CTAS][2];
    int seg[MAX_CTAS][2];             // segment of cta[i][0] (began earlier) and cta[i][1] (began here, goes on), or -1
};

// NT: n8 tiles of rows.  One tile's registers allow 12 warps, with two blocks each; two allow 8, with three.
template <int D, int NT>
struct Ring {
    static constexpr int NW = NT == 1 ? 12 : 8;
    static constexpr int ST = (NT == 2 ? 3 : 2) * (128 / D);   // blocks in the ring of a warp: 192 KB a CTA
    static constexpr int TILE = BLK * D;                       // bytes of a block's keys or values
    static constexpr int WARP = ST * 2 * TILE;
    static constexpr int BYTES = NW * WARP;
    static_assert(WARP >= NT * 8 * D * 4 + 2 * ROWS * 4 && NW <= MAX_NW, "a partial fits a warp's memory");
    static_assert(WARP % 1024 == 0, "alignment of swizzled copies");
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

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 4 bytes to shared memory; `bar` gets this thread's arrival when they are there.
__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src, uint32_t bar) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n\tcp.async.mbarrier.arrive.noinc.shared::cta.b64 [%2];"
                 ::"r"(dst), "l"(src), "r"(bar) : "memory");
}

// The result of a warp: lane (g, t) holds rows 8 n + 2 t, + 1 and channels g D/8 .. + D/8 - 1.
template <int D, int NT>
struct Acc {
    static constexpr int DL = D / 8;   // channels of a lane
    float o[NT][D / 16][4];            // tile i: channel 2 i of rows 2 t, 2 t + 1, channel 2 i + 1 of the same
    float m[NT][2], l[NT][2];
    __device__ __forceinline__ float ch(int n, int k, int c) const { return o[n][c / 2][2 * (c & 1) + k]; }
};

template <int D, int NT>
__device__ __forceinline__ void write_part(Part<D>* p, const Acc<D, NT>& c, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 8 * n + 2 * t + k;
            if (r >= rows) continue;
            float4* o = reinterpret_cast<float4*>(&p->o[r][g * Acc<D, NT>::DL]);
#pragma unroll
            for (int i = 0; i < Acc<D, NT>::DL / 4; ++i)
                o[i] = make_float4(c.ch(n, k, 4 * i), c.ch(n, k, 4 * i + 1), c.ch(n, k, 4 * i + 2), c.ch(n, k, 4 * i + 3));
            if (g == 0) {
                p->m[r] = c.m[n][k];
                p->l[r] = c.l[n][k];
            }
        }
}

// The accumulators join the sum of the segment's windows so far (none: first), and start afresh.
template <int D, int NT>
__device__ __forceinline__ void write_sum(Part<D>* p, Acc<D, NT>& c, int rows, bool first) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 8 * n + 2 * t + k;
            const float keep = first || r >= rows ? 0.f : since(p->m[r], c.m[n][k]);
            float4* o = reinterpret_cast<float4*>(&p->o[r][g * Acc<D, NT>::DL]);
#pragma unroll
            for (int i = 0; i < Acc<D, NT>::DL / 4; ++i) {
                const float4 z = first || r >= rows ? make_float4(0.f, 0.f, 0.f, 0.f) : o[i];
                if (r < rows)
                    o[i] = make_float4(fmaf(z.x, keep, c.ch(n, k, 4 * i)), fmaf(z.y, keep, c.ch(n, k, 4 * i + 1)),
                                       fmaf(z.z, keep, c.ch(n, k, 4 * i + 2)), fmaf(z.w, keep, c.ch(n, k, 4 * i + 3)));
            }
        }
    __syncwarp();                      // all have read the old maxima
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (g == 0 && 8 * n + 2 * t + k < rows) p->m[8 * n + 2 * t + k] = c.m[n][k];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) c.o[n][i][k] = c.o[n][i][2 + k] = 0.f;
        }
    __syncwarp();
}
// The sum comes back to the accumulators.
template <int D, int NT>
__device__ __forceinline__ void read_sum(const Part<D>* p, Acc<D, NT>& c, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 8 * n + 2 * t + k;
            if (r >= rows) continue;
            const float keep = since(p->m[r], c.m[n][k]);
#pragma unroll
            for (int i = 0; i < Acc<D, NT>::DL / 4; ++i) {
                const float4 z = *reinterpret_cast<const float4*>(&p->o[r][g * Acc<D, NT>::DL + 4 * i]);
                c.o[n][2 * i][k] = fmaf(z.x, keep, c.o[n][2 * i][k]);
                c.o[n][2 * i][2 + k] = fmaf(z.y, keep, c.o[n][2 * i][2 + k]);
                c.o[n][2 * i + 1][k] = fmaf(z.z, keep, c.o[n][2 * i + 1][k]);
                c.o[n][2 * i + 1][2 + k] = fmaf(z.w, keep, c.o[n][2 * i + 1][2 + k]);
            }
        }
}

template <int D, int NT>
__device__ __forceinline__ void write_out(const AttnArgs& a, const Acc<D, NT>& c, const Seq& s, int h) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, G = a.Hq / a.c.Hkv, first = first_seeing(a, s.n, s.L);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 8 * n + 2 * t + k;
            if (r >= s.n * G) continue;
            const int row = s.q0 + r / G, head = h * G + r % G;
            const float l = row_sum(c.l[n][k], r, first), f = inv_sum(l);
            const int64_t at = row * a.ldo + (int64_t)head * D + g * Acc<D, NT>::DL;
#pragma unroll
            for (int i = 0; i < Acc<D, NT>::DL / 4; ++i)
                store_out4(a.O, at + 4 * i, a.yt, c.ch(n, k, 4 * i) * f, c.ch(n, k, 4 * i + 1) * f,
                           c.ch(n, k, 4 * i + 2) * f, c.ch(n, k, 4 * i + 3) * f);
            if (a.lse && g == 0) a.lse[(int64_t)row * a.Hq + head] = lse_of(c.m[n][k], l);
        }
}

// PT: fp16 terms that carry a weight (one for 16-bit outputs, two for f32).
template <int D, int NT, int PT, bool WIN>
__global__ void __launch_bounds__(Ring<D, NT>::NW * 32, 1) k_attn_decode(const __grid_constant__ Maps maps,
                                                                         const AttnArgs a, uint64_t wait_ns) {
    using R = Ring<D, NT>;
    constexpr int NW = R::NW, KS = D / 16;   // k16 steps of a score
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[NW][R::ST];
    __shared__ float2 scales[NW][R::ST]; // the staged blocks' key scale and value scale
    __shared__ int64_t pre[NW * 32 + 1]; // units before each thread's sequences
    __shared__ int64_t wsum[NW];
    __shared__ int wseg[NW * 2];         // segment of each warp's two partials, or -1
    __shared__ bool wfrom[NW * 2];       // that partial has its segment's first unit
    __shared__ bool wend[NW * 2];        // and its last
    __shared__ uint32_t runs[NW * 2];    // the CTA's runs of partials of one segment
    __shared__ int nruns;
    __shared__ int stop;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t ring0 = smem_u32(ring) + warp * R::WARP;
    // a warp's partial of the segment that its share ends in goes to its ring, which is done by then
    auto last_part = [&](int w) { return reinterpret_cast<Part<D>*>(ring + w * R::WARP); };
    Space<D>* sp = static_cast<Space<D>*>(a.ws);
    if (lane == 0)
        for (int i = 0; i < R::ST; ++i) mbar_init(smem_u32(&bars[warp][i]), 3);   // the copies' bytes, two scales
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
        if (!rows_ok(qs, qe, a.b.T, a.max_q) || !length_ok(a.c, L)) bad = true;
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
    const int64_t c0 = blockIdx.x < ctas ? total * blockIdx.x / ctas : 0;
    const int64_t c1 = blockIdx.x < ctas ? total * (blockIdx.x + 1) / ctas : 0;
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

    if (lane < 2) wseg[warp * 2 + lane] = -1;
    if (u0 < u1) {
        Cursor cons, prod;
        seek(u0, cons);
        prod = cons;
        int64_t pu = u0;                         // next unit to load
        int pstage = 0;
        // 32 blocks' places in the pools at a time, one per lane
        int have = 0, used = 0, row = 0;

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
                    }
                }
                const int r = __shfl_sync(0xffffffffu, row, used);
                const uint32_t bar = smem_u32(&bars[warp][pstage]);
                if (lane < 2 && !a.stall) copy4_async(smem_u32(&scales[warp][pstage]) + 4 * lane, a.c.s[lane] + r / BLK, bar);
                if (lane == 0 && !a.stall) {
                    const uint32_t dst = ring0 + pstage * 2 * R::TILE;
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
            uint32_t q[NT][KS][2];
            float qf[NT][2];                      // score to log2 units, without the block's scale
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = 8 * n + g;          // this lane holds row r of Q
                const bool in = r < s.n * G;
                const char* src = static_cast<const char*>(a.Q) +
                                  2 * ((s.q0 + r / G) * a.ldq + (int64_t)(h * G + r % G) * D + t * (D / 4));
                uint4 w[KS / 2];
#pragma unroll
                for (int j = 0; j < KS / 2; ++j) w[j] = in ? __ldcg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
                float f = a.scale * LOG2E;
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
                    f *= pow2i(-sh);
                    const float up = pow2i(sh);
#pragma unroll
                    for (int j = 0; j < KS * 2; ++j)
                        v[j] = pack_f16(__uint_as_float(v[j] << 16) * up, __uint_as_float(v[j] & 0xFFFF0000u) * up);
                }
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    q[n][j][0] = v[2 * j];
                    q[n][j][1] = v[2 * j + 1];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)       // and its scores and outputs are of rows 2 t, 2 t + 1
                    qf[n][k] = __shfl_sync(0xffffffffu, f, (2 * t + k) * 4);
            }
            // blocks in [free_lo, free_hi) tokens need no mask
            const int free_hi = row_hi(0, s.n, s.L, a.causal), free_lo = row_lo(s.n - 1, s.n, s.L, a.window);
            Acc<D, NT> acc;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) acc.o[n][i][0] = acc.o[n][i][1] = acc.o[n][i][2] = acc.o[n][i][3] = 0.f;
                acc.m[n][0] = acc.m[n][1] = -INFINITY;
                acc.l[n][0] = acc.l[n][1] = 0.f;
            }
            int hi = -64;                         // largest value exponent so far, seen or not

            // in windows (two-term weights' products are added outside the tensor cores: in one)
            Part<D>* sum = &sp->sum[blockIdx.x * NW + warp];
            for (int i0 = from, end; i0 < until && s.L > 0 && alive; i0 = end) {
                end = WIN ? min(until, i0 + WINDOW) : until;
                if (WIN && i0 > from) write_sum<D, NT>(sum, acc, s.n * G, i0 == from + WINDOW);
                for (int i = i0; i < end; ++i) {
                    // one answer for the warp, as what follows takes all its lanes: it joins the vote on the maxima, and
                    // what is computed until then from a block that did not come is dropped
                    const bool here = wait_bar(smem_u32(&bars[warp][stage]), parity, wait_ns, &stop);
                    const uint32_t kt = ring0 + stage * 2 * R::TILE, vt = kt + R::TILE;
                    const float2 bs = scales[warp][stage];
                    const int tok0 = (s.first + i) * BLK;
                    float x[NT][2][4];                // tokens 16 mt + g (rows 2 t, 2 t + 1), + 8 (the same)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) x[n][mt][0] = x[n][mt][1] = x[n][mt][2] = x[n][mt][3] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            uint4 w[2];               // tokens 16 mt + g, + 8: four k16 steps
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int r = 16 * mt + 8 * e + g;
                                w[e] = lds128(D == 128 ? kt + r * 128 + (((2 * t + c) ^ (r & 7)) << 4) : kt + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
                            }
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                uint32_t ka[2][4];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const uint32_t y0 = (jj ? (j ? w[0].w : w[0].z) : (j ? w[0].y : w[0].x)) ^ 0x80808080u;
                                    const uint32_t y1 = (jj ? (j ? w[1].w : w[1].z) : (j ? w[1].y : w[1].x)) ^ 0x80808080u;
                                    ka[j][0] = codes_f16(y0, 0x4140u);
                                    ka[j][1] = codes_f16(y1, 0x4140u);
                                    ka[j][2] = codes_f16(y0, 0x4342u);
                                    ka[j][3] = codes_f16(y1, 0x4342u);
                                }
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    const int j0 = 4 * c + 2 * jj;
                                    mma_16816_f16(x[n][mt], ka[0], q[n][j0][0], q[n][j0][1]);
                                    mma_16816_f16(x[n][mt], ka[1], q[n][j0 + 1][0], q[n][j0 + 1][1]);
                                }
                            }
                        }
                    // z = score in log2 units + value exponent; a value scale of NaN spoils it like a key scale of NaN
                    const float ks = bs.y == bs.y ? bs.x : bs.y;
                    const int lv = value_exp(bs.y);
                    hi = max(hi, lv);
                    const bool masked = tok0 < free_lo || tok0 + BLK > free_hi;
                    float mx[NT][2];
                    bool grows = !here;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float f = qf[n][k] * ks;
                            float m = acc.m[n][k];
                            int lo = 0, hi = 0;
                            if (masked) {
                                const int rr = 8 * n + 2 * t + k, row = rr / G;
                                hi = rr < s.n * G ? row_hi(row, s.n, s.L, a.causal) : 0;
                                lo = row_lo(row, s.n, s.L, a.window);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float& y = x[n][e >> 1][2 * (e & 1) + k];
                                y = fmaf(y, f, (float)lv);
                                if (masked) {
                                    const int tok = tok0 + 8 * e + g;
                                    if (tok < lo || tok >= hi) y = -INFINITY;
                                }
                                m = fmaxf(m, y);
                            }
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            mx[n][k] = m;
                            grows |= m > acc.m[n][k];
                        }
                    if (__any_sync(0xffffffffu, grows)) {
                        if (!__all_sync(0xffffffffu, here)) {
                            alive = false;
                            break;
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float root = mx[n][k] > acc.m[n][k] ? root_of(acc.m[n][k] - mx[n][k]) : 1.f, f = root * root;
                                acc.m[n][k] = mx[n][k];
                                acc.l[n][k] = acc.l[n][k] * root * root;
#pragma unroll
                                for (int i2 = 0; i2 < D / 16; ++i2) {
                                    acc.o[n][i2][k] *= f;
                                    acc.o[n][i2][2 + k] *= f;
                                }
                            }
                    }
                    const bool far = lv < hi - APART;
                    const float back = far ? 0.f : pow2i(-lv);
                    if (far)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc.l[n][k] += ex2((x[n][e >> 1][2 * (e & 1) + k] - (acc.m[n][k] == -INFINITY ? 0.f : acc.m[n][k])) + (float)(P_EXP - lv));
                    uint32_t p[NT][PT][4];            // weights of tokens 8 e + 2 t, + 1, row g
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float m0 = acc.m[n][k] == -INFINITY ? 0.f : acc.m[n][k];
                            float sum = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float& y = x[n][e >> 1][2 * (e & 1) + k];
                                y = ex2((y - m0) + (float)P_EXP);      // (beside a huge m0 the exponent would be rounded away)
                                sum += y;
                            }
                            acc.l[n][k] = fmaf(sum, back, acc.l[n][k]);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float y0 = x[n][e >> 1][2 * (e & 1)], y1 = x[n][e >> 1][2 * (e & 1) + 1];
                            const uint32_t hi = pack_f16(y0, y1);
                            p[n][0][e] = transpose8(hi);
                            if (PT == 2) {
                                const float2 r = unpack_f16(hi);
                                p[n][PT - 1][e] = transpose8(pack_f16(y0 - r.x, y1 - r.y));
                            }
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
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t sel = e ? 0x7362u : 0x5140u;
                                const uint32_t ya = prmt(v[0][j], v[1][j], sel), yb = prmt(v[2][j], v[3][j], sel);
                                const uint32_t va[4] = {codes_f16(ya, 0x4140u), codes_f16(ya, 0x4342u), codes_f16(yb, 0x4140u), codes_f16(yb, 0x4342u)};
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    float(&o)[4] = acc.o[n][2 * j + e];
                                    if (PT == 1) {
                                        mma_16816_f16(o, va, p[n][0][2 * kk], p[n][0][2 * kk + 1]);
                                    } else {          // the products truncate what they add up: long sums are added here
                                        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                        for (int z = 0; z < PT; ++z) mma_16816_f16(y, va, p[n][z][2 * kk], p[n][z][2 * kk + 1]);
#pragma unroll
                                        for (int i = 0; i < 4; ++i) o[i] += y[i];
                                    }
                                }
                            }
                        }
                    }
                    __syncwarp();                     // the stage is free
                    stage = stage + 1 == R::ST ? 0 : stage + 1;
                    parity ^= stage == 0;
                    produce();
                }
            }
            if (s.L == 0) produce();
            if (!alive) break;
            if (WIN && until - from > WINDOW && s.L > 0) read_sum<D, NT>(sum, acc, s.n * G);
            // ---- the segment's end, or the share's
            u += until - from;
            const float un = pow2i(-P_EXP);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc.o[n][i][e] *= un;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    acc.l[n][k] += __shfl_xor_sync(0xffffffffu, acc.l[n][k], 4);
                    acc.l[n][k] += __shfl_xor_sync(0xffffffffu, acc.l[n][k], 8);
                    acc.l[n][k] += __shfl_xor_sync(0xffffffffu, acc.l[n][k], 16);
                    acc.l[n][k] *= un;
                }
            }
            if (from == 0 && until == s.units) {
                write_out<D, NT>(a, acc, s, h);
            } else {
                const int slot = u == u1 ? 1 : 0;     // the share's last segment, or one that began before it
                write_part<D, NT>(slot ? last_part(warp) : &sp->warp[blockIdx.x * NW + warp], acc, s.n * G);
                if (lane == 0) {
                    wseg[warp * 2 + slot] = s.b * a.c.Hkv + h;
                    wend[warp * 2 + slot] = until == s.units;
                    wfrom[warp * 2 + slot] = from == 0;
                }
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
                wait_bar(smem_u32(&bars[warp][stage]), parity, wait_ns, &never);
                stage = stage + 1 == R::ST ? 0 : stage + 1;
                parity ^= stage == 0;
            }
        }
    }
    __syncthreads();
    // ---- the CTA's partials, in order: runs of one segment are joined, all at once
    if (warp == 0) {
        const int seg = lane < 2 * NW ? wseg[lane] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, seg);
        const bool first = seg >= 0 && (same & ((1u << lane) - 1)) == 0;
        const uint32_t firsts = __ballot_sync(0xffffffffu, first);
        if (first) runs[__popc(firsts & ((1u << lane) - 1))] = same;
        if (lane == 0) {
            nruns = __popc(firsts);
            sp->seg[blockIdx.x][0] = sp->seg[blockIdx.x][1] = -1;
        }
    }
    __syncthreads();
    if (stop) return;
    const int quads = a.max_q * (a.Hq / a.c.Hkv) * (D / 4);    // of a run, at most
    for (int k = threadIdx.x; k < nruns * quads; k += NW * 32) {
        const uint32_t run = runs[k / quads];
        const int i = __ffs(run) - 1, seg = wseg[i], h = seg % a.c.Hkv;
        const Seq s = seq_of(a, seg / a.c.Hkv);
        const int r = k % quads / (D / 4), d = k % (D / 4) * 4;
        if (r >= s.n * (a.Hq / a.c.Hkv)) continue;
        const bool begins = wfrom[i], ends = wend[31 - __clz(run)];
        uint32_t left = run;
        auto part = [&](int) {               // called in order
            const int w = __ffs(left) - 1;
            left &= left - 1;
            return (const Part<D>*)(w & 1 ? last_part(w >> 1) : &sp->warp[blockIdx.x * NW + (w >> 1)]);
        };
        join<false, D, 1, 8>(a, s.q0, first_seeing(a, s.n, s.L), h, r, r, d, __popc(run), part, begins && ends ? nullptr : &sp->cta[blockIdx.x][begins ? 1 : 0]);
        if (!(begins && ends) && r == 0 && d == 0) sp->seg[blockIdx.x][begins ? 1 : 0] = seg;
    }
}

// Joins the segments that lie across CTAs: the CTAs (i, .) take the one that began in share i, four channels a thread.
constexpr int JOIN_THREADS = 128;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) k_attn_join(const AttnArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const Space<D>* sp = static_cast<const Space<D>*>(a.ws);
    const int i = blockIdx.x, lane = threadIdx.x & 31, seg = __ldcg(&sp->seg[i][1]);
    int cnt = 1;
    while (true) {                     // the shares after it that go on with the segment
        const int j = i + cnt + lane;
        const bool more = j < (int)gridDim.x && __ldcg(&sp->seg[j][0]) == seg;
        const int k = __ffs(~__ballot_sync(0xffffffffu, more));
        cnt += k ? k - 1 : 32;
        if (k) break;
    }
    if (seg < 0) return;
    const Seq s = seq_of(a, seg / a.c.Hkv);
    const int k = blockIdx.y * JOIN_THREADS + threadIdx.x, r = k / (D / 4);
    if (r < s.n * (a.Hq / a.c.Hkv))
        join<true, D, 1, 8>(a, s.q0, first_seeing(a, s.n, s.L), seg % a.c.Hkv, r, r, k % (D / 4) * 4, cnt,
                            [&](int j) { return j == 0 ? &sp->cta[i][1] : &sp->cta[i + j][0]; }, (Part<D>*)nullptr);
}

template <int D, int NT, int PT, bool WIN>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    using R = Ring<D, NT>;
    Maps maps;
    const uint64_t dims[2] = {(uint64_t)D, (uint64_t)a.c.pages * a.c.Hkv * a.c.page}, strides[1] = {(uint64_t)D};
    const uint32_t box[2] = {(uint32_t)D, (uint32_t)BLK};
    for (int i = 0; i < 2; ++i)
        if (!encode_tiled(&maps.t[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.c.q[i], dims, strides, box,
                          D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    constexpr size_t smem = R::BYTES + 1024;
    cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, NT, PT, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)std::min(num_sms(), MAX_CTAS);
    e = launch_pdl(k_attn_decode<D, NT, PT, WIN>, dim3(ctas), dim3(R::NW * 32), smem, s, maps, a, (uint64_t)options().wait_ns.load());
    if (e != cudaSuccess) return e;
    return launch_pdl(k_attn_join<D>, dim3(ctas, NT * 8 * (D / 4) / JOIN_THREADS), dim3(JOIN_THREADS), 0, s, a);
}

template <int D, int NT>
cudaError_t run_as(const AttnArgs& a, cudaStream_t s) {
    if (a.yt == CQ_F32) return run<D, NT, 2, false>(a, s);
    return a.c.ldt * a.c.page > WINDOW * BLK ? run<D, NT, 1, true>(a, s) : run<D, NT, 1, false>(a, s);
}
template <int D>
cudaError_t run_d(const AttnArgs& a, cudaStream_t s) {
    return a.max_q * (a.Hq / a.c.Hkv) <= 8 ? run_as<D, 1>(a, s) : run_as<D, 2>(a, s);
}

}  // namespace

bool decode_serves(int64_t rows) { return rows <= ROWS; }
size_t decode_workspace(int64_t D) { return D == 128 ? sizeof(Space<128>) : sizeof(Space<64>); }

cudaError_t launch_decode(const AttnArgs& a, cudaStream_t s) { return a.D == 128 ? run_d<128>(a, s) : run_d<64>(a, s); }

}  // namespace kv8
}  // namespace cq

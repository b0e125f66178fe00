// Attention over the 8-bit cache for many query rows: 128-row x 128-token tiles on the
// 5th-generation tensor cores.
//
// A row is a (token, head of the group) pair, so the heads that share a KV head share its
// tiles.  Per 128 tokens (a step) and tile S = Q K^T (Q and K in shared memory, S in tensor
// memory) and O += P V (P in tensor memory over S, V in shared memory token-major).  A CTA
// keeps two tiles going, so that the tensor cores have one while the other's softmax runs:
// two row tiles (TILES 2, items of 256 rows), or, where no sequence has more than 128 rows,
// the even and the odd steps of one row tile (TILES 1), whose two results are joined at the end.
//   warps 0, 2      issue the products of the two tiles (an elected lane each: a wait or a commit costs
//                   about 100 cycles, which the other's products cover), in turns: left to
//                   themselves the tiles fall into step, and both softmaxes run while no products do
//   warp 1          TMA loads of the codes by page, 32 tokens a box, and their scales
//   warps 4-7, 8-11 softmax of the two tiles, one row a thread; queries in, outputs out
//   warps 12-15     codes -> fp16 (exactly), into the 128-byte-swizzled operand tiles
// A key block's scale joins the scores in f32, a value block's scale 2^lv the exponent:
// w = 2^(s + lv - m + 10), with m at most 5 below the row's largest s + lv (O is only rescaled
// when that has grown by more); the normaliser takes w 2^-lv.  For f32 outputs P goes in two
// fp16 terms, two products each.
//
// The work is the list of all (row tile, KV head, step), cut into one equal share per SM.  A
// first small kernel lays the list out (only the device knows the lengths), a third joins the
// row tiles that lie across shares, in share order.
//
// TREE: in steps that reach a sequence's last tokens a row's mask words, shifted to the step's tokens, tell what it sees.
//
// Measured, 128 channels, bf16 outputs: a 16384-token prompt of 32 heads over 8 KV heads 1803 us, 1220 TFLOP/s; prompts
// of up to 2000 tokens behind up to 3000 260 us, 876; 2 x 1024 rows against 4500 to 5100 tokens, 24 heads, 136 us, 889.  f32
// outputs: the ragged prompts 435 us; 64 channels: 217.  80 rows of 8 heads over 300 to 9000 tokens (TILES 1): 110 us; 26 rows
// of 4 heads of a group of 32 trees (TILES 1 with a mask) over 1000 to 16000 tokens 180 us, 3.2 TB/s.  A step of two tiles takes 1.85 us where its products alone would take 1.1: a tile's
// products wait for its exponentials (four cycles a warp and scheduler each) and each hand-over between the two costs a few
// hundred cycles, which the other tile covers only in part.
#pragma once
#include "tiles_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int MMA_WARP = 0, LOAD_WARP = 1, MMA_WARP2 = 2, SOFT_WARP = 4, CONV_WARP = 12;
constexpr int THREADS = 512;           // four warpgroups of 128 registers a thread at launch
constexpr int REGS_SOFTMAX = 200, REGS_CONV = 56, REGS_ISSUE = 56;
static_assert(2 * REGS_SOFTMAX + REGS_CONV + REGS_ISSUE <= 4 * 128, "what the launch has");

// An unfinished result, channels in fours with the rows side by side, as the threads hold them.
template <int D, int TILES>
struct Part {
    float4 o[D / 4][TILES * TM];
    float m[TILES * TM], l[TILES * TM];
    __device__ __forceinline__ const float4* quad(int r, int d) const { return &o[d / 4][r]; }
};
// Workspace: partials, then the list.
template <int D, int TILES>
struct Space {
    Part<D, TILES> cta[MAX_CTAS][2];
    Part<D, TILES> odd[TILES == 1 ? MAX_CTAS : 1];   // TILES 1: the odd steps' result
    List list;
};

// ---- shared memory -------------------------------------------------------------------------------------------------
template <int D, int TILES>
struct Smem {
    static constexpr int RS = TILES == 1 ? 4 : 2; // code tiles in the ring (keys and values alternate)
    static constexpr int QT = TM * D * 2;         // a query tile: D/64 chunks of [128 rows][128 B], swizzled
    static constexpr int HT = TN * D * 2;         // an fp16 operand tile, the same
    static constexpr int RT = TN * D;             // codes
    static constexpr int Q = 0, H = TILES * QT, R = H + HS * HT, MISC = R + RS * RT;
    static constexpr int NBAR = 2 * RS + 2 * HS + SS + 13;
    static constexpr int SC = (MISC + NBAR * 8 + 15) / 16 * 16;   // Block [SS][NB]
    static constexpr int END = SC + SS * NB * (int)sizeof(Block) + 16;
};

// Two weights join the sum and become one (or two) fp16 terms.
template <int PT>
__device__ __forceinline__ void weights(float y0, float y1, uint64_t& sum, uint32_t& p, uint32_t& p2) {
    sum = add2(sum, pair(y0, y1));
    p = pack_f16(y0, y1);
    if (PT == 2) {
        const float2 h = unpack_f16(p);
        p2 = pack_f16(y0 - h.x, y1 - h.y);
    }
}
// TREE: with a mask.
// AHEAD: codes a tile ahead in the converters' registers, which shortens a step and lengthens an item's begin.  Trees of one row
// tile (140 shapes of 1 to 48 sequences, 500 to 40000 tokens, both sides): 64 channels 0 to 8 % faster, 128 with f32
// outputs 0 to 4 %, with fp16 ones 3 % slower (32 trees of up to 2000 tokens, 57.5 us to 59.1) to 10 % faster (up to 40000, 403 to 361),
// with bf16 ones 4 % slower (5000, 106 to 111; 12000, 75.1 to 78.3) to 9 % faster (40000, 438 to 397).  Without a mask 80 rows over 300 to 9000 tokens take
// 115 us so and 110 without, two row tiles 2 % more.
template <int D, int PT, int TILES, bool WIN, bool TREE>
__global__ void __launch_bounds__(THREADS, 1) k_tiles(const __grid_constant__ Maps maps, const AttnArgs a, uint64_t wait_ns) {
    using M = Smem<D, TILES>;
    constexpr bool AHEAD = TREE && TILES == 1;
    constexpr int WINDOW = window<PT>();
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem), raw_full = sb + M::MISC, raw_empty = raw_full + 8 * M::RS,
                   h_full = raw_empty + 8 * M::RS, h_empty = h_full + 8 * HS, sc_full = h_empty + 8 * HS,
                   q_ready = sc_full + 8 * SS, s_full = q_ready + 16, p_ready = s_full + 16, o_full = p_ready + 16,
                   odd_full = o_full + 16, turn = odd_full + 8, drain = turn + 16;
    Block* scales = reinterpret_cast<Block*>(smem + M::SC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::END - 16);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const volatile int* never = reinterpret_cast<const volatile int*>(tmem_slot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_ready + 8 * i, 4);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_ready + 8 * i, 4);
            mbar_init(o_full + 8 * i, 1);
            mbar_init(turn + 8 * i, 1);
            mbar_init(drain + 8 * i, 1);
        }
        mbar_init(odd_full, 4);
        for (int i = 0; i < M::RS; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 4);
        }
        for (int i = 0; i < HS; ++i) {
            mbar_init(h_full + 8 * i, 4);
            mbar_init(h_empty + 8 * i, TILES);                    // TILES 1: a step belongs to one tile
        }
        for (int i = 0; i < SS; ++i) mbar_init(sc_full + 8 * i, 1);
        tmem_slot[1] = tmem_slot[2] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto tm_s = [&](int x) { return tmem + x * TN; };            // scores; block c's weights over its own columns
    auto tm_o = [&](int x) { return tmem + 2 * TN + x * D; };
    pdl_launch_dependents();
    pdl_wait();

    Space<D, TILES>* sp = static_cast<Space<D, TILES>*>(a.ws);
    const int G = a.Hq / a.c.Hkv;
    List* list = &sp->list;
    Walk w;
    w.begin(list);
    // Every wait is bounded; the first to give up stops the CTA.
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive && !wait_bar(bar, parity, wait_ns, stop)) {
            alive = false;
            *stop = 1;
            set_err(a.b.err, DEV_TIMEOUT);
        }
        return alive;
    };
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {     // the same answer for all lanes
        wait(bar, parity);
        return alive = __all_sync(0xffffffffu, alive);
    };
    // Steps of a part that tile x takes (TILES 2: whether it has rows), out of n.
    auto steps_of = [&](const Item& it, int n, int x) {
        if (TILES == 1) return (n + 1 - x) / 2;
        const int nq = __ldg(a.b.q_start + it.b + 1) - __ldg(a.b.q_start + it.b);
        return (int64_t)nq * G - it.f0 > x * TM ? n : 0;
    };
    constexpr int EACH = TILES == 1 ? 2 : 1;      // tile x takes steps x0, x0 + EACH, ..

    if (warp >= CONV_WARP) {
        regs_down<REGS_CONV>();
        // ---- codes -> fp16: thread = token; keys and values of a step alternate
        const int tok = threadIdx.x & 127;
        uint32_t k = 0;                          // operand tiles so far
        uint4 v[AHEAD ? D / 16 : 1];
        auto arrived = [&]() { return wait_warp(raw_full + 8 * (k % M::RS), k / M::RS & 1); };
        auto fetch = [&]() {
            if (arrived())
#pragma unroll
                for (int c = 0; c < (AHEAD ? D / 16 : 0); ++c) v[c] = fetch_chunk<D>(smem + M::R + k % M::RS * M::RT + tok * D, tok, c);
        };
        for (bool first = true; alive && w.next(a, list, first); first = false) {
            const uint32_t end = k + 2 * (w.until - w.from);
            if (AHEAD) fetch();
            while (k < end && alive) {
                const uint32_t rs = k % M::RS, hs = k % HS;
                if ((!AHEAD && !arrived()) || !wait_warp(h_empty + 8 * hs, (k / HS & 1) ^ 1)) break;
                if constexpr (AHEAD) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) convert_chunk(v[c], smem + M::H + hs * M::HT + tok * 128, tok, c);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(raw_empty + 8 * rs);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(h_full + 8 * hs);
                } else {
                    convert_tile<D>(smem + M::R + rs * M::RT, smem + M::H + hs * M::HT, tok);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(raw_empty + 8 * rs);
                        mbar_arrive(h_full + 8 * hs);
                    }
                }
                ++k;
                if (AHEAD && k < end) fetch();
            }
        }
    } else if (warp >= SOFT_WARP) {
        regs_up<REGS_SOFTMAX>();
        // ---- softmax: thread = row of tile x
        const int x = (warp - SOFT_WARP) >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // tensor-memory lane of the warp's first row
        uint32_t steps = 0, odds = 0, parts = 0, tile0 = 0;       // of this tile: steps, joined parts, parts; of the CTA: steps
        // A part's place in the batch; its queries are on their way to registers while the part before it ends.
        struct Rows {
            int q0, nq, L, r, f, wf, wl;     // the sequence; this thread's row; the warp's rows (none: wl < wf)
            int64_t rows;                    // of the item
            bool in;
        } t;
        constexpr int QLPR = D / 8, QRPI = 32 / QLPR;             // lanes a row of queries, rows a load
        uint4 v[D / 8];
        auto enter = [&]() {
            t.q0 = __ldg(a.b.q_start + w.it.b);
            t.nq = __ldg(a.b.q_start + w.it.b + 1) - t.q0;
            t.L = __ldg(a.b.lens + w.it.b);
            t.rows = (int64_t)t.nq * G - w.it.f0;
            t.r = (TILES == 1 ? 0 : x * TM) + row;
            t.f = w.it.f0 + t.r;
            t.in = t.r < t.rows;
            t.wf = t.f - lane;
            t.wl = (int)min((int64_t)t.wf + 31, w.it.f0 + t.rows - 1);
            const uint16_t* Q = static_cast<const uint16_t*>(a.Q) + (int64_t)w.at.h * G * D;
            if (TILES == 2 || x == 0) {      // neighbouring lanes read neighbouring chunks of a row
                int ff = t.wf + lane / QLPR, tok = ff / G, g = ff % G;
#pragma unroll
                for (int k = 0; k < 32 / QRPI; ++k) {
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (ff <= t.wl) v[k] = __ldcg(reinterpret_cast<const uint4*>(Q + (t.q0 + tok) * a.ldq + g * D) + lane % QLPR);
                    ff += QRPI;
                    for (g += QRPI; g >= G; g -= G) ++tok;
                }
            } else if (a.xt == CQ_BF16) {    // the row's own chunks, for its guard
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    v[c] = make_uint4(0, 0, 0, 0);
                    if (t.in) v[c] = __ldcg(reinterpret_cast<const uint4*>(Q + (t.q0 + t.f / G) * a.ldq + t.f % G * D) + c);
                }
            }
        };
        // The next part that this tile has steps of.
        auto advance = [&](bool first) {
            while (w.next(a, list, first)) {
                if (steps_of(w.it, w.until - w.from, x)) return true;
                tile0 += w.until - w.from;
                first = false;
            }
            return false;
        };
        bool more = advance(true);
        if (more) enter();
        while (more && alive) {
            const int n = w.until - w.from, mine = steps_of(w.it, n, x);
            float qf = a.scale * LOG2E;
            auto guard = [&]() {             // bf16: the row's shift, from its chunks in v
                uint32_t mx = 0;
                auto top = [&](uint32_t y) { mx = max(mx, max((y << 16) & 0x7FFFFFFFu, y & 0x7FFF0000u)); };
#pragma unroll
                for (int c = 0; c < D / 8; ++c) top(v[c].x), top(v[c].y), top(v[c].z), top(v[c].w);
                const int sh = guard_of(__uint_as_float(mx));
                qf *= pow2i(-sh);
                return pow2i(sh);
            };
            if (TILES == 2 || x == 0) {
                uint8_t* q = smem + M::Q + x * M::QT;
                auto chunk = [&](int rr, int c) { return reinterpret_cast<uint4*>(q + (c >> 3) * (TM * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)); };
#pragma unroll
                for (int k = 0; k < 32 / QRPI; ++k) *chunk((row & 96) + k * QRPI + lane / QLPR, lane % QLPR) = v[k];
                __syncwarp();
                if (a.xt == CQ_BF16) {       // each row's own thread sees to its guard
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) v[c] = *chunk(row, c);
                    const float up = guard();
                    auto cv = [&](uint32_t y) { return pack_f16(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xFFFF0000u) * up); };
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) *chunk(row, c) = make_uint4(cv(v[c].x), cv(v[c].y), cv(v[c].z), cv(v[c].w));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(q_ready + 8 * x);
                    if (TILES == 1 && n > 1) mbar_arrive(q_ready + 8);
                }
            } else if (a.xt == CQ_BF16) {
                guard();
            }

            const Rows u0 = t;               // of this part; t goes on to the next
            const int i = u0.f / G;
            const int rhi = u0.in ? row_hi(i, u0.nq, u0.L, a.causal) : 0, rlo = u0.in ? row_lo(i, u0.nq, u0.L, a.window) : 0;
            // steps inside [free_lo, free_hi) need no mask in this warp (rows past the item's take no part)
            const int own = u0.L - u0.nq;    // TREE: from here on the mask tells
            const int free_hi = u0.wf > u0.wl ? INT32_MAX : TREE ? own : row_hi(u0.wf / G, u0.nq, u0.L, a.causal);
            const int free_lo = u0.wf <= u0.wl ? row_lo(u0.wl / G, u0.nq, u0.L, a.window) : 0;
            float m = -INFINITY, l = 0.f;    // of z; the normaliser (with the weights' 2^10)
            // this tile's partial, and its sum in the meantime: against the maximum m_sum
            Part<D, TILES>* part = TILES == 1 && x == 1 ? &sp->odd[blockIdx.x] : &sp->cta[blockIdx.x][w.from == 0 ? 1 : 0];
            float m_sum = -INFINITY;
            bool summed = false;
            for (int j0 = 0; j0 < mine; j0 += WIN ? WINDOW : mine) {
                // A part's first scores are waited for before its first scales: a tile that takes no part in some items
                // does not see every phase of the scales' barriers, and these scores come after all phases but the last.
                if (!wait_warp(s_full + 8 * x, steps & 1)) break;
                if (WIN && j0 > 0 && u0.wf <= u0.wl) {  // the next window: its scores came after all products so far
                    tc_fence_after();
                    const float un = acc_unit<PT>(WINDOW), keep = since(m_sum, m);
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t y[32];
                        tmem_ld_32x32b_x32(tm_o(x) + lanes + 32 * c, y);
                        tmem_ld_wait();
                        if (u0.in)
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float4* o = &part->o[8 * c + e][u0.r];
                                const float4 z = summed ? *o : make_float4(0.f, 0.f, 0.f, 0.f);
                                *o = make_float4(fmaf(z.x, keep, __uint_as_float(y[4 * e]) * un),
                                                 fmaf(z.y, keep, __uint_as_float(y[4 * e + 1]) * un),
                                                 fmaf(z.z, keep, __uint_as_float(y[4 * e + 2]) * un),
                                                 fmaf(z.w, keep, __uint_as_float(y[4 * e + 3]) * un));
                            }
                    }
                    m_sum = m;
                    summed = true;
                }
                for (int j = j0; j < (WIN ? min(j0 + WINDOW, mine) : mine); ++j, ++steps) {
                    const uint32_t tile = tile0 + j * EACH + (TILES == 1 ? x : 0);
                    if (!wait_warp(sc_full + 8 * (tile % SS), tile / SS & 1)) break;
                    const int t0 = w.it.tok0 + (w.from + (int)(tile - tile0)) * TN;
                    const Block* sc = scales + tile % SS * NB;
                    uint32_t odd_k = 0;          // blocks whose factor is no positive number: their scores are taken in full below
                    bool far = false;
#pragma unroll
                    for (int c = 0; c < NB; ++c) {
                        const float k = qf * sc[c].k;
                        if (!(k > 0.f && k < INFINITY)) odd_k |= 1u << c;
                        far |= sc[c].far;
                    }
                    const bool prep = __any_sync(0xffffffffu, t0 < free_lo || t0 + TN > free_hi || odd_k != 0);
                    bool again = PT == 2 || far || __any_sync(0xffffffffu, !(fabsf(m) <= 1048576.f));
                    if (j > j0 && !wait_warp(s_full + 8 * x, steps & 1)) break;
                    if (u0.wl < u0.wf) {         // no rows: whatever lies there as weights only meets its own rows
                        if (lane == 0) mbar_arrive(p_ready + 8 * x);
                        continue;
                    }
                    tc_fence_after();
                    const bool fresh = j == j0;
                    // Scores that a row does not see become -inf.  Blocks with an odd factor are multiplied here; or all become z - m.
                    auto prepare = [&](uint32_t full, bool less, float off) {
                        // TREE: the words that hold token t0's bit and on
                        int word = TREE ? (t0 - own) >> 5 : 0;
                        uint32_t w0 = 0, w1 = 0;
                        if (TREE && u0.in) w0 = mask_word(a, u0.q0 + i, word, u0.nq), w1 = mask_word(a, u0.q0 + i, word + 1, u0.nq);
#pragma unroll 1
                        for (int c = 0; c < TN / 16; ++c) {
                            uint32_t y[16];
                            tmem_ld_32x32b_x16(tm_s(x) + lanes + 16 * c, y);
                            tmem_ld_wait();
                            const float k = full >> (c >> 1) & 1 ? qf * sc[c >> 1].k : 1.f;
                            const float lv = less ? sc[c >> 1].lv : 0.f;
                            const int lo = rlo - t0 - 16 * c, hi = rhi - t0 - 16 * c;
                            uint32_t sees = 0;
                            if (TREE) {
                                const int at = t0 + 16 * c - own;    // the first token's number among the last ones
                                if (at >> 5 != word) {
                                    ++word;
                                    w0 = w1;
                                    w1 = u0.in ? mask_word(a, u0.q0 + i, word + 1, u0.nq) : 0u;
                                }
                                sees = __funnelshift_r(w0, w1, at & 31);
                                if (at < 0) sees |= at <= -16 ? 0xFFFFu : (1u << -at) - 1;
                                if (hi < 16) sees &= hi > 0 ? (1u << hi) - 1 : 0u;
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                y[e] = (TREE ? sees >> e & 1 : e >= lo && e < hi) ? __float_as_uint(fmaf(__uint_as_float(y[e]), k, lv) - off) : 0xFF800000u;
                            tmem_st_32x32b_x16(tm_s(x) + lanes + 16 * c, y);
                        }
                        tmem_st_wait();
                    };
                    uint32_t full = 0;
                    if (prep) {
                        // one choice of blocks for the warp: a factor that is odd in one row is taken in full in all
                        full = __reduce_or_sync(0xffffffffu, odd_k);
                        prepare(full, false, 0.f);
                    }
                    bool less = false;           // m has been taken off
                    // One pass: weights against the m so far, kept in registers until the step's maximum is known.  Where
                    // that has grown by more than GROW (and at first) the maximum comes before them.  f32 outputs
                    // (whose weights take twice the registers) always take the maximum first.
                    while (true) {
                        if (again) {
                            float top = -INFINITY;
#pragma unroll 1
                            for (int c = 0; c < NB; ++c) {
                                uint32_t y[32];
                                tmem_ld_32x32b_x32(tm_s(x) + lanes + 32 * c, y);
                                tmem_ld_wait();
                                float mx = -INFINITY;
#pragma unroll
                                for (int e = 0; e < 32; e += 2) mx = max3(mx, __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                                top = fmaxf(top, fmaf(mx, full >> c & 1 ? 1.f : qf * sc[c].k, sc[c].lv));
                            }
                            const bool grow = top > m + GROW;
                            if (__any_sync(0xffffffffu, grow)) {
                                const float root = grow ? root_of(m - top) : 1.f, fo = root * root;
                                m = grow ? top : m;
                                l = l * root * root;
                                if (!fresh) {
#pragma unroll 1
                                    for (int c = 0; c < D / 32; ++c) {
                                        uint32_t y[32];
                                        tmem_ld_32x32b_x32(tm_o(x) + lanes + 32 * c, y);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * fo);
                                        tmem_st_32x32b_x32(tm_o(x) + lanes + 32 * c, y);
                                    }
                                }
                            }
                            // From 2^20 on z is rounded before m is taken off, as it was for m, and the exponent is
                            // added after that: a fused step would leave its own rounding, which is then no longer small.
                            if (__any_sync(0xffffffffu, fabsf(m) > 1048576.f && fabsf(m) < INFINITY)) {
                                prepare(~full & ((1u << NB) - 1), true, m == -INFINITY ? 0.f : m);
                                full = (1u << NB) - 1;
                                less = true;
                            }
                            if (far) {           // m is settled: their part of the normaliser
#pragma unroll 1
                                for (int c = 0; c < TN / 16; ++c) {
                                    const Block b = sc[c >> 1];
                                    if (!b.far) continue;
                                    uint32_t y[16];
                                    tmem_ld_32x32b_x16(tm_s(x) + lanes + 16 * c, y);
                                    tmem_ld_wait();
                                    const float kc = full >> (c >> 1) & 1 ? 1.f : qf * b.k;
                                    const float sub = W_EXP - (less ? b.lv : m == -INFINITY ? 0.f : m);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) l += ex2(fmaf(__uint_as_float(y[e]), kc, sub));
                                }
                            }
                        }
                        const float m0 = less || m == -INFINITY ? 0.f : m;
                        float top = -INFINITY, add = 0.f;
                        uint32_t s[2][32], p[PT == 1 ? NB : 1][16], p2[16];
                        tmem_ld_32x32b_x32(tm_s(x) + lanes, s[0]);
#pragma unroll
                        for (int c = 0; c < NB; ++c) {
                            tmem_ld_wait();
                            if (c + 1 < NB) tmem_ld_32x32b_x32(tm_s(x) + lanes + 32 * (c + 1), s[(c + 1) & 1]);
                            const Block b = sc[c];
                            const float kc = full >> c & 1 ? 1.f : qf * b.k;
                            const float sub = W_EXP + (less ? 0.f : b.lv - m0);
                            const uint64_t k2 = pair(kc, kc), sub2 = pair(sub, sub);
                            const uint32_t(&y)[32] = s[c & 1];
                            uint32_t(&pc)[16] = p[PT == 1 ? c : 0];
                            uint64_t sum = 0;
                            float mx = -INFINITY;
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float a0 = __uint_as_float(y[2 * e]), a1 = __uint_as_float(y[2 * e + 1]);
                                if (PT == 1) mx = max3(mx, a0, a1);
                                const float2 z = unpair(fma2(pair(a0, a1), k2, sub2));
                                weights<PT>(ex2(z.x), ex2(z.y), sum, pc[e], p2[e]);
                            }
                            top = fmaxf(top, fmaf(mx, kc, b.lv));
                            const float2 z = unpair(sum);
                            add = fmaf(z.x + z.y, b.back, add);
                            if (PT == 2) {
                                tmem_st_32x32b_x16(tm_s(x) + lanes + 32 * c, pc);
                                tmem_st_32x32b_x16(tm_s(x) + lanes + 32 * c + 16, p2);
                            }
                        }
                        if (PT == 1 && !again && __any_sync(0xffffffffu, top > m + GROW)) {
                            again = true;
                            continue;
                        }
                        l += add;
                        if (PT == 1) {
#pragma unroll
                            for (int c = 0; c < NB; ++c) tmem_st_32x32b_x16(tm_s(x) + lanes + 32 * c, p[PT == 1 ? c : 0]);
                        }
                        break;
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_ready + 8 * x);
                }
                if (!alive) break;
            }
            const Walk cur = w;              // this part; w goes on to the next
            tile0 += n;
            more = alive && advance(false);
            if (more) enter();
            if (!wait_warp(o_full + 8 * x, parts & 1)) break;
            ++parts;
            tc_fence_after();
            const bool begins = cur.from == 0, ends = cur.until == cur.it.steps, whole = begins && ends;
            const float un = acc_unit<PT>((mine - 1) % WINDOW + 1);
            l *= pow2i(-(int)W_EXP);
            // TILES 1: the odd steps' result goes to the even steps' threads
            Part<D, TILES>* odd = &sp->odd[TILES == 1 ? blockIdx.x : 0];
            const bool both = TILES == 1 && n > 1;
            float w0 = un, w1 = 0.f, ws = since(m_sum, m);
            if (both && x == 0) {
                if (!wait_warp(odd_full, odds++ & 1)) break;
                if (u0.in) {
                    const float m1 = odd->m[u0.r], l1 = odd->l[u0.r], top = fmaxf(m, m1);
                    const float r0 = m == -INFINITY ? 1.f : root_of(m - top), r1 = m1 == -INFINITY ? 1.f : root_of(m1 - top);
                    w0 = un * r0 * r0;
                    ws = ws * r0 * r0;
                    w1 = r1 * r1;
                    l = l * r0 * r0 + l1 * r1 * r1;
                    m = top;
                }
            }
            const bool direct = whole && !(both && x == 1);
            if (direct) {
                if (u0.in) l = end_sum<TREE>(a, l, u0.f, u0.q0, u0.nq, u0.L);
                const float inv = inv_sum(l);
                w0 *= inv;
                ws *= inv;
                w1 *= inv;
            }
            // Outputs go through the query tile (its products are done), so that neighbouring lanes store
            // neighbouring chunks of a row: 16-bit rows whole, f32 rows half at a time.  They lie as the queries do, so
            // that a warp stays inside its own rows: another may have its next queries there already.
            constexpr int RB = 2 * D, LPR = RB / 16, RPI = 32 / LPR;  // staged bytes and chunks of a row, rows a store
            uint8_t* stage = smem + M::Q + (TILES == 1 ? 0 : x) * M::QT;
            auto chunk = [&](int rr, int c) { return reinterpret_cast<uint4*>(stage + (c >> 3) * (TM * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)); };
            const int es = a.yt == CQ_F32 ? 4 : 2;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(tm_o(x) + lanes + 32 * c, v);
                tmem_ld_wait();
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(v[e]) * w0;
                if (WIN && summed && u0.in) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 z = part->o[8 * c + e][u0.r];
                        y[4 * e] = fmaf(z.x, ws, y[4 * e]);
                        y[4 * e + 1] = fmaf(z.y, ws, y[4 * e + 1]);
                        y[4 * e + 2] = fmaf(z.z, ws, y[4 * e + 2]);
                        y[4 * e + 3] = fmaf(z.w, ws, y[4 * e + 3]);
                    }
                }
                if (both && x == 0 && u0.in) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 z = odd->o[8 * c + e][u0.r];
                        y[4 * e] = fmaf(z.x, w1, y[4 * e]);
                        y[4 * e + 1] = fmaf(z.y, w1, y[4 * e + 1]);
                        y[4 * e + 2] = fmaf(z.z, w1, y[4 * e + 2]);
                        y[4 * e + 3] = fmaf(z.w, w1, y[4 * e + 3]);
                    }
                }
                if (!direct) {
                    if (u0.in)
#pragma unroll
                        for (int e = 0; e < 8; ++e) part->o[8 * c + e][u0.r] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    continue;
                }
                if (a.yt == CQ_F32) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(chunk(row, c % (D / 64) * 8 + e)) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                } else {
                    uint32_t h[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) h[e] = a.yt == CQ_F16 ? pack_f16(y[2 * e], y[2 * e + 1]) : pack_bf16(y[2 * e], y[2 * e + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) *chunk(row, 4 * c + e) = make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                }
                const int done = (c + 1) * 32 * es;                   // bytes of the row so far
                if (done % RB == 0) {
                    __syncwarp();
                    int ff = u0.wf + lane / LPR, tok = ff / G, g = ff % G;
                    char* out = static_cast<char*>(a.O) + (int64_t)cur.at.h * G * D * es + (done - RB) + lane % LPR * 16;
#pragma unroll 4
                    for (int k = 0; k < 32 / RPI; ++k) {
                        if (ff <= u0.wl)
                            *reinterpret_cast<uint4*>(out + ((u0.q0 + tok) * a.ldo + g * D) * es) = *chunk((row & 96) + k * RPI + lane / LPR, lane % LPR);
                        ff += RPI;
                        for (g += RPI; g >= G; g -= G) ++tok;
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            if (u0.in) {
                if (direct) {
                    if (a.lse) a.lse[(int64_t)(u0.q0 + i) * a.Hq + cur.at.h * G + u0.f % G] = lse_of(m, l);
                } else {
                    part->m[u0.r] = m;
                    part->l[u0.r] = l;
                }
            }
            if (both && x == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(odd_full);
            }
            if (!whole && x == 0 && row == 0) list->seg[blockIdx.x][begins ? 1 : 0] = cur.at.slot * a.c.Hkv + cur.at.h;
        }
    } else {
        regs_down<REGS_ISSUE>();
        if (warp == MMA_WARP || warp == MMA_WARP2) {
            // ---- products of tile x
            constexpr uint32_t id_qk = idesc_f16(TM, TN, 0), id_pv = idesc_f16(TM, D, 0) | (1u << 16);
            const int x = warp == MMA_WARP2;
            const uint32_t d_s = uniform(tm_s(x)), d_o = uniform(tm_o(x));
            const uint32_t qa = uniform(desc_inner(sb + M::Q + (TILES == 1 ? 0 : x) * M::QT));
            uint32_t k0 = 0, parts = 0, steps = 0, turns = 0;     // k0: operand tiles before the part
            // The first turn is tile 0's; the last of a part hands it back to tile 0.  (TILES 1 measured 5 % slower
            // with turns: its loads set the pace.)
            auto take = [&](bool both) { return !both || wait_warp(turn + 8 * x, (turns++ + (x == 0)) & 1); };
            auto pass = [&](bool both, bool last) {
                if (both) mbar_arrive(turn + 8 * (last ? 0 : 1 - x));
            };
            auto h_wait = [&](uint32_t kt) { return wait_warp(h_full + 8 * (kt % HS), kt / HS & 1); };
            auto release = [&](uint32_t kt) { tc_commit(h_empty + 8 * (kt % HS)); };
            auto qk = [&](uint32_t kt, bool both) {
                const uint32_t ka = uniform(desc_inner(sb + M::H + (kt % HS) * M::HT));
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint32_t off = ((s >> 2) * (TM * 128) + (s & 3) * 32) >> 4;
                        tc_mma_f16(d_s, desc_of(qa + off, DESC_SW128), desc_of(ka + off, DESC_SW128), id_qk, s > 0);
                        if (s == D / 32 - 1) pass(both, false);   // the turn takes 300 cycles to reach the other thread
                    }
                    tc_commit(s_full + 8 * x);
                }
                __syncwarp();
            };
            auto pv = [&](uint32_t vt, uint32_t acc) {
                const uint32_t va = uniform(desc_outer(sb + M::H + (vt % HS) * M::HT, TN * 128));
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int z = 0; z < PT; ++z)
#pragma unroll
                        for (int s = 0; s < TN / 16; ++s)
                            tc_mma_f16_ts(d_o, d_s + (s >> 1) * 32 + (s & 1) * 8 + z * 16, desc_of(va + s * (2048 >> 4), DESC_SW128),
                                          id_pv, s > 0 || z > 0 ? 1u : acc);
                }
                __syncwarp();
            };
            for (bool first = true; alive && w.next(a, list, first); first = false) {
                const int n = w.until - w.from, mine = steps_of(w.it, n, x);
                if (mine == 0) {
                    if (TILES == 2)                               // not this tile's: the operands go back from here at once
                        for (int j = 0; j < 2 * n && h_wait(k0 + j); ++j)
                            if (lane == 0) mbar_arrive(h_empty + 8 * ((k0 + j) % HS));
                } else {
                    const bool both = TILES == 2 && steps_of(w.it, n, 1) > 0;
                    uint32_t kt = k0 + (TILES == 1 ? 2 * x : 0);  // the step's keys; its values are kt + 1
                    if (!wait_warp(q_ready + 8 * x, parts++ & 1) || !h_wait(kt) || !take(both)) break;
                    qk(kt, both);
                    if (elect_one()) release(kt);
                    for (int j = 0; j < mine; ++j, kt += 2 * EACH) {
                        // the values are mostly there already and waited for first: each such wait takes 100 cycles, which
                        // would come between the weights and their product.  The next keys often are not, and the
                        // conversion that brings them may wait for the place of these values: their product goes first, and
                        // hands it back by itself (one row tile of 80 rows 123 us to 110, 1024-row blocks 137.4 to 136.3)
                        const uint32_t next = kt + 2 * EACH;
                        if (!h_wait(kt + 1) || !take(both)) break;
                        if (!wait_warp(p_ready + 8 * x, steps++ & 1)) break;
                        pv(kt + 1, WIN ? j % WINDOW != 0 : j > 0);
                        if (j + 1 < mine) {
                            if (elect_one()) release(kt + 1);
                            __syncwarp();
                            if (!h_wait(next)) break;
                            qk(next, both);
                            if (elect_one()) release(next);
                        } else if (elect_one()) {
                            tc_commit(o_full + 8 * x);
                            pass(both, x == 1);
                            release(kt + 1);
                        }
                        __syncwarp();
                    }
                }
                k0 += 2 * n;
            }
            if (!alive) {      // let the products in flight end before the tensor memory goes: nothing else waits for this
                if (elect_one()) tc_commit(drain + 8 * x);
                wait_bar(drain + 8 * x, 0, 10000000, never);
            }
            __syncwarp();
        } else if (warp == LOAD_WARP) {
            load_codes<D, M::RS>(a, list, w, maps, sb + M::R, raw_full, raw_empty, scales, sc_full, wait_warp, alive);
            if (!alive) {      // copies in flight land in memory that must still be this CTA's
                for (int i = 0; i < M::RS; ++i)
                    for (uint32_t par = 0; par < 2; ++par) wait_bar(raw_full + 8 * i, par, 10000000, never);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// Joins the items that lie across shares: CTA (i, y) takes rows 32 y .. of the one that began in share i, a warp an
// eighth of the channels.
template <int D, int TILES, bool TREE>
__global__ void __launch_bounds__(256) k_tiles_join(const AttnArgs a, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    const Space<D, TILES>* sp = static_cast<const Space<D, TILES>*>(a.ws);
    const List* list = &sp->list;
    const int i = blockIdx.x, seg = __ldcg(&list->seg[i][1]), cnt = shares_of(list, i, ctas, seg);
    if (seg < 0) return;
    const int4 it = __ldcg(reinterpret_cast<const int4*>(&list->item[seg / a.c.Hkv]));
    const int q0 = __ldg(a.b.q_start + it.x), n = __ldg(a.b.q_start + it.x + 1) - q0;
    const int rows = (int)min((int64_t)TILES * TM, (int64_t)n * (a.Hq / a.c.Hkv) - it.y);
    const int r = blockIdx.y * 32 + threadIdx.x % 32;
    if (r < rows)
        join<true, TREE, D, D / 32, 4>(a, q0, n, __ldg(a.b.lens + it.x), seg % a.c.Hkv, it.y + r, r, threadIdx.x / 32 * (D / 8), cnt,
                                 [&](int j) { return j == 0 ? &sp->cta[i][1] : &sp->cta[i + j][0]; }, (Part<D, TILES>*)nullptr);
}

template <int D, int PT, int TILES, bool WIN, bool TREE>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    Maps maps;
    if (!make_maps(a, maps)) return cudaErrorInvalidValue;
    constexpr size_t smem = Smem<D, TILES>::END + 1024;
    static_assert(smem <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(k_tiles<D, PT, TILES, WIN, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(num_sms(), MAX_CTAS), G = a.Hq / a.c.Hkv, rows = TILES * TM;
    e = launch_pdl(k_tiles_plan<TILES * TM>, dim3(1), dim3(PLAN_THREADS), 0, s, a, &static_cast<Space<D, TILES>*>(a.ws)->list, (int)slots_of(a.b.T, G, a.c.B, rows), ctas);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_tiles<D, PT, TILES, WIN, TREE>, dim3(ctas), dim3(THREADS), smem, s, maps, a, (uint64_t)options().wait_ns.load());
    if (e != cudaSuccess) return e;
    const unsigned y = (unsigned)((std::min<int64_t>(rows, (int64_t)a.max_q * G) + 31) / 32);
    return launch_pdl(k_tiles_join<D, TILES, TREE>, dim3(ctas, y), dim3(256), 0, s, a, ctas);
}

template <int D, int TILES, bool TREE>
cudaError_t run_as(const AttnArgs& a, cudaStream_t s) {
    if (a.yt == CQ_F32) return run<D, 2, TILES, true, TREE>(a, s);
    return needs_windows(a) ? run<D, 1, TILES, true, TREE>(a, s) : run<D, 1, TILES, false, TREE>(a, s);
}
template <int D, bool TREE>
cudaError_t run_d(const AttnArgs& a, cudaStream_t s) {
    return (int64_t)a.max_q * (a.Hq / a.c.Hkv) <= TM ? run_as<D, 1, TREE>(a, s) : run_as<D, 2, TREE>(a, s);
}
template <bool TREE>
cudaError_t run_tiles(const AttnArgs& a, cudaStream_t s) { return a.D == 128 ? run_d<128, TREE>(a, s) : run_d<64, TREE>(a, s); }

}  // namespace
}  // namespace kv8
}  // namespace cq

// Attention over the 8-bit cache for 17 to 32 query rows of a KV head (wide groups, short
// guesses), on the 5th-generation tensor cores with the rows as the narrow side.
//
// Bound by HBM.  Per 128 tokens (a step) S^T = K Q^T (128 tokens x 32 rows) and O^T += V^T P^T
// (D channels x 32 rows): 16 products of 128 x 32 x 16, about 800 cycles, where tiles of 128 rows
// would take 2048 and a softmax of four times the size.  A thread of the softmax has one token
// and its 32 rows: no exchange between threads but for the rows' maxima, and those only when one
// has grown by more than 5 (a vote per step).
//   warp 0          issues the products
//   warp 1          TMA loads of the codes by page, 32 tokens a box, and their scales
//   warps 4-7, 8-11 softmax of the even and the odd steps
//   warps 12-15, 16-19  keys and values -> fp16 (exactly), into the operand tiles
// Both softmax groups work against one maximum per row, kept in shared memory: a step's
// decision to move it follows the decision of the step before (a barrier hands it on; the
// exponentials of neighbouring steps overlap), and whoever moves it rescales O^T in tensor memory.
// Scales, weights and the list of work as in the kernel for many rows.
//
// Measured: 25 rows of 8 heads of 128 channels, 24 sequences of 300 to 9000 tokens: 80 us, 2.8 TB/s; f32 outputs 98 us.
// 64 channels: 72 us.
// Bound by a step's chain (scores, vote, weights to shared memory, product), two of which are under way at a time, and by
// 10 us for the list and the joins.
#include <cfloat>

#include "tiles_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int NR = 32;                 // rows
constexpr int THREADS = 640;           // five warpgroups of 96 registers a thread at launch
constexpr int MMA_WARP = 0, LOAD_WARP = 1, SOFT_WARP = 4, CONV_WARP = 12;
constexpr int REGS_SOFTMAX = 136, REGS_CONV = 56, REGS_ISSUE = 96;
static_assert(2 * REGS_SOFTMAX + 2 * REGS_CONV + REGS_ISSUE <= 5 * 96, "what the launch has");

template <int D>
using Part = PartOf<D, NR>;
template <int D>
struct Space {
    Part<D> cta[MAX_CTAS][2];
    List list;
};

// What the softmax groups share of a part.
struct Rows {
    float2 rc[NR];                     // score factor; minus the maximum of z (FLT_MAX: nothing seen yet, which keeps -inf apart)
    int2 lim[NR];                      // visible tokens
    float fac[NR];                     // the root of what the last move of the maxima scaled sums by
    float wmax[2][4][NR];              // maxima of the warps' tokens
    float sum[8][NR];                  // row sums of the warps
    float m_sum[NR];                   // maxima of the sum in the workspace
    int moves;                         // moves of the maxima so far
};

template <int D, int PT>
struct Smem {
    static constexpr int RS = 4;                  // code tiles in the ring (keys and values alternate)
    static constexpr int PBUF = PT == 1 ? 2 : 1;  // steps of weights (two terms a step: one step's room)
    static constexpr int QT = NR * D * 2;         // queries: D/64 chunks of [32 rows][128 B], swizzled
    static constexpr int HT = TN * D * 2, RT = TN * D, PT_BYTES = TN * NR * 2;
    static constexpr int H = 0, R = H + HS * HT, P = R + RS * RT, Q = P + PBUF * PT * PT_BYTES, BARS = Q + QT;
    static constexpr int NBAR = 2 * RS + 2 * HS + SS + 10;
    static constexpr int SC = BARS + NBAR * 8, ROWS = SC + SS * NB * (int)sizeof(Block), END = ROWS + (int)sizeof(Rows) + 16;
    static_assert(Q % 1024 == 0 && SC % 16 == 0 && ROWS % 16 == 0, "alignment");
};

// Second operand with N = 32 contiguous (64-byte rows, one per k; 64-byte swizzle): 8-row groups 512 bytes apart.
constexpr uint32_t DESC_SW64 = (512u >> 4) | (1u << 14) | (4u << 29);

// Lane r gets the maximum (or sum) over the warp of v[r].
template <bool MAX>
__device__ __forceinline__ float across(const float (&v)[NR]) {
    const int lane = threadIdx.x & 31;
    float t[16];
    auto both = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const bool up = lane & 16;
        t[i] = both(up ? v[i + 16] : v[i], __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 16], 16));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? t[i + o] : t[i], give = up ? t[i] : t[i + o];
            t[i] = both(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    return t[0];
}

template <int D, int PT, bool WIN>
__global__ void __launch_bounds__(THREADS, 1) k_narrow(const __grid_constant__ Maps maps, const AttnArgs a, uint64_t wait_ns) {
    using M = Smem<D, PT>;
    extern __shared__ __align__(1024) uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem), raw_full = sb + M::BARS, raw_empty = raw_full + 8 * M::RS,
                   h_full = raw_empty + 8 * M::RS, h_empty = h_full + 8 * HS, sc_full = h_empty + 8 * HS,
                   q_ready = sc_full + 8 * SS, s_full = q_ready + 8, p_ready = s_full + 16, decided = p_ready + 16,
                   pv_done = decided + 16, o_full = pv_done + 8, drain = o_full + 8;
    Block* scales = reinterpret_cast<Block*>(smem + M::SC);
    Rows* rows = reinterpret_cast<Rows*>(smem + M::ROWS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::END - 16);
    volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const volatile int* never = reinterpret_cast<const volatile int*>(tmem_slot + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < M::RS; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 4);
        }
        for (int i = 0; i < HS; ++i) {
            mbar_init(h_full + 8 * i, 4);
            mbar_init(h_empty + 8 * i, 1);
        }
        for (int i = 0; i < SS; ++i) mbar_init(sc_full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_ready + 8 * i, 4);
            mbar_init(decided + 8 * i, 4);
        }
        mbar_init(q_ready, 4);
        mbar_init(pv_done, 1);
        mbar_init(o_full, 1);
        mbar_init(drain, 1);
        tmem_slot[1] = tmem_slot[2] = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot, tm_o = tmem + 2 * NR;
    pdl_launch_dependents();
    pdl_wait();

    Space<D>* sp = static_cast<Space<D>*>(a.ws);
    List* list = &sp->list;
    const int G = a.Hq / a.c.Hkv;
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

    if (warp >= CONV_WARP) {
        regs_down<REGS_CONV>();
        // ---- codes -> fp16: thread = token; one warpgroup has the keys, one the values
        const int tok = threadIdx.x & 127;
        uint32_t k = (warp - CONV_WARP) >> 2;    // operand tile
        for (bool first = true; alive && w.next(a, list, first); first = false)
            for (int j = w.from; j < w.until && alive; ++j, k += 2) {
                const uint32_t rs = k % M::RS, hs = k % HS;
                if (!wait_warp(raw_full + 8 * rs, k / M::RS & 1) || !wait_warp(h_empty + 8 * hs, (k / HS & 1) ^ 1)) break;
                convert_tile<D>(smem + M::R + rs * M::RT, smem + M::H + hs * M::HT, tok);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(raw_empty + 8 * rs);
                    mbar_arrive(h_full + 8 * hs);
                }
            }
    } else if (warp >= SOFT_WARP) {
        regs_up<REGS_SOFTMAX>();
        // ---- softmax of the steps j % 2 == x: thread = token
        const int x = (warp - SOFT_WARP) >> 2, tid = threadIdx.x & 127, quarter = warp & 3;
        const uint32_t lanes = (uint32_t)quarter << 21, ts = tmem + x * NR + lanes, to = tm_o + lanes;
        // Meetings of this group's 128 threads (ids 1, 2) or of both groups (3).  Whoever has given up still comes, so
        // that nobody waits here for a thread that has gone; then all leave together.
        auto any_of = [&](bool mine, int id, int count) {
            uint32_t any;
            asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.or.aligned.pred q, %2, %3, p;\n"
                         " selp.u32 %0, 1, 0, q;\n}" : "=r"(any) : "r"((uint32_t)mine), "r"(id), "r"(count) : "memory");
            return any != 0;
        };
        uint32_t steps = 0, took = 0, parts = 0, done0 = 0, tile0 = 0;   // own steps and decisions taken; of the CTA: parts, steps
        for (bool first = true; alive && w.next(a, list, first); first = false) {
            const int n = w.until - w.from;
            const int q0 = __ldg(a.b.q_start + w.it.b), nq = __ldg(a.b.q_start + w.it.b + 1) - q0, L = __ldg(a.b.lens + w.it.b);
            const int nrows = (int)min((int64_t)NR, (int64_t)nq * G - w.it.f0);
            if (x == 0) {
                // queries: four threads a row
                const int r = tid >> 2, qd = tid & 3, f = w.it.f0 + r;
                const bool in = r < nrows;
                uint4 v[D / 32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    v[c] = make_uint4(0, 0, 0, 0);
                    if (in)
                        v[c] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.Q) + (q0 + f / G) * a.ldq +
                                                                    (int64_t)(w.at.h * G + f % G) * D + qd * (D / 4)) + c);
                }
                float qf = in ? a.scale * LOG2E : 0.f;
                if (a.xt == CQ_BF16) {
                    uint32_t mx = 0;
                    auto top = [&](uint32_t y) { mx = max(mx, max((y << 16) & 0x7FFFFFFFu, y & 0x7FFF0000u)); };
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) top(v[c].x), top(v[c].y), top(v[c].z), top(v[c].w);
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const int sh = guard_of(__uint_as_float(mx));
                    const float up = pow2i(sh);
                    qf *= pow2i(-sh);
                    auto cv = [&](uint32_t y) { return pack_f16(__uint_as_float(y << 16) * up, __uint_as_float(y & 0xFFFF0000u) * up); };
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) v[c] = make_uint4(cv(v[c].x), cv(v[c].y), cv(v[c].z), cv(v[c].w));
                }
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const int ch = qd * (D / 32) + c;
                    *reinterpret_cast<uint4*>(smem + M::Q + (ch >> 3) * (NR * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v[c];
                }
                if (qd == 0) {
                    rows->rc[r] = make_float2(qf, in ? FLT_MAX : -INFINITY);     // (no row: no weights)
                    rows->lim[r] = in ? make_int2(row_lo(f / G, nq, L, a.window), row_hi(f / G, nq, L, a.causal)) : make_int2(0, 0);
                }
                if (tid == 0) rows->moves = 0;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
            }
            alive = !any_of(!alive, 3, 256);
            if (!alive) break;
            // tokens inside [free_lo, free_hi) need no mask
            const int free_hi = row_hi(w.it.f0 / G, nq, L, a.causal), free_lo = row_lo((w.it.f0 + nrows - 1) / G, nq, L, a.window);
            float l[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) l[r] = 0.f;
            int moves = 0;
            Part<D>* part = &sp->cta[blockIdx.x][w.from == 0 ? 1 : 0];
            // the step before has decided, and perhaps moved the maxima
            auto follow = [&]() {
                wait_warp(decided + 8 * x, took++ & 1);
                if (moves != rows->moves) {
                    moves = rows->moves;
#pragma unroll 1
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int r = 0; r < NR; ++r) l[r] *= rows->fac[r];
                }
            };
            bool gone = false;
            for (int j0 = 0; j0 < n && !gone; j0 += WIN ? window<PT>() : n) {
                if (WIN && __builtin_expect(j0 > 0 && x == 0, PT == 2)) {    // the next window: what the last one holds goes to the sum
                    // (the window's first scores come after all products but the last, whose phase follows on theirs)
                    wait_warp(s_full, steps & 1);
                    follow();
                    wait_warp(pv_done, (done0 + j0 - 1) & 1);
                    tc_fence_after();
                    const float un = acc_unit<PT>(window<PT>());
#pragma unroll 1
                    for (int c = 0; c < NR / 16; ++c) {
                        uint32_t y[16];
                        tmem_ld_32x32b_x16(to + 16 * c, y);
                        tmem_ld_wait();
                        if (tid < D)
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int r = 16 * c + e;
                                float* o = &part->o[r][tid];
                                const float z = j0 > window<PT>() ? *o * since(rows->m_sum[r], -rows->rc[r].y) : 0.f;
                                *o = fmaf(__uint_as_float(y[e]), un, z);
                            }
                    }
                    any_of(false, 1 + x, 128);               // all have read the old maxima
                    if (quarter == 0) rows->m_sum[lane] = -rows->rc[lane].y;
                }
                for (int j = j0 + x; j < (WIN ? min(j0 + window<PT>(), n) : n); j += 2, ++steps) {
                    const uint32_t tile = tile0 + j;
                    wait_warp(sc_full + 8 * (tile % SS), tile / SS & 1);
                    const Block blk = scales[tile % SS * NB + quarter];   // this warp's 32 tokens are one block
                    const int tok = w.it.tok0 + (w.from + j) * TN + tid;
                    wait_warp(s_full + 8 * x, steps & 1);
                    tc_fence_after();
                    float s[NR];
                    {
                        uint32_t y[32];
                        tmem_ld_32x32b_x32(ts, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int r = 0; r < NR; ++r) s[r] = __uint_as_float(y[r]);
                    }
                    if (j > j0) follow();
                    const bool fresh = j == j0;      // (the even steps' group only)
                    const bool masked = __any_sync(0xffffffffu, tok < free_lo || tok >= free_hi);
                    float over = -INFINITY;
#pragma unroll
                    for (int r = 0; r < NR; r += 2) {
                        const float4 c = *reinterpret_cast<const float4*>(&rows->rc[r]);
                        s[r] = fmaf(s[r], blk.k * c.x, blk.lv);            // z, rounded as for the maximum: a fused step on to z - m
                        s[r + 1] = fmaf(s[r + 1], blk.k * c.z, blk.lv);    // would leave a huge score's rounding
                        if (masked) {
                            const int4 lim = *reinterpret_cast<const int4*>(&rows->lim[r]);
                            if (tok < lim.x || tok >= lim.y) s[r] = -INFINITY;
                            if (tok < lim.z || tok >= lim.w) s[r + 1] = -INFINITY;
                        }
                        over = max3(over, s[r] + c.y, s[r + 1] + c.w);
                    }
                    if (any_of(over > GROW || !alive, 1 + x, 128)) {
                        alive = !any_of(!alive, 1 + x, 128);
                        if ((gone = !alive)) break;
                        // Move the maxima: lane r has row r.
                        rows->wmax[x][quarter][lane] = across<true>(s);
                        any_of(false, 1 + x, 128);
                        const float m = -rows->rc[lane].y;
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = fmaxf(top, rows->wmax[x][i][lane]);
                        const bool grow = top > m + GROW;
                        const float nm = grow ? top : m, fac = grow ? root_of(m - nm) : 1.f, fo = fac * fac;
                        if (!fresh) {                // all products so far are in O^T
                            wait_warp(pv_done, (done0 + j - 1) & 1);
                            tc_fence_after();
                            uint32_t y[32];
                            tmem_ld_32x32b_x32(to, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int r = 0; r < NR; ++r) y[r] = __float_as_uint(__uint_as_float(y[r]) * __shfl_sync(0xffffffffu, fo, r));
                            tmem_st_32x32b_x32(to, y);
                            tmem_st_wait();
                        }
#pragma unroll 1
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int r = 0; r < NR; ++r) l[r] *= __shfl_sync(0xffffffffu, fac, r);
                        alive = !any_of(!alive, 1 + x, 128);     // all have read the old maxima
                        if ((gone = !alive)) break;
                        if (quarter == 0) {
                            rows->rc[lane].y = -nm;
                            rows->fac[lane] = fac;
                            if (lane == 0) rows->moves = moves + 1;
                        }
                        any_of(false, 1 + x, 128);
                        ++moves;
                    }
                    // the maxima come off before the next step may move them
#pragma unroll
                    for (int r = 0; r < NR; r += 2) {
                        const float4 c = *reinterpret_cast<const float4*>(&rows->rc[r]);
                        s[r] += c.y;
                        s[r + 1] += c.w;
                    }
                    __syncwarp();
                    if (j + 1 < n && lane == 0) mbar_arrive(decided + 8 * (1 - x));
                    uint32_t p[NR / 2], p2[NR / 2];
                    // (a far block's part of the normaliser comes in a round before the weights: a loop, as more code would
                    // push this one out of the instruction cache)
                    float base = blk.far ? W_EXP - blk.lv : W_EXP, back = blk.far ? 1.f : blk.back;
#pragma unroll 1
                    for (int i = blk.far ? 2 : 1; i > 0; --i) {
#pragma unroll
                        for (int r = 0; r < NR; r += 2) {
                            const float y0 = ex2(s[r] + base), y1 = ex2(s[r + 1] + base);
                            l[r] = fmaf(y0, back, l[r]);
                            l[r + 1] = fmaf(y1, back, l[r + 1]);
                            p[r / 2] = pack_f16(y0, y1);
                            if (PT == 2) {
                                const float2 h = unpack_f16(p[r / 2]);
                                p2[r / 2] = pack_f16(y0 - h.x, y1 - h.y);
                            }
                        }
                        base = W_EXP;
                        back = 0.f;
                    }
                    if (M::PBUF == 1 && j > 0) wait_warp(pv_done, (done0 + j - 1) & 1);   // (a failure shows at the next meeting)
                    uint8_t* buf = smem + M::P + (M::PBUF == 1 ? 0 : x) * PT * M::PT_BYTES + tid * 64;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4* at = reinterpret_cast<uint4*>(buf + ((c ^ ((tid >> 1) & 3)) << 4));
                        *at = make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
                        if (PT == 2) *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(at) + M::PT_BYTES) = make_uint4(p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3]);
                    }
                    tc_fence_before();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_ready + 8 * x);
                }
            }
            done0 += n;
            tile0 += n;
            wait_warp(o_full, parts & 1);
            ++parts;
            // (a group whose last step came before the other's last move)
            if (any_of(!alive, 3, 256)) break;
            if (moves != rows->moves) {
#pragma unroll 1
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < NR; ++r) l[r] *= rows->fac[r];
            }
            rows->sum[x * 4 + quarter][lane] = across<false>(l);
            any_of(false, 3, 256);
            tc_fence_after();
            // O^T: thread = channel; this group's half of the rows
            const bool whole = w.from == 0 && w.until == w.it.steps;
            const float un = acc_unit<PT>((n - 1) % window<PT>() + 1);
            // (a loop: what runs once a part should not push the loops of every step out of the instruction cache)
#pragma unroll 1
            for (int r = 16 * x; r < min(16 * x + 16, nrows); ++r) {
                const int f = w.it.f0 + r;
                uint32_t y;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(y) : "r"(to + r));
                tmem_ld_wait();
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += rows->sum[i][r];
                sum *= pow2i(-(int)W_EXP);
                const float m = -rows->rc[r].y;
                float o = __uint_as_float(y) * un;
                if (WIN && n > window<PT>() && tid < D) o = fmaf(part->o[r][tid], since(rows->m_sum[r], m), o);
                if (whole) {
                    sum = row_sum(sum, f, first_seeing(a, nq, L));
                    const int64_t row = q0 + f / G, head = w.at.h * G + f % G;
                    if (tid < D) store_out(a.O, row * a.ldo + head * D + tid, a.yt, o * inv_sum(sum));
                    if (tid == 0 && a.lse) a.lse[row * a.Hq + head] = lse_of(m, sum);
                } else {
                    if (tid < D) part->o[r][tid] = o;
                    if (tid == 0) {
                        part->m[r] = sum == 0.f ? -INFINITY : m;
                        part->l[r] = sum;
                    }
                }
            }
            if (!whole && x == 0 && tid == 0) list->seg[blockIdx.x][w.from == 0 ? 1 : 0] = w.at.slot * a.c.Hkv + w.at.h;
            tc_fence_before();
            alive = !any_of(!alive, 3, 256);     // the shared rows are read
        }
    } else {
        regs_down<REGS_ISSUE>();
        if (warp == MMA_WARP) {
            // ---- products
            // S^T: 128 tokens x 32 rows, both along the channels; O^T: 128 channels x 32 rows, both across the tokens
            constexpr uint32_t id_qk = idesc_f16(TN, NR, 0), id_pv = idesc_f16(TM, NR, 0) | (1u << 15) | (1u << 16);
            const uint32_t qa = uniform(desc_inner(sb + M::Q)), d_s = uniform(tmem), d_o = uniform(tm_o);
            uint32_t k0 = 0, parts = 0, steps[2] = {0, 0};
            auto h_wait = [&](uint32_t kt) { return wait_warp(h_full + 8 * (kt % HS), kt / HS & 1); };
            auto qk = [&](int x, uint32_t kt) {
                const uint32_t ka = uniform(desc_inner(sb + M::H + (kt % HS) * M::HT)), d = uniform(d_s + x * NR);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        tc_mma_f16(d, desc_of(ka + (((s >> 2) * (TN * 128) + (s & 3) * 32) >> 4), DESC_SW128),
                                   desc_of(qa + (((s >> 2) * (NR * 128) + (s & 3) * 32) >> 4), DESC_SW128), id_qk, s > 0);
                    tc_commit(s_full + 8 * x);
                    tc_commit(h_empty + 8 * (kt % HS));
                }
                __syncwarp();
            };
            for (bool first = true; alive && w.next(a, list, first); first = false) {
                const int n = w.until - w.from;
                if (!wait_warp(q_ready, parts++ & 1)) break;
                for (int j = 0; j < min(n, 2); ++j) {
                    if (!h_wait(k0 + 2 * j)) break;
                    qk(j, k0 + 2 * j);
                }
                for (int j = 0; j < n && alive; ++j) {
                    const int x = j & 1;
                    const uint32_t vt = k0 + 2 * j + 1;
                    if (!h_wait(vt) || !wait_warp(p_ready + 8 * x, steps[x]++ & 1)) break;
                    tc_fence_after();
                    // (D 64: the tile's upper 64 channels are the lower ones again, and unused)
                    const uint32_t va = uniform(desc_outer(sb + M::H + (vt % HS) * M::HT, D == 128 ? TN * 128 : 0));
                    const uint32_t pb = uniform(desc_outer(sb + M::P + (M::PBUF == 1 ? 0 : x) * PT * M::PT_BYTES, 0));
                    const uint32_t acc = WIN ? j % window<PT>() != 0 : j > 0;
                    if (elect_one()) {
#pragma unroll
                        for (int z = 0; z < PT; ++z)
#pragma unroll
                            for (int s = 0; s < TN / 16; ++s)
                                tc_mma_f16(d_o, desc_of(va + s * (2048 >> 4), DESC_SW128),
                                           desc_of(pb + ((z * M::PT_BYTES + s * 1024) >> 4), DESC_SW64), id_pv, s > 0 || z > 0 ? 1u : acc);
                        tc_commit(pv_done);
                        if (j + 1 == n) tc_commit(o_full);
                        tc_commit(h_empty + 8 * (vt % HS));
                    }
                    __syncwarp();
                    if (j + 2 < n) {
                        if (!h_wait(vt + 3)) break;
                        qk(x, vt + 3);
                    }
                }
                k0 += 2 * n;
            }
            if (!alive) {      // let the products in flight end before the tensor memory goes: nothing else waits for this
                if (elect_one()) tc_commit(drain);
                wait_bar(drain, 0, 10000000, never);
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
    if (warp == MMA_WARP) tmem_dealloc(tmem, 128);
}

// Joins the items that lie across shares: the CTAs (i, .) take the one that began in share i, four channels a thread.
template <int D>
__global__ void __launch_bounds__(256) k_narrow_join(const AttnArgs a, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    const Space<D>* sp = static_cast<const Space<D>*>(a.ws);
    const List* list = &sp->list;
    const int i = blockIdx.x, seg = __ldcg(&list->seg[i][1]), cnt = shares_of(list, i, ctas, seg);
    if (seg < 0) return;
    const int4 it = __ldcg(reinterpret_cast<const int4*>(&list->item[seg / a.c.Hkv]));
    const int q0 = __ldg(a.b.q_start + it.x), n = __ldg(a.b.q_start + it.x + 1) - q0;
    const int rows = (int)min((int64_t)NR, (int64_t)n * (a.Hq / a.c.Hkv) - it.y);
    const int k = blockIdx.y * 256 + threadIdx.x, r = k / (D / 4);
    if (r < rows)
        join<true, D, 1, 8>(a, q0, first_seeing(a, n, __ldg(a.b.lens + it.x)), seg % a.c.Hkv, it.y + r, r, k % (D / 4) * 4, cnt,
                            [&](int j) { return j == 0 ? &sp->cta[i][1] : &sp->cta[i + j][0]; }, (Part<D>*)nullptr);
}

template <int D, int PT, bool WIN>
cudaError_t run(const AttnArgs& a, cudaStream_t s) {
    Maps maps;
    if (!make_maps(a, maps)) return cudaErrorInvalidValue;
    constexpr size_t smem = Smem<D, PT>::END + 1024;
    static_assert(smem <= 232448, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(k_narrow<D, PT, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(num_sms(), MAX_CTAS), G = a.Hq / a.c.Hkv;
    e = launch_pdl(k_tiles_plan<NR>, dim3(1), dim3(PLAN_THREADS), 0, s, a, &static_cast<Space<D>*>(a.ws)->list,
                   (int)slots_of(a.b.T, G, a.c.B, NR), ctas);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_narrow<D, PT, WIN>, dim3(ctas), dim3(THREADS), smem, s, maps, a, (uint64_t)options().wait_ns.load());
    if (e != cudaSuccess) return e;
    return launch_pdl(k_narrow_join<D>, dim3(ctas, NR * (D / 4) / 256), dim3(256), 0, s, a, ctas);
}

template <int D>
cudaError_t run_d(const AttnArgs& a, cudaStream_t s) {
    if (a.yt == CQ_F32) return run<D, 2, true>(a, s);
    return needs_windows(a) ? run<D, 1, true>(a, s) : run<D, 1, false>(a, s);
}

}  // namespace

bool narrow_serves(int64_t rows) { return rows <= NR; }
size_t narrow_workspace(int64_t T, int64_t G, int64_t D, int64_t B) {
    return (D == 128 ? sizeof(Space<128>) : sizeof(Space<64>)) + slots_of(T, G, B, NR) * sizeof(Item);
}
cudaError_t launch_narrow(const AttnArgs& a, cudaStream_t s) { return a.D == 128 ? run_d<128>(a, s) : run_d<64>(a, s); }

}  // namespace kv8
}  // namespace cq

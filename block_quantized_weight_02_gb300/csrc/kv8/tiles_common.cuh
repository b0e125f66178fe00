// What the tensor-core attention kernels share: the list of work, the loading and the
// conversion of codes, operand descriptors.
#pragma once
#include "attn_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int TM = 128;                // rows or channels of a tensor-core tile
constexpr int TN = 128;                // tokens of a step
constexpr int NB = TN / BLK;           // blocks of a step
constexpr int MAX_CTAS = 160;          // workspace bound: a full GB300 has no more SMs (and no more than a plan's threads)
constexpr int PLAN_THREADS = 1024;
// Beginning and ending an item counts as so many steps in the shares.  Counted too low, the shares of many short items end
// last: a 16384-token prompt took 2234 us with 3, 1811 with 5, 1824 with 7, 1867 with 12; 25 rows of 24 sequences 106, 92, 82
// and 88 us.
constexpr int ITEM_COST = 7;
constexpr int SS = 8;                  // steps whose scales are kept
constexpr int LB = 32 / NB;            // steps that the loading warp looks up at a time
constexpr int HS = 4;                  // fp16 operand tiles in the ring (keys and values alternate)
// The tensor cores truncate what they add to an accumulator, a product of 16 tokens at a time, towards zero: what is lost goes with
// what the accumulator holds already.  So it is nothing where a weight or two make the sum, and on average 2.3e-8 of the whole
// a product where it grows evenly (values of one sign; half of it where they have both): measured, f32 outputs over 40960
// tokens, 3.0e-6 with windows of 8 steps, 1.4e-6 with 4, 0.7e-6 with 2.  Hence windows: an accumulator starts afresh every window<PT>()
// of a tile's steps, and what it held is added, rounded to nearest, to a sum in the workspace.
// f32 outputs: 8 steps (trees of 64 rows over 70000 and 100000 tokens 255 us; 281 with 4, 338 with 2), and LOST a product is put
// back, the middle between nothing and 2.3e-8, so that 1.6e-6 is left on either side; the same with a mask and without.
// 16-bit outputs (half the products): 128 steps, 7e-5 at most, under their own rounding.
template <int PT>
constexpr int window() { return PT == 2 ? 8 : 128; }
constexpr float LOST = 1.1e-8f;
// 16-bit outputs whose sequences have no room for more than a window are served without (WIN false): 24 sequences of 25 rows
// 79.4 against 79.9 us (64 channels: 72.5 against 74), ragged prompts 258 against 270.
inline bool needs_windows(const AttnArgs& a) { return a.yt == CQ_F32 || a.c.ldt * a.c.page > window<1>() * TN; }
// From an accumulator that holds `steps` steps to O.
template <int PT>
__device__ __forceinline__ float acc_unit(int steps) { return PT == 2 ? fmaf((float)steps, LOST * (PT * TN / 16), 1.f) * 0x1p-10f : 0x1p-10f; }
constexpr float W_EXP = 10.f, GROW = 5.f;   // weights carry 2^10 (acc_unit takes it off) and grow by 2^5 before the maximum moves

// What the softmax needs of a block (written by the loading warp, which has the time).
struct alignas(16) Block {
    float k;               // the keys' scale (NaN if either scale is)
    float lv;              // the values' exponent
    float back;            // 2^-lv, or 0 if far
    int far;               // lv is more than APART below the part's largest so far
};

struct Maps {
    CUtensorMap t[2];                  // keys, values: {D, pages * Hkv * page}, box {D, 32}
};
inline bool make_maps(const AttnArgs& a, Maps& maps) {
    const uint64_t dims[2] = {(uint64_t)a.D, (uint64_t)a.c.pages * a.c.Hkv * a.c.page}, strides[1] = {(uint64_t)a.D};
    const uint32_t box[2] = {(uint32_t)a.D, (uint32_t)BLK};
    for (int i = 0; i < 2; ++i)
        if (!encode_tiled(&maps.t[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.c.q[i], dims, strides, box,
                          a.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return false;
    return true;
}

struct alignas(16) Item {
    int b, f0, tok0, steps;            // sequence, first row, first token, steps (none visible: 1)
};
struct Start {
    int slot, h, step;                 // where a CTA's share begins
};
// The list of work, and which segments (slot * Hkv + h) the CTAs left unfinished: one that began in an earlier
// share, one that began in their own and goes on, or -1.
struct alignas(16) List {
    int seg[MAX_CTAS][2];
    Start start[MAX_CTAS + 1];
    int ok;                            // the list stands
    Item item[1];                      // [slots]
};

inline int64_t slots_of(int64_t T, int64_t G, int64_t B, int rows) { return T * G / rows + B; }

// ---- the list ------------------------------------------------------------------------------------------------------
// One block, bound by the latency of its loads: 2.4 us.  Threads price the items they hold, then each share finds where it
// begins (the thread of an item writing all shares in it took 11 us for 38 heads).
// Sequence b owns the slots floor(q_start[b] G / ROWS) + b .., since n tokens make at most floor(n G / ROWS) + 1 items.
template <int ROWS>
__global__ void __launch_bounds__(PLAN_THREADS) k_tiles_plan(const AttnArgs a, List* sp, int slots, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int64_t wsum[PLAN_THREADS / 32];
    const int G = a.Hq / a.c.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    for (int b = threadIdx.x; b < a.c.B; b += PLAN_THREADS) {
        const int L = __ldg(a.b.lens + b);
        if (!rows_ok(__ldg(a.b.q_start + b), __ldg(a.b.q_start + b + 1), a.b.T, a.max_q) || !length_ok(a.c, L)) bad = true;
    }
    for (int i = threadIdx.x; i < MAX_CTAS; i += PLAN_THREADS) sp->seg[i][0] = sp->seg[i][1] = -1;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) {
            set_err(a.b.err, DEV_INDEX);
            sp->ok = 0;
        }
        return;
    }
    const int per = (slots + PLAN_THREADS - 1) / PLAN_THREADS;      // neighbouring slots of a thread
    const int s0 = min(threadIdx.x * per, slots), s1 = min(s0 + per, slots);
    auto key = [&](int b) { return (int64_t)__ldg(a.b.q_start + b) * G / ROWS + b; };
    int64_t mine = 0;
    int b = 0, n = a.c.B;
    if (s0 < s1)
        while (n > 1) {                                            // the largest b whose slots start at or before s0
            const int half = n / 2;
            if (key(b + half) <= s0) b += half, n -= half; else n = half;
        }
    for (int s = s0; s < s1; ++s) {
        while (b + 1 < a.c.B && key(b + 1) <= s) ++b;
        Item it = {b, 0, 0, 0};
        const int q0 = __ldg(a.b.q_start + b), nq = __ldg(a.b.q_start + b + 1) - q0, L = __ldg(a.b.lens + b);
        const int64_t f0 = (s - key(b)) * ROWS, rows = (int64_t)nq * G;
        if (f0 >= 0 && f0 < rows) {
            const int first = (int)f0 / G, last = (int)(min(f0 + ROWS, rows) - 1) / G;
            const int lo = row_lo(first, nq, L, a.window) / BLK * BLK, hi = row_hi(last, nq, L, a.causal);
            it.f0 = (int)f0;
            it.tok0 = lo;
            it.steps = hi > lo ? (hi - lo + TN - 1) / TN : 1;
        }
        sp->item[s] = it;
        if (it.steps) mine += (int64_t)(it.steps + ITEM_COST) * a.c.Hkv;
    }
    __shared__ int64_t before[PLAN_THREADS + 1];                   // cost of the slots ahead of each thread's
    auto scan = [&](int64_t v) {
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    const int64_t inc = scan(mine);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    const int64_t sums = scan(wsum[lane]);
    const int64_t ahead = __shfl_sync(0xffffffffu, sums, warp) - wsum[warp], total = __shfl_sync(0xffffffffu, sums, 31);
    before[threadIdx.x] = ahead + inc - mine;
    if (threadIdx.x == 0) {
        before[PLAN_THREADS] = total;
        sp->ok = 1;
        sp->start[ctas] = {slots, 0, 0};
    }
    __syncthreads();
    // a thread finds where share i begins: at cost i q + min(i, rem)
    const int i = threadIdx.x;
    if (i >= ctas) return;
    const int64_t u = i * (total / ctas) + min((int64_t)i, total % ctas);
    Start at = {slots, 0, 0};                                      // (past the list: there are more CTAs than cost)
    if (u < total) {
        int t = 0;                                                 // the last thread with before[t] <= u: it has slots
        for (int o = PLAN_THREADS / 2; o; o >>= 1)
            if (before[t + o] <= u) t += o;
        int64_t rest = u - before[t];
        for (int s = min(t * per, slots);; ++s) {
            const int cost = sp->item[s].steps + ITEM_COST;
            if (cost == ITEM_COST) continue;
            const int64_t all = (int64_t)cost * a.c.Hkv;
            if (rest < all) {
                const int h = (int)(rest / cost);
                at = {s, h, max((int)(rest - (int64_t)h * cost) - ITEM_COST, 0)};
                break;
            }
            rest -= all;
        }
    }
    sp->start[i] = at;
}

// ---- issuing products.  A whole warp runs the issuing loops and one elected lane the instructions, on values the
// compiler can keep in uniform registers: with one lane in a branch of its own each product took 44 instructions and
// about 100 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Operand descriptors as (low, high) words; the low word moves by (bytes >> 4).
// Rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart.  Inner operands (rows = M or N) lie along k; outer
// ones (rows = k) have the next 64 elements of M or N `next` bytes on.
constexpr uint32_t DESC_SW128 = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_inner(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_outer(uint32_t saddr, uint32_t next) { return ((saddr & 0x3FFFFu) >> 4) | ((next >> 4) << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }

// The parts of items that a CTA's share is made of, in order; every role walks the same list.
struct Walk {
    Start at, end;
    Item it;
    int from, until;      // steps of the current part
    __device__ __forceinline__ void begin(const List* sp) {
        auto get = [&](int i) {
            const Start* p = &sp->start[i];
            return Start{__ldcg(&p->slot), __ldcg(&p->h), __ldcg(&p->step)};
        };
        at = get(blockIdx.x);
        end = get(blockIdx.x + 1);
        if (!__ldcg(&sp->ok)) at = end = {0, 0, 0};
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, const List* sp, bool first) {
        if (!first) {
            at.step = until;
            if (until == it.steps) {
                at.step = 0;
                if (++at.h == a.c.Hkv) {
                    at.h = 0;
                    ++at.slot;
                }
            }
        }
        while (true) {
            const bool last = at.slot == end.slot && at.h == end.h;
            if (at.slot > end.slot || (at.slot == end.slot && at.h > end.h) || (last && at.step >= end.step)) return false;
            const int4 v = __ldcg(reinterpret_cast<const int4*>(&sp->item[at.slot]));
            if (v.w != 0) {
                it = {v.x, v.y, v.z, v.w};
                from = at.step;
                until = last ? end.step : v.w;
                return true;
            }
            ++at.slot;
        }
    }
};

// ---- loads by one warp: lane NB i + c has block c of step i of a batch of LB steps.  RS code tiles in the ring, keys
// and values in turn; `wait` is a bounded wait with one answer for the warp.
template <int D, int RS, class W>
__device__ __forceinline__ void load_codes(const AttnArgs& a, const List* list, Walk w, const Maps& maps, uint32_t ring,
                                           uint32_t raw_full, uint32_t raw_empty, Block* scales, uint32_t sc_full, W wait,
                                           const bool& alive) {
    const int lane = threadIdx.x & 31;
    uint32_t k = 0, tile = 0;
    for (bool first = true; alive && w.next(a, list, first); first = false) {
        const int L = __ldg(a.b.lens + w.it.b);
        int row1 = 0;
        float2 s1;
        auto look_up = [&](int j) {       // of the batch that begins at step j
            const int tok = w.it.tok0 + j * TN + lane * BLK;
            row1 = -1;
            s1 = make_float2(1.f, pow2i(-64));
            if (j + lane / NB < w.until && tok < L) {
                int pid = __ldg(a.c.table + w.it.b * a.c.ldt + tok / a.c.page);
                if (pid < 0 || pid >= a.c.pages) {       // read some page instead: the result is void
                    set_err(a.b.err, DEV_INDEX);
                    pid = 0;
                }
                row1 = (pid * a.c.Hkv + w.at.h) * a.c.page + tok % a.c.page;
                s1 = make_float2(__ldcg(a.c.s[0] + row1 / BLK), __ldcg(a.c.s[1] + row1 / BLK));
            }
        };
        look_up(w.from);
        int hi = -64;                     // largest value exponent of the part up to this batch
        for (int j0 = w.from; j0 < w.until && alive; j0 += LB) {
            const int row = row1;
            const float2 s = s1;
            Block blk;
            if (j0 + LB < w.until) look_up(j0 + LB);
            for (int i = 0; i < min(LB, w.until - j0) && alive; ++i, ++tile) {
                const bool me = lane / NB == i, have = me && row >= 0;
                const uint32_t blocks = __popc(__ballot_sync(0xffffffffu, have));
                for (int z = 0; z < 2 && alive; ++z, ++k) {
                    const uint32_t rs = k % RS, bar = raw_full + 8 * rs;
                    if (!wait(raw_empty + 8 * rs, (k / RS & 1) ^ 1)) break;
                    const bool issue = !a.stall || k == 0;
                    if (lane == 0 && issue) mbar_arrive_expect_tx(bar, blocks * BLK * D);
                    __syncwarp();
                    if (have && issue) tma_load_2d(ring + rs * (TN * D) + lane % NB * BLK * D, &maps.t[z], bar, 0, row);
                }
                if (!alive) break;
                if (i == 0) {                       // of the whole batch (now that the first copies are on their way)
                    const int lv = value_exp(s.y);
                    hi = max(hi, __reduce_max_sync(0xffffffffu, lv));
                    const bool far = row >= 0 && lv < hi - APART;
                    blk = {s.y == s.y ? s.x : s.y, (float)lv, far ? 0.f : pow2i(-lv), far};
                }
                if (me) scales[tile % SS * NB + lane % NB] = blk;
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full + 8 * (tile % SS));
            }
        }
    }
}

// ---- a tile of codes [128 tokens][D] -> fp16 (exactly), chunks of 64 channels [128][128 B], swizzled; one token a thread
template <int D>
__device__ __forceinline__ uint4 fetch_chunk(const uint8_t* src, int tok, int c) {
    const int at = D == 128 ? (c ^ (tok & 7)) : (c ^ ((tok >> 1) & 3));
    return *reinterpret_cast<const uint4*>(src + at * 16);
}
__device__ __forceinline__ void convert_chunk(uint4 v, uint8_t* dst, int tok, int c) {
    const uint32_t u[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int ch = (2 * c + e) & 7;       // 16-byte chunk of the 64-channel row
        *reinterpret_cast<uint4*>(dst + (c >> 2) * (TN * 128) + ((ch ^ (tok & 7)) << 4)) =
            make_uint4(codes_f16(u[2 * e], 0x4140u), codes_f16(u[2 * e], 0x4342u), codes_f16(u[2 * e + 1], 0x4140u),
                       codes_f16(u[2 * e + 1], 0x4342u));
    }
}
template <int D>
__device__ __forceinline__ void convert_tile(const uint8_t* raw, uint8_t* out, int tok) {
    const uint8_t* src = raw + tok * D;
    uint8_t* dst = out + tok * 128;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) convert_chunk(fetch_chunk<D>(src, tok, c), dst, tok, c);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Registers of a warpgroup from here on (a multiple of 8; the groups' shares add up to the launch's).
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// The shares after share i that go on with its last segment, and itself.
__device__ __forceinline__ int shares_of(const List* list, int i, int ctas, int seg) {
    const int lane = threadIdx.x & 31;
    int cnt = 1;
    while (true) {
        const int j = i + cnt + lane;
        const bool more = j < ctas && __ldcg(&list->seg[j][0]) == seg;
        const int k = __ffs(~__ballot_sync(0xffffffffu, more));
        cnt += k ? k - 1 : 32;
        if (k) return cnt;
    }
}

}  // namespace
}  // namespace kv8
}  // namespace cq

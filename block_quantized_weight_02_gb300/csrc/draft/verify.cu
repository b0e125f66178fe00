// Check of drafted tokens against the target's probabilities.
//
// A cluster of CTAs has one sequence.  Each of them gathers what the walk needs of the rows (tokens, parents, their
// two probabilities) and walks by itself, one warp, 32 rows a look; what is left of the probabilities is then summed by the
// whole cluster, a contiguous share a warp, and the CTA whose share holds the drawn number looks again at that share alone.
// So a sequence costs one pass over one row of P (and of Q), which bounds it for large batches; a rejection costs another
// pass only where a sibling drawn from the same Q follows.
//
// After k rejected children drawn from q what is left is max(P - A q, 0): with w_k = max(P - A_k q, 0) and m_k its sum (m_0 = 1)
//   w_{k+1} = max(w_k - m_k q, 0) = max(P - (A_k + m_k) q, 0),
// so a pass needs A alone, however many were rejected.
//
// Measured: 64 chains over 152001 entries, f32, 19.5 us (78 MB if every chain ends early: 4.0 TB/s, of which 8 us are
// latency); one chain over 32000 7.4 us; 16 trees of 26 chosen tokens over 131072 bf16 entries 10.5 us.  A pass after a
// rejection, of one tree and of 16: over 32000 f32 entries 4.1 and 4.9 us, over 128000 7.5 and 10.
//
// A border of the drawn number may lie anywhere, so sums carry 2^-40 and better: each term is the difference
// in two floats, sums add the rounding errors that two floats lose (Knuth's two-sum), two elements an instruction.  64-bit
// arithmetic, one warp instruction in 16 cycles of an SM, is left to the walk.
#include "draft.cuh"

namespace cq {
namespace draft {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, MAX_CLUSTER = 8, MAX_ROWS = 1024, UNROLL = 4;
constexpr int SHARES = MAX_CLUSTER * WARPS;

struct Row {
    int token, parent;     // parent: place in the sequence, or -1
    float p, q, u;         // the target's and the draft's probability of the token after its parent
};

// A number in two floats, lo at most half a last place of hi.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const float t = a.hi + b.hi, v = t - a.hi;
    const float e = ((a.hi - (t - v)) + (b.hi - v)) + (a.lo + b.lo), h = t + e;
    return {h, e - (h - t)};
}
__device__ __forceinline__ bool operator>(Two a, Two b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.f; }
__device__ __forceinline__ Two times(Two a, float x) {
    const float t = __fmul_rn(a.hi, x), e = fmaf(a.lo, x, fmaf(a.hi, x, -t)), h = t + e;
    return {h, e - (h - t)};
}
__device__ __forceinline__ double wide(Two a) { return (double)a.hi + (double)a.lo; }

struct Shared {
    Two sum[2][SHARES];    // the cluster's shares, of even and odd passes
    Two part[WARPS];       // of a look at one share
    Two aim;               // what the drawn number leaves within its share
    double mass, less;
    int what, last, next, stand, fell, pass, share;
    int path[MAX_ROWS];    // places of the rows that stand
    int gone[MAX_ROWS];    // rejected tokens that were not drawn
    Row row[MAX_ROWS];
};

template <class X>
constexpr int VEC = 16 / (int)sizeof(X);
template <class X>
__device__ __forceinline__ void widen(uint4 v, float (&f)[VEC<X>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(X) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (std::is_same<X, __half>::value) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
template <class X>
__device__ __forceinline__ float one(const X* p) {
    if constexpr (sizeof(X) == 4) return fmaxf(__ldcg(p), 0.f);
    else if constexpr (std::is_same<X, __half>::value) return fmaxf(__half2float(__ldcg(p)), 0.f);
    else return fmaxf(__bfloat162float(__ldcg(p)), 0.f);
}

// What is left at a row of P: max(P - a q, 0), a in two floats.  Negative entries and NaN count as 0 (the maxima drop them).
enum { NOTHING_OFF = 0, Q_OFF = 1, MORE_OFF = 2 };       // a = 0; a = 1: one rejection; any a
template <class X, bool DRAWN>
struct Left {
    static constexpr int N = VEC<X>;
    const X *p, *q;
    Two a;
    int off, V, ngone;
    const int* gone;
    __device__ __forceinline__ Left(const VerifyArgs& v, const Shared& sm, int q0, bool whole) {
        p = static_cast<const X*>(v.P) + (q0 + sm.last) * v.ldp;
        q = DRAWN ? static_cast<const X*>(v.Q) + (q0 + sm.last) * v.ldq : nullptr;
        const double less = whole ? 0.0 : sm.less;
        a.hi = (float)less;
        a.lo = (float)(less - (double)a.hi);
        off = !DRAWN || less == 0.0 ? NOTHING_OFF : less == 1.0 ? Q_OFF : MORE_OFF;
        V = v.V;
        ngone = whole ? 0 : sm.fell;
        gone = sm.gone;
    }
    // The warp's entries will be those in [lo, hi): most have none of the rejected tokens.
    __device__ __forceinline__ void narrow(int lo, int hi) {
        if (DRAWN || ngone == 0) return;
        bool mine = false;
        for (int k = threadIdx.x & 31; k < ngone; k += 32) mine |= gone[k] >= lo && gone[k] < hi;
        if (!__any_sync(0xffffffffu, mine)) ngone = 0;
    }
    // A row's last vector may be a part of one, of which nothing past the row is read.
    __device__ __forceinline__ uint4 load(const X* r, int at) const {
        if (at + N <= V) return __ldcg(reinterpret_cast<const uint4*>(r + at));
        uint32_t w[4] = {0, 0, 0, 0};
        if (at < V)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (at + i < V) {
                    if constexpr (sizeof(X) == 4) w[i] = __ldcg(reinterpret_cast<const uint32_t*>(r + at) + i);
                    else w[i / 2] |= (uint32_t)__ldcg(reinterpret_cast<const uint16_t*>(r + at) + i) << 16 * (i & 1);
                }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 load_q(int at) const { return DRAWN && off ? load(q, at) : make_uint4(0, 0, 0, 0); }
    // The vector's entries, with what was rejected as chosen taken out.
    __device__ __forceinline__ void entries(uint4 pv, uint4 qv, int at, float (&f)[N], float (&g)[N]) const {
        widen<X>(pv, f);
        widen<X>(qv, g);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = DRAWN ? fmaxf(g[i], 0.f) : 0.f;
        if (!DRAWN)
            for (int k = 0; k < ngone; ++k)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (gone[k] == at + i) f[i] = 0.f;
    }
    // One entry: exact for a up to 1 (with f >= g the difference's rounding error is (f - d) - g), else to 2^-45 of the larger term.
    // The float f may lie next to the product's own float, on either side, and the two rests decide: so the difference is
    // taken with both (Knuth's two-sum, twice), and its first float is positive where the entry is.
    __device__ __forceinline__ Two term(float f, float g) const {
        if (!DRAWN || off != MORE_OFF) {
            const float h = fmaxf(f, g), d = h - g;
            return {d, (h - d) - g};
        }
        const float t = __fmul_rn(g, a.hi), tl = fmaf(g, a.lo, fmaf(g, a.hi, -t));
        const float d = f - t, b = d - f, e = ((f - (d - b)) - (t + b)) - tl;
        const float h = d + e, c = h - d;
        return h > 0.f ? Two{h, (d - (h - c)) + (e - c)} : Two{0.f, 0.f};
    }
    // Adds a vector to running sums of the even and the odd entries.
    __device__ __forceinline__ void add(uint4 pv, uint4 qv, int at, uint64_t& hi, uint64_t& lo) const {
        float f[N], g[N];
        entries(pv, qv, at, f, g);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            uint64_t d, e = 0;
            if (!DRAWN || off != MORE_OFF) {
                const uint64_t h = pair(fmaxf(f[i], g[i]), fmaxf(f[i + 1], g[i + 1])), t = pair(g[i], g[i + 1]);
                d = DRAWN ? sub2(h, t) : h;
                if (DRAWN) e = sub2(sub2(h, d), t);
            } else {
                const Two x = term(f[i], g[i]), y = term(f[i + 1], g[i + 1]);
                d = pair(x.hi, y.hi);
                e = pair(x.lo, y.lo);
            }
            const uint64_t t = add2(hi, d), v = sub2(t, hi);
            lo = add2(lo, add2(sub2(hi, sub2(t, v)), sub2(d, v)));
            if (DRAWN) lo = add2(lo, e);
            hi = t;
        }
    }
};

__device__ __forceinline__ Two shuffle_up(Two x, int o) { return {__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)}; }
__device__ __forceinline__ Two shuffle(Two x, int l) { return {__shfl_sync(0xffffffffu, x.hi, l), __shfl_sync(0xffffffffu, x.lo, l)}; }
__device__ __forceinline__ Two warp_sum(Two x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = x + Two{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
    return x;
}
// The sum of the lanes before this one; *all gets that of all.
__device__ __forceinline__ Two warp_before(Two x, Two* all) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two y = shuffle_up(x, o);
        if (lane >= o) x = y + x;
    }
    *all = shuffle(x, 31);
    const Two y = shuffle_up(x, 1);
    return lane ? y : Two{0.f, 0.f};
}
__device__ __forceinline__ void st_cluster(uint32_t addr, Two x) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x.hi), "f"(x.lo) : "memory");
}

template <class X, bool DRAWN>
__global__ void __launch_bounds__(THREADS, 4) k_verify(const VerifyArgs a, int cluster) {
    constexpr int N = VEC<X>, LOOK = 8 / N;              // LOOK: vectors of a thread that looks at a share again
    __shared__ Shared sm;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int q0 = __ldcg(a.q_start + b), n = __ldcg(a.q_start + b + 1) - q0;
    const float u_last = __ldcg(a.u_last + b);
    int32_t* out = a.out + b * a.ldo;
    int32_t* path = a.path + b * a.ldo;
    const bool ok = kv8::rows_ok(q0, q0 + n, a.T, a.max_q);
    if (!ok || n == 0) {                                 // (the same for the whole cluster)
        if (!ok && tid == 0) kv8::set_err(a.err, DEV_INDEX);
        if (rank == 0) {
            for (int i = tid; i < a.max_q; i += THREADS) out[i] = path[i] = -1;
            if (tid == 0) a.count[b] = 0;
        }
        return;
    }
    const X* P = static_cast<const X*>(a.P) + (int64_t)q0 * a.ldp;
    const X* Q = static_cast<const X*>(a.Q) + (DRAWN ? (int64_t)q0 * a.ldq : 0);

    // ---- the rows
    bool bad = false;
    for (int j = tid; j < n; j += THREADS) {
        Row r = {0, j - 1, 0.f, 0.f, 0.f};
        if (j > 0) {
            r.token = __ldcg(a.tokens + q0 + j);
            r.u = __ldcg(a.u + q0 + j);
            if (r.u < 0.f) r.u = 0.f;                    // (what has no probability must not stand; NaN rejects)
            if (a.mask) {
                r.parent = -1;
                const uint32_t* m = a.mask + (q0 + j) * a.ldm;
                for (int i = (j - 1) >> 5; i >= 0 && r.parent < 0; --i) {
                    uint32_t w = __ldcg(m + i);
                    if (i == j >> 5) w &= (1u << (j & 31)) - 1;
                    if (w) r.parent = 32 * i + 31 - __clz(w);
                }
            }
            if (r.token < 0 || r.token >= a.V) {
                bad = true;
                r.token = 0;
            } else if (r.parent >= 0) {
                r.p = one(P + r.parent * a.ldp + r.token);
                if (DRAWN) r.q = one(Q + r.parent * a.ldq + r.token);
            }
        }
        sm.row[j] = r;
    }
    if (tid == 0) {
        sm.mass = 1.0;
        sm.less = 0.0;
        sm.last = sm.fell = sm.stand = sm.pass = 0;
        sm.next = 1;
        sm.path[0] = 0;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) kv8::set_err(a.err, DEV_INDEX);
    }
    // (every CTA of the cluster has begun before another writes to it: waited for before the first sums go out)
    __syncwarp();
    if (cluster > 1) cluster_arrive_relaxed();

    const int vecs = (a.V + N - 1) / N, per = (vecs + cluster * WARPS - 1) / (cluster * WARPS);   // vectors of a share
    bool whole = false;                                  // nothing was left: P as it is
    while (true) {
        // ---- the walk, up to where it needs a sum
        if (warp == 0 && !whole) {
            int last = sm.last, j = sm.next, stand = sm.stand, fell = sm.fell, what = 0;
            double mass = sm.mass, less = sm.less;
            bool waits = sm.pass > 0;                    // the sum after a rejection came in
            for (; j < n; ) {
                const int c = j + lane;
                const uint32_t kids = __ballot_sync(0xffffffffu, c < n && sm.row[c].parent == last);
                if (!kids) {
                    j += 32;
                    continue;
                }
                j += __ffs(kids) - 1;
                const Row r = sm.row[j];
                const double p = r.p, q = r.q;
                bool stands;
                if (mass == 1.0 && less == 0.0 && fell == 0) {
                    // nothing rejected yet: u q < p, exactly: in 32 bits (t < p leaves no room for a rounding in between) unless the
                    // product's rounding error may be none of their numbers
                    const float g = DRAWN ? r.q : 1.f, t = __fmul_rn(r.u, g);
                    stands = t >= 0x1p-100f ? t < r.p || (t == r.p && fmaf(r.u, g, -t) < 0.f) : r.u * (double)g < p;
                    if (!stands && DRAWN) less = 1.0;
                    if (!stands && !DRAWN) {
                        mass -= p;
                        if (lane == 0) sm.gone[0] = r.token;
                        __syncwarp();
                        fell = 1;
                    }
                } else if (DRAWN) {
                    if (less > 0.0 && !waits) {          // a sibling was rejected: what is left of the mass?
                        what = 1;
                        break;
                    }
                    waits = false;
                    stands = r.u * q * mass < fmax(p - less * q, 0.0);
                    if (!stands) less += mass;
                } else {
                    bool again = false;
                    for (int k = lane; k < fell; k += 32) again |= sm.gone[k] == r.token;
                    const double w = __any_sync(0xffffffffu, again) ? 0.0 : p;
                    stands = r.u * fmax(mass, 0.0) < w;  // (numbers above 1 may have taken more than there was)
                    if (!stands) {
                        mass -= w;
                        if (lane == 0) sm.gone[fell] = r.token;
                        __syncwarp();
                        ++fell;
                    }
                }
                if (stands) {
                    last = j;
                    ++stand;
                    if (lane == 0) sm.path[stand] = j;
                    mass = 1.0;
                    less = 0.0;
                    fell = 0;
                }
                ++j;
            }
            __syncwarp();
            if (lane == 0) {
                sm.last = last;
                sm.next = j;
                sm.stand = stand;
                sm.fell = fell;
                sm.what = what;
                sm.mass = mass;
                sm.less = less;
            }
        }
        __syncthreads();
        // ---- a pass over what is left at the last row that stands
        const int turn = sm.pass & 1;
        Left<X, DRAWN> left(a, sm, q0, whole);
        const int mine = rank * WARPS + warp;
        const int v0 = min(mine * per, vecs), v1 = min(v0 + per, vecs);
        left.narrow(v0 * N, v1 * N);
        uint64_t hi = 0, lo = 0;
        for (int v = v0 + lane; v < v1; v += 32 * UNROLL) {
            uint4 pv[UNROLL], qv[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int at = v + 32 * i < v1 ? (v + 32 * i) * N : a.V;
                pv[i] = left.load(left.p, at);
                qv[i] = left.load_q(at);
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) left.add(pv[i], qv[i], (v + 32 * i) * N, hi, lo);
            const uint64_t h = add2(hi, lo);             // (lo stays below a last place of hi, however many there are)
            lo = sub2(lo, sub2(h, hi));
            hi = h;
        }
        const float2 h = unpair(hi), l = unpair(lo);
        const Two sum = warp_sum(Two{h.x, l.x} + Two{h.y, l.y});
        if (cluster > 1) {
            if (sm.pass == 0) cluster_wait_acquire();
            if (lane < cluster) st_cluster(mapa_shared(smem_u32(&sm.sum[turn][mine]), lane), sum);
            __syncwarp();
            cluster_sync_all();
        } else {
            if (lane == 0) sm.sum[turn][mine] = sum;
            __syncthreads();
        }
        // ---- all shares' sums, and the share that holds the drawn number
        if (warp == 0) {
            const int shares = cluster * WARPS, k = (shares + 31) / 32;      // lane l has shares l k .. l k + k - 1
            Two own = {0.f, 0.f}, total;
            for (int i = 0; i < k; ++i)
                if (lane * k + i < shares) own = own + sm.sum[turn][lane * k + i];
            Two at = warp_before(own, &total);
            const Two aim = times(total, u_last);
            int found = -1, some = -1;                   // the share; the last one that has anything
            Two before = at, before_some = at;
            for (int i = 0; i < k; ++i)
                if (lane * k + i < shares) {
                    const Two x = sm.sum[turn][lane * k + i];
                    if (x.hi > 0.f) {
                        some = lane * k + i;
                        before_some = at;
                        if (found < 0 && at + x > aim) {
                            found = some;
                            before = at;
                        }
                    }
                    at = at + x;
                }
            const uint32_t who = __ballot_sync(0xffffffffu, found >= 0), any = __ballot_sync(0xffffffffu, some >= 0);
            const int src = who ? __ffs(who) - 1 : any ? 31 - __clz(any) : 0;
            const int share = __shfl_sync(0xffffffffu, who ? found : some, src);
            const Two base = shuffle(who ? before : before_some, src);
            if (lane == 0) {
                if (sm.what == 1) sm.mass = wide(total);
                sm.share = any ? share : -1;
                sm.aim = aim + Two{-base.hi, -base.lo};
                ++sm.pass;
            }
        }
        __syncthreads();
        const bool walks = !whole && sm.what == 1, empty = sm.share < 0 && !whole && (sm.less > 0.0 || sm.fell > 0);
        if (!walks && !empty) break;
        whole = empty && !walks;
        __syncthreads();                                 // all have read what the next round writes
    }

    // ---- outputs
    const int stand = sm.stand;
    if (rank == 0) {
        for (int i = tid; i < a.max_q; i += THREADS) {
            path[i] = i <= stand ? q0 + sm.path[i] : -1;
            if (i != stand) out[i] = i < stand ? sm.row[sm.path[i + 1]].token : -1;
        }
        if (tid == 0) {
            a.count[b] = stand;
            if (sm.share < 0) out[stand] = -1;
        }
    }
    if (sm.share < 0 || sm.share / WARPS != rank) return;
    // The share again, neighbouring vectors a thread: the first x whose running sum passes the aim, or the last one with a weight.
    Left<X, DRAWN> left(a, sm, q0, whole);
    const int v0 = sm.share * per, v1 = min(v0 + per, vecs);
    left.narrow(v0 * N, v1 * N);
    const Two aim = sm.aim;
    Two base = {0.f, 0.f};
    int newest = -1;                                     // the last x with a weight so far
    for (int c = v0; c < v1; c += THREADS * LOOK) {
        const int v = c + tid * LOOK;
        uint4 pv[LOOK], qv[LOOK];
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            const int at = v + k < v1 ? (v + k) * N : a.V;
            pv[k] = left.load(left.p, at);
            qv[k] = left.load_q(at);
        }
        Two all, t[LOOK * N];
        int tail = -1, hit = INT32_MAX;
#pragma unroll
        for (int k = 0; k < LOOK; ++k) {
            float f[N], g[N];
            left.entries(pv[k], qv[k], (v + k) * N, f, g);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                t[k * N + i] = left.term(f[i], g[i]);
                if (t[k * N + i].hi > 0.f) tail = (v + k) * N + i;
            }
        }
#pragma unroll
        for (int o = 1; o < LOOK * N; o *= 2)            // (in pairs: a chain of sums takes 50 cycles each)
#pragma unroll
            for (int i = 0; i < LOOK * N; i += 2 * o) t[i] = t[i] + t[i + o];
        const Two own = t[0];
        Two r = warp_before(own, &all);
        __syncthreads();                                 // (the look before is read)
        if (lane == 0) sm.part[warp] = all;
        if (tid == 0) sm.what = INT32_MAX, sm.next = -1;
        __syncthreads();
        Two ahead = base;
        for (int i = 0; i < WARPS; ++i) {
            if (i == warp) r = ahead + r;
            ahead = ahead + sm.part[i];
        }
        base = ahead;
        if (r + own > aim || c + THREADS * LOOK >= v1) { // (its number may lie here)
#pragma unroll
            for (int k = 0; k < LOOK; ++k) {
                float f[N], g[N];
                left.entries(pv[k], qv[k], (v + k) * N, f, g);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const Two x = left.term(f[i], g[i]);
                    r = r + x;
                    if (hit == INT32_MAX && x.hi > 0.f && r > aim) hit = (v + k) * N + i;
                }
            }
        }
        if (hit != INT32_MAX) atomicMin(&sm.what, hit);
        if (tail >= 0) atomicMax(&sm.next, tail);
        __syncthreads();
        newest = max(newest, sm.next);
        if (sm.what != INT32_MAX) {
            newest = sm.what;
            break;
        }
    }
    if (tid == 0) out[stand] = newest;
}

template <class X, bool DRAWN>
cudaError_t run(const VerifyArgs& a, cudaStream_t s) {
    // CTAs of a sequence: twice as many, as long as the SMs hold them all at once, four each (but not four on every one, which clusters
    // do not fill: another wave of them would begin with its latencies again), and a warp's share keeps 64 vectors, or 128
    // where SMs have more than one.  Of 216 shapes (1 to 300 sequences over 2000 to 152064 entries) within 0.4 % of the best of 1,
    // 2, 4 and 8 CTAs on average, 14 % at worst (76 sequences over 32000 f32 entries 12.2 us with 4, 10.7 with 2): 64 chains over 152064
    // f32 entries 19.5 us with 8, 24.9 with 4; 152 over 8000 bf16 entries 8.0 with one, 15.1 with 4; one over 32000 7.4 with 8, 11.5 with one.
    const int64_t vecs = (a.V + VEC<X> - 1) / VEC<X>;
    int cluster = 1;
    for (int64_t ctas = 2LL * a.B; cluster < MAX_CLUSTER && ctas < 4 * num_sms() && vecs > (int64_t)cluster * WARPS * (ctas <= num_sms() ? 128 : 256); ctas *= 2)
        cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return counted(cudaLaunchKernelEx(&cfg, k_verify<X, DRAWN>, a, cluster));
}
template <class X>
cudaError_t run_as(const VerifyArgs& a, cudaStream_t s) { return a.Q ? run<X, true>(a, s) : run<X, false>(a, s); }

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
    if (a.pt == CQ_F16) return run_as<__half>(a, s);
    if (a.pt == CQ_BF16) return run_as<__nv_bfloat16>(a, s);
    return run_as<float>(a, s);
}

}  // namespace draft
}  // namespace cq

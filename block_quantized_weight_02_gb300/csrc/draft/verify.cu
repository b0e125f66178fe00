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
// A border of the drawn number may lie anywhere, so sums carry 2^-40 and better: each term is the exact difference
// in two floats, sums add the rounding errors that two floats lose (Knuth's two-sum), and the warps' sums are joined in 64
// bits.  (Sums in 64 bits throughout would take one warp instruction in 16 cycles of an SM.)
#include <cfloat>

#include "draft.cuh"

namespace cq {
namespace draft {
namespace {

constexpr int THREADS = 512, WARPS = THREADS / 32, MAX_CLUSTER = 16, MAX_ROWS = 1024;
constexpr int SHARES = MAX_CLUSTER * WARPS;

struct Row {
    int token, parent;     // parent: place in the sequence, or -1
    float p, q, u;         // the target's and the draft's probability of the token after its parent
};

struct Shared {
    double sum[2][SHARES]; // the cluster's shares, of even and odd passes
    double part[WARPS];    // of a look at one share
    double total, mass, less;
    int what, last, next, stand, fell, pass, share, bad;
    int path[MAX_ROWS];    // places of the rows that stand
    int gone[MAX_ROWS];    // rejected tokens that were not drawn
    Row row[MAX_ROWS];
};

// A positive finite number, or 0.
__device__ __forceinline__ float weight(float x) { return __float_as_uint(x) - 1u < 0x7F7FFFFFu ? x : 0.f; }

template <class X>
constexpr int VEC = 16 / (int)sizeof(X);
template <class X>
__device__ __forceinline__ void widen(uint4 v, float (&f)[VEC<X>]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(X) == 4) {
            f[i] = weight(__uint_as_float(w[i]));
        } else if constexpr (std::is_same<X, __half>::value) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = weight(p.x);
            f[2 * i + 1] = weight(p.y);
        } else {
            f[2 * i] = weight(__uint_as_float(w[i] << 16));
            f[2 * i + 1] = weight(__uint_as_float(w[i] & 0xFFFF0000u));
        }
    }
}
template <class X>
__device__ __forceinline__ float one(const X* p) {
    if constexpr (sizeof(X) == 4) return weight(__ldcg(p));
    else if constexpr (std::is_same<X, __half>::value) return weight(__half2float(__ldcg(p)));
    else return weight(__bfloat162float(__ldcg(p)));
}

struct Two {
    float hi, lo;
};
// max(p - a q, 0), a in two floats, to 2^-46 of the larger term.
__device__ __forceinline__ Two left_of(float p, float q, Two a) {
    const float t = __fmul_rn(q, a.hi), tl = fmaf(q, a.lo, fmaf(q, a.hi, -t));
    const float d = p - t, v = d - p;
    const float e = ((p - (d - v)) - (t + v)) - tl;
    const bool some = d + e > 0.f;
    return {some ? d : 0.f, some ? e : 0.f};
}
__device__ __forceinline__ void add(Two& s, Two x) {
    const float t = s.hi + x.hi, v = t - s.hi;
    s.lo += ((s.hi - (t - v)) + (x.hi - v)) + x.lo;
    s.hi = t;
}

// Terms of one vector of a row: elements from `at` on.  A row's last vector may be a part of one, of which nothing past
// the row is read.
template <class X, bool DRAWN>
struct Left {
    const X *p, *q;
    Two a;
    bool less;             // a > 0
    int V, ngone;
    const int* gone;
    __device__ __forceinline__ uint4 load(const X* r, int at) const {
        if (at + VEC<X> <= V) return __ldcg(reinterpret_cast<const uint4*>(r + at));
        uint32_t w[4] = {0, 0, 0, 0};
        if (at < V)
#pragma unroll
            for (int i = 0; i < VEC<X>; ++i)
                if (at + i < V) {
                    if constexpr (sizeof(X) == 4) w[i] = __ldcg(reinterpret_cast<const uint32_t*>(r + at) + i);
                    else w[i / 2] |= (uint32_t)__ldcg(reinterpret_cast<const uint16_t*>(r + at) + i) << 16 * (i & 1);
                }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void terms(uint4 pv, uint4 qv, int at, Two (&w)[VEC<X>]) const {
        constexpr int N = VEC<X>;
        float f[N], g[N];
        widen<X>(pv, f);
        if (DRAWN) widen<X>(qv, g);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = DRAWN && less ? left_of(f[i], g[i], a) : Two{f[i], 0.f};
        if (!DRAWN)
            for (int k = 0; k < ngone; ++k)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (gone[k] == at + i) w[i] = {0.f, 0.f};
    }
};

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ double warp_scan(double x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double x) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(x) : "memory");
}

template <class X, bool DRAWN>
__global__ void __launch_bounds__(THREADS) k_verify(const VerifyArgs a, int cluster) {
    constexpr int N = VEC<X>;
    __shared__ Shared sm;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int q0 = __ldcg(a.q_start + b), n = __ldcg(a.q_start + b + 1) - q0;
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
    // every CTA of the cluster has begun before another writes to it
    if (cluster > 1) cluster_sync_all();

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
                if (DRAWN) {
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
                    stands = r.u * mass < w;
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
        const double less = whole ? 0.0 : sm.less;
        Left<X, DRAWN> left = {P + sm.last * a.ldp, DRAWN ? Q + sm.last * a.ldq : nullptr, {(float)less, (float)(less - (double)(float)less)},
                               less > 0.0, a.V, whole ? 0 : sm.fell, sm.gone};
        const int mine = rank * WARPS + warp;
        const int v0 = min(mine * per, vecs), v1 = min(v0 + per, vecs);
        Two s = {0.f, 0.f};
        constexpr int UN = 4;
        for (int v = v0 + lane; v < v1; v += 32 * UN) {
            uint4 pv[UN], qv[UN];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int at = v + 32 * i < v1 ? (v + 32 * i) * N : a.V;
                pv[i] = left.load(left.p, at);
                qv[i] = DRAWN && left.less ? left.load(left.q, at) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                Two w[N];
                left.terms(pv[i], qv[i], v + 32 * i < v1 ? (v + 32 * i) * N : a.V, w);
#pragma unroll
                for (int k = 0; k < N; ++k) add(s, w[k]);
            }
        }
        const double sum = warp_sum((double)s.hi + (double)s.lo);
        if (cluster > 1) {
            if (lane < cluster) st_cluster_f64(mapa_shared(smem_u32(&sm.sum[turn][mine]), lane), sum);
            cluster_sync_all();
        } else {
            if (lane == 0) sm.sum[turn][mine] = sum;
            __syncthreads();
        }
        // ---- all shares' sums, and the share that holds the drawn number
        if (warp == 0) {
            const int shares = cluster * WARPS;          // lane l has shares l k .. l k + k - 1
            const int k = (shares + 31) / 32;
            double own = 0.0;
            for (int i = 0; i < k; ++i)
                if (lane * k + i < shares) own += sm.sum[turn][lane * k + i];
            const double upto = warp_scan(own), total = __shfl_sync(0xffffffffu, upto, 31);
            const double aim = (double)__ldcg(a.u_last + b) * total;
            double at = upto - own;
            int found = -1, some = -1;
            double before = 0.0, before_some = 0.0;
            for (int i = 0; i < k; ++i)
                if (lane * k + i < shares) {
                    const double x = sm.sum[turn][lane * k + i];
                    if (x > 0.0) {
                        some = lane * k + i;
                        before_some = at;
                        if (found < 0 && at + x > aim) {
                            found = some;
                            before = at;
                        }
                    }
                    at += x;
                }
            const uint32_t who = __ballot_sync(0xffffffffu, found >= 0), any = __ballot_sync(0xffffffffu, some >= 0);
            const int src = who ? __ffs(who) - 1 : any ? 31 - __clz(any) : 0;
            const int share = __shfl_sync(0xffffffffu, who ? found : some, src);
            const double base = __shfl_sync(0xffffffffu, who ? before : before_some, src);
            if (lane == 0) {
                if (sm.what == 1) sm.mass = total;
                sm.share = any ? share : -1;
                sm.total = aim - base;                   // what is to be passed within the share
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
    // The share again, a vector a thread: the first x whose running sum passes the aim, or the last one with a weight.
    const double less = whole ? 0.0 : sm.less;
    Left<X, DRAWN> left = {P + sm.last * a.ldp, DRAWN ? Q + sm.last * a.ldq : nullptr, {(float)less, (float)(less - (double)(float)less)},
                           less > 0.0, a.V, whole ? 0 : sm.fell, sm.gone};
    const int v0 = sm.share * per, v1 = min(v0 + per, vecs);
    double aim = sm.total;
    int newest = -1;                                     // the last x with a weight so far
    for (int c = v0; c < v1; c += THREADS) {
        const int v = c + tid, at = v < v1 ? v * N : a.V;
        Two w[N];
        left.terms(left.load(left.p, at), DRAWN && left.less ? left.load(left.q, at) : make_uint4(0, 0, 0, 0), at, w);
        double own = 0.0;
        int tail = -1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            own += (double)w[i].hi + (double)w[i].lo;
            if (w[i].hi + w[i].lo > 0.f) tail = at + i;
        }
        const double upto = warp_scan(own);
        __syncthreads();                                 // (the look before is read)
        if (lane == 31) sm.part[warp] = upto;
        if (tid == 0) sm.what = INT32_MAX, sm.next = -1;
        __syncthreads();
        double run = upto - own, all = 0.0;
        for (int i = 0; i < WARPS; ++i) {
            if (i < warp) run += sm.part[i];
            all += sm.part[i];
        }
        int hit = INT32_MAX;
        double r = run;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double x = (double)w[i].hi + (double)w[i].lo;
            r += x;
            if (hit == INT32_MAX && x > 0.0 && r > aim) hit = at + i;
        }
        if (hit != INT32_MAX) atomicMin(&sm.what, hit);
        if (tail >= 0) atomicMax(&sm.next, tail);
        __syncthreads();
        newest = max(newest, sm.next);
        if (sm.what != INT32_MAX) {
            newest = sm.what;
            break;
        }
        aim -= all;
    }
    if (tid == 0) out[stand] = newest;
}

template <class X, bool DRAWN>
cudaError_t run(const VerifyArgs& a, cudaStream_t s) {
    // CTAs of a sequence: enough for every SM to have one, as long as a warp's share keeps 32 vectors
    const int64_t vecs = (a.V + VEC<X> - 1) / VEC<X>;
    int cluster = 1;
    while (cluster < MAX_CLUSTER && cluster * a.B < num_sms() && vecs >= (int64_t)cluster * 2 * WARPS * 32) cluster *= 2;
    if (cluster > 8) {
        const cudaError_t e = cudaFuncSetAttribute(k_verify<X, DRAWN>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
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

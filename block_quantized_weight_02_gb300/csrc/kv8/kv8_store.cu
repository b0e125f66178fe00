// Writing keys and values to the 8-bit cache, and reading them back.
//
// Both are one pass over the data and bound by HBM.  The unit of work is one block
// of 32 tokens of one head of the keys or of the values, and one warp takes it: it
// has the whole block in registers (up to 32 loads of 16 bytes a lane in flight),
// takes the largest magnitude with shuffles, and stores the codes, so no shared
// memory, barrier or second pass is needed.  Consecutive warps take consecutive
// heads, whose rows are neighbours in the token-major tensors.
//
// Measured: four documents of 32768 tokens written and read back in bf16 (8 heads of 128 channels) take 275 us for
// the two calls, 5.9 TB/s.
//
// Sequences are ragged and only the device knows their lengths, so the grid covers
// the most blocks that T rows of B sequences can touch: sequence b owns the slots
// floor(q_start[b] / 32) + 2 b .., since n rows touch at most floor(n / 32) + 2
// blocks; a warp finds its sequence by a 32-way search and leaves if its slot is
// one too many.
#include "kv8.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int WARPS = 4;

// Exponent of the scale: the smallest e >= -64 with a <= 127 * 2^e.  127 = 1.984375 * 2^6,
// so the mantissa field's distance to the next power carries into the exponent exactly
// when a's mantissa is above 1.984375.
__device__ __forceinline__ int scale_exp(float a) {
    return max((int)((__float_as_uint(a) + 0x1FFFFu) >> 23) - 127 - 6, -64);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// x / 2^e rounded to the nearest integer, ties to even, in the low byte: the product is
// exact and the sum with 1.5 * 2^23 rounds once.
__device__ __forceinline__ uint32_t code_of(float x, float inv) {
    return __float_as_uint(fmaf(x, inv, 12582912.0f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
}
__device__ __forceinline__ float byte_f(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

template <class X>
struct In;   // 16 bytes of a row
template <>
struct In<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(uint4 u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <>
struct In<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct In<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(uint4 u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// One block of one head: which rows, where in the cache.
struct Item {
    int kv, head;
    int row0;        // tensor row of the block's row `lo`
    int lo, hi;      // block rows that the call writes or reads
    int64_t block;   // global block number: the scale's index; the codes start at block * 32 * D
    bool ok;
};

// Sequence b's tokens [first, last) that the call writes or reads; false if an entry is out of range.
template <bool WRITE>
__device__ __forceinline__ bool tokens_of(const Cache& c, const Batch& b, int seq, int& qs, int64_t& first,
                                          int64_t& last) {
    qs = __ldg(b.q_start + seq);
    const int qe = __ldg(b.q_start + seq + 1), n = qe - qs;
    if (WRITE) {
        last = __ldg(b.lens + seq);
        first = last - n;
    } else {
        first = b.first ? __ldg(b.first + seq) : 0;
        last = first + n;
    }
    return rows_ok(qs, qe, b.T, b.T) && first >= 0 && last <= c.ldt * c.page;
}

// The warp's item: (slot, head, keys or values) with the head running fastest.
// The first block also looks at every sequence's entries: a warp's search need not
// come past a wrong one.
template <bool WRITE>
__device__ __forceinline__ Item find_item(const Cache& c, const Batch& b) {
    Item it;
    it.ok = false;
    int64_t w = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    it.head = (int)(w % c.Hkv);
    w /= c.Hkv;
    it.kv = (int)(w & 1);
    const int64_t slot = w >> 1;
    auto start = [&](int i) { return (int64_t)(__ldg(b.q_start + i) >> 5) + 2 * i; };
    const int seq = warp_find(c.B, slot, start);
    int qs;
    int64_t first, last;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < c.B; i += WARPS * 32)
            if (!tokens_of<WRITE>(c, b, i, qs, first, last)) set_err(b.err, DEV_INDEX);
    if (!tokens_of<WRITE>(c, b, seq, qs, first, last)) return it;
    const int64_t blk = first / BLK + (slot - start(seq));
    if (first == last || slot < start(seq) || blk * BLK >= last) return it;
    const int pid = __ldg(c.table + seq * c.ldt + blk * BLK / c.page);
    if (pid < 0 || pid >= c.pages) {
        if ((threadIdx.x & 31) == 0) set_err(b.err, DEV_INDEX);
        return it;
    }
    it.lo = (int)max((int64_t)0, first - blk * BLK);
    it.hi = (int)min((int64_t)BLK, last - blk * BLK);
    it.row0 = (int)(qs + (blk * BLK + it.lo - first));
    it.block = ((int64_t)pid * c.Hkv + it.head) * (c.page / BLK) + (blk * BLK % c.page) / BLK;
    it.ok = true;
    return it;
}

template <class X, int D>
__global__ void __launch_bounds__(WARPS * 32) k_kv8_write(const Cache c, const Batch b, const X* K, const X* V,
                                                          int64_t ldk, int64_t ldv) {
    pdl_launch_dependents();
    pdl_wait();
    const Item it = find_item<true>(c, b);
    if (!it.ok) return;
    constexpr int N = In<X>::N, LPR = D / N, RPI = 32 / LPR, IT = BLK / RPI;   // lanes a row, rows a step
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, col = (lane % LPR) * N;
    const int64_t ld = it.kv ? ldv : ldk;
    const X* src = (it.kv ? V : K) + it.row0 * ld + (int64_t)it.head * D + col;
    uint4 u[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub;
        u[i] = make_uint4(0, 0, 0, 0);
        if (r >= it.lo && r < it.hi) u[i] = __ldcs(reinterpret_cast<const uint4*>(src + (r - it.lo) * ld));
    }
    float* sp = c.s[it.kv] + it.block;
    const float s0 = it.lo > 0 ? *sp : 0.f;
    // largest magnitude, as bits: an infinity or NaN is larger than every finite value
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        float f[N];
        In<X>::get(u[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const bool bad = m >= 0x7F800000u || s0 != s0;
    const float s1 = bad ? __uint_as_float(0x7FC00000u) : fmaxf(s0, pow2(scale_exp(__uint_as_float(m))));
    const float inv = bad ? 0.f : 1.0f / s1;      // exact: a power of two
    int8_t* dst = c.q[it.kv] + it.block * (BLK * D) + col;
    if (it.lo > 0 && s1 > s0) {                   // the kept codes move to the larger scale
        const float ratio = s0 * inv;
        for (int i = 0; i < IT; ++i) {
            const int r = i * RPI + sub;
            if (r < it.lo) {
                uint32_t* p = reinterpret_cast<uint32_t*>(dst + r * D);
#pragma unroll
                for (int j = 0; j < N / 4; ++j) {
                    const uint32_t w = p[j];
                    p[j] = pack4(code_of(byte_f(w, 0), ratio), code_of(byte_f(w, 1), ratio),
                                 code_of(byte_f(w, 2), ratio), code_of(byte_f(w, 3), ratio));
                }
            }
        }
    }
    __syncwarp();   // every lane has read the old scale
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub;
        float f[N];
        In<X>::get(u[i], f);
        uint32_t w[N / 4];
#pragma unroll
        for (int j = 0; j < N / 4; ++j)
            w[j] = bad ? 0u
                       : pack4(code_of(f[4 * j], inv), code_of(f[4 * j + 1], inv), code_of(f[4 * j + 2], inv),
                               code_of(f[4 * j + 3], inv));
        if (r >= it.lo && r < it.hi) {
            if constexpr (N == 8) *reinterpret_cast<uint2*>(dst + r * D) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t*>(dst + r * D) = w[0];
        }
    }
    if (lane == 0) *sp = s1;
}

template <class Y, int D>
__global__ void __launch_bounds__(WARPS * 32) k_kv8_read(const Cache c, const Batch b, Y* K, Y* V, int64_t ldk,
                                                         int64_t ldv) {
    pdl_launch_dependents();
    pdl_wait();
    const Item it = find_item<false>(c, b);
    if (!it.ok) return;
    constexpr int N = In<Y>::N, LPR = D / N, RPI = 32 / LPR, IT = BLK / RPI;
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, col = (lane % LPR) * N;
    const int64_t ld = it.kv ? ldv : ldk;
    Y* dst = (it.kv ? V : K) + it.row0 * ld + (int64_t)it.head * D + col;
    const int8_t* src = c.q[it.kv] + it.block * (BLK * D) + col;
    const float s = c.s[it.kv][it.block];
    uint2 u[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub;
        u[i] = make_uint2(0, 0);
        if (r >= it.lo && r < it.hi) {
            if constexpr (N == 8) u[i] = *reinterpret_cast<const uint2*>(src + r * D);
            else u[i].x = *reinterpret_cast<const uint32_t*>(src + r * D);
        }
    }
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + sub;
        float f[N];
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] = byte_f(j < 4 ? u[i].x : u[i].y, j & 3) * s;
        if (r >= it.lo && r < it.hi) __stcs(reinterpret_cast<uint4*>(dst + (r - it.lo) * ld), In<Y>::put(f));
    }
}

dim3 store_grid(const Cache& c, const Batch& b) {
    const int64_t slots = b.T / BLK + 2 * (int64_t)c.B;
    return dim3((unsigned)((slots * c.Hkv * 2 + WARPS - 1) / WARPS));
}

template <class X>
cudaError_t write_as(const Cache& c, const Batch& b, int D, const void* K, const void* V, int64_t ldk, int64_t ldv,
                     cudaStream_t s) {
    const X *k = static_cast<const X*>(K), *v = static_cast<const X*>(V);
    if (D == 128) return launch_pdl(k_kv8_write<X, 128>, store_grid(c, b), dim3(WARPS * 32), 0, s, c, b, k, v, ldk, ldv);
    return launch_pdl(k_kv8_write<X, 64>, store_grid(c, b), dim3(WARPS * 32), 0, s, c, b, k, v, ldk, ldv);
}
template <class Y>
cudaError_t read_as(const Cache& c, const Batch& b, int D, void* K, void* V, int64_t ldk, int64_t ldv,
                    cudaStream_t s) {
    Y *k = static_cast<Y*>(K), *v = static_cast<Y*>(V);
    if (D == 128) return launch_pdl(k_kv8_read<Y, 128>, store_grid(c, b), dim3(WARPS * 32), 0, s, c, b, k, v, ldk, ldv);
    return launch_pdl(k_kv8_read<Y, 64>, store_grid(c, b), dim3(WARPS * 32), 0, s, c, b, k, v, ldk, ldv);
}

}  // namespace

cudaError_t launch_write(const Cache& c, const Batch& b, int D, const void* K, const void* V, int xt, int64_t ldk,
                         int64_t ldv, cudaStream_t s) {
    if (xt == CQ_F16) return write_as<__half>(c, b, D, K, V, ldk, ldv, s);
    if (xt == CQ_BF16) return write_as<__nv_bfloat16>(c, b, D, K, V, ldk, ldv, s);
    return write_as<float>(c, b, D, K, V, ldk, ldv, s);
}
cudaError_t launch_read(const Cache& c, const Batch& b, int D, void* K, void* V, int yt, int64_t ldk, int64_t ldv,
                        cudaStream_t s) {
    if (yt == CQ_F16) return read_as<__half>(c, b, D, K, V, ldk, ldv, s);
    if (yt == CQ_BF16) return read_as<__nv_bfloat16>(c, b, D, K, V, ldk, ldv, s);
    return read_as<float>(c, b, D, K, V, ldk, ldv, s);
}

}  // namespace kv8
}  // namespace cq

// Writing keys and values to the 8-bit cache, and reading them back.
//
// Both are one pass over the data and bound by HBM.  The unit of work is one block
// of 32 tokens of one head of the keys or of the values, and one warp takes it: it
// has the whole block in registers (up to 32 loads of 16 bytes a lane in flight),
// takes the largest magnitude with shuffles, and stores the codes, so no shared
// memory, barrier or second pass is needed.  Consecutive warps take consecutive
// heads, whose rows are neighbours in the token-major tensors.
//
// Measured: four documents of 32768 tokens written and read back in bf16 (8 heads of 128 channels) take 265 us for
// the two calls, 6.1 TB/s.
#include "store_common.cuh"

namespace cq {
namespace kv8 {
namespace {

constexpr int WARPS = 4;

// The warp's item: (slot, head, keys or values) with the head running fastest.
template <bool WRITE>
__device__ __forceinline__ Item my_item(const Cache& c, const Batch& b) {
    int64_t w = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
    const int head = (int)(w % c.Hkv);
    w /= c.Hkv;
    return find_item<WRITE>(c, b, w >> 1, (int)(w & 1), head);
}

// A warp stores block `it` and its scale: u holds this lane's channels of rows i RPI + lane / LPR, 0 in rows that are not the call's.
// (A function of its own takes up to 24 registers less than the same lines in the kernel, which wrote four prompts of 16000 to
// 16384 tokens, 8 heads of 128 channels, in 90 us for 79 (fp16), 75 for 73 (bf16).)
template <class X, int D>
__device__ __forceinline__ void store_block(const Cache& c, const Item& it, const uint4 (&u)[BLK * D / In<X>::N / 32]) {
    constexpr int N = In<X>::N, LPR = D / N, RPI = 32 / LPR, IT = BLK / RPI;   // lanes a row, rows a step
    const int lane = threadIdx.x & 31, sub = lane / LPR, col = (lane % LPR) * N;
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

template <class X, int D>
__global__ void __launch_bounds__(WARPS * 32) k_kv8_write(const Cache c, const Batch b, const X* K, const X* V,
                                                          int64_t ldk, int64_t ldv) {
    pdl_launch_dependents();
    pdl_wait();
    const Item it = my_item<true>(c, b);
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
    store_block<X, D>(c, it, u);
}

template <class Y, int D>
__global__ void __launch_bounds__(WARPS * 32) k_kv8_read(const Cache c, const Batch b, Y* K, Y* V, int64_t ldk,
                                                         int64_t ldv) {
    pdl_launch_dependents();
    pdl_wait();
    const Item it = my_item<false>(c, b);
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
    return dim3((unsigned)((store_slots(c, b) * c.Hkv * 2 + WARPS - 1) / WARPS));
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

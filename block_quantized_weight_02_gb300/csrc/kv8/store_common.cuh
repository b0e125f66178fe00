// What writing to the 8-bit cache and reading from it share: scales and codes, rows as
// vectors of 16 bytes, and where a block of a ragged batch lies.
//
// Sequences are ragged and only the device knows their lengths, so a grid covers
// the most blocks that T rows of B sequences can touch: sequence b owns the slots
// floor(q_start[b] / 32) + 2 b .., since n rows touch at most floor(n / 32) + 2
// blocks; a warp finds its sequence by a 32-way search and leaves if its slot is
// one too many.
#pragma once
#include "kv8.cuh"

namespace cq {
namespace kv8 {
namespace {

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
    int tok0;        // and its place in the sequence
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

// Head `head` of the keys (kv 0) or values (1) of the block in a slot.
// The first block of the grid also looks at every sequence's entries: a warp's search need not
// come past a wrong one.
template <bool WRITE>
__device__ __forceinline__ Item find_item(const Cache& c, const Batch& b, int64_t slot, int kv, int head) {
    Item it;
    it.ok = false;
    it.kv = kv;
    it.head = head;
    auto start = [&](int i) { return (int64_t)(__ldg(b.q_start + i) >> 5) + 2 * i; };
    const int seq = warp_find(c.B, slot, start);
    int qs;
    int64_t first, last;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < c.B; i += blockDim.x)
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
    it.tok0 = (int)(blk * BLK + it.lo);
    it.block = ((int64_t)pid * c.Hkv + it.head) * (c.page / BLK) + (blk * BLK % c.page) / BLK;
    it.ok = true;
    return it;
}

inline int64_t store_slots(const Cache& c, const Batch& b) { return b.T / BLK + 2 * (int64_t)c.B; }

}  // namespace
}  // namespace kv8
}  // namespace cq

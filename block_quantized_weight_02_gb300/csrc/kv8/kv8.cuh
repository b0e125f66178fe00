// Shared declarations of the 8-bit key/value cache: the cache as kernels see
// it, the ragged batch's bookkeeping, and the launchers of its translation units.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "../../../include/cq_kv8.h"
#include "../cq_internal.h"
#include "../cq_ptx.cuh"
#include "f32x2.cuh"

namespace cq {
namespace kv8 {

constexpr int BLK = CQ_KV8_BLOCK;   // tokens per scale

struct Cache {
    int8_t* q[2];          // keys, values
    float* s[2];
    const int32_t* table;
    int64_t ldt;
    int pages, Hkv, page, B;
};

// One ragged batch: rows q_start[b] .. of sequence b, its length and the device error word.
struct Batch {
    const int32_t* q_start;
    const int32_t* lens;   // tokens held (write, attention)
    const int32_t* first;  // read back: first token (nullable)
    int T;
    int* err;
};

struct AttnArgs {
    Cache c;
    Batch b;
    const void* Q;
    void* O;
    float* lse;
    int64_t ldq, ldo;
    int xt, yt, Hq, D, max_q, causal;
    int64_t window;
    float scale;
    void* ws;
    int stall;             // test only: copies are left out (few rows: all; else all but a CTA's first tile), so that a wait runs out
    const uint32_t* mask;  // trees: which of a sequence's last tokens its rows see, ldm words a row (causal = 0 and no window then)
    int64_t ldm;
};

cudaError_t launch_write(const Cache& c, const Batch& b, int D, const void* K, const void* V, int xt, int64_t ldk,
                         int64_t ldv, cudaStream_t s);
cudaError_t launch_read(const Cache& c, const Batch& b, int D, void* K, void* V, int yt, int64_t ldk, int64_t ldv,
                        cudaStream_t s);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_tree(const AttnArgs& a, cudaStream_t s);   // with a mask
bool decode_serves(int64_t rows);                     // rows: query rows of a sequence that share a KV head
size_t decode_workspace(int64_t D);
cudaError_t launch_decode(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_decode_tree(const AttnArgs& a, cudaStream_t s);
bool narrow_serves(int64_t rows);
size_t narrow_workspace(int64_t T, int64_t G, int64_t D, int64_t B);
cudaError_t launch_narrow(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_narrow_tree(const AttnArgs& a, cudaStream_t s);
size_t tiles_workspace(int64_t T, int64_t G, int64_t D, int64_t B, int64_t max_q);
cudaError_t launch_tiles(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_tiles_tree(const AttnArgs& a, cudaStream_t s);
size_t attn_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q);        // of a call
size_t attn_workspace_upto(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q);   // and of any smaller one

// A kernel that starts under the ones before it.  What those may have written (queries, codes, scales, the workspace) is read
// after pdl_wait() and not through the read-only path (__ldg), which is for data that no kernel writes while this one runs;
// q_start, lens and the table come from the caller.
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return counted(cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...));
}

// First writer wins.
__device__ __forceinline__ void set_err(int* err, int code) { atomicCAS(err, 0, code); }

// The largest b in [0, B) with key(b) <= x, for an ascending key with key(0) <= x: the
// warp's 32 lanes probe 32 places at a time (one round of loads up to 32 sequences, two
// up to 1024).  Whatever the keys hold, the result is in [0, B).
template <class Key>
__device__ __forceinline__ int warp_find(int B, int64_t x, Key key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;                              // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane == 0 || (at < lo + n && key(at) <= x);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));
        const int end = min(lo + n, lo + (k + 1) * step);
        lo += k * step;
        n = end - lo;
    }
    return lo;
}

// A length that attention takes: its pages are in the table, and the tokens that a kernel looks up ahead of it (up to 1024
// past the last) have 31-bit numbers.
constexpr int MAX_LEN = INT32_MAX - 2047;
__device__ __forceinline__ bool length_ok(const Cache& c, int L) { return L >= 0 && L <= MAX_LEN && L <= c.ldt * c.page; }

// A ragged batch's entry b: rows [qs, qe) in [0, T], at most max_rows of them.
__device__ __forceinline__ bool rows_ok(int qs, int qe, int T, int max_rows) {
    return qs >= 0 && qe >= qs && qe <= T && qe - qs <= max_rows;
}

}  // namespace kv8
}  // namespace cq

// Attention over the 8-bit cache: one warp per query row and head, a softmax with a
// running maximum and sum over blocks of 32 tokens.
#include "kv8.cuh"

namespace cq {
namespace kv8 {
namespace {

__device__ __forceinline__ float load_f(const void* p, int64_t i, int t) {
    if (t == CQ_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_f(void* p, int64_t i, int t, float v) {
    if (t == CQ_F32) static_cast<float*>(p)[i] = v;
    else if (t == CQ_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <int D>
__global__ void __launch_bounds__(128) k_attn_rows(const AttnArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.c.B; i += 128) {
            const int n = __ldg(a.b.lens + i);
            if (!rows_ok(__ldg(a.b.q_start + i), __ldg(a.b.q_start + i + 1), a.b.T, a.max_q) || n < 0 || n > a.c.ldt * a.c.page)
                set_err(a.b.err, DEV_INDEX);
        }
    const int64_t w = (int64_t)blockIdx.x * 4 + warp;
    const int row = (int)(w / a.Hq), h = (int)(w % a.Hq), hk = h / (a.Hq / a.c.Hkv);
    if (row >= a.b.T) return;
    const int seq = warp_find(a.c.B, row, [&](int i) { return (int64_t)__ldg(a.b.q_start + i); });
    const int q0 = __ldg(a.b.q_start + seq), q1 = __ldg(a.b.q_start + seq + 1), len = __ldg(a.b.lens + seq);
    if (row < q0 || row >= q1) return;
    if (!rows_ok(q0, q1, a.b.T, a.max_q) || len < 0 || len > a.c.ldt * a.c.page) return;
    const int64_t pos = (int64_t)len - (q1 - q0) + (row - q0);
    const int64_t hi = a.causal ? pos + 1 : len;
    const int64_t lo = a.window ? max((int64_t)0, pos - a.window + 1) : 0;
    for (int d = lane; d < D; d += 32) qs[warp][d] = load_f(a.Q, row * a.ldq + (int64_t)h * D + d, a.xt);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[D / 32];
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    for (int64_t t0 = lo / BLK * BLK; t0 < hi; t0 += BLK) {
        const int pid = __ldg(a.c.table + seq * a.c.ldt + t0 / a.c.page);
        if (pid < 0 || pid >= a.c.pages) {
            if (lane == 0) set_err(a.b.err, DEV_INDEX);
            return;
        }
        const int64_t blk = ((int64_t)pid * a.c.Hkv + hk) * (a.c.page / BLK) + t0 % a.c.page / BLK;
        const bool in = t0 + lane >= lo && t0 + lane < hi;
        float s = -INFINITY;
        if (in) {
            const int8_t* k = a.c.q[0] + (blk * BLK + lane) * D;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot += qs[warp][d] * (float)k[d];
            s = dot * (a.c.s[0][blk] * a.scale);
        }
        float bm = s;
        for (int o = 16; o; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
        const float mn = fmaxf(m, bm);
        const float p = in ? expf(s - mn) : 0.f, f = m == mn ? 1.f : expf(m - mn);
        float ps = p;
        for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l = l * f + ps;
        m = mn;
        const float sv = a.c.s[1][blk];
        for (int i = 0; i < D / 32; ++i) acc[i] *= f;
        for (int j = 0; j < BLK; ++j) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
            if (t0 + j < lo || t0 + j >= hi) continue;
            const int8_t* v = a.c.q[1] + (blk * BLK + j) * D;
            for (int i = 0; i < D / 32; ++i) acc[i] += pj * sv * (float)v[lane + 32 * i];
        }
    }
    for (int i = 0; i < D / 32; ++i)
        store_f(a.O, row * a.ldo + (int64_t)h * D + lane + 32 * i, a.yt, hi > lo ? acc[i] / l : 0.f);
    if (a.lse && lane == 0) a.lse[(int64_t)row * a.Hq + h] = hi > lo ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t attn_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t, int64_t max_q) {
    if (decode_serves(std::min(max_q, T) * (Hq / Hkv))) return decode_workspace(D);
    return 256;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    if (decode_serves((int64_t)a.max_q * (a.Hq / a.c.Hkv))) return launch_decode(a, s);
    const dim3 grid((unsigned)(((int64_t)a.b.T * a.Hq + 3) / 4));
    if (a.D == 128) return launch_pdl(k_attn_rows<128>, grid, dim3(128), 0, s, a);
    return launch_pdl(k_attn_rows<64>, grid, dim3(128), 0, s, a);
}

}  // namespace kv8
}  // namespace cq

// The C entry points of the 8-bit key/value cache: argument checks and launches.
#include "kv8_checks.h"

using namespace cq;
using namespace cq::kv8;

extern "C" {

cq_status cq_kv8_write(const cq_kv8_cache* cache, const void* K, const void* V, int xt, int64_t T, int64_t ldk,
                       int64_t ldv, const int32_t* q_start, const int32_t* lens, void* stream) {
    clear_last_error();
    if (!lens) return fail(CQ_ERR_NULL, "cq_kv8_write: null pointer");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Cache c;
    int* err = nullptr;
    cq_status st = check_store("cq_kv8_write", cache, &c, K, V, xt, T, ldk, ldv, q_start, lens, s, &err);
    if (st) return st;
    const Batch b = {q_start, lens, nullptr, (int)T, err};
    return launched(launch_write(c, b, (int)cache->D, K, V, xt, ldk, ldv, s), "cache write");
}

cq_status cq_kv8_read(const cq_kv8_cache* cache, const int32_t* first, const int32_t* out_start, void* K, void* V,
                      int yt, int64_t T, int64_t ldk, int64_t ldv, void* stream) {
    clear_last_error();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Cache c;
    int* err = nullptr;
    cq_status st = check_store("cq_kv8_read", cache, &c, K, V, yt, T, ldk, ldv, out_start, first, s, &err);
    if (st) return st;
    const Batch b = {out_start, nullptr, first, (int)T, err};
    return launched(launch_read(c, b, (int)cache->D, K, V, yt, ldk, ldv, s), "cache read-back");
}

size_t cq_attn_kv8_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    if (T < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || D < 1 || B < 1 || max_q < 1) return 0;
    return attn_workspace_upto(T, Hq, Hkv, D, B, max_q);
}

cq_status cq_attn_kv8(const void* Q, int xt, int64_t T, int64_t Hq, int64_t ldq, const cq_kv8_cache* cache,
                      const int32_t* q_start, const int32_t* lens, int64_t max_q, float scale, int causal,
                      int64_t window, void* O, int yt, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                      void* stream) {
    const char* who = "cq_attn_kv8";
    clear_last_error();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnArgs a;
    cq_status st = attn_args(who, Q, xt, T, Hq, ldq, cache, q_start, lens, max_q, scale, causal, window, O, yt, ldo, lse, ws, ws_bytes, s, &a);
    if (st) return st;
    a.stall = (int)options().test_stall.exchange(0);
    return launched(launch_attn(a, s), "attention");
}

}  // extern "C"

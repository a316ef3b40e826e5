// What the attention kernels (fp8blk_attn.hip, fp8blk_latent.hip) share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {

struct AttnArgs {
    const char* k;
    const char* v;
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // bytes
    const char* q;
    char* out;
    int64_t q_token, q_head, out_token, out_head;  // bytes
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    const float* sinks;
    float* ws;
    int64_t max_pages;
    int32_t N, seqs, heads, group;  // group: heads that share a key head
    int32_t pages, page_shift;
    int32_t max_new, window, causal;
    float z_scale;    // scale * k_scale * log2(e): weights are powers of 2
    float out_scale;  // v_scale
};

constexpr float kLog2e = 1.44269504088896340736f;

// A sequence's rows and keys as a call gives them, cut to what exists.
struct Seq {
    int32_t first, rows;  // its new tokens among the rows of q
    int32_t keys;         // keys that its table holds
    int32_t at;           // position of its first new token (below 0: more new tokens than keys)
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int s) {
    Seq q;
    const int32_t b = a.starts[s], e = a.starts[s + 1], len = max(a.lens[s], 0);
    q.first = min(max(b, 0), a.N);
    q.rows = max(min(e, a.N) - q.first, 0);
    const int64_t held = a.max_pages << a.page_shift;
    q.keys = len < held ? len : (int32_t)held;
    q.at = len - q.rows;
    q.rows = min(q.rows, a.max_new);
    return q;
}

// The keys that the row at position p sees: [lo, hi).
__device__ __forceinline__ int first_key(const AttnArgs& a, int p) { return a.window > 0 ? max(p - a.window + 1, 0) : 0; }
__device__ __forceinline__ int end_key(const AttnArgs& a, const Seq& s, int p) {
    return a.causal ? min(max(p + 1, 0), s.keys) : s.keys;
}

// The page that holds key j, -1 if none does. j is inside the table.
__device__ __forceinline__ int page_of(const AttnArgs& a, int s, int j) {
    const int p = a.table[(int64_t)s * a.max_pages + (j >> a.page_shift)];
    return (uint32_t)p < (uint32_t)a.pages ? p : -1;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Checks the arguments of an attention call and writes its AttnArgs (the workspace
// apart); FP8BLK_OK or what the call returns.
int attn_args(AttnArgs& a, const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
              int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window, const float* sinks,
              uint16_t* out, int64_t out_token, int64_t out_head);

}  // namespace fp8blk

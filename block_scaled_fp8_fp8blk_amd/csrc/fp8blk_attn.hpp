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
    float z_scale;    // |scale| * k_scale * log2(e): weights are powers of 2
    float out_scale;  // v_scale
    uint32_t q_and, q_xor;  // on two bf16 of q: its sign turned where scale < 0, 0 where it is 0 (then z_scale is 1)
    int32_t splits, chunk;  // workgroups along a sequence's keys, and their keys
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
    const int32_t b = a.starts[s], e = a.starts[s + 1], len = min(max(a.lens[s], 0), 1 << 30);
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

// The part of a sequence's keys that split c takes: whole chunks at multiples of
// `chunk` from the first that a row of it sees (the last split takes what is left),
// so which keys are summed together depends neither on the rows nor on the batch.
struct Split {
    int32_t n;       // splits of the sequence that have keys
    int32_t lo, hi;  // this one's keys
};
__device__ __forceinline__ Split split_of(const AttnArgs& a, const Seq& s, int c) {
    const int lo = first_key(a, s.at), hi = end_key(a, s, s.at + s.rows - 1);
    Split t;
    const int first = lo / a.chunk;
    t.n = hi <= lo ? 0 : min((hi - 1) / a.chunk - first + 1, a.splits);
    t.lo = (first + c) * a.chunk;
    t.hi = c + 1 >= t.n ? max(hi, t.lo) : t.lo + a.chunk;
    return t;
}

// Split c's unnormalised sums, maximum and sum of weights of a row and head.
__device__ __forceinline__ int64_t partial(const AttnArgs& a, int s, int i, int head, int c) {
    return (((int64_t)s * a.max_new + i) * a.heads + head) * a.splits + c;
}
__device__ __forceinline__ float* partial_ml(const AttnArgs& a, int v_cols) {
    return a.ws + (int64_t)a.seqs * a.max_new * a.heads * a.splits * v_cols;
}

// --- tiles of 32 keys on the matrix cores -----------------------------------------
//
// v_mfma_f32_32x32x16_bf16 takes A [32 x 16] and B [16 x 32] as 8 values of one
// row (column) l % 32 a lane, k = 8 (l / 32) + i, and leaves C[r][l % 32], r = (i &
// 3) + 8 (i >> 2) + 4 (l / 32), in register i of lane l. Scores are formed
// transposed, C = K Q^T: a lane holds 16 of the 32 keys' scores of one row of q, so
// maximum and sum are 15 steps in the lane and one exchange of lane halves, and
// what rescales a row is one value a lane. The weights of registers 8 s .. 8 s + 7
// are B of the product out^T = V^T P^T as they lie, if its k-th key is the one that
// lies there: 16 s + 4 (l / 32) + i for i < 4 and 8 more for the others, which is
// how V^T is read.

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kTile = 32;

// Rows in LDS are chunks of 16 bytes, and within every 8 chunks (128 bytes, all
// banks once) row r holds chunk c at c ^ swizzle(r): 8 rows' reads of one chunk, and
// 4 rows' of two, as the products need them, then meet in no bank.
__device__ __forceinline__ int swizzle(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }

// Key (lane, register i) of a tile's scores.
__device__ __forceinline__ int key_of(int lane, int i) { return (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5); }

// 16 bytes a lane from global memory to LDS at lds + 16 * lane, past the registers.
// The wait is the caller's: the compiler does not see the load.
__device__ __forceinline__ void load_lds16(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void load_lds4(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N loads to LDS are still on their way
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char*)p);
}

// C += K Q^T of a tile: K's rows in LDS, Q's columns in registers.
template <int DK>
__device__ __forceinline__ v16f tile_scores(const char* k, const v8bf (&q)[DK / 16], int lane) {
    const int row = lane & 31, h = lane >> 5, s = swizzle(row);
    const char* at = k + row * DK * 2;
    v16f c = {};
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) {
        const v8bf a = *(const v8bf*)(at + (t >> 2) * 128 + (((2 * (t & 3) + h) ^ s) << 4));
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, q[t], c, 0, 0, 0);
    }
    return c;
}

// out^T += V^T P^T of a tile: V's rows in LDS, P as tile_scores leaves it. A read
// gives a lane four rows of one column: lanes 16 g .. 16 g + 15 read four rows of 16
// columns, and are handed a column each.
template <int DV>
__device__ __forceinline__ void tile_sums(const char* v, const v8bf (&p)[2], v16f (&o)[DV / 32], int lane) {
    const int h = lane >> 5, row = 4 * h + ((lane & 15) >> 2), s = swizzle(row);
    const int chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const char* at = v + row * DV * 2 + (lane & 1) * 8;
#pragma unroll
    for (int t = 0; t < DV / 32; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const char* b = at + (t >> 1) * 128 + (((4 * (t & 1) + chunk) ^ s) << 4) + 16 * k * DV * 2;
            typedef __attribute__((address_space(3))) v4s lds_v4s;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)b);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(b + 8 * DV * 2));
            const v8bf a = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, p[k], o[t], 0, 0, 0);
        }
    }
}

__device__ __forceinline__ bool not_finite(uint32_t d) {  // one of two bf16
    return (d & 0x7f80u) == 0x7f80u || (d & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t d) {  // each of two bf16
    const uint32_t lo = (d & 0x7f80u) == 0x7f80u ? 0u : d & 0xffffu;
    return ((d & 0x7f800000u) == 0x7f800000u ? 0u : d & 0xffff0000u) | lo;
}

// A value that is not finite, in a key that some rows of a tile see and others do
// not, would reach the latter as 0 * inf. Such tiles (found by tile_not_finite) take
// two steps more: these values times their weights for the rows that see them, and
// zeros in their place for tile_sums, which then gives every row the bits that
// it has without them.
template <int DV>
__device__ __forceinline__ bool tile_not_finite(const char* v, int lane) {  // for the whole wave
    bool odd = false;
#pragma unroll 1
    for (int n = 0; n < DV * kTile * 2 / 1024; ++n) {
        const uint4 d = *(const uint4*)(v + n * 1024 + lane * 16);
        odd = odd || not_finite(d.x) || not_finite(d.y) || not_finite(d.z) || not_finite(d.w);
    }
    return __any(odd);
}
template <int DV>
__device__ __forceinline__ void tile_make_finite(char* v, int lane) {
#pragma unroll 1
    for (int n = 0; n < DV * kTile * 2 / 1024; ++n) {
        uint4* p = (uint4*)(v + n * 1024 + lane * 16);
        const uint4 d = *p;
        *p = make_uint4(finite_or_zero(d.x), finite_or_zero(d.y), finite_or_zero(d.z), finite_or_zero(d.w));
    }
}
template <int DV>
__device__ __forceinline__ void tile_add_not_finite(const char* v, v16f w, uint32_t seen, v16f (&o)[DV / 32], int lane) {
    const int h = lane >> 5;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {  // register i of the weights, which move down one by one
        const float own = w[0];
#pragma unroll
        for (int r = 0; r < 15; ++r) w[r] = w[r + 1];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
            const float f = __shfl(own, (lane & 31) + 32 * half);
            const int row = (i & 3) + 8 * (i >> 2) + 4 * half, s = swizzle(row);
            if (!(seen >> row & 1)) continue;
#pragma unroll
            for (int t = 0; t < DV / 32; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int chunk = 4 * t + j;  // columns 32 t + 8 j + 4 h ..
                    const uint2 d = *(const uint2*)(v + row * DV * 2 + (chunk >> 3) * 128 + (((chunk & 7) ^ s) << 4) + 8 * h);
                    if (!not_finite(d.x) && !not_finite(d.y)) continue;
                    float e[4];
                    widen2_bf16(d.x, e), widen2_bf16(d.y, e + 2);
#pragma unroll
                    for (int n = 0; n < 4; ++n) o[t][4 * j + n] += __builtin_isfinite(e[n]) ? 0.0f : f * e[n];
                }
        }
    }
}

__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return fmaxf(as_f32(r[0]), as_f32(r[1]));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi}); }

// 8 columns of a row's output from its sums v of weights times values and `sum` of
// weights, both relative to its maximum `top`. A row that sees keys has a weight of 1.
__device__ __forceinline__ void write_out(const AttnArgs& a, int row, int head, int col, const float (&v)[8], float top, float sum) {
    const float base = top == -INFINITY ? 0.0f : top;
    const bool none = sum == 0.0f;
    if (a.sinks) sum += exp2_fast(__builtin_fmaf(a.sinks[head], kLog2e, -base));
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = none ? 0.0f : v[i] * a.out_scale / sum;
    *(__attribute__((address_space(1))) v4u*)(a.out + row * a.out_token + head * a.out_head + 2 * col) =
        v4u{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

// A row's 8 values of q at `p` as an operand.
__device__ __forceinline__ v8bf q_operand(const AttnArgs& a, const char* p) {
    uint4 d = load_global16(p);
    d.x = (d.x & a.q_and) ^ a.q_xor, d.y = (d.y & a.q_and) ^ a.q_xor;
    d.z = (d.z & a.q_and) ^ a.q_xor, d.w = (d.w & a.q_and) ^ a.q_xor;
    return __builtin_bit_cast(v8bf, d);
}

// Bits of the keys of the tile at `base` that lie in [lo, hi).
__device__ __forceinline__ uint32_t keys_between(int base, int lo, int hi) {
    const int b = min(max(lo - base, 0), kTile), e = min(max(hi - base, 0), kTile);
    return (uint32_t)(((uint64_t)1 << e) - 1) & ~(uint32_t)(((uint64_t)1 << b) - 1);
}

// Scores of keys that the lane's row does not see: -inf.
__device__ __forceinline__ void hide(v16f& z, uint32_t seen, int lane) {
    seen >>= 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = seen >> ((i & 3) + 8 * (i >> 2)) & 1 ? z[i] : -INFINITY;
}

// A tile's scores become weights: running maximum m and the lane's part l of the
// running sum; returns the factor of what was summed before.
struct Running {
    float m, l;
};
__device__ __forceinline__ float tile_weights(v16f& z, float scale, Running& r) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] *= scale;
    float top = z[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, z[i]);
    top = fmaxf(max_halves(top), r.m);
    const float base = top == -INFINITY ? 0.0f : top;
    const float keep = exp2_fast(r.m - base);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        z[i] = exp2_fast(z[i] - base);
        sum += z[i];
    }
    r.l = __builtin_fmaf(r.l, keep, sum);
    r.m = top;
    return keep;
}

// Checks the arguments of an attention call and writes its AttnArgs (the workspace
// apart); FP8BLK_OK or what the call returns.
int attn_args(AttnArgs& a, const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
              int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window, const float* sinks,
              uint16_t* out, int64_t out_token, int64_t out_head);

}  // namespace fp8blk

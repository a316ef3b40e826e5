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
    float z_back;     // 1 / z_scale
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

// The split that a unit works on, `of` being what it is a split of. Units go round the
// XCDs, and a short sequence's last splits are empty: the splits of each next one begin
// one further (of less than 8 splits, one more each time round), or a number of them that
// shares a factor with the 8 XCDs left all the work to some of those (3 sequences of 500
// new tokens, 16 heads over 4, up to 6000 keys in 4 splits: 68 us, without 100).
__device__ __forceinline__ int split_at(const AttnArgs& a, int unit, int of) {
    return (unit + of + (a.splits < 8 ? of * a.splits / 8 : 0)) % a.splits;
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
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr int kTile = 32;

// Rows of COLS bf16 lie in LDS as blocks of 8 rows by 64 columns, 1 KB, what one load
// of a wave brings; in a block, row r holds its 16-byte chunk c at c ^ swizzle(r): 8
// rows' reads of one chunk, and 4 rows' of two, as the products need them, then meet
// in no bank.
__device__ __forceinline__ int swizzle(int row) { return ((row & 3) << 1) | ((row >> 2) & 1); }
template <int COLS>
__device__ __forceinline__ int row_at(int row) { return (row >> 3) * (COLS / 64 * 1024) + (row & 7) * 128; }
__device__ __forceinline__ int chunk_at(int chunk, int row) { return (chunk >> 3) * 1024 + (((chunk & 7) ^ swizzle(row)) << 4); }

// Key (lane, register i) of a tile's scores.
__device__ __forceinline__ int key_of(int lane, int i) { return (i & 3) + 8 * (i >> 2) + 4 * (lane >> 5); }

// 16 bytes a lane from global memory to LDS at lds + 16 * lane, past the registers.
// The wait is the caller's: the compiler does not see the load.
__device__ __forceinline__ void load_lds16(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void load_lds16(const char* p, uint32_t off, uint32_t lds) {  // p: the same for all lanes
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(p) : "memory");
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

// Operands are read from LDS one group ahead of the products that take them: left to
// itself the compiler reads each right before its product, and a wave waits for LDS
// between any two. Vector and scalar instructions may move past this, reads of LDS and
// products may not.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x7); }

// C += K Q^T of a tile: K's rows in LDS, Q's columns in registers.
template <int DK>
__device__ __forceinline__ v16f tile_scores(const char* k, const v8bf (&q)[DK / 16], int lane) {
    constexpr int kAhead = DK == 256 ? 2 : 4, kGroups = DK / 16 / kAhead;  // 256: what registers are left for
    const int row = lane & 31, h = lane >> 5;
    const char* at = k + row_at<DK>(row);
    v8bf x[2][kAhead];
    v16f c = {};
    auto read = [&](int g) {
#pragma unroll
        for (int t = g * kAhead; t < (g + 1) * kAhead; ++t)
            x[g & 1][t % kAhead] = *(const v8bf*)(at + (t >> 2) * 1024 + chunk_at(2 * (t & 3) + h, row));
    };
    read(0);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (g + 1 < kGroups) read(g + 1);
        keep_order();
#pragma unroll
        for (int t = 0; t < kAhead; ++t) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[g & 1][t], q[g * kAhead + t], c, 0, 0, 0);
        keep_order();
    }
    return c;
}

// Values as the operand of a tile's sums: columns 32 t .. and keys 16 k .. of V's rows
// of COLS in LDS, transposed. A read gives a lane four rows of one column: lanes 16 g .. 16 g
// + 15 read four rows of 16 columns, and are handed a column each.
template <int COLS>
__device__ __forceinline__ v8bf values_operand(const char* v, int t, int k, int lane) {
    const int row = 4 * (lane >> 5) + ((lane & 15) >> 2), chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const char* at = v + row_at<COLS>(16 * k) + row * 128 + (lane & 1) * 8 + (t >> 1) * 1024 + chunk_at(4 * (t & 1) + chunk, row);
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + row_at<COLS>(8)));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// out^T += V^T P^T of a tile: V's rows in LDS, P as tile_scores leaves it.
template <int DV>
__device__ __forceinline__ void tile_sums(const char* v, const v8bf (&p)[2], v16f (&o)[DV / 32], int lane) {
    v8bf x[2][2];
    auto read = [&](int t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) x[t & 1][k] = values_operand<DV>(v, t, k, lane);
    };
    read(0);
#pragma unroll
    for (int t = 0; t < DV / 32; ++t) {
        if (t + 1 < DV / 32) read(t + 1);
        keep_order();
#pragma unroll
        for (int k = 0; k < 2; ++k) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[t & 1][k], p[k], o[t], 0, 0, 0);
        keep_order();
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
// not, would reach the latter as 0 * inf. In tiles that not all rows see whole it is
// made a 0 in LDS before the product, so that every row has the bits that it has
// without it, and add_not_finite gives it to those that see it at the end.
template <int COLS, int ROWS>
__device__ __forceinline__ bool make_finite(char* v, int lane) {  // whether there was one, for the whole wave
    bool odd = false;
#pragma unroll 1
    for (int n = 0; n < COLS * ROWS / 512; ++n) {
        uint4* p = (uint4*)(v + n * 1024 + lane * 16);
        const uint4 d = *p;
        if (not_finite(d.x) || not_finite(d.y) || not_finite(d.z) || not_finite(d.w)) {
            *p = make_uint4(finite_or_zero(d.x), finite_or_zero(d.y), finite_or_zero(d.z), finite_or_zero(d.w));
            odd = true;
        }
    }
    return __any(odd);
}

// What make_finite took from the tiles of KEYS keys from `from` on that lie in [lo,
// hi) and not whole in [all_lo, all_hi): infinities and NaN in 8 columns, from `col`,
// of the keys in [own_lo, own_hi), read again where they come from.
template <int KEYS>
__device__ __forceinline__ void add_not_finite(const AttnArgs& a, int s, const char* v_base, bool e4m3, int col, int from, int lo, int hi,
                                               int all_lo, int all_hi, int own_lo, int own_hi, float (&v)[8]) {
#pragma unroll 1
    for (int j = max(lo, own_lo); j < min(hi, own_hi); ++j) {
        const int tile = from + (j - from) / KEYS * KEYS;
        if (tile >= all_lo && tile + KEYS <= all_hi) {
            j = tile + KEYS - 1;
            continue;
        }
        const int page = page_of(a, s, j);
        if (page < 0) continue;
        const char* p = v_base + page * a.v_page + (j & ((1 << a.page_shift) - 1)) * a.v_slot + (e4m3 ? col : 2 * col);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const float x = e4m3 ? __builtin_amdgcn_cvt_f32_fp8((int)((const uint8_t*)p)[i], 0) : as_f32((uint32_t)((const uint16_t*)p)[i] << 16);
            if (!__builtin_isfinite(x))
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += k == i ? x : 0.0f;
        }
    }
}

// Bits of the keys of the tile at `base` that lie in [lo, hi).
__device__ __forceinline__ uint32_t keys_between(int base, int lo, int hi) {
    const int b = min(max(lo - base, 0), kTile), e = min(max(hi - base, 0), kTile);
    return (uint32_t)(((uint64_t)1 << e) - 1) & ~(uint32_t)(((uint64_t)1 << b) - 1);
}

// Where a wave's next ROWS rows lie. ONE: pages hold at least as many, so that they
// are neighbours in one, all lanes agree and addresses are a scalar's business; else
// lane l has the byte offsets of row l % 32.
template <bool ONE>
struct TileRows {
    int64_t k, v;
    uint32_t held;  // bit: a key that a page holds and the workgroup's rows may see
};
template <bool ONE, int ROWS = kTile>
__device__ __forceinline__ TileRows<ONE> tile_rows(const AttnArgs& a, int page, int base, int lo, int hi, int lane) {
    constexpr uint32_t kAll = (uint32_t)(((uint64_t)1 << ROWS) - 1);
    const int j = ONE ? base : base + (lane & 31);
    const bool there = (uint32_t)page < (uint32_t)a.pages, ok = ONE ? there : there && j >= lo && j < hi;
    const int64_t p = ok ? page : 0, slot = ok ? j & ((1 << a.page_shift) - 1) : 0;
    TileRows<ONE> t;
    t.k = p * a.k_page + slot * a.k_slot;
    t.v = p * a.v_page + slot * a.v_slot;
    t.held = (ONE ? ok ? keys_between(base, lo, hi) : 0u : (uint32_t)__ballot(ok)) & kAll;
    return t;
}
__device__ __forceinline__ int64_t of_row(int64_t v, int row) {
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)v, row), hi = (uint32_t)__shfl((int)(v >> 32), row);
    return (int64_t)((uint64_t)hi << 32 | lo);
}
// The table's entry for key j, or some other where that lies outside.
__device__ __forceinline__ const int32_t* entry(const AttnArgs& a, int s, int j) {
    const int64_t i = min((int64_t)(j >> a.page_shift), a.max_pages - 1);
    return a.table + s * a.max_pages + i;
}
// The entries for the rows from key j on, as tile_rows takes them.
template <bool ONE>
__device__ __forceinline__ int page_at(const AttnArgs& a, int s, int j, int lane) {
    if constexpr (ONE) return *(const __attribute__((address_space(4))) int32_t*)entry(a, s, j);
    else return *entry(a, s, j + (lane & 31));
}

// ROWS rows of COLS bf16 to LDS, a block a load: lanes 8 r .. 8 r + 7 a row's 128 bytes.
// `lane_off` (ONE): load_offset of the rows' distance.
__device__ __forceinline__ uint32_t load_offset(int64_t slot, int lane) {
    return (uint32_t)((lane >> 3) * slot) + (((lane & 7) ^ swizzle(lane >> 3)) << 4);
}
template <int COLS, int ROWS, bool ONE>
__device__ __forceinline__ void load_tile(const char* base, int64_t rows, int64_t slot, uint32_t lane_off, uint32_t lds, int lane) {
#pragma unroll
    for (int r = 0; r < ROWS / 8; ++r) {
        const char* p = ONE ? base + rows + 8 * r * slot : base + of_row(rows, 8 * r + (lane >> 3)) + (((lane & 7) ^ swizzle(lane >> 3)) << 4);
#pragma unroll
        for (int c = 0; c < COLS / 64; ++c) {
            const uint32_t to = lds + (r * (COLS / 64) + c) * 1024;
            if constexpr (ONE) load_lds16(p + 128 * c, lane_off, to);
            else load_lds16(p + 128 * c, to);
        }
    }
}

// Rows of a tile in LDS that hold no key: zeros, for 0 * what lies there is 0.
template <int COLS, int ROWS = kTile>
__device__ __forceinline__ void clear_rows(char* lds, uint32_t held, int lane) {
#pragma unroll 1
    for (int n = 0; n < COLS * ROWS / 512; ++n)
        if (!(held >> (n / (COLS / 64) * 8 + (lane >> 3)) & 1)) *(uint4*)(lds + n * 1024 + lane * 16) = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return fmaxf(as_f32(r[0]), as_f32(r[1]));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) { return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi}); }

// What a row's sums of weights times values are multiplied by, from its maximum `top`
// and the sum of its weights, both relative to that. A row that sees keys has a
// weight of 1; one that sees none, or only scores of -inf, gives 0 whatever its sums are
// (0 * inf among the latter's): its factor is kNone, which no other is.
constexpr float kNone = -1.0f;
__device__ __forceinline__ float out_factor(const AttnArgs& a, int head, float top, float sum) {
    if (sum == 0.0f) return kNone;
    if (a.sinks) sum += exp2_fast(__builtin_fmaf(a.sinks[head], kLog2e, top == -INFINITY ? 0.0f : -top));
    return a.out_scale / sum;
}

// 8 columns of a row's output.
__device__ __forceinline__ void write_out(char* p, const float (&v)[8], float f) {
    const v4u d = {pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f), pack_bf16(v[4] * f, v[5] * f), pack_bf16(v[6] * f, v[7] * f)};
    *(__attribute__((address_space(1))) v4u*)p = f == kNone ? v4u{} : d;
}

// A row's values of q, 8 at `p` and every `step` bytes on, as operands; as_operands,
// once they have arrived, turns their sign or makes them 0 where scale asks for it.
template <int N>
__device__ __forceinline__ void load_q(const char* p, int step, v8bf (&q)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) q[t] = __builtin_bit_cast(v8bf, load_global16(p + t * step));
}
template <int N>
__device__ __forceinline__ void as_operands(const AttnArgs& a, v8bf (&q)[N]) {
    if (!(a.q_xor | ~a.q_and)) return;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        uint4 d = __builtin_bit_cast(uint4, q[t]);
        d.x = (d.x & a.q_and) ^ a.q_xor, d.y = (d.y & a.q_and) ^ a.q_xor;
        d.z = (d.z & a.q_and) ^ a.q_xor, d.w = (d.w & a.q_and) ^ a.q_xor;
        q[t] = __builtin_bit_cast(v8bf, d);
    }
}

// Scores of keys that the lane's row does not see: -inf.
__device__ __forceinline__ void hide(v16f& z, uint32_t seen, int lane) {
    seen >>= 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = seen >> ((i & 3) + 8 * (i >> 2)) & 1 ? z[i] : -INFINITY;
}

// a + x[0] + x[1]
__device__ __forceinline__ float add2(v2bf x, float a) {
    return __builtin_amdgcn_fdot2_f32_bf16(x, v2bf{(__bf16)1.0f, (__bf16)1.0f}, a, false);
}

// Of scores above 2^24 a step of f32 is 2 or more: z * scale, which weights 2^(z * scale -
// m) take unrounded, is then as far from the rounded maximum m, and past 2^31 the highest
// weight is 2^128 or 0 for it. In rows of such an m, z becomes (z * scale - m) / scale, the
// product rounded like m's, and 0 is left to subtract (m else). A row's own m decides, so
// that its bits do not depend on the others. One comparison a tile where there is none.
template <int N, typename Z>
__device__ __forceinline__ float less_coarse(const AttnArgs& a, Z (&z)[N], float m) {
    const bool coarse = __builtin_fabsf(m) > 0x1p24f;
    if (__any(coarse)) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < (int)(sizeof(Z) / sizeof(float)); ++i) z[n][i] = coarse ? (z[n][i] * a.z_scale - m) * a.z_back : z[n][i];
    }
    return coarse ? 0.0f : m;
}

// The scores of N tiles become weights 2^(z - m), as bf16 for their product with the
// values: m is the row's maximum (in units of log 2) when it was last set, l the
// lane's part of the running sum; returns the factor of what was summed before. The sum
// is of the rounded weights, so that they stay weights: their mean of equal values is
// that value, and what rounding does to a row that few keys decide is less (the sum of
// unrounded ones took 16 additions where this takes 8 instructions). m follows the
// maximum only where that has grown by more than 8: weights of up to 2^8 lose nothing,
// and the outputs are hardly ever multiplied (not at all is what `rescale` checks for).
struct Running {
    float m, l;
};
template <int N>
__device__ __forceinline__ float tile_weights(const AttnArgs& a, v16f (&z)[N], Running& r, v8bf (&p)[N][2]) {
    float top = z[0][0];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, z[n][i]);
    top = max_halves(top) * a.z_scale;
    top = top > r.m + 8.0f ? top : r.m;
    const float base = top == -INFINITY ? 0.0f : top;
    const float keep = top == r.m ? 1.0f : exp2_fast(r.m - base);
    const float less = less_coarse(a, z, base);
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const v2bf w = {(__bf16)exp2_fast(__builtin_fmaf(z[n][i], a.z_scale, -less)), (__bf16)exp2_fast(__builtin_fmaf(z[n][i + 1], a.z_scale, -less))};
            p[n][i >> 3][i & 7] = w[0], p[n][i >> 3][(i & 7) + 1] = w[1];
            sum = add2(w, sum);
        }
    r.l = __builtin_fmaf(r.l, keep, sum);
    r.m = top;
    return keep;
}

template <int T>
__device__ __forceinline__ void rescale(v16f (&o)[T], float keep) {
    if (!__any(keep != 1.0f)) return;
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] *= keep;
}

// Joins the splits of rows and heads: kOnes threads of 8 columns of a row for every
// WAYS-th chunk of its keys, which they add in order; then those sums, in order. Which
// chunks go together depends on the keys alone. A launch and two reads, the second of
// which waits for the first: 5 us; few splits take a wave a row (64 new tokens of 8192,
// 16 splits of 2048 rows: attention and join 30 us, with a workgroup a row 34).
template <int DV, int WAYS>
static __global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    constexpr int kCols = DV < 128 ? DV : 128, kOnes = kCols / 8, kRows = 256 / kOnes / WAYS;
    static_assert(kOnes * WAYS % 64 == 0, "a wave for a row, or for a part of one");
    __shared__ __attribute__((aligned(16))) float sums[kRows][WAYS][kCols];
    __shared__ float weights[kRows][WAYS];
    const int one = threadIdx.x % kOnes, way = threadIdx.x / kOnes % WAYS, r = threadIdx.x / (kOnes * WAYS);
    const int64_t id = (int64_t)blockIdx.x * kRows + r;
    const int head = (int)(id % a.heads), i = (int)(id / a.heads % a.max_new), s = (int)min(id / a.heads / a.max_new, (int64_t)a.seqs - 1);
    const Seq seq = sequence(a, s);
    const Split split = split_of(a, seq, 0);
    const bool there = id < (int64_t)a.seqs * a.max_new * a.heads && i < seq.rows && split.n > 1;
    const int col = blockIdx.y * kCols + one * 8;
    const int64_t at = partial(a, s, i, head, 0);
    const float2* ml = (const float2*)partial_ml(a, DV) + at;
    const float* part = a.ws + at * DV + col;
    float top = -INFINITY, sum = 0.0f, v[8] = {};
    if (there) {
        for (int c = threadIdx.x & 63; c < split.n; c += 64) top = fmaxf(top, ml[c].x);  // a wave has one row's threads
        for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int c = (way - split.lo / a.chunk) & (WAYS - 1); c < split.n; c += WAYS) {
            const float2 t = ml[c];
            const float4 x = *(const float4*)(part + (int64_t)c * DV), y = *(const float4*)(part + (int64_t)c * DV + 4);
            const float f = exp2_fast(t.x - base);
            sum = __builtin_fmaf(f, t.y, sum);
            const float e[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __builtin_fmaf(f, e[k], v[k]);
        }
    }
    float* const mine = &sums[r][way][one * 8];
    *(float4*)mine = make_float4(v[0], v[1], v[2], v[3]);
    *(float4*)(mine + 4) = make_float4(v[4], v[5], v[6], v[7]);
    if (one == 0) weights[r][way] = sum;
    __syncthreads();
    if (way > 0 || !there) return;
#pragma unroll 4
    for (int w = 1; w < WAYS; ++w) {
        sum += weights[r][w];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += mine[w * kCols + k];
    }
    write_out(a.out + (seq.first + i) * a.out_token + head * a.out_head + 2 * col, v, out_factor(a, head, top, sum));
}

template <int DV>
void launch_join(const AttnArgs& a, hipStream_t s) {
    if (a.splits < 2) return;
    constexpr int kAll = DV < 128 ? 32 : 16, kBlocks = DV < 128 ? 1 : DV / 128;
    const int64_t rows = (int64_t)a.seqs * a.max_new * a.heads;
    if (a.splits <= kAll / 4) k_attn_join<DV, kAll / 4><<<dim3((unsigned)ceil_div(rows, 4), kBlocks), 256, 0, s>>>(a);
    else k_attn_join<DV, kAll><<<dim3((unsigned)rows, kBlocks), 256, 0, s>>>(a);
}

// A grid of units (splits of a key head's keys) and their row tiles: workgroup b runs
// on XCD b % 8, and a unit's row tiles, which read the same keys, on `spread` XCDs, as
// few as leave no more than a sixteenth of the places empty (or the fewest).
struct Deal {
    unsigned grid;
    int spread;
};
inline Deal deal(int64_t units, int64_t tiles) {
    Deal best = {};
    for (int spread = 1; spread <= 8; spread *= 2) {
        const int64_t grid = 8 * ceil_div(units, 8 / spread) * ceil_div(tiles, spread);
        if (spread == 1 || grid < best.grid) best = {(unsigned)grid, spread};
        if (grid * 16 <= units * tiles * 17) break;
    }
    return best;
}

// Latent attention (fp8blk_latent.hip): rows of a workgroup, value columns, and the launch.
constexpr int kLatentRows = 64, kLatent = 512;
void launch_latent(const AttnArgs& a, int64_t k_cols, bool few, hipStream_t s);

// Whether `rows` neighbours in a page lie near enough for 32-bit offsets (see TileRows).
inline bool one_page(const AttnArgs& a, int rows) {
    return 1 << a.page_shift >= rows && a.k_slot < (INT64_C(1) << 26) && a.v_slot < (INT64_C(1) << 26);
}

// Checks the arguments of an attention call and writes its AttnArgs (the workspace
// apart); FP8BLK_OK or what the call returns.
int attn_args(AttnArgs& a, const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
              int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window, const float* sinks,
              uint16_t* out, int64_t out_token, int64_t out_head);

}  // namespace fp8blk

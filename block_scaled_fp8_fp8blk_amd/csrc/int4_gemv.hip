// Matrix-vector products with unsigned 4-bit weights and a scale and zero
// point per group of columns.
//
// For token m and weight row r the sum over a group is taken apart as
//   sum_c (q - z) s x = s * (D - z X),  D = sum_c q x,  X = sum_c x,
// so that the matrix instruction (v_mfma_f32_16x16x32_bf16) runs on the codes
// themselves: q = 0 .. 15 is a bf16 value, z and s (whose product with q is
// not one) are applied to a group's f32 sum. X comes from the same
// instruction with a column of ones and is shared by a wave's row tiles.
// Where every code equals a zero point of 8, or another power of two, D and
// z X are the same sums scaled and cancel exactly.
//
// Codes to bf16: byte values 0 .. 15 are e4m3's subnormals and first binade,
// which are linear (code * 2^-9), so two masks spread a dword's nibbles over
// bytes and one scaled conversion turns two of them into bf16: 7 instructions
// for 8 weights.
//
// Many rows (k_int4): the token panel lies in LDS in the order the
// instruction's operand takes it, so that a step's four reads are 16 bytes per
// lane without bank conflicts; panels larger than kPanelBytes are staged in
// pieces. Workgroups are persistent, one per compute unit; a wave takes a tile
// of 16 weight rows x 512 columns at a time: lane (n, k) = (l % 16, l / 16)
// loads 16 bytes, 32 codes, of row n in each 128-column step, and the loads of
// its next 512 columns are in flight while it computes. Where a group is
// shorter than a step, dwords change places between lane groups so that one
// instruction stays inside a group (gather_groups). `split` waves share a row
// tile's columns, in turn, and add their sums in wave order through LDS. Few
// rows (k_int4_shot): a workgroup a tile, no staging. Which way, and split,
// depend on rows, cols and group alone, so a token's bits do not depend on M.
//
// What bounds it: one token, the codes' way from memory (129280 x 4096 in
// groups of 128: 51 us, 5.4 TB/s; a plain read of that much reaches 6 TB/s);
// 16 tokens, besides, 21 vector instructions for each matrix instruction (in
// groups of 64: 65 us, 4.5 TB/s; of 32: 79 us, 3.9 TB/s); few rows, the launch
// and one chain of load, sum, join and store (4096 x 4096, 1 token: 5.7 us, 1.5
// TB/s, 16 tokens 8.0 us), and at 16 tokens the panel, which every tile of 16
// rows reads again, 16 bytes of a token at a time (4096 x 16384: 134 MB for 34
// MB of codes, 23.5 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u32 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16;               // weight rows of a matrix instruction
constexpr int kStep = 128;              // columns of one 16-byte load per lane
constexpr int kSuper = 512;             // columns a wave takes at a time
constexpr int kSteps = kSuper / kStep;
constexpr int kPanelBytes = 128 * 1024; // LDS for the token panel

constexpr int kWaves = 16;              // of a workgroup, at most
constexpr int kPlanCUs = 256;           // compute units that a plan is made for

struct Int4Args {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* x;
    float* y;
    int64_t rows;
    int32_t cols, M, split, piece;  // piece: columns of the panel in LDS at a time (a multiple of kSuper)
};

// The 8 codes of a dword (columns 0 .. 7, low nibble first) as bf16 values in
// the order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ v8bf codes_bf16(uint32_t d) {
    const uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false);
    const v2bf e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// 8 consecutive bf16 values in that order.
__device__ __forceinline__ v8bf even_odd(const uint4& v) {
    const v4u32 o = {__builtin_amdgcn_perm(v.y, v.x, 0x05040100u), __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                     __builtin_amdgcn_perm(v.y, v.x, 0x07060302u), __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
    return __builtin_bit_cast(v8bf, o);
}

// Hand the lane groups (k = lane / 16, each with 32 columns of a step) dwords
// of 8 columns so that dword j of all four lies in one group of G columns.
// G = 128: nothing to do. G = 64: the upper two lane groups' first two dwords
// change places with the lower two's last two. G = 32: the dword index changes
// places with the lane group.
template <int G>
__device__ __forceinline__ void gather_groups(uint4& v) {
    if constexpr (G < kStep) {
        const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
        v = make_uint4(a[0], b[0], a[1], b[1]);
    }
    if constexpr (G < 64) {
        const auto a = __builtin_amdgcn_permlane16_swap(v.x, v.y, false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(v.z, v.w, false, false);
        v = make_uint4(a[0], a[1], b[0], b[1]);
    }
}
// The first column, in a step, of dword j of lane group k after that.
template <int G>
__device__ __forceinline__ int gathered_column(int j, int k) {
    if constexpr (G == kStep) return 32 * k + 8 * j;
    if constexpr (G == 64) return 64 * (j >> 1) + 8 * (j & 1) + 32 * (k & 1) + 16 * (k >> 1);
    return 32 * j + 8 * k;
}

// The scales and zero points of N groups of a row; zeros past the row's end.
template <int N>
struct Groups {
    uint32_t s[N / 2];
    uint32_t z[(N + 3) / 4];
};

template <int N, bool ZERO>
__device__ __forceinline__ void load_groups(Groups<N>& g, const uint16_t* s, const uint8_t* z, int left) {
    if (left >= N) {
        __builtin_memcpy(g.s, s, 2 * N);
        if constexpr (ZERO) __builtin_memcpy(g.z, z, N);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) g.s[i] = 0;
#pragma unroll
        for (int i = 0; i < (N + 3) / 4; ++i) g.z[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) {
                g.s[i / 2] |= (uint32_t)s[i] << (16 * (i % 2));
                if constexpr (ZERO) g.z[i / 4] |= (uint32_t)z[i] << (8 * (i % 4));
            }
    }
}

// A lane's two weight rows of a tile (rows past the last are the last): bytes
// from the tile's first, which is the same for the whole wave.
struct Rows {
    const uint8_t* codes;
    uint32_t lo, hi;
    __device__ __forceinline__ Rows(const Int4Args& a, int64_t row0, int lane) {
        const uint32_t wide = a.cols / 2;
        const int last = (int)min(a.rows - 1 - row0, (int64_t)kTile);
        codes = a.codes + row0 * wide;
        lo = min(lane & 7, last) * wide;
        hi = min(8 + (lane & 7), last) * wide;
    }
};

// One wave's loads of a tile's 512 columns; WIDE: without the scales, which
// come as a block (below).
template <int G, bool WIDE>
struct Load {
    uint4 q[kSteps];
    Groups<WIDE ? 2 : kSuper / G> g;
};

template <int G, bool ZERO, bool WIDE>
__device__ __forceinline__ void issue(Load<G, WIDE>& b, const Int4Args& a, const Rows& rows, int64_t row, int lane, int c0) {
#pragma unroll
    for (int s = 0; s < kSteps; s += 2) {  // columns past the end meet zeros of the panel: any code will do
        const uint32_t c = min(c0 + s * kStep + 16 * (lane & 8) + 32 * (lane >> 4), a.cols - 32) / 2;
        b.q[s] = load_stream16(rows.codes + (rows.lo + c));
        b.q[s + 1] = load_stream16(rows.codes + (rows.hi + c));
    }
    if constexpr (!WIDE) {
        const int64_t g = row * (a.cols / G) + c0 / G;
        load_groups<kSuper / G, ZERO>(b.g, a.scales + g, ZERO ? a.zeros + g : nullptr, (a.cols - c0) / G);
    }
}

// The scales and zero points of 32 groups of a tile's 16 rows, 64 and 32 bytes
// a row. Read row by row where they are used, they would ask for 16 lines with
// every load, and for each line many times; so a wave reads a block as it lies
// and hands it out through its own part of LDS.
constexpr int kBlockGroups = 32, kBlockScales = 16 * 2 * kBlockGroups, kBlockBytes = kBlockScales + 16 * kBlockGroups;
struct Block {
    uint32_t s[4], z[2];  // lane: 8 groups of row lane / 4
};

template <int N>
__device__ __forceinline__ void load_inside(uint32_t* d, const uint8_t* p, int64_t at, int64_t end) {
    if (at + 4 * N <= end) {
        __builtin_memcpy(d, p + at, 4 * N);
    } else {  // across the array's end: its last dword, shifted
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t from = min(at + 4 * k, end - 4);
            uint32_t v;
            __builtin_memcpy(&v, p + from, 4);
            d[k] = v >> (8 * (int)(at + 4 * k - from) & 31);
        }
    }
}

template <bool ZERO>
__device__ __forceinline__ void issue_block(Block& b, const Int4Args& a, int groups, int64_t row0, int lane, int first) {
    const int64_t at = min(row0 + (lane >> 2), a.rows - 1) * groups + first + 8 * (lane & 3), end = a.rows * groups;
    load_inside<4>(b.s, reinterpret_cast<const uint8_t*>(a.scales), 2 * at, 2 * end);
    if constexpr (ZERO) load_inside<2>(b.z, a.zeros, at, end);
}

// Zeros past the row's last group, whose neighbours are another row's.
template <bool ZERO>
__device__ __forceinline__ void place_block(const Block& b, uint8_t* to, int groups, int lane, int first) {
    const int left = groups - first - 8 * (lane & 3);
    uint32_t s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = left >= 2 * k + 2 ? b.s[k] : left == 2 * k + 1 ? b.s[k] & 0xFFFFu : 0;
    *reinterpret_cast<uint4*>(to + 16 * lane) = make_uint4(s[0], s[1], s[2], s[3]);
    if constexpr (ZERO) *reinterpret_cast<uint2*>(to + kBlockScales + 8 * lane) = make_uint2(b.z[0], b.z[1]);
}

// acc += the 512 columns of b times the panel's columns from x on (LDS).
template <int G, bool ZERO, int NI, bool WIDE>
__device__ __forceinline__ void compute(Load<G, WIDE>& b, const uint4* x, const float* xsum, const uint8_t* sb, const uint8_t* zb,
                                        float (&acc)[NI]) {
    constexpr int N = kSuper / G;
    Groups<N> gr;
    if constexpr (WIDE) {  // the lane's row of the block, from these columns' groups on
        __builtin_memcpy(gr.s, __builtin_assume_aligned(sb, 8), 2 * N);
        if constexpr (ZERO) __builtin_memcpy(gr.z, __builtin_assume_aligned(zb, 4), N);
    } else {
        gr = b.g;
    }
    constexpr int per_step = kStep / G;  // groups of a step
    constexpr int per_group = 4 / per_step;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        if (s % 2 == 0) {
            swap_lane_bit3(b.q[s].x, b.q[s + 1].x);
            swap_lane_bit3(b.q[s].y, b.q[s + 1].y);
            swap_lane_bit3(b.q[s].z, b.q[s + 1].z);
            swap_lane_bit3(b.q[s].w, b.q[s + 1].w);
        }
        gather_groups<G>(b.q[s]);
        const uint32_t d[4] = {b.q[s].x, b.q[s].y, b.q[s].z, b.q[s].w};
#pragma unroll
        for (int g = 0; g < per_step; ++g) {
            v4f D = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = g * per_group; j < (g + 1) * per_group; ++j) {
                const v8bf xb = __builtin_bit_cast(v8bf, x[(s * 4 + j) * 16 * NI]);
                D = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, codes_bf16(d[j]), D, 0, 0, 0);
            }
            const int i = s * per_step + g;
            const uint32_t sc = gr.s[i / 2];
            const float scale = as_f32(i % 2 ? sc & 0xFFFF0000u : sc << 16);
            const float zero = ZERO ? (float)((gr.z[i / 4] >> (8 * (i % 4))) & 0xFFu) : 8.0f;
#pragma unroll
            for (int k = 0; k < NI; ++k)
                acc[k] = __builtin_fmaf(scale, __builtin_fmaf(-zero, xsum[i * 4 * NI + k], D[k]), acc[k]);
        }
    }
}

// NI: registers of a result tile that hold tokens. The instruction's operand
// row n carries token 4 (n % NI) + n / 4 (rows repeat where NI < 4), so that
// token t ends in register t / 4 of lane group t % 4.
template <int G, bool ZERO, int NI, bool WIDE>
__global__ __launch_bounds__(1024) void k_int4(Int4Args a) {
    extern __shared__ uint4 lds[];  // the panel's piece: [step][j][lane group][token]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n = lane & 15, kg = lane >> 4;
    const int side = wave / a.split, part = wave % a.split, across = waves / a.split;  // across: tiles a workgroup takes at once
    const int64_t tiles = (a.rows + kTile - 1) / kTile;
    const uint4* x = lds + kg * 4 * NI + 4 * (n & (NI - 1)) + (n >> 2);
    float* const xsums = reinterpret_cast<float*>(lds + a.piece / 8 * 4 * NI);  // [group][lane group][NI]
    float* const sums = xsums + a.piece / G * 4 * NI;
    const float* xsum = xsums + kg * NI;
    // WIDE (split == 1): the wave's block of scales
    uint8_t* const block = reinterpret_cast<uint8_t*>(sums) + wave * kBlockBytes;
    constexpr int SPAN = kBlockGroups * G;  // its columns
    const int groups = a.cols / G;
    Block next;
    if constexpr (WIDE)
        if ((int64_t)blockIdx.x * across + side < tiles)
            issue_block<ZERO>(next, a, groups, ((int64_t)blockIdx.x * across + side) * kTile, lane, 0);
    const int pieces = (a.cols + a.piece - 1) / a.piece;

    auto stage = [&](int p0, int cols) {
        for (int o = threadIdx.x; o < cols / 8 * 4 * NI; o += blockDim.x) {
            const int t = o % (4 * NI), k = o / (4 * NI) % 4, j = o / (16 * NI) % 4, s = o / (64 * NI);
            const int c = p0 + s * kStep + gathered_column<G>(j, k);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (t < a.M && c < a.cols) v = load_global16(a.x + (int64_t)t * a.cols + c);
            lds[o] = __builtin_bit_cast(uint4, even_odd(v));
        }
        __syncthreads();
        const v8bf ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                           (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
        for (int g = wave; g < cols / G; g += waves) {
            v4f X = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < G / 32; ++j)
                X = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x[(g * (G / 32) + j) * 16 * NI]), ones, X,
                                                            0, 0, 0);
            if (n < NI) xsums[(g * 4 + kg) * NI + n] = n == 0 ? X[0] : n == 1 ? X[1] : n == 2 ? X[2] : X[3];
        }
    };

    for (int64_t first = (int64_t)blockIdx.x * across; first < tiles; first += (int64_t)gridDim.x * across) {
        const int64_t tile = first + side;
        const int64_t row0 = min(tile, tiles - 1) * kTile, row = min(row0 + n, a.rows - 1);
        const Rows rows(a, row0, lane);
        float acc[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = 0.0f;
        for (int p = 0; p < pieces; ++p) {
            const int p0 = p * a.piece, p1 = min(p0 + a.piece, a.cols);
            int c0 = p0 + part * kSuper;
            Load<G, WIDE> A, B;
            if (c0 < p1) issue<G, ZERO, WIDE>(A, a, rows, row, lane, c0);
            if (pieces > 1 || first == (int64_t)blockIdx.x * across) {
                if (pieces > 1) __syncthreads();
                stage(p0, (p1 - p0 + kSuper - 1) / kSuper * kSuper);
                __syncthreads();
            }
            const int stride = a.split * kSuper;
            while (c0 < p1) {
                const int c1 = c0 + stride;
                if (c1 < p1) issue<G, ZERO, WIDE>(B, a, rows, row, lane, c1);
                if constexpr (WIDE)
                    if (c0 % SPAN == 0) {  // the next block: this row's, or the next tile's first
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                        __builtin_amdgcn_wave_barrier();
                        place_block<ZERO>(next, block, groups, lane, c0 / G);
                        const bool more = c0 + SPAN < a.cols;
                        const int64_t t = more ? tile : tile + (int64_t)gridDim.x * across;
                        if (t < tiles) issue_block<ZERO>(next, a, groups, t * kTile, lane, more ? (c0 + SPAN) / G : 0);
                        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                        __builtin_amdgcn_wave_barrier();
                    }
                const uint8_t *sb = block + n * 2 * kBlockGroups, *zb = block + kBlockScales + n * kBlockGroups;
                compute<G, ZERO, NI, WIDE>(A, x + (c0 - p0) / 8 * 4 * NI, xsum + (c0 - p0) / G * 4 * NI, sb + c0 % SPAN / G * 2,
                                           zb + c0 % SPAN / G, acc);
                if (c1 >= p1) break;
                c0 = c1 + stride;
                if (c0 < p1) issue<G, ZERO, WIDE>(A, a, rows, row, lane, c0);
                compute<G, ZERO, NI, WIDE>(B, x + (c1 - p0) / 8 * 4 * NI, xsum + (c1 - p0) / G * 4 * NI, sb + c1 % SPAN / G * 2,
                                           zb + c1 % SPAN / G, acc);
            }
        }
        if (!WIDE && a.split > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NI; ++i) sums[(wave * NI + i) * 64 + lane] = acc[i];
            __syncthreads();
            if (part != 0) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                for (int v = 1; v < a.split; ++v) acc[i] += sums[((wave + v) * NI + i) * 64 + lane];
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int m = kg + 4 * i;
            const int64_t r = tile * kTile + n;
            if (m < a.M && r < a.rows) store_global_f32(a.y + (int64_t)m * a.rows + r, acc[i]);
        }
    }
}

// Few tiles: one workgroup per tile, each wave taking NS steps of its columns
// (more only where there are more than 16 waves' worth), the panel read where
// it is needed instead of staged, every load issued before any is used.
template <int G, bool ZERO, int NI, int NS>
__global__ __launch_bounds__(1024) void k_int4_shot(Int4Args a) {
    __shared__ float sums[16 * NI * 64];
    constexpr int per_step = kStep / G, per_group = 4 / per_step, N = NS * per_step;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int n = lane & 15, kg = lane >> 4, last = a.cols - 32;
    const int64_t row0 = (int64_t)blockIdx.x * kTile, row = min(row0 + n, a.rows - 1);
    const uint8_t* lo = a.codes + min(row0 + (lane & 7), a.rows - 1) * (a.cols / 2);
    const uint8_t* hi = a.codes + min(row0 + 8 + (lane & 7), a.rows - 1) * (a.cols / 2);
    const uint16_t* x = a.x + (int64_t)min(4 * (n & (NI - 1)) + (n >> 2), a.M - 1) * a.cols;
    const v8bf ones = {(__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f,
                       (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f, (__bf16)1.0f};
    float acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.0f;
    for (int c0 = wave * NS * kStep; c0 < a.cols; c0 += waves * NS * kStep) {
        uint4 q[NS], v[NS][4];
        Groups<N> g;
        const auto load_codes = [&]() {
#pragma unroll
            for (int s = 0; s < NS; s += 2) {
                const int c = min(c0 + s * kStep + 16 * (lane & 8) + 32 * kg, last) / 2;
                q[s] = load_stream16(lo + c);
                q[s + 1] = load_stream16(hi + c);
            }
        };
        const auto load_x = [&]() {
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // A group past the row's end reads the last one, whose columns it
                    // so holds once each: its sums are f32s where that group's are,
                    // and its scale of 0 leaves nothing of them.
                    const int at = gathered_column<G>(j, kg);
                    v[s][j] = load_global16(x + min(c0 + s * kStep + at, a.cols - G + at % G));
                }
        };
        // Loads arrive in order: 4 steps' codes are asked for last, to be used one
        // by one as they come (16 tokens, 8192 rows x 4096: 12.7 us against 13.7,
        // 4096 x 16384 23.6 against 25.6); 2 steps' first, being the longest wait
        // (2001 x 2080 4.9 against 5.2).
        if constexpr (NS == 2) load_codes();
        else load_x();
        const int64_t g0 = row * (a.cols / G) + c0 / G;
        load_groups<N, ZERO>(g, a.scales + g0, ZERO ? a.zeros + g0 : nullptr, (a.cols - c0) / G);
        if constexpr (NS == 2) load_x();
        else load_codes();
        if constexpr (NS == 4) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            if (s % 2 == 0) {
                swap_lane_bit3(q[s].x, q[s + 1].x);
                swap_lane_bit3(q[s].y, q[s + 1].y);
                swap_lane_bit3(q[s].z, q[s + 1].z);
                swap_lane_bit3(q[s].w, q[s + 1].w);
            }
            gather_groups<G>(q[s]);
            const uint32_t d[4] = {q[s].x, q[s].y, q[s].z, q[s].w};
#pragma unroll
            for (int h = 0; h < per_step; ++h) {
                v4f D = {0.0f, 0.0f, 0.0f, 0.0f}, X = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = h * per_group; j < (h + 1) * per_group; ++j) {
                    const v8bf xb = even_odd(v[s][j]);
                    D = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, codes_bf16(d[j]), D, 0, 0, 0);
                    X = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb, ones, X, 0, 0, 0);
                }
                const int i = s * per_step + h;
                const float scale = as_f32(i % 2 ? g.s[i / 2] & 0xFFFF0000u : g.s[i / 2] << 16);
                const float zero = ZERO ? (float)((g.z[i / 4] >> (8 * (i % 4))) & 0xFFu) : 8.0f;
#pragma unroll
                for (int k = 0; k < NI; ++k) acc[k] = __builtin_fmaf(scale, __builtin_fmaf(-zero, X[k], D[k]), acc[k]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) sums[(wave * NI + i) * 64 + lane] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < NI * 64; o += blockDim.x) {
        float s = sums[o];
        for (int v = 1; v < waves; ++v) s += sums[v * NI * 64 + o];
        const int m = (o >> 4 & 3) + 4 * (o >> 6);
        const int64_t r = row0 + (o & 15);
        if (m < a.M && r < a.rows) store_global_f32(a.y + (int64_t)m * a.rows + r, s);
    }
}

// How a workgroup's waves share the tiles: `split` waves per tile, `across`
// tiles at once. Chosen for the least work of the busiest of kPlanCUs compute
// units, counted in tiles x 512 columns, of which one with fewer than kWaves
// waves does less at a time; a join counts as two. Always 16 tiles across takes
// 21.9 us where this takes 10.9 (12288 rows x 4096, 1 token), 26.1 against 17.0
// (16384 rows, 16 tokens); always 4 waves a tile 64 us against 51 (129280
// rows, 1 token), 54 against 43 (28672 x 8192, 16 tokens).
struct Plan {
    int split, across;
};
Plan plan(int64_t tiles, int supers) {
    Plan best = {1, 1};
    double least = 1e300;
    for (int split = 1; split <= 8 && split <= supers; split *= 2)
        for (int across = 1; across * split <= kWaves; ++across) {
            const int w = split * across;
            const int64_t rounds = ceil_div(ceil_div(tiles, across), kPlanCUs);
            const double busy = (double)(rounds * across * ceil_div(supers, split) * split);
            const double cost = busy * (0.7 + 0.3 * kWaves / w) + (double)rounds * (split > 1 ? 2.0 : 0.0);
            if (cost < least) {
                least = cost;
                best = {split, across};
            }
        }
    return best;
}

template <int G, bool ZERO, int NI>
void launch(Int4Args a, int cus, hipStream_t s) {
    const int64_t tiles = ceil_div(a.rows, kTile);
    const int supers = (int)ceil_div(a.cols, kSuper);
    // Up to two tiles a compute unit, a workgroup for each tile: there is too
    // little for a persistent one to run through (1 token, 8192 rows x 4096: 8.1
    // us against 8.5, 16 tokens 12.7 against 13.0; 16 tokens x 2048 columns 7.7
    // against 10.0), and beyond that the other way round (12288 rows x 4096, 16
    // tokens 19.8 against 16.1; 16384 rows, 1 token 14.5 against 12.5, 16
    // tokens 24.8 against 17.0).
    if (tiles <= 2 * kPlanCUs) {
        // Of 4 steps a wave where that gives at least 4 waves that all have 4 and
        // few scales (2048 rows x 2048 columns in groups of 128: 3.7 us against
        // 3.9 with 2 steps, 1024 x 7168 6.4 against 7.0, 4096 x 4096 5.7 against
        // 5.9 and of 16 tokens 8.0 against 9.0), else 2 (2001 x 2080 in groups
        // of 32 4.9 against 5.8, 2880 x 2880 in groups of 64 5.0 against 6.4,
        // 8192 x 1024 3.8 against 4.2, 4096 x 4096 in groups of 32 6.2 against 6.6).
        const bool two = a.cols % kSuper != 0 || supers < 4 || (G == 32 && supers <= 8);
        const int64_t w = ceil_div(a.cols, (two ? 2 : 4) * kStep);
        const int grid = (int)tiles, threads = 64 * (int)(w < kWaves ? w : kWaves);
        if (two) k_int4_shot<G, ZERO, NI, 2><<<grid, threads, 0, s>>>(a);
        else k_int4_shot<G, ZERO, NI, 4><<<grid, threads, 0, s>>>(a);
        return;
    }
    const Plan p = plan(tiles, supers);
    a.split = p.split;
    const int64_t padded = (int64_t)supers * kSuper, most = kPanelBytes / (8 * NI);
    a.piece = (int)(padded < most ? padded : most);
    const int waves = p.split * p.across;
    const size_t lds = (size_t)a.piece * 8 * NI + (size_t)(a.piece / G) * 16 * NI +
                       (p.split > 1 ? (size_t)waves * NI * 256 : (size_t)waves * kBlockBytes);
    const int64_t groups = ceil_div(tiles, p.across);
    const int grid = (int)(groups < cus ? groups : cus);
    // A wave that has a tile to itself reads its scales as blocks: 57399 rows x
    // 352 in groups of 32 8.1 us against 10.1 row by row, 129280 x 4096 in
    // groups of 128 51 against 56, of 64 with 16 tokens 65 against 69.
    if (p.split > 1) k_int4<G, ZERO, NI, false><<<grid, 64 * waves, lds, s>>>(a);
    else k_int4<G, ZERO, NI, true><<<grid, 64 * waves, lds, s>>>(a);
}

template <int G, bool ZERO>
void run(const Int4Args& a, int cus, hipStream_t s) {
    if (a.M <= 4) launch<G, ZERO, 1>(a, cus, s);
    else if (a.M <= 8) launch<G, ZERO, 2>(a, cus, s);
    else launch<G, ZERO, 4>(a, cus, s);
}

template <int G>
void run_zeros(const Int4Args& a, int cus, hipStream_t s) {
    if (a.zeros) run<G, true>(a, cus, s);
    else run<G, false>(a, cus, s);
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" int int4_gemv(const uint8_t* codes, const uint16_t* scales_bf16, const uint8_t* zeros, int group,
                         int64_t rows, int64_t cols, const uint16_t* x_bf16, int64_t M, float* y,
                         fp8blk_stream_t stream) {
    if ((group != 32 && group != 64 && group != 128) || !shape_ok(rows, cols) || cols % group != 0 || M < 1 ||
        M > FP8BLK_MAX_M)
        return FP8BLK_ERR_ARG;
    if (!codes || !scales_bf16 || !x_bf16 || !y || !aligned(codes, 16) || !aligned(scales_bf16, 2) ||
        !aligned(x_bf16, 16) || !aligned(y, 4))
        return FP8BLK_ERR_ARG;
    const Int4Args a = {codes, scales_bf16, zeros, x_bf16, y, rows, (int32_t)cols, (int32_t)M, 1, kSuper};
    const int cus = device_cus();
    if (cus < 1) return FP8BLK_ERR_HIP;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (group == 32) run_zeros<32>(a, cus, s);
    else if (group == 64) run_zeros<64>(a, cus, s);
    else run_zeros<128>(a, cus, s);
    return launch_status();
}

// A whole mixture-of-experts layer over FP4 experts for a few tokens: gate and
// up with silu, down, and the weighted sum over a token's experts.
//
// A choice of an expert by a token is a slot. Gate and up, and down, are two
// launches of one kernel (k_moe): a workgroup takes an expert's tiles of 16
// weight rows for up to four slots that go to it, so that the tokens that share
// an expert read it once; which slots those are every workgroup finds from the
// ids, and those that are not the first of theirs end at once. No list of
// tokens by expert is built, and nothing goes to the host.
//
// The sums are v_mfma_f32_16x16x32_bf16 on weights widened to bf16, exact for
// both formats. MXFP4: with their scale, a power of two, in the conversion. An
// operand of 16 rows holds 4 slots, and for down every slot's h as three bf16
// pieces, which hold all its bits (below 2^-110, where the last piece is a
// subnormal bf16, all down to 2^-133). NVFP4: an e4m3 scale times a code is a
// bf16 value, but a conversion takes powers of two only, so the instruction
// runs on the codes, with the 16-column blocks of 32 columns in rows of their
// own (the operand's other half zero), and f32 scales its results. More
// instructions for every byte, hence NVFP4's distance from MXFP4 below.
//
// What bounds it: the experts' weights. 16 tokens, 8 of 128 experts of
// 4096x2048 MXFP4, 1.1 GB: 196 us, 5.6 TB/s (a plain read of that much
// reaches 6 to 6.9); NVFP4 230 us, 5.0 TB/s. One token, 8 of 64: 29.5 and 33.7
// us, 3.6 and 3.4 TB/s, where gate/up and down each ask for all that they read
// at once, and the sum is a launch of its own. Tokens that share experts: a
// workgroup takes 4 slots of an expert (2 in NVFP4's down), as many as the
// operand holds, so its weights are read, exchanged and widened again for every
// 4 (16 tokens, 4 of 8 of 2048x4096 MXFP4: 70 us, 21 by its bytes; 14 tokens, 5
// of 6 of 2560x1024 NVFP4: 47 us, 5 by its bytes; the waves wait half of their
// time, vector units are 18 to 28% busy). Small layers are latency (2 tokens, 2
// of 8 of 512x512: 7.7 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMX = FP8BLK_FMT_MXFP4, kNV = FP8BLK_FMT_NVFP4;
constexpr int64_t kMoeAlign = 256;
constexpr int kTile = 16;   // weight rows of a matrix instruction
constexpr int kStep = 128;  // columns of one 16-byte load per lane
constexpr int kWaves = 8;   // of a workgroup, at most
constexpr int kBusy = 512;  // workgroups with work: two a compute unit
// Up to so many weights of down (tokens x experts of a token x slab), down and
// the sum over the experts are one launch, which saves a launch's start and end
// but lets tokens read an expert that they share once each. One launch against
// two, us: 2 tokens, 2 of 8 experts of 512x512 MXFP4 7.7, 10.3; 6 tokens, 4 of
// 32 of 1440x736 (25e6 weights) 18.8, 21.6; 4 tokens, 8 of 128 of 2048x768
// (50e6) 23.9, 26.2, NVFP4 26.9, 29.3; 4 tokens, 2 of 8 of 4096x2048 (67e6)
// 32.7, 28.1; 8 tokens, 6 of 64 of 2048x1024 (101e6) 40.4, 36.7.
constexpr int64_t kFewWeights = 50 << 20;
constexpr int kPieces = 3;  // bf16 values that hold an f32 h
constexpr int kSlots = FP8BLK_MAX_M * FP8BLK_MAX_TOP_K;

// A choice of an expert by a token is a slot, slot = m * K + k.
struct MoeArgs {
    const uint8_t* w[2];   // codes: gate, up; or down
    const uint8_t* sc[2];  // block scales
    const float* top[2];   // global scales, or null
    const uint16_t* in;    // x [M, cols]; or the pieces of h [slot][piece][cols]
    const int32_t* ids;
    uint16_t* pieces;      // of h [slot][piece][rows] (gate and up)
    float* part;           // a slot's output [slot][rows] (down)
    int64_t experts;
    int32_t rows, cols;
    int32_t slots, K;
    int32_t most;          // slots of one expert that a workgroup takes
    int32_t turns;         // tiles (of R * 16 rows) that it takes, one after another
    float limit;
};

// What a wave takes at a time: one tile of gate and one of up, or four tiles
// of down, NS steps of each.
template <int FMT, bool DOWN, int NS>
struct Unit {
    static constexpr int MATS = DOWN ? 1 : 2, R = DOWN ? 4 : 1, T = MATS * R;
    static constexpr int PER = FMT == kNV && DOWN ? 2 : 4;  // slots of a matrix operand
    static constexpr int LANES = DOWN ? kPieces : 1;        // operand rows of a slot in LDS
    static constexpr int SLICE = NS * kStep;                // columns
    static constexpr int B = FMT == kMX ? 32 : 16;          // columns of a block scale
    static constexpr int ROW = SLICE / B;                   // block scales of a row, and of a pair of steps
    static constexpr int PAIR = 2 * kStep / B;
    static constexpr int CHUNK = ROW < 16 ? ROW : 16, LOADS = (T * kTile * ROW / CHUNK + 63) / 64;  // a lane's scale loads
};

// The weights of two steps.
template <int T>
struct Pair {
    uint4 q[T][2];
};

// Where tile t of a unit lies. A workgroup of one expert takes tiles side by
// side, one of one token the same rows of the experts that it goes to.
struct Where {
    int expert, row;  // rows of this expert's from this one on
};
template <typename U>
struct SideBySide {
    int expert, tile;
    __device__ __forceinline__ Where operator()(int t) const { return {expert, (tile * U::R + t % U::R) * kTile}; }
};

template <typename U, typename F>
__device__ __forceinline__ void issue(Pair<U::T>& b, const MoeArgs& a, const F& where, int lane, int c0) {
    const uint32_t wide = a.cols / 2;  // bytes of a row: an expert's slab is less than 2^31 bytes
    // columns past the end meet zeros of the operand: any code will do
    const uint32_t c = min(c0 + 16 * (lane & 8) + 32 * (lane >> 4), a.cols - 32) / 2;
#pragma unroll
    for (int t = 0; t < U::T; ++t) {
        const Where at = where(t);
        const uint8_t* w = a.w[t / U::R] + (int64_t)at.expert * a.rows * wide;
        b.q[t][0] = load_stream16(w + (min(at.row + (lane & 7), a.rows - 1) * wide + c));
        b.q[t][1] = load_stream16(w + (min(at.row + 8 + (lane & 7), a.rows - 1) * wide + c));
    }
}

// The block scales of a unit. A lane's matrix column is one weight row, and
// reading that row's few scales in place would ask for 16 lines per load and
// every line many times over (measured: a third of the whole time). So a load
// takes them as they lie, and they change places in LDS, [tile][row][block].
template <typename U>
struct Scales {
    uint32_t d[U::LOADS][U::CHUNK / 4];
};

template <typename U, typename F>
__device__ __forceinline__ void issue_scales(Scales<U>& b, const MoeArgs& a, const F& where, int lane, int c0) {
    constexpr int PER_ROW = U::ROW / U::CHUNK;
    const uint32_t blocks = a.cols / U::B;
#pragma unroll
    for (int i = 0; i < U::LOADS; ++i) {
        const int o = min(i * 64 + lane, U::T * kTile * PER_ROW - 1), t = o / (kTile * PER_ROW);
        const Where w = where(t);
        const int row = min(w.row + o / PER_ROW % kTile, a.rows - 1);
        const uint8_t* sc = (U::MATS == 2 && t ? a.sc[1] : a.sc[0]) + (int64_t)w.expert * a.rows * blocks;
        const uint32_t at = row * blocks + c0 / U::B + o % PER_ROW * U::CHUNK;
        const int64_t end = (a.experts - w.expert) * a.rows * blocks;  // of the array, from this expert's scales
        // past a row's end come other rows' scales, which place_scales leaves out
        if (at + U::CHUNK <= end) {
            __builtin_memcpy(b.d[i], sc + at, U::CHUNK);
        } else {  // past the array's end there are none: its last dword, shifted
#pragma unroll
            for (int k = 0; k < U::CHUNK / 4; ++k) {
                const int64_t from = min((int64_t)at + 4 * k, end - 4);
                uint32_t v;
                __builtin_memcpy(&v, sc + from, 4);
                b.d[i][k] = v >> (8 * (int)(at + 4 * k - from) & 31);
            }
        }
    }
}

// left: blocks of the row from the slice's first on. The columns past the end
// are codes times a zero operand, but a code times a scale that was not chosen
// for it may be infinite: there the scale is the smallest (code 0).
template <typename U>
__device__ __forceinline__ void place_scales(Scales<U>& b, uint8_t* to, int lane, int left) {
    if (left < U::ROW) {
#pragma unroll
        for (int i = 0; i < U::LOADS; ++i)
#pragma unroll
            for (int k = 0; k < U::CHUNK / 4; ++k) {
                const int in = left - (i * 64 + lane) % (U::ROW / U::CHUNK) * U::CHUNK - 4 * k;
                b.d[i][k] = in >= 4 ? b.d[i][k] : in > 0 ? b.d[i][k] & ((1u << 8 * in) - 1) : 0;
            }
    }
#pragma unroll
    for (int i = 0; i < U::LOADS; ++i)
        if (i * 64 + lane < U::T * kTile * U::ROW / U::CHUNK) __builtin_memcpy(to + (i * 64 + lane) * U::CHUNK, b.d[i], U::CHUNK);
}

// Exchange the dword index with the lane group: afterwards dword j of lane
// group k is what dword k of lane group j was.
__device__ __forceinline__ void transpose_groups(uint4& v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v = make_uint4(c[0], c[1], d[0], d[1]);
}

// The 8 codes of a dword times a power-of-two scale, as bf16 values.
__device__ __forceinline__ v8bf codes_bf16(uint32_t d, float scale) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
    const v2bf e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
}

// acc += two steps of weights times the operand's columns (LDS; `stride`
// 16-byte units from one 32-column read to the next); sc: the lane's row of
// scales of the steps. OWN: every tile has an operand of its own, kPieces rows
// from one to the next.
template <int FMT, bool DOWN, typename U, bool OWN = false>
__device__ __forceinline__ void compute(Pair<U::T>& b, const uint4* in, int stride, const uint8_t* sc, int kg, bool live, v4f* acc) {
    uint32_t e[U::T][U::PAIR / 4];
#pragma unroll
    for (int t = 0; t < U::T; ++t) {
        __builtin_memcpy(e[t], __builtin_assume_aligned(sc + t * kTile * U::ROW, U::PAIR), U::PAIR);
        swap_lane_bit3(b.q[t][0].x, b.q[t][1].x);
        swap_lane_bit3(b.q[t][0].y, b.q[t][1].y);
        swap_lane_bit3(b.q[t][0].z, b.q[t][1].z);
        swap_lane_bit3(b.q[t][0].w, b.q[t][1].w);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        if constexpr (FMT == kNV) {
#pragma unroll
            for (int t = 0; t < U::T; ++t) transpose_groups(b.q[t][s]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 v = in[(s * 4 + j) * stride];
#pragma unroll
            for (int t = 0; t < U::T; ++t) {
                if constexpr (OWN)
                    if (t > 0) v = in[(s * 4 + j) * stride + t * kPieces];
                if (FMT == kNV && (OWN || t == 0)) v = live ? v : make_uint4(0, 0, 0, 0);
                const v8bf x = __builtin_bit_cast(v8bf, v);
                const uint32_t d[4] = {b.q[t][s].x, b.q[t][s].y, b.q[t][s].z, b.q[t][s].w};
                if constexpr (FMT == kMX) {
                    // byte kg of the step's dword into the exponent field
                    const uint32_t f = __builtin_amdgcn_alignbit(e[t][s], e[t][s], (uint32_t)(8 * kg + 9));
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, codes_bf16(d[j], as_f32(f)), acc[t], 0, 0, 0);
                } else {
                    const v4f D = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, codes_bf16(d[j], 1.0f), v4f{0.0f, 0.0f, 0.0f, 0.0f},
                                                                          0, 0, 0);
                    const int i = s * 8 + 2 * j;
                    const v2f f = i % 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e[t][i / 4], 1.0f, true)
                                        : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(e[t][i / 4], 1.0f, false);
                    float r = __builtin_fmaf(f.y, D[1], __builtin_fmaf(f.x, D[0], acc[t][0]));
                    if constexpr (DOWN) r = __builtin_fmaf(f.y, D[3], __builtin_fmaf(f.x, D[2], r));
                    acc[t][0] = r;
                }
            }
            if constexpr (FMT == kNV) {
                // keep the sums where they are: taken later, every result of
                // the matrix instruction would wait for them in registers
#pragma unroll
                for (int t = 0; t < U::T; ++t) asm volatile("" : "+v"(acc[t][0]));
            }
        }
    }
}

__device__ __forceinline__ int ceil_step(int n, int step) { return (n + step - 1) / step * step; }

// bf16 value nearest to f, as an f32.
__device__ __forceinline__ float head_bf16(float f) { return as_f32(bf16_of_scaled(1.0f, as_u32(f)) << 16); }

// A tile's sums over the waves that share its columns, and its outputs: every
// wave calls it as often.
template <int FMT, bool DOWN, typename U>
__device__ __forceinline__ void finish(const MoeArgs& a, const float (&top)[U::MATS], int tile, int member, int count, float* sums, v4f* acc) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
    for (int t = 0; t < U::T; ++t) {
        sums[(wave * U::T + t) * 64 + lane] = DOWN && FMT == kMX ? acc[t][0] + (acc[t][1] + acc[t][2]) : acc[t][0];
        acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();
    for (int r = wave; r < U::R; r += waves) {
        const int row = (tile * U::R + r) * kTile + (lane & 15), of = (lane >> 4) / (4 / U::PER);
        float v[U::MATS];
#pragma unroll
        for (int m = 0; m < U::MATS; ++m) {
            for (int w = 0; w < waves; ++w) {
                const float* p = sums + (w * U::T + m * U::R + r) * 64;
                const float x = U::PER == 2 ? p[lane] + p[lane ^ 16] : p[lane];
                v[m] = w == 0 ? x : v[m] + x;
            }
            v[m] *= top[m];
        }
        const int sl = __shfl(member, of & 63);
        if (row >= a.rows || of >= count) continue;
        if constexpr (DOWN) {
            if (U::PER == 4 || !(lane & 16)) a.part[(int64_t)sl * a.rows + row] = v[0];
        } else {
            float g1 = v[0], u = v[U::MATS - 1];
            if (a.limit > 0.0f) {  // a NaN stays one
                g1 = g1 > a.limit ? a.limit : g1;
                u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
            }
            float h = g1 / (1.0f + expf(-g1)) * u;
            uint16_t* to = a.pieces + (int64_t)sl * kPieces * a.rows + row;
            const bool number = fabsf(h) < __builtin_inff();
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                float bf = head_bf16(h);
                // bf16's largest, where the nearest would be an infinity
                if (p == 0 && number) bf = __builtin_amdgcn_fmed3f(bf, as_f32(0xFF7F0000u), as_f32(0x7F7F0000u));
                to[(int64_t)p * a.rows] = (uint16_t)(as_u32(bf) >> 16);
                h = p > 0 || number ? h - bf : 0.0f;  // an infinity or NaN is its first piece
            }
        }
    }
}

template <int FMT, bool DOWN, int NS>
__global__ __launch_bounds__(64 * kWaves, 3) void k_moe(MoeArgs a) {
    using U = Unit<FMT, DOWN, NS>;
    constexpr int SLICE = U::SLICE;
    extern __shared__ uint4 lds[];  // the operand, the waves' block scales and their sums
    const int lane = threadIdx.x & 63, n = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int slot = blockIdx.y, tiles = (a.rows + kTile * U::R - 1) / (kTile * U::R);
    const int end = min((int)(blockIdx.x + 1) * a.turns, tiles);

    // The slots of this slot's expert; the workgroup is theirs if `slot` is
    // the first, or (a.most)-th, ... of them.
    int ids[kSlots / 64];
#pragma unroll
    for (int q = 0; q < kSlots / 64; ++q) ids[q] = 64 * q < a.slots ? a.ids[min(64 * q + lane, a.slots - 1)] : 0;
    int expert = 0;
#pragma unroll
    for (int q = 0; q < kSlots / 64; ++q)
        if (slot >> 6 == q) expert = __builtin_amdgcn_readlane(ids[q], slot & 63);
    if (expert < 0 || expert >= a.experts) return;
    float top[U::MATS];  // the global scales
#pragma unroll
    for (int m = 0; m < U::MATS; ++m) top[m] = a.top[m] ? a.top[m][expert] : 1.0f;
    int before = 0, count = 0, member = 0;  // member: lane t holds the t-th slot
#pragma unroll
    for (int q = 0; q < kSlots / 64; ++q) {
        if (64 * q >= a.slots) continue;
        uint64_t same = __ballot(64 * q + lane < a.slots && ids[q] == expert);
        if (slot >= 64 * q) {
            const uint64_t below = slot - 64 * q < 64 ? (1ull << (slot - 64 * q)) - 1 : ~0ull;
            before += __popcll(same & below);
            same &= ~below;
        }
        while (same && count < a.most) {
            const int at = 64 * q + __builtin_ctzll(same);
            member = lane == count ? at : member;
            ++count;
            same &= same - 1;
        }
    }
    if (before % a.most != 0) return;

    int tile = blockIdx.x * a.turns, c0 = wave * SLICE;
    // The operand: [step][32 columns][lane group][row], zeros past the last
    // column; a wave reads only the slices that it has staged itself. Its first
    // rows are asked for before the weights and so are there before them.
    const int rows_in = a.most * U::LANES, live_rows = count * U::LANES;
    const auto operand_at = [&](int p0, int o) {  // column of 8 that unit o of a slice holds
        const int k = o % 4, j = o / 4 % 4;
        return p0 + o / 16 * kStep + (FMT == kMX ? 32 * k + 8 * j : 32 * j + 8 * k);
    };
    const auto load_operand = [&](int r, int c) {
        const int sl = __builtin_amdgcn_readlane(member, r / U::LANES);
        const int64_t at = DOWN ? (int64_t)sl * kPieces + r % kPieces : (int64_t)(sl / a.K);
        return load_global16(a.in + at * a.cols + min(c, a.cols - 8));
    };
    constexpr int FIRST = DOWN ? kPieces : 2, ROUNDS = (NS * 16 + 63) / 64;
    uint4 first[ROUNDS][FIRST];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i)
#pragma unroll
        for (int r = 0; r < FIRST; ++r)
            if (DOWN || r < live_rows) first[i][r] = load_operand(r, operand_at(c0, i * 64 + lane));
    Pair<U::T> b[NS / 2];
    Scales<U> sr;
    issue_scales<U>(sr, a, SideBySide<U>{expert, tile}, lane, c0);
#pragma unroll
    for (int s = 0; s < NS / 2; ++s) issue<U>(b[s], a, SideBySide<U>{expert, tile}, lane, c0 + 2 * s * kStep);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
        const int o = i * 64 + lane;
        const bool in = operand_at(c0, o) < a.cols;
#pragma unroll
        for (int r = 0; r < FIRST; ++r)
            if (o < NS * 16 && (DOWN || r < live_rows)) lds[(c0 / 8 + o) * rows_in + r] = in ? first[i][r] : make_uint4(0, 0, 0, 0);
    }
    for (int p0 = c0; p0 < a.cols; p0 += waves * SLICE)
        for (int r0 = p0 == c0 ? FIRST : 0; r0 < live_rows; r0 += 4)
            for (int i = 0; i < NS * 16; i += 64) {
                uint4 v[4];
                const int o = i + lane, c = operand_at(p0, o);
#pragma unroll
                for (int p = 0; p < 4; ++p) v[p] = load_operand(min(r0 + p, live_rows - 1), c);
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    if (r0 + p < live_rows && o < NS * 16)
                        lds[(p0 / 8 + o) * rows_in + r0 + p] = c < a.cols ? v[p] : make_uint4(0, 0, 0, 0);
            }
    // the wave's own lanes read what the others wrote
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    int row_in;  // the lane's operand row
    if constexpr (!DOWN) row_in = n >> 2;
    else if constexpr (FMT == kMX) row_in = kPieces * (n >> 2) + min(n & 3, 2);
    else row_in = kPieces * (n >> 3) + min((n & 7) >> 1, 2);
    const uint4* in = lds + kg * rows_in + min(row_in, rows_in - 1);
    // NVFP4: an operand row holds one 16-column block of each 32 columns, row
    // bit 0 says which; a down operand's rows 6 and 7 of 8 hold nothing.
    const bool live = (kg >> 1) == (n & 1) && (!DOWN || (n & 7) < 6);
    const int64_t operand = ceil_step(a.cols, SLICE) / 8 * (int64_t)rows_in;
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds + operand) + wave * U::T * kTile * U::ROW;  // [wave][tile][row][block]
    float* const sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lds + operand) + waves * U::T * kTile * U::ROW);

    v4f acc[U::T];
#pragma unroll
    for (int t = 0; t < U::T; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int turn = 0; tile < end;) {
        int t1 = tile, c1 = c0 + waves * SLICE;
        if (c1 >= a.cols) c1 = wave * SLICE, ++t1;
        place_scales<U>(sr, scales, lane, (a.cols - c0) / U::B);
        if (t1 < end) issue_scales<U>(sr, a, SideBySide<U>{expert, t1}, lane, c1);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int s = 0; s < NS / 2; ++s) {
            compute<FMT, DOWN, U>(b[s], in + (c0 / 8 + 32 * s) * rows_in, 4 * rows_in, scales + n * U::ROW + s * U::PAIR, kg,
                                  live, acc);
            if (t1 < end) issue<U>(b[s], a, SideBySide<U>{expert, t1}, lane, c1 + 2 * s * kStep);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        c0 = c1;
        if (t1 == tile) continue;
        finish<FMT, DOWN, U>(a, top, tile, member, count, sums + (turn & 1) * waves * U::T * 64, acc);
        tile = t1;
        ++turn;
    }
}

// Down and the weighted sum in one, for a few tokens: a workgroup takes 16 rows
// of the output of one token, of all its experts at once, a wave four of them
// and a slice of columns, so that their sum stays in the workgroup. Every sum is taken
// as k_moe and k_moe_sum take it. (Tokens read an expert that they share once
// each, which is why many tokens go the other way.)
template <int FMT, int NS>
__global__ __launch_bounds__(64 * kWaves, 2) void k_moe_token(MoeArgs a, const float* __restrict__ weights, const float* base,
                                                              float* y) {
    using U = Unit<FMT, true, NS>;
    constexpr int ROWS = U::T * kPieces;  // operand rows in LDS
    extern __shared__ uint4 lds[];        // the waves' operands, block scales and sums
    const int lane = threadIdx.x, n = lane & 15, kg = lane >> 4, slices = blockDim.y, waves = blockDim.z * slices;
    const int slice = __builtin_amdgcn_readfirstlane(threadIdx.y), group = __builtin_amdgcn_readfirstlane(threadIdx.z);
    const int wave = group * slices + slice;
    const int m = blockIdx.y, row0 = blockIdx.x * kTile, c0 = slice * U::SLICE, k0 = group * U::T;
    uint4* const own = lds + wave * NS * 16 * ROWS;
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds + waves * NS * 16 * ROWS) + wave * U::T * kTile * U::ROW;
    float* const sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lds + waves * NS * 16 * ROWS) +
                                                 waves * U::T * kTile * U::ROW);  // [slice][k][lane group 0, 1][row]
    const int padded = blockDim.z * U::T;  // K, up to whole waves' experts
    // A choice that is none takes part as expert 0 and is left out of the sum.
    const auto from = [&](int t) {
        const int e = a.ids[m * a.K + min(k0 + t, a.K - 1)];
        return Where{e >= 0 && e < a.experts ? e : 0, row0};
    };
    const uint4* in = own + kg * ROWS + (FMT == kMX ? min(n & 3, 2) : min((n & 7) >> 1, 2));
    const bool live = (kg >> 1) == (n & 1) && (n & 7) < 6;  // as in k_moe
    uint4 v[U::T][kPieces];
    const int k = lane % 4, j = lane / 4 % 4, c = c0 + lane / 16 * kStep + (FMT == kMX ? 32 * k + 8 * j : 32 * j + 8 * k);
    const bool mine = lane < NS * 16;
#pragma unroll
    for (int t = 0; t < U::T; ++t)
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
            v[t][p] = load_global16(a.in + (int64_t)((m * a.K + min(k0 + t, a.K - 1)) * kPieces + p) * a.cols + min(c, a.cols - 8));
    Pair<U::T> b[NS / 2];
    Scales<U> sr;
    issue_scales<U>(sr, a, from, lane, c0);
#pragma unroll
    for (int s = 0; s < NS / 2; ++s) issue<U>(b[s], a, from, lane, c0 + 2 * s * kStep);
    __builtin_amdgcn_sched_barrier(0);  // every load goes out before the first is waited for
    if (mine)
#pragma unroll
        for (int t = 0; t < U::T; ++t)
#pragma unroll
            for (int p = 0; p < kPieces; ++p) own[lane * ROWS + t * kPieces + p] = c < a.cols ? v[t][p] : make_uint4(0, 0, 0, 0);
    place_scales<U>(sr, scales, lane, (a.cols - c0) / U::B);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    v4f acc[U::T];
#pragma unroll
    for (int t = 0; t < U::T; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < NS / 2; ++s)
        compute<FMT, true, U, true>(b[s], in + 32 * s * ROWS, 4 * ROWS, scales + n * U::ROW + s * U::PAIR, kg, live, acc);
#pragma unroll
    for (int t = 0; t < U::T; ++t)
        if (lane < 32) sums[(slice * padded + k0 + t) * 32 + lane] = FMT == kMX ? acc[t][0] + (acc[t][1] + acc[t][2]) : acc[t][0];
    // The first wave joins: lane (k, row) the slices of expert k of every four,
    // then the first 16 lanes the experts.
    constexpr int ROUNDS = FP8BLK_MAX_TOP_K / U::T;
    const int row = row0 + n;
    bool is[ROUNDS];
    float top[ROUNDS], weight[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
        if (i * U::T >= a.K) break;
        const int slot = m * a.K + min(i * U::T + kg, a.K - 1), e = a.ids[slot];
        is[i] = e >= 0 && e < a.experts;
        top[i] = a.top[0] && is[i] ? a.top[0][e] : 1.0f;
        weight[i] = weights[slot];
    }
    float s = base && row < a.rows ? base[(int64_t)m * a.rows + row] : 0.0f;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
        if (i * U::T >= a.K) break;
        float f = 0.0f;
        for (int w = 0; w < slices; ++w) {
            const float* p = sums + (w * padded + i * U::T + kg) * 32 + n;
            const float g = U::PER == 2 ? p[0] + p[16] : p[0];
            f = w == 0 ? g : f + g;
        }
        f *= top[i];
#pragma unroll
        for (int t = 0; t < U::T; ++t) {
            const float ft = __shfl(f, kTile * t + n), wt = __shfl(weight[i], kTile * t);
            if (__shfl((int)is[i], kTile * t) && i * U::T + t < a.K) s = __builtin_fmaf(wt, ft, s);
        }
    }
    if (lane < kTile && row < a.rows) y[(int64_t)m * a.rows + row] = s;
}

// y = base + the weighted sum of a token's experts, in order of k. All loads
// are issued before the first is used: a choice that is none reads what lies
// in its place and leaves it.
__global__ __launch_bounds__(64) void k_moe_sum(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                const float* __restrict__ weights, const float* base, int64_t experts,
                                                int hidden, int K, float* y) {
    const int m = blockIdx.y, c = (blockIdx.x * 64 + threadIdx.x) * 4;
    if (c >= hidden) return;
    const int64_t o = (int64_t)m * hidden + c;
    v4f s = base ? *reinterpret_cast<const v4f*>(base + o) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < K; k0 += 8) {
        v4f v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = *reinterpret_cast<const v4f*>(part + (int64_t)(m * K + min(k0 + k, K - 1)) * hidden + c);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int slot = m * K + min(k0 + k, K - 1), e = ids[slot];
            const float w = weights[slot];
            if (k0 + k >= K || e < 0 || e >= experts) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = __builtin_fmaf(w, v[k][i], s[i]);
        }
    }
    *reinterpret_cast<v4f*>(y + o) = s;
}

// How many slots' workgroups have something to do, to be expected of tokens
// that choose freely: one for every expert that is chosen, or for every `most`
// slots where they are more.
inline double busy_slots(const MoeArgs& a) {
    const double idle = a.K < a.experts ? 1.0 - (double)a.K / (double)a.experts : 0.0;
    double none = 1.0;  // that no token goes to an expert
    for (int m = 0; m < a.slots / a.K; ++m) none *= idle;
    const double chosen = (double)a.experts * (1.0 - none), full = (double)a.slots / a.most;
    return chosen > full ? chosen : full;
}

template <int FMT, bool DOWN, int NS>
void launch_steps(MoeArgs a, hipStream_t s) {
    using U = Unit<FMT, DOWN, NS>;
    const int64_t slices = ceil_div(a.cols, NS * kStep), tiles = ceil_div(a.rows, kTile * U::R);
    const int waves = (int)(slices < kWaves ? slices : kWaves);
    const int64_t row_bytes = slices * NS * kStep * 2 * U::LANES;
    // LDS for the operand, besides the waves' scales and sums: at least 1 row of
    // FP8BLK_MAX_COLS columns of x or 3 of FP8BLK_MAX_INTER of h. All of it goes
    // to slots that share an expert's weights, although fewer workgroups then
    // fit a compute unit (16 tokens, 4 of 8 experts of 2048x4096 MXFP4: 70 us,
    // 82 with at most 64 KB; 8 tokens, 6 of 32 of 5120x8192 NVFP4: 458 against 493).
    const int64_t own = waves * U::T * (kTile * U::ROW + 512), room = 160 * 1024 - own;
    static_assert((DOWN ? FP8BLK_MAX_INTER : FP8BLK_MAX_COLS) * 2 * U::LANES + kWaves * U::T * (kTile * U::ROW + 512) <= 160 * 1024,
                  "LDS of a workgroup");
    a.most = a.slots / a.K < U::PER ? a.slots / a.K : U::PER;
    while (a.most > 1 && a.most * row_bytes > room) a.most /= 2;
    // Several tiles a workgroup, for whose operand and start it pays once while
    // the next tile's loads are in flight, where about two workgroups with work
    // for each compute unit are left. us for 1, 2, 4 and 8 tiles at most: 16
    // tokens, 8 of 128 experts of 4096x2048 MXFP4 228, 195, 196, 202; 4 tokens,
    // 8 of 128 of 4096x1536 NVFP4 82, 83, 74, 74; where it leaves too few, 14
    // tokens, 5 of 6 of 2560x1024 NVFP4, 4 tiles 59 and this rule's 2 47.
    const double turns = (double)tiles * busy_slots(a) / kBusy;
    a.turns = turns >= 3.0 ? 4 : turns >= 1.5 ? 2 : 1;
    const dim3 grid((unsigned)ceil_div(tiles, a.turns), (unsigned)a.slots);
    k_moe<FMT, DOWN, NS><<<grid, 64 * waves, (size_t)(a.most * row_bytes + own), s>>>(a);
}

// Steps a wave takes at a time: fewer where the columns are few. us for both
// sides, of experts of 4096x2048 where no other size is named.
// Down: 2 wherever 8 waves then cover the row, else 4. With 4 there too, 1 token,
// 8 of 64 NVFP4 35.0 against 33.8, MXFP4 29.9 against 29.6; 4 tokens NVFP4 89.2
// against 87.7; from 8 tokens on the other way round or the same (NVFP4 128.6
// against 131.6; 16 tokens, 8 of 128 229 against 233, MXFP4 197 against 198), but
// a token's bits are those of any panel, so the tokens do not choose.
// Gate and up: 2 up to 1024 columns (16 tokens, 8 of 64 of 512x256 MXFP4 13.3,
// with 4 14.1), 4 up to 2048 (8 of 64 of 2048x1408 73.5, with 2 79.1), else 8
// (16 tokens, 8 of 128 MXFP4 196, with 4 207, NVFP4 228 and 236; 4 tokens, 6 of
// 32 of 5120x1536 MXFP4 62.9 and 68.1, NVFP4 71.8 and 71.6; 1 token, 8 of 64
// MXFP4 the same, NVFP4 34.6 and 33.8).
constexpr int down_steps(int cols) { return cols <= 2 * kStep * kWaves ? 2 : 4; }

template <int FMT>
void launch_up(const MoeArgs& a, hipStream_t s) {
    if (a.cols <= 8 * kStep) launch_steps<FMT, false, 2>(a, s);
    else if (a.cols <= 16 * kStep) launch_steps<FMT, false, 4>(a, s);
    else launch_steps<FMT, false, 8>(a, s);
}

template <int FMT>
void launch_down(const MoeArgs& a, hipStream_t s) {
    if (down_steps(a.cols) == 2) launch_steps<FMT, true, 2>(a, s);
    else launch_steps<FMT, true, 4>(a, s);
}

template <int FMT, int NS>
void launch_token(const MoeArgs& a, int M, const float* weights, const float* base, float* y, hipStream_t s) {
    using U = Unit<FMT, true, NS>;
    const dim3 block(64, (unsigned)ceil_div(a.cols, U::SLICE), (unsigned)ceil_div(a.K, U::T));
    const size_t lds = (size_t)(block.y * block.z) * (NS * 256 * U::T * kPieces + U::T * kTile * U::ROW + U::T * 128);
    k_moe_token<FMT, NS><<<dim3((unsigned)ceil_div(a.rows, kTile), (unsigned)M), block, lds, s>>>(a, weights, base, y);
}

template <int FMT>
void run(const fp4_moe_layer& l, const uint16_t* x, int M, const int32_t* ids, const float* weights, int K,
         const float* base, float* y, uint16_t* pieces, float* part, hipStream_t s) {
    const int H = (int)l.hidden, I = (int)l.inter;
    MoeArgs a = {{l.gate, l.up}, {l.gate_scales, l.up_scales}, {l.gate_global, l.up_global}, x, ids, pieces, nullptr,
                 l.experts, I, H, M * K, K, 1, 1, l.limit};
    launch_up<FMT>(a, s);
    a = {{l.down, nullptr}, {l.down_scales, nullptr}, {l.down_global, nullptr}, pieces, ids, nullptr, part,
         l.experts, H, I, M * K, K, 1, 1, 0.0f};
    const int NS = down_steps(I);
    const int64_t waves = ceil_div(I, NS * kStep) * ceil_div(K, Unit<FMT, true, 4>::T);
    if ((int64_t)M * K * H * I <= kFewWeights && waves <= kWaves) {
        if (NS == 2) launch_token<FMT, 2>(a, M, weights, base, y, s);
        else launch_token<FMT, 4>(a, M, weights, base, y, s);
        return;
    }
    launch_down<FMT>(a, s);
    k_moe_sum<<<dim3((unsigned)ceil_div(H, 256), (unsigned)M), 64, 0, s>>>(part, ids, weights, base, l.experts, H, K, y);
}

bool width_ok(int64_t n, int64_t most) { return n >= 32 && n <= most && n % 32 == 0; }

// The workspace: the pieces of h, then the slots' outputs (room for any hidden).
size_t pieces_bytes(int64_t inter, int64_t slots) {
    return (size_t)(ceil_div(slots * kPieces * inter * 2, kMoeAlign) * kMoeAlign);
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp4_moe_bytes(int64_t inter, int64_t M, int top_k) {
    if (!width_ok(inter, FP8BLK_MAX_INTER) || M < 1 || M > FP8BLK_MAX_M || top_k < 1 || top_k > FP8BLK_MAX_TOP_K) return 0;
    return pieces_bytes(inter, M * top_k) + (size_t)(M * top_k) * FP8BLK_MAX_COLS * sizeof(float);
}

extern "C" int fp4_moe(const fp4_moe_layer* layer, const uint16_t* x_bf16, int64_t M, const int32_t* ids,
                       const float* weights, int top_k, const float* base, float* y, void* ws, size_t ws_bytes,
                       fp8blk_stream_t stream) {
    if (!layer || (layer->fmt != FP8BLK_FMT_MXFP4 && layer->fmt != FP8BLK_FMT_NVFP4)) return FP8BLK_ERR_ARG;
    const fp4_moe_layer& l = *layer;
    if (l.experts < 1 || l.experts > FP8BLK_MAX_EXPERTS || !width_ok(l.hidden, FP8BLK_MAX_COLS) ||
        !width_ok(l.inter, FP8BLK_MAX_INTER) || !(l.limit >= 0.0f) || std::isinf(l.limit) || M < 1 ||
        M > FP8BLK_MAX_M || top_k < 1 || top_k > FP8BLK_MAX_TOP_K)
        return FP8BLK_ERR_ARG;
    const uintptr_t sa = l.fmt == kMX ? 4 : 8;
    const void* codes[] = {l.gate, l.up, l.down, x_bf16, y};
    const void* scales[] = {l.gate_scales, l.up_scales, l.down_scales};
    const void* words[] = {l.gate_global, l.up_global, l.down_global, ids, weights};
    for (const void* p : codes)
        if (!p || !aligned(p, 16)) return FP8BLK_ERR_ARG;
    for (const void* p : scales)
        if (!p || !aligned(p, sa)) return FP8BLK_ERR_ARG;
    for (const void* p : words)
        if (!aligned(p, 4)) return FP8BLK_ERR_ARG;
    if (!ids || !weights || !aligned(base, 16)) return FP8BLK_ERR_ARG;
    const int64_t yb = 4 * M * l.hidden, slots = M * top_k;
    if (ranges_meet(y, yb, x_bf16, 2 * M * l.hidden) || ranges_meet(y, yb, ids, 4 * slots) ||
        ranges_meet(y, yb, weights, 4 * slots) || (base != y && ranges_meet(y, yb, base, yb)))
        return FP8BLK_ERR_ARG;
    if (!ws || !aligned(ws, kMoeAlign) || ws_bytes < fp4_moe_bytes(l.inter, M, top_k)) return FP8BLK_ERR_WORKSPACE;
    uint16_t* pieces = static_cast<uint16_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pieces_bytes(l.inter, slots));
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (l.fmt == kMX) run<kMX>(l, x_bf16, (int)M, ids, weights, top_k, base, y, pieces, part, s);
    else run<kNV>(l, x_bf16, (int)M, ids, weights, top_k, base, y, pieces, part, s);
    return launch_status();
}

// A whole mixture-of-experts layer over FP4 experts for a few tokens: two
// launches of one kernel template (gate and up with silu; down), and the
// weighted sum over a token's experts.
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
    float limit;
};

// A wave's weights: one tile of gate and one of up, or four tiles of down,
// NS steps of each, all loaded before any is used.
template <int FMT, bool DOWN, int NS>
struct Load {
    static constexpr int MATS = DOWN ? 1 : 2, R = DOWN ? 4 : 1, T = MATS * R;
    static constexpr int SB = NS * kStep / (FMT == kMX ? 32 : 16);  // block scales of a row
    static constexpr int PER = FMT == kNV && DOWN ? 2 : 4;          // slots of a matrix operand
    static constexpr int LANES = DOWN ? kPieces : 1;                // operand rows of a slot in LDS
    uint4 q[T][NS];
    uint32_t sc[T][SB / 4];
};

template <int FMT, bool DOWN, int NS>
__device__ __forceinline__ void issue(Load<FMT, DOWN, NS>& b, const MoeArgs& a, int64_t expert, int tile, int lane, int c0) {
    using L = Load<FMT, DOWN, NS>;
    constexpr int B = FMT == kMX ? 32 : 16;
    const uint32_t wide = a.cols / 2, blocks = a.cols / B;  // bytes of a row: an expert's slab is less than 2^31 bytes
    const int64_t slab = expert * a.rows;
#pragma unroll
    for (int t = 0; t < L::T; ++t) {
        const int m = t / L::R, r0 = (tile * L::R + t % L::R) * kTile;
        const uint8_t* w = a.w[m] + slab * wide;
        const uint32_t lo = min(r0 + (lane & 7), a.rows - 1) * wide, hi = min(r0 + 8 + (lane & 7), a.rows - 1) * wide;
#pragma unroll
        for (int s = 0; s < NS; s += 2) {  // columns past the end meet zeros of the operand: any code will do
            const uint32_t c = min(c0 + s * kStep + 16 * (lane & 8) + 32 * (lane >> 4), a.cols - 32) / 2;
            b.q[t][s] = load_stream16(w + (lo + c));
            b.q[t][s + 1] = load_stream16(w + (hi + c));
        }
    }
#pragma unroll
    for (int t = 0; t < L::T; ++t) {
        const int m = t / L::R, r0 = (tile * L::R + t % L::R) * kTile;
        const uint8_t* sc = a.sc[m] + slab * blocks;
        const uint32_t at = min(r0 + (lane & 15), a.rows - 1) * blocks + c0 / B;
        if (c0 + NS * kStep <= a.cols) {
            __builtin_memcpy(b.sc[t], sc + at, L::SB);
        } else {
            // Past the row's end other rows' scales are as good (the operand
            // is zero there), past the last row's there are none: the last
            // dword, shifted.
            const uint32_t last = (uint32_t)min((a.experts - expert) * a.rows * blocks, (int64_t)INT32_MAX) - 4;
#pragma unroll
            for (int i = 0; i < L::SB / 4; ++i) {
                const uint32_t from = min(at + 4 * i, last);
                uint32_t d;
                __builtin_memcpy(&d, sc + from, 4);
                b.sc[t][i] = d >> (8 * (at + 4 * i - from) & 31);
            }
        }
    }
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

// acc += the wave's weights times the operand's columns (LDS; `stride` 16-byte
// units from one 32-column read to the next).
template <int FMT, bool DOWN, int NS>
__device__ __forceinline__ void compute(Load<FMT, DOWN, NS>& b, const uint4* in, int stride, int kg, bool live, v4f* acc) {
    using L = Load<FMT, DOWN, NS>;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int t = 0; t < L::T; ++t) {
            if (s % 2 == 0) {
                swap_lane_bit3(b.q[t][s].x, b.q[t][s + 1].x);
                swap_lane_bit3(b.q[t][s].y, b.q[t][s + 1].y);
                swap_lane_bit3(b.q[t][s].z, b.q[t][s + 1].z);
                swap_lane_bit3(b.q[t][s].w, b.q[t][s + 1].w);
            }
            if constexpr (FMT == kNV) transpose_groups(b.q[t][s]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 v = in[(s * 4 + j) * stride];
            if constexpr (FMT == kNV) v = live ? v : make_uint4(0, 0, 0, 0);
            const v8bf x = __builtin_bit_cast(v8bf, v);
#pragma unroll
            for (int t = 0; t < L::T; ++t) {
                const uint32_t d[4] = {b.q[t][s].x, b.q[t][s].y, b.q[t][s].z, b.q[t][s].w};
                if constexpr (FMT == kMX) {
                    // byte kg of the step's dword into the exponent field
                    const uint32_t e = __builtin_amdgcn_alignbit(b.sc[t][s], b.sc[t][s], (uint32_t)(8 * kg + 9));
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, codes_bf16(d[j], as_f32(e)), acc[t], 0, 0, 0);
                } else {
                    const v4f D = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, codes_bf16(d[j], 1.0f), v4f{0.0f, 0.0f, 0.0f, 0.0f},
                                                                          0, 0, 0);
                    const int i = s * 8 + 2 * j;
                    const v2f sc = i % 4 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b.sc[t][i / 4], 1.0f, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b.sc[t][i / 4], 1.0f, false);
                    float f = __builtin_fmaf(sc.y, D[1], __builtin_fmaf(sc.x, D[0], acc[t][0]));
                    if constexpr (DOWN) f = __builtin_fmaf(sc.y, D[3], __builtin_fmaf(sc.x, D[2], f));
                    acc[t][0] = f;
                }
            }
            if constexpr (FMT == kNV) {
                // keep the sums where they are: taken later, every result of
                // the matrix instruction would wait for them in registers
#pragma unroll
                for (int t = 0; t < L::T; ++t) asm volatile("" : "+v"(acc[t][0]));
            }
        }
    }
}

// bf16 value nearest to f, as an f32.
__device__ __forceinline__ float head_bf16(float f) { return as_f32(bf16_of_scaled(1.0f, as_u32(f)) << 16); }

template <int FMT, bool DOWN, int NS>
__global__ __launch_bounds__(64 * kWaves, 3) void k_moe(MoeArgs a) {
    using L = Load<FMT, DOWN, NS>;
    constexpr int CHUNKS = NS * 16;  // 16-byte reads of an operand row
    extern __shared__ uint4 lds[];   // each wave's operand rows, then the waves' sums
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, n = lane & 15, kg = lane >> 4;
    const int slot = blockIdx.y, tile = blockIdx.x;

    // The slots of this slot's expert; the workgroup is theirs if `slot` is
    // the first, or (a.most)-th, ... of them.
    const int expert = a.ids[slot];
    if (expert < 0 || expert >= a.experts) return;
    int before = 0, count = 0, member = 0;  // member: lane t holds the t-th slot
#pragma unroll
    for (int q = 0; q < kSlots / 64; ++q) {
        if (64 * q >= a.slots) continue;
        const int s = 64 * q + lane;
        uint64_t same = __ballot(s < a.slots && a.ids[min(s, a.slots - 1)] == expert);
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

    const int rows_in = a.most * L::LANES, live_rows = count * L::LANES;
    uint4* own = lds + wave * CHUNKS * rows_in;
    int row_in;  // the lane's operand row
    if constexpr (!DOWN) row_in = n >> 2;
    else if constexpr (FMT == kMX) row_in = kPieces * (n >> 2) + min(n & 3, 2);
    else row_in = kPieces * (n >> 3) + min((n & 7) >> 1, 2);
    const uint4* in = own + kg * rows_in + min(row_in, rows_in - 1);
    // NVFP4: an operand row holds one 16-column block of each 32 columns, row
    // bit 0 says which; a down operand's rows 6 and 7 of 8 hold nothing.
    const bool live = (kg >> 1) == (n & 1) && (!DOWN || (n & 7) < 6);

    v4f acc[L::T];
#pragma unroll
    for (int t = 0; t < L::T; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int c0 = wave * NS * kStep; c0 < a.cols; c0 += waves * NS * kStep) {
        L b;
        issue<FMT, DOWN, NS>(b, a, expert, tile, lane, c0);
        // The operand: [step][j][lane group][row], zeros past the last column.
        constexpr int AT_ONCE = CHUNKS < 64 ? 64 / CHUNKS : 1, TIMES = CHUNKS < 64 ? 1 : CHUNKS / 64;  // rows, loads
        constexpr int BATCH = 4 / TIMES * AT_ONCE;                                                   // rows of four loads
        for (int r0 = 0; r0 < live_rows; r0 += BATCH) {
            uint4 v[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int r = r0 + p / TIMES * AT_ONCE + lane / CHUNKS, o = (p % TIMES * 64 + lane) % CHUNKS;
                const int sl = __shfl(member, min(r / L::LANES, count - 1)), k = o % 4, j = o / 4 % 4;
                const int64_t at = DOWN ? (int64_t)sl * kPieces + r % kPieces : (int64_t)(sl / a.K);
                const int c = c0 + o / 16 * kStep + (FMT == kMX ? 32 * k + 8 * j : 32 * j + 8 * k);
                v[p] = make_uint4(0, 0, 0, 0);
                if (c < a.cols && r < live_rows) v[p] = load_global16(a.in + at * a.cols + c);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int r = r0 + p / TIMES * AT_ONCE + lane / CHUNKS, o = (p % TIMES * 64 + lane) % CHUNKS;
                if (r < live_rows) own[o * rows_in + r] = v[p];
            }
        }
        // the wave's own lanes read what the others wrote
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        compute<FMT, DOWN, NS>(b, in, 4 * rows_in, kg, live, acc);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    float* sums = reinterpret_cast<float*>(lds + waves * CHUNKS * rows_in);  // [wave][tile][lane]
#pragma unroll
    for (int t = 0; t < L::T; ++t)
        sums[(wave * L::T + t) * 64 + lane] = DOWN && FMT == kMX ? acc[t][0] + (acc[t][1] + acc[t][2]) : acc[t][0];
    __syncthreads();
    for (int o = threadIdx.x; o < L::R * 64; o += blockDim.x) {
        const int l = o & 63, r = o / 64;
        const int row = (tile * L::R + r) * kTile + (l & 15), of = (l >> 4) / (4 / L::PER);
        float v[L::MATS];
#pragma unroll
        for (int m = 0; m < L::MATS; ++m) {
            for (int w = 0; w < waves; ++w) {
                const float* p = sums + (w * L::T + m * L::R + r) * 64;
                const float x = L::PER == 2 ? p[l] + p[l ^ 16] : p[l];
                v[m] = w == 0 ? x : v[m] + x;
            }
            if (a.top[m]) v[m] *= a.top[m][expert];
        }
        const int sl = __shfl(member, of & 63);
        if (row >= a.rows || of >= count) continue;
        if constexpr (DOWN) {
            if (L::PER == 4 || !(l & 16)) a.part[(int64_t)sl * a.rows + row] = v[0];
        } else {
            float g1 = v[0], u = v[L::MATS - 1];
            if (a.limit > 0.0f) {
                g1 = fminf(g1, a.limit);
                u = fminf(fmaxf(u, -a.limit), a.limit);
            }
            float h = g1 / (1.0f + expf(-g1)) * u;
            uint16_t* to = a.pieces + (int64_t)sl * kPieces * a.rows + row;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const float bf = head_bf16(h);
                to[(int64_t)p * a.rows] = (uint16_t)(as_u32(bf) >> 16);
                h -= bf;
            }
        }
    }
}

// y = base + the weighted sum of a token's experts, in order of k.
__global__ __launch_bounds__(256) void k_moe_sum(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                 const float* __restrict__ weights, const float* base, int64_t experts,
                                                 int hidden, int K, float* y) {
    const int m = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (c >= hidden) return;
    const int64_t o = (int64_t)m * hidden + c;
    v4f s = base ? *reinterpret_cast<const v4f*>(base + o) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < K; ++k) {
        const int slot = m * K + k, e = ids[slot];
        if (e < 0 || e >= experts) continue;
        const v4f v = *reinterpret_cast<const v4f*>(part + (int64_t)slot * hidden + c);
        const float w = weights[slot];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __builtin_fmaf(w, v[i], s[i]);
    }
    *reinterpret_cast<v4f*>(y + o) = s;
}

template <int FMT, bool DOWN, int NS>
void launch_steps(MoeArgs a, hipStream_t s) {
    using L = Load<FMT, DOWN, NS>;
    a.most = a.slots / a.K < L::PER ? a.slots / a.K : L::PER;
    const int64_t slices = ceil_div(a.cols, NS * kStep);
    const int waves = (int)(slices < kWaves ? slices : kWaves);
    const size_t lds = (size_t)waves * (NS * 256 * a.most * L::LANES + L::T * 256);
    const dim3 grid((unsigned)ceil_div(a.rows, kTile * L::R), (unsigned)a.slots);
    k_moe<FMT, DOWN, NS><<<grid, 64 * waves, lds, s>>>(a);
}

template <int FMT, bool DOWN>
void launch(const MoeArgs& a, hipStream_t s) {
    constexpr int NS = DOWN ? 4 : 8;
    if (a.cols <= 2 * NS * kStep) launch_steps<FMT, DOWN, NS / 2>(a, s);
    else launch_steps<FMT, DOWN, NS>(a, s);
}

template <int FMT>
void run(const fp4_moe_layer& l, const uint16_t* x, int M, const int32_t* ids, const float* weights, int K,
         const float* base, float* y, uint16_t* pieces, float* part, hipStream_t s) {
    const int H = (int)l.hidden, I = (int)l.inter;
    MoeArgs a = {{l.gate, l.up}, {l.gate_scales, l.up_scales}, {l.gate_global, l.up_global}, x, ids, pieces, nullptr,
                 l.experts, I, H, M * K, K, 1, l.limit};
    launch<FMT, false>(a, s);
    a = {{l.down, nullptr}, {l.down_scales, nullptr}, {l.down_global, nullptr}, pieces, ids, nullptr, part,
         l.experts, H, I, M * K, K, 1, 0.0f};
    launch<FMT, true>(a, s);
    k_moe_sum<<<dim3((unsigned)ceil_div(H, 1024), (unsigned)M), 256, 0, s>>>(part, ids, weights, base, l.experts, H, K, y);
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

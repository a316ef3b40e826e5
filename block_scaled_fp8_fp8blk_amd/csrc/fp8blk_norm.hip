// Norms around a block: the RMS norm of a block's output, its gate and scale,
// the residual sum, and the RMS norm that forms the next block's bf16 input.
//
// r' = resid + scale * gate * (y / rms(y) * post_w), x_next = r' / rms(r') * pre_w.
// The second mean square is that of the unrounded r', which no sum over y and
// resid gives beforehand, so a row takes two sums over the workgroup; it stays in
// registers from the first load to the last store, and every array is read or
// written once. Bound by memory for many rows (8192 rows of 4096, bf16 stream: 61
// us, 5.5 TB/s; two passes over y and r' took 208), by the launch for few (1 row of
// 4096 2.8 us, an empty launch 2.6; 16 rows of 7168 4.8).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

struct NormArgs {
    const void* resid;
    const float* y;
    const uint16_t* post_w;
    const uint16_t* gate;
    void* resid_out;
    const uint16_t* pre_w;
    uint16_t* x_next;
    int64_t gate_stride;
    int32_t cols;
    float scale, eps;
};

// Columns are taken 8 at a time, chunk 64 g + l by lane l of a wave: group g's
// sum of squares is 8 squares in order in each lane, then a tree over the
// lanes; a row's is four runs over the groups g % 4 = 0, 1, 2, 3 and the tree
// of those. So a row's bits depend neither on how many threads take it nor on
// the other rows.
constexpr int kChunkCols = 8, kGroupCols = 64 * kChunkCols, kMaxGroups = FP8BLK_MAX_COLS / kGroupCols;

struct Chunk {
    float v[kChunkCols];
};

__device__ __forceinline__ void widen(const uint4& d, Chunk& c) { widen8_bf16(d, c.v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ uint4 narrow(const Chunk& c) {
    return make_uint4(pack_bf16(c.v[0], c.v[1]), pack_bf16(c.v[2], c.v[3]), pack_bf16(c.v[4], c.v[5]), pack_bf16(c.v[6], c.v[7]));
}

__device__ __forceinline__ void load_f32(const float* p, Chunk& c) {
    const uint4 a = load_global16(p), b = load_global16(p + 4);
    const uint32_t d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) c.v[i] = as_f32(d[i]);
}

__device__ __forceinline__ void store16(void* p, const uint4& v) {
    *(__attribute__((address_space(1))) v4u*)p = v4u{v.x, v.y, v.z, v.w};
}

template <typename T>
__device__ __forceinline__ void load_resid(const T* p, Chunk& c) {
    if constexpr (sizeof(T) == 4) load_f32(p, c);
    else widen(load_global16(p), c);
}

template <typename T>
__device__ __forceinline__ void store_resid(T* p, const Chunk& c) {
    if constexpr (sizeof(T) == 4) {
        store16(p, make_uint4(as_u32(c.v[0]), as_u32(c.v[1]), as_u32(c.v[2]), as_u32(c.v[3])));
        store16(p + 4, make_uint4(as_u32(c.v[4]), as_u32(c.v[5]), as_u32(c.v[6]), as_u32(c.v[7])));
    } else {
        store16(p, narrow(c));
    }
}

// A group's sum over its wave, in every lane.
__device__ __forceinline__ float sum_group(const Chunk& c) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunkCols; ++i) s = __builtin_fmaf(c.v[i], c.v[i], s);
    return tree_row16(bfly16(bfly32(s)));
}

// 1 / sqrt(mean square + eps) of the row whose groups' sums lie in LDS.
__device__ __forceinline__ float inverse_rms(const float* sums, int groups, int cols, float eps) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int g = 0; g < groups; g += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] += sums[g + k];
    return 1.0f / sqrtf(((s[0] + s[1]) + (s[2] + s[3])) / (float)cols + eps);
}

// One workgroup per row; thread t takes chunks t, t + threads, ... V of them,
// and holds their values from the first load to the last store: one pass over
// every array. What can be loaded before the first sum is (EARLY).
template <typename T, int V, bool EARLY>
__global__ __launch_bounds__(1024) void k_block_norm(NormArgs a) {
    __shared__ __attribute__((aligned(16))) float sums[2][kMaxGroups];
    const int64_t o = (int64_t)blockIdx.x * a.cols;
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
    const int groups = (a.cols + kGroupCols - 1) / kGroupCols, padded = (groups + 3) & ~3;
    const T* resid = static_cast<const T*>(a.resid) + o;
    const float* y = a.y + o;
    T* resid_out = static_cast<T*>(a.resid_out) + o;
    uint16_t* x_next = a.x_next + o;
    const uint16_t* gate = a.gate ? a.gate + (int64_t)blockIdx.x * a.gate_stride : nullptr;
    if ((int)threadIdx.x < padded - groups) sums[0][groups + threadIdx.x] = sums[1][groups + threadIdx.x] = 0.0f;

    const uint32_t step = blockDim.x * kChunkCols;
    uint32_t c0 = threadIdx.x * kChunkCols;
    auto in = [&](int v) { return c0 + v * step < (uint32_t)a.cols; };
    auto col = [&](int v) { return in(v) ? c0 + v * step : 0u; };
    Chunk r[V];  // y, then r'
    Chunk res[EARLY ? V : 1];
    uint4 wpost[EARLY ? V : 1], wgate[EARLY ? V : 1], wpre[EARLY ? V : 1];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.y) load_f32(y + col(v), r[v]);
        else load_resid(resid + col(v), r[v]);
        if constexpr (EARLY) {
            if (a.y) load_resid(resid + col(v), res[v]);
            if (a.post_w) wpost[v] = load_global16(a.post_w + col(v));
            if (gate) wgate[v] = load_global16(gate + col(v));
            if (a.pre_w) wpre[v] = load_global16(a.pre_w + col(v));
        }
    }
    if constexpr (V > 4) asm volatile("" : "+v"(c0));  // columns are formed again: kept, they would not fit the registers
    if (a.y) {
        float inv = 1.0f;
        if (a.post_w) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!in(v))
#pragma unroll
                    for (int i = 0; i < kChunkCols; ++i) r[v].v[i] = 0.0f;
                const float s = sum_group(r[v]);
                if (lane == 0 && v * waves + wave < groups) sums[0][v * waves + wave] = s;
            }
            __syncthreads();
            inv = inverse_rms(sums[0], groups, a.cols, a.eps);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Chunk w;
            if (a.post_w) {
                if constexpr (EARLY) widen(wpost[v], w);
                else widen(load_global16(a.post_w + col(v)), w);
#pragma unroll
                for (int i = 0; i < kChunkCols; ++i) r[v].v[i] = r[v].v[i] * inv * w.v[i];
            }
            if (gate) {
                if constexpr (EARLY) widen(wgate[v], w);
                else widen(load_global16(gate + col(v)), w);
#pragma unroll
                for (int i = 0; i < kChunkCols; ++i) r[v].v[i] *= w.v[i];
            }
            if constexpr (EARLY) w = res[v];
            else load_resid(resid + col(v), w);
#pragma unroll
            for (int i = 0; i < kChunkCols; ++i) r[v].v[i] = __builtin_fmaf(a.scale, r[v].v[i], w.v[i]);
            if (in(v)) store_resid(resid_out + col(v), r[v]);
            if constexpr (!EARLY) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (!a.x_next) return;
    if constexpr (V > 4) asm volatile("" : "+v"(c0));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (!in(v))
#pragma unroll
            for (int i = 0; i < kChunkCols; ++i) r[v].v[i] = 0.0f;
        const float s = sum_group(r[v]);
        if (lane == 0 && v * waves + wave < groups) sums[1][v * waves + wave] = s;
    }
    __syncthreads();
    const float inv = inverse_rms(sums[1], groups, a.cols, a.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Chunk w;
        if constexpr (EARLY) widen(wpre[v], w);
        else widen(load_global16(a.pre_w + col(v)), w);
#pragma unroll
        for (int i = 0; i < kChunkCols; ++i) w.v[i] = r[v].v[i] * inv * w.v[i];
        if (in(v)) store16(x_next + col(v), narrow(w));
        if constexpr (!EARLY) __builtin_amdgcn_sched_barrier(0);
    }
}

template <typename T>
void launch(const NormArgs& a, int64_t N, hipStream_t s) {
    // One chunk a thread, for few rows (latency) with up to 16 waves (4 rows of
    // 12288 columns 5.2 us, 8.1 with 8; 1 of 16384 5.8, 8.0); more rows than there
    // is room for run better as workgroups of at most 8 (4096 rows of 8192 columns:
    // 62.8 us, against 65.1 with 16 and 70.6 with 4). All loads are issued before
    // the first sum where registers hold them, up to 2 chunks a thread.
    const int waves = (a.cols + kGroupCols - 1) / kGroupCols, most = N >= 512 ? 8 : 16;
    const int v = (waves + most - 1) / most;
    auto threads = [&](int V) { return 64 * ((waves + V - 1) / V); };
    const unsigned n = (unsigned)N;
    if (v <= 1) k_block_norm<T, 1, true><<<n, threads(1), 0, s>>>(a);
    else if (v <= 2) k_block_norm<T, 2, true><<<n, threads(2), 0, s>>>(a);
    else if (waves <= 64) k_block_norm<T, 4, false><<<n, threads(4), 0, s>>>(a);
    else k_block_norm<T, 8, false><<<n, threads(8), 0, s>>>(a);
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_block_norm(const void* resid, int resid_type, const float* y, int64_t N, int64_t cols,
                                 const uint16_t* post_w, const uint16_t* gate, int64_t gate_rows, float scale,
                                 void* resid_out, const uint16_t* pre_w, float eps, uint16_t* x_next,
                                 fp8blk_stream_t stream) {
    if (N < 1 || N > FP8BLK_MAX_PANEL || !shape_ok(N, cols)) return FP8BLK_ERR_ARG;
    if (resid_type != FP8BLK_F32 && resid_type != FP8BLK_BF16) return FP8BLK_ERR_ARG;
    if (!resid || !pre_w != !x_next || !(eps >= 0.0f) || std::isinf(eps)) return FP8BLK_ERR_ARG;
    if (y ? !resid_out : (post_w || gate || resid_out || !x_next)) return FP8BLK_ERR_ARG;
    if (gate ? gate_rows != 1 && gate_rows != N : gate_rows != 0) return FP8BLK_ERR_ARG;
    const void* all[] = {resid, y, post_w, gate, resid_out, pre_w, x_next};
    for (const void* p : all)
        if (!aligned(p, 16)) return FP8BLK_ERR_ARG;
    const int64_t n = N * cols, rb = n * (resid_type == FP8BLK_F32 ? 4 : 2);
    const struct {
        const void* p;
        int64_t bytes;
    } in[] = {{y, 4 * n}, {post_w, 2 * cols}, {gate, 2 * gate_rows * cols}, {pre_w, 2 * cols}};
    for (const auto& i : in)
        if (ranges_meet(x_next, 2 * n, i.p, i.bytes) || ranges_meet(resid_out, rb, i.p, i.bytes)) return FP8BLK_ERR_ARG;
    if (ranges_meet(x_next, 2 * n, resid, rb) || ranges_meet(x_next, 2 * n, resid_out, rb) ||
        (resid_out != resid && ranges_meet(resid_out, rb, resid, rb)))
        return FP8BLK_ERR_ARG;
    const NormArgs a = {resid,  y, post_w, gate, resid_out, pre_w, x_next, gate_rows > 1 ? cols : 0, (int32_t)cols,
                        scale, eps};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (resid_type == FP8BLK_F32) launch<float>(a, N, s);
    else launch<uint16_t>(a, N, s);
    return launch_status();
}

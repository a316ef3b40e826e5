// Norms around a block: the RMS norm of a block's output, its gate and scale,
// the residual sum, and the RMS norm that forms the next block's bf16 input.
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

__device__ __forceinline__ uint16_t to_bf16(float f) { return (uint16_t)bf16_of_scaled(1.0f, as_u32(f)); }
__device__ __forceinline__ float from_bf16(uint16_t h) { return as_f32((uint32_t)h << 16); }

constexpr int kNormThreads = 256;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ float sum_block(float v, float* part) {
    v = tree64(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < kNormThreads / 64; ++i) s += part[i];
    return s;
}

template <typename T>
__device__ __forceinline__ float load_as_f32(const T* p) {
    if constexpr (sizeof(T) == 4) return *p;
    else return from_bf16(*p);
}

// One workgroup per row, three passes over it.
template <typename T>
__global__ __launch_bounds__(kNormThreads) void k_block_norm(NormArgs a) {
    __shared__ float part[kNormThreads / 64];
    const int64_t row = blockIdx.x, o = row * a.cols;
    const T* r = static_cast<const T*>(a.resid) + o;
    const uint16_t* gate = a.gate ? a.gate + row * a.gate_stride : nullptr;
    float inv_post = 1.0f;
    if (a.post_w) {
        float q = 0.0f;
        for (int c = threadIdx.x; c < a.cols; c += kNormThreads) q = __builtin_fmaf(a.y[o + c], a.y[o + c], q);
        inv_post = 1.0f / sqrtf(sum_block(q, part) / (float)a.cols + a.eps);
    }
    auto next = [&](int c) {
        float v = load_as_f32(r + c);
        if (a.y) {
            float n = a.y[o + c];
            if (a.post_w) n = n * inv_post * from_bf16(a.post_w[c]);
            if (gate) n *= from_bf16(gate[c]);
            v = __builtin_fmaf(a.scale, n, v);
        }
        return v;
    };
    float q = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float v = next(c);
        q = __builtin_fmaf(v, v, q);
    }
    const float inv_pre = 1.0f / sqrtf(sum_block(q, part) / (float)a.cols + a.eps);
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
        const float v = next(c);
        if (a.x_next) a.x_next[o + c] = to_bf16(v * inv_pre * from_bf16(a.pre_w[c]));
        if (a.resid_out) {
            if constexpr (sizeof(T) == 4) static_cast<T*>(a.resid_out)[o + c] = v;
            else static_cast<T*>(a.resid_out)[o + c] = to_bf16(v);
        }
    }
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
    if (resid_type == FP8BLK_F32) k_block_norm<float><<<(int)N, kNormThreads, 0, s>>>(a);
    else k_block_norm<uint16_t><<<(int)N, kNormThreads, 0, s>>>(a);
    return launch_status();
}

// Router: the experts each token goes to and their weights, in 64 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

constexpr size_t kRouteAlign = 256;

struct RouteArgs {
    const float* bias;
    const double* logits;  // [M, E]
    int32_t* ids;
    float* weights;
    int32_t E, K, score, normalize;
    float scale;
};

__device__ __forceinline__ double shfl_xor64(double v, int m) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)u, m), hi = (uint32_t)__shfl_xor((int)(uint32_t)(u >> 32), m);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// One wave per (expert, token).
__global__ __launch_bounds__(64) void k_route_logits(const uint16_t* __restrict__ w, const uint16_t* __restrict__ x,
                                                     int cols, int E, double* __restrict__ logits) {
    const int64_t e = blockIdx.x, m = blockIdx.y;
    double s = 0.0;
    for (int c = threadIdx.x; c < cols; c += 64)
        s = __builtin_fma((double)as_f32((uint32_t)w[e * cols + c] << 16), (double)as_f32((uint32_t)x[m * cols + c] << 16), s);
    for (int h = 32; h >= 1; h >>= 1) s += shfl_xor64(s, h);
    if (threadIdx.x == 0) logits[m * E + e] = s;
}

// One wave per token; lane l holds experts l, l + 64, ...
template <int NE>
__global__ __launch_bounds__(64) void k_route_choose(RouteArgs a) {
    const int64_t m = blockIdx.x;
    const int lane = threadIdx.x;
    const double lowest = -__builtin_inf();
    double s[NE], pick[NE], top = lowest;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        s[i] = e < a.E ? a.logits[m * a.E + e] : lowest;
        top = s[i] > top ? s[i] : top;
    }
    if (a.score == FP8BLK_SCORE_SOFTMAX) {
        for (int h = 32; h >= 1; h >>= 1) top = fmax(top, shfl_xor64(top, h));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = exp(s[i] - top);
            sum += lane + 64 * i < a.E ? s[i] : 0.0;
        }
        for (int h = 32; h >= 1; h >>= 1) sum += shfl_xor64(sum, h);
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i)
            s[i] = a.score == FP8BLK_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-s[i]))
                                                   : sqrt(fmax(s[i], 0.0) + log1p(exp(-fabs(s[i]))));
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        pick[i] = e < a.E ? s[i] + (a.bias ? (double)a.bias[e] : 0.0) : lowest;
        if (!(pick[i] > lowest)) pick[i] = lowest;  // NaN: never chosen
    }
    double mine = 0.0, total = 0.0;  // lane k: the k-th choice's score
    int my_id = -1;
    for (int k = 0; k < a.K; ++k) {
        double best = lowest, score = 0.0;
        int id = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (pick[i] > best) best = pick[i], score = s[i], id = lane + 64 * i;
        for (int h = 32; h >= 1; h >>= 1) {
            const double b = shfl_xor64(best, h), sc = shfl_xor64(score, h);
            const int j = __shfl_xor(id, h);
            if (b > best || (b == best && j < id)) best = b, score = sc, id = j;
        }
        const bool none = !(best > lowest);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (id == lane + 64 * i) pick[i] = lowest;
        if (lane == k) mine = none ? 0.0 : score, my_id = none ? -1 : id;
        total += none ? 0.0 : score;
    }
    if (lane < a.K) {
        if (a.normalize) mine = total > 0.0 ? mine / total : 0.0;
        a.ids[m * a.K + lane] = my_id;
        a.weights[m * a.K + lane] = (float)(mine * (double)a.scale);
    }
}

bool route_shape_ok(int64_t experts, int64_t cols, int64_t M) {
    return experts >= 1 && experts <= FP8BLK_MAX_EXPERTS && M >= 1 && M <= FP8BLK_MAX_PANEL && shape_ok(experts, cols);
}

}  // namespace

size_t route_workspace_bytes(int64_t experts, int64_t cols, int64_t M) {
    if (!route_shape_ok(experts, cols, M)) return 0;
    return (size_t)ceil_div(M * experts * (int64_t)sizeof(double), kRouteAlign) * kRouteAlign;
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_moe_route(const uint16_t* w_bf16, const float* bias, int64_t experts, int64_t cols,
                                const uint16_t* x_bf16, int64_t M, int score, int top_k, int normalize, float scale,
                                int32_t* ids, float* weights, void* ws, size_t ws_bytes, fp8blk_stream_t stream) {
    if (!route_shape_ok(experts, cols, M) || top_k < 1 || top_k > FP8BLK_MAX_TOP_K || top_k > experts ||
        score < FP8BLK_SCORE_SOFTMAX || score > FP8BLK_SCORE_SQRT_SOFTPLUS)
        return FP8BLK_ERR_ARG;
    if (!w_bf16 || !x_bf16 || !ids || !weights || !aligned(w_bf16, 16) || !aligned(x_bf16, 16) || !aligned(bias, 4) ||
        !aligned(ids, 4) || !aligned(weights, 4))
        return FP8BLK_ERR_ARG;
    if (!ws || !aligned(ws, kRouteAlign) || ws_bytes < route_workspace_bytes(experts, cols, M)) return FP8BLK_ERR_WORKSPACE;
    double* logits = static_cast<double*>(ws);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    k_route_logits<<<dim3((unsigned)experts, (unsigned)M), 64, 0, s>>>(w_bf16, x_bf16, (int)cols, (int)experts, logits);
    const RouteArgs a = {bias, logits, ids, weights, (int32_t)experts, top_k, score, normalize != 0, scale};
    if (experts <= 64) k_route_choose<1><<<(unsigned)M, 64, 0, s>>>(a);
    else if (experts <= 256) k_route_choose<4><<<(unsigned)M, 64, 0, s>>>(a);
    else k_route_choose<16><<<(unsigned)M, 64, 0, s>>>(a);
    return launch_status();
}

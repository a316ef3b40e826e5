// A whole mixture-of-experts layer over FP4 experts for a few tokens.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

constexpr int kMX = FP8BLK_FMT_MXFP4;
constexpr int64_t kMoeAlign = 256;

struct MoeArgs {
    fp4_moe_layer l;
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const float* base;
    float* y;
    float* h;  // [M * K, inter]
    int32_t M, K;
};

// Two e2m1 codes (a byte, low nibble first) times their block scale.
template <int FMT>
__device__ __forceinline__ v2f weight_pair(const uint8_t* codes, const uint8_t* scales, int64_t row, int cols, int c) {
    const v2f w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[row * (cols / 2) + c / 2], 1.0f, 0);
    const uint32_t sc = scales[row * (cols / (FMT == kMX ? 32 : 16)) + c / (FMT == kMX ? 32 : 16)];
    const v2f s8 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(sc, 1.0f, false);
    const float s = FMT == kMX ? e8m0_to_f32(sc) : s8.x;
    return v2f{w.x * s, w.y * s};
}

// One wave per (choice, row of the expert's gate and up).
template <int FMT>
__global__ __launch_bounds__(64) void k_moe_up(MoeArgs a) {
    const int64_t i = blockIdx.x, slot = blockIdx.y;
    const int e = a.ids[slot], H = (int)a.l.hidden;
    if (e < 0 || e >= a.l.experts) return;
    const int64_t row = e * a.l.inter + i;
    float g = 0.0f, u = 0.0f;
    for (int c = 2 * threadIdx.x; c < H; c += 128) {
        float x[2];
        widen2_bf16(*reinterpret_cast<const uint32_t*>(a.x + slot / a.K * H + c), x);
        const v2f wg = weight_pair<FMT>(a.l.gate, a.l.gate_scales, row, H, c);
        const v2f wu = weight_pair<FMT>(a.l.up, a.l.up_scales, row, H, c);
        g = __builtin_fmaf(wg.y, x[1], __builtin_fmaf(wg.x, x[0], g));
        u = __builtin_fmaf(wu.y, x[1], __builtin_fmaf(wu.x, x[0], u));
    }
    g = tree64(g);
    u = tree64(u);
    if (a.l.gate_global) g *= a.l.gate_global[e];
    if (a.l.up_global) u *= a.l.up_global[e];
    if (a.l.limit > 0.0f) {
        g = fminf(g, a.l.limit);
        u = fminf(fmaxf(u, -a.l.limit), a.l.limit);
    }
    if (threadIdx.x == 0) a.h[slot * a.l.inter + i] = g / (1.0f + expf(-g)) * u;
}

// One wave per (output column, token).
template <int FMT>
__global__ __launch_bounds__(64) void k_moe_down(MoeArgs a) {
    const int64_t n = blockIdx.x, m = blockIdx.y;
    const int I = (int)a.l.inter;
    float y = a.base ? a.base[m * a.l.hidden + n] : 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int64_t slot = m * a.K + k;
        const int e = a.ids[slot];
        if (e < 0 || e >= a.l.experts) continue;
        float s = 0.0f;
        for (int c = 2 * threadIdx.x; c < I; c += 128) {
            const v2f w = weight_pair<FMT>(a.l.down, a.l.down_scales, e * a.l.hidden + n, I, c);
            s = __builtin_fmaf(w.y, a.h[slot * I + c + 1], __builtin_fmaf(w.x, a.h[slot * I + c], s));
        }
        s = tree64(s);
        if (a.l.down_global) s *= a.l.down_global[e];
        y = __builtin_fmaf(a.weights[slot], s, y);
    }
    if (threadIdx.x == 0) a.y[m * a.l.hidden + n] = y;
}

template <int FMT>
void launch_moe(const MoeArgs& a, hipStream_t s) {
    k_moe_up<FMT><<<dim3((unsigned)a.l.inter, (unsigned)(a.M * a.K)), 64, 0, s>>>(a);
    k_moe_down<FMT><<<dim3((unsigned)a.l.hidden, (unsigned)a.M), 64, 0, s>>>(a);
}

bool width_ok(int64_t n) { return n >= 32 && n <= FP8BLK_MAX_COLS && n % 32 == 0; }

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp4_moe_bytes(int64_t inter, int64_t M, int top_k) {
    if (!width_ok(inter) || M < 1 || M > FP8BLK_MAX_M || top_k < 1 || top_k > FP8BLK_MAX_TOP_K) return 0;
    return (size_t)(ceil_div(M * top_k * inter * (int64_t)sizeof(float), kMoeAlign) * kMoeAlign);
}

extern "C" int fp4_moe(const fp4_moe_layer* layer, const uint16_t* x_bf16, int64_t M, const int32_t* ids,
                       const float* weights, int top_k, const float* base, float* y, void* ws, size_t ws_bytes,
                       fp8blk_stream_t stream) {
    if (!layer || (layer->fmt != FP8BLK_FMT_MXFP4 && layer->fmt != FP8BLK_FMT_NVFP4)) return FP8BLK_ERR_ARG;
    const fp4_moe_layer& l = *layer;
    if (l.experts < 1 || l.experts > FP8BLK_MAX_EXPERTS || !width_ok(l.hidden) || !width_ok(l.inter) ||
        !(l.limit >= 0.0f) || std::isinf(l.limit) || M < 1 || M > FP8BLK_MAX_M || top_k < 1 || top_k > FP8BLK_MAX_TOP_K)
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
    const MoeArgs a = {l, x_bf16, ids, weights, base, y, static_cast<float*>(ws), (int32_t)M, top_k};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (l.fmt == kMX) launch_moe<FP8BLK_FMT_MXFP4>(a, s);
    else launch_moe<FP8BLK_FMT_NVFP4>(a, s);
    return launch_status();
}

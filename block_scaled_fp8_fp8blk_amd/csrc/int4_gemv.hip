// Matrix-vector products with unsigned 4-bit weights and a scale and zero
// point per group of columns.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

struct Int4Args {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* x;
    float* y;
    int64_t rows;
    int32_t cols, group;
};

// One wave per (weight row, token).
__global__ __launch_bounds__(64) void k_int4(Int4Args a) {
    const int64_t r = blockIdx.x, m = blockIdx.y, groups = a.cols / a.group;
    float s = 0.0f;
    for (int c = 2 * threadIdx.x; c < a.cols; c += 128) {
        const uint32_t b = a.codes[r * (a.cols / 2) + c / 2];
        const int64_t g = r * groups + c / a.group;
        const float z = a.zeros ? (float)a.zeros[g] : 8.0f, sc = as_f32((uint32_t)a.scales[g] << 16);
        float w[2];
        widen2_bf16(*reinterpret_cast<const uint32_t*>(a.x + m * a.cols + c), w);
        s = __builtin_fmaf(((float)(b & 15u) - z) * sc, w[0], s);
        s = __builtin_fmaf(((float)(b >> 4) - z) * sc, w[1], s);
    }
    s = tree64(s);
    if (threadIdx.x == 0) a.y[m * a.rows + r] = s;
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
    if (rows > INT32_MAX) return FP8BLK_ERR_ARG;
    const Int4Args a = {codes, scales_bf16, zeros, x_bf16, y, rows, (int32_t)cols, group};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    k_int4<<<dim3((unsigned)rows, (unsigned)M), 64, 0, s>>>(a);
    return launch_status();
}

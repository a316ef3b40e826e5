// Router: the experts each token goes to and their weights, in 64 bits.
//
// A choice is a decision, and neighbours around the border have to fall the
// same way wherever they are computed, so the logits are sums in 64 bits of
// products that are exact (bf16 x bf16), on v_mfma_f64_16x16x4_f64: 16 tokens
// by 16 experts. What bounds it:
//   - a large panel: that instruction. Alone it runs in 74 cycles with two or
//     more waves a SIMD (86 with one), and the conversion of its inputs to 64
//     bits is not hidden behind it: 2 more vector instructions for each make it
//     88. 2048 tokens, 256 experts, 4096 columns: 78 us, 55 TFLOP/s (a library's
//     64-bit product of inputs that are converted already: 125 us; of 4096^3:
//     74 TFLOP/s).
//   - some hundred tokens: rounds of whole tiles over the compute units, each
//     tile with all its columns (300 tokens 31 us, 700 44, 1024 46, 1500 74: 1.6
//     to 3.6 times their products at 74 TFLOP/s).
//   - a few tokens: latency, of two launches, a chain of 32 instructions and a
//     choice (1 token, 256 experts, 4096 columns: 8.7 us, of which an empty
//     launch takes 2.6 each).
//
// Order of a logit, whatever the panel: chunks of 128 columns (of 64, 1 token
// takes 10.7 us for the chunks to add, of 256 9.5 for the chain), each a chain
// of matrix instructions from 0; eight sums over the chunks c % 8 = 0 .. 7 in
// order; then their tree. Few tiles: every chunk is a wave of its own, the
// chunks' sums go to the workspace, and the kernel that chooses adds them.
// Many tiles: the eight waves of a workgroup each walk an eighth of the chunks
// and add in LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));

constexpr int64_t kRouteAlign = 256;
constexpr int kTile = 16, kStepCols = 32, kChunkCols = 128;
constexpr int kWaves = 8;       // sums of a logit, and waves that share a tile's chunks
constexpr int kSplitWaves = 4;  // chunks of a workgroup where each has a wave of its own
// Up to so many 16 x 16 tiles each chunk has a wave of its own: 256 experts of
// 4096 columns, against eight waves a tile, 128 tokens (128 tiles) 15.8 against
// about 19 us, 200 tokens 20.9 against 19.5, 256 tokens 23.1 against 19.6.
constexpr int kSplitTiles = 128;

inline int route_chunks(int64_t cols) { return (int)ceil_div(cols, kChunkCols); }
inline bool route_split(int64_t experts, int64_t M) { return ceil_div(experts, kTile) * ceil_div(M, kTile) <= kSplitTiles; }

struct RouteArgs {
    const uint16_t* w;
    const uint16_t* x;
    const float* bias;
    double* logits;  // [M, E], or [chunk][M, E] where the chunks are added later
    int32_t* ids;
    float* weights;
    int32_t E, M, cols, K, score, normalize, chunks;
    float scale;
};

__device__ __forceinline__ double tree(const double (&s)[kWaves]) {
    return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// The inputs of RX by RW tiles (tokens by experts). Lane (n, k) of a wave holds
// 8 columns, k-th of four, of token or expert n in a 32-column step;
// instruction j takes column j of each. The loads of AHEAD steps are in flight.
constexpr int kSteps = kChunkCols / kStepCols;
template <int RX, int RW, int AHEAD>
struct Steps {
    const uint8_t *x, *w;        // the first rows
    uint32_t xrow[RX], wrow[RW];  // the lane's rows from there, in bytes
    uint4 xd[AHEAD][RX], wd[AHEAD][RW];
    int cols, kg;

    __device__ __forceinline__ void start(const RouteArgs& a, int m0, int e0, int lane) {
        x = reinterpret_cast<const uint8_t*>(a.x + (int64_t)m0 * a.cols);
        w = reinterpret_cast<const uint8_t*>(a.w + (int64_t)e0 * a.cols);
        cols = a.cols;
        kg = lane >> 4;
#pragma unroll
        for (int i = 0; i < RX; ++i) xrow[i] = 2u * a.cols * min(i * kTile + (lane & 15), a.M - 1 - m0);
#pragma unroll
        for (int i = 0; i < RW; ++i) wrow[i] = 2u * a.cols * min(i * kTile + (lane & 15), a.E - 1 - e0);
    }
    __device__ __forceinline__ void load(int slot, int c) {
        // a last step has 16 columns, which both halves of the wave then read
        const uint32_t in = c + kStepCols <= cols ? 16 * kg : 16 * (kg & 1);
        const int64_t at = 2 * (c < cols ? c : 0);
#pragma unroll
        for (int i = 0; i < RX; ++i) xd[slot][i] = load_global16(x + at + (xrow[i] + in));
#pragma unroll
        for (int i = 0; i < RW; ++i) wd[slot][i] = load_global16(w + at + (wrow[i] + in));
    }
    static __device__ __forceinline__ double value(const uint4& d, int k) {
        const uint32_t q[4] = {d.x, d.y, d.z, d.w};
        return (double)as_f32(k % 2 ? q[k / 2] & 0xFFFF0000u : q[k / 2] << 16);
    }
    // acc += the step in `slot`, columns c on; that slot then takes the step at `next`.
    __device__ __forceinline__ void multiply(int slot, int c, bool more, int next, v4d (&acc)[RX][RW]) {
        if (c + kStepCols > cols) {  // zeros past the last column
            const uint32_t keep = c + 8 * kg < cols ? ~0u : 0u;
#pragma unroll
            for (int i = 0; i < RX; ++i)
                xd[slot][i] = make_uint4(xd[slot][i].x & keep, xd[slot][i].y & keep, xd[slot][i].z & keep, xd[slot][i].w & keep);
#pragma unroll
            for (int i = 0; i < RW; ++i)
                wd[slot][i] = make_uint4(wd[slot][i].x & keep, wd[slot][i].y & keep, wd[slot][i].z & keep, wd[slot][i].w & keep);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            double xe[RX], we[RW];
#pragma unroll
            for (int i = 0; i < RX; ++i) xe[i] = value(xd[slot][i], k);
#pragma unroll
            for (int i = 0; i < RW; ++i) we[i] = value(wd[slot][i], k);
            if (k == 7) {
                if (more) load(slot, next);
                __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not where they are used
            }
#pragma unroll
            for (int i = 0; i < RX; ++i)
#pragma unroll
                for (int j = 0; j < RW; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(xe[i], we[j], acc[i][j], 0, 0, 0);
        }
    }
};

// Register i of lane l of a result tile is token 4 i + l / 16, expert l % 16.
template <int RX, int RW, bool SPLIT>
__global__ __launch_bounds__(64 * kWaves) void k_route_logits(RouteArgs a) {
    constexpr int T = RX * RW;
    __shared__ double sums[SPLIT ? 1 : kWaves][SPLIT ? 1 : T * 4 * 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, kg = lane >> 4;
    // Many tiles: workgroups that follow each other, on one L2 after the other,
    // take other tokens, so that an L2 reads its tokens once (2048 tokens 79.6 ->
    // 78.3 us; 146 -> 34 MB read).
    const int e0 = (SPLIT ? blockIdx.x : blockIdx.y) * RW * kTile, m0 = (SPLIT ? blockIdx.y : blockIdx.x) * RX * kTile;
    constexpr int AHEAD = T < 4 ? kSteps : 2;
    Steps<RX, RW, AHEAD> steps;
    steps.start(a, m0, e0, lane);
    v4d acc[RX][RW], total[RX][RW];
    const auto clear = [](v4d(&t)[RX][RW]) {
#pragma unroll
        for (int i = 0; i < RX; ++i)
#pragma unroll
            for (int j = 0; j < RW; ++j) t[i][j] = v4d{0.0, 0.0, 0.0, 0.0};
    };
    const auto store = [&](double* out, int tile, int k, double v) {
        const int m = m0 + tile / RW * kTile + 4 * k + kg, e = e0 + tile % RW * kTile + n;
        if (m < a.M && e < a.E) out[(int64_t)m * a.E + e] = v;
    };
    if constexpr (SPLIT) {
        const int chunk = blockIdx.z * kSplitWaves + wave, c0 = chunk * kChunkCols;
        if (chunk >= a.chunks) return;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) steps.load(s, c0 + s * kStepCols);
        __builtin_amdgcn_sched_barrier(0);
        clear(acc);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) steps.multiply(s, c0 + s * kStepCols, false, 0, acc);
#pragma unroll
        for (int k = 0; k < 4; ++k) store(a.logits + (int64_t)chunk * a.M * a.E, 0, k, acc[0][0][k]);
    } else {
        clear(total);
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) steps.load(s, wave * kChunkCols + s * kStepCols);
        for (int chunk = wave; chunk < a.chunks; chunk += kWaves) {
            clear(acc);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int t = s + AHEAD, c0 = chunk * kChunkCols;
                steps.multiply(s % AHEAD, c0 + s * kStepCols, true, c0 + t / kSteps * kWaves * kChunkCols + t % kSteps * kStepCols, acc);
            }
#pragma unroll
            for (int i = 0; i < RX; ++i)
#pragma unroll
                for (int j = 0; j < RW; ++j) total[i][j] += acc[i][j];
        }
#pragma unroll
        for (int t = 0; t < T * 4; ++t) sums[wave][t * 64 + lane] = total[t / 4 / RW][t / 4 % RW][t % 4];
        __syncthreads();
        for (int t = wave; t < T * 4; t += kWaves) {
            double s[kWaves];
#pragma unroll
            for (int v = 0; v < kWaves; ++v) s[v] = sums[v][t * 64 + lane];
            store(a.logits, t / 4, t % 4, tree(s));
        }
    }
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A reduction over the wave, the same bits in every lane.
template <typename F>
__device__ __forceinline__ double reduce64(double v, F f) {
    const auto halves = [&](bool by32) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
        const auto a = by32 ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false) : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
        const auto b = by32 ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false) : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        return f(__builtin_bit_cast(double, (uint64_t)b[0] << 32 | a[0]), __builtin_bit_cast(double, (uint64_t)b[1] << 32 | a[1]));
    };
    v = halves(true);
    v = halves(false);
    v = f(v, dpp64<kRowRor8>(v));
    v = f(v, dpp64<kRowRor4>(v));
    v = f(v, dpp64<kQuadXor2>(v));
    v = f(v, dpp64<kQuadXor1>(v));
    return v;
}

// Largest of one value per lane, the same in every lane.
__device__ __forceinline__ uint32_t most_of_wave(uint32_t v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(b[0], b[1]);
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kRowRor8, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kRowRor4, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kQuadXor2, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kQuadXor1, 0xF, 0xF, false));
    return v;
}

// A number as an unsigned one that orders the same way, never 0.
__device__ __forceinline__ uint64_t rank_of(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 as 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double lane_value64(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A logit from its chunks' sums, N loads at a time, and behind the first of
// them its expert's bias.
template <int N>
__device__ __forceinline__ double add_chunks(const RouteArgs& a, int64_t at, int e, float& bias) {
    const int64_t n = (int64_t)a.M * a.E;
    double s[kWaves] = {};
    for (int c = 0; c < a.chunks; c += N) {
        double v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = a.logits[at + min(c + k, a.chunks - 1) * n];
        if (c == 0 && a.bias) bias = a.bias[e];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (c + k < a.chunks) s[k % kWaves] += v[k];
    }
    return tree(s);
}

// sigmoid(l) or sqrt(log(1 + exp(l))), which is exp(l / 2) to the last bit far
// below 0, where exp(l) is no normal number any more but its root still is.
__device__ __forceinline__ double own_score(int score, double l) {
    const double t = exp(-fabs(l));  // at most 1
    if (score == FP8BLK_SCORE_SIGMOID) return l >= 0.0 ? 1.0 / (1.0 + t) : t / (1.0 + t);
    if (l < -700.0) return exp(0.5 * l);
    return sqrt((l > 0.0 ? l : 0.0) + log1p(t));
}

// One wave per token; lane l holds experts l, l + 64, ... WIDE: the logits are
// first added by a workgroup, a thread each.
template <int NE, bool WIDE>
__global__ __launch_bounds__(WIDE ? 64 * NE : 256) void k_route_choose(RouteArgs a) {
    __shared__ double whole[WIDE ? FP8BLK_MAX_EXPERTS : 1];
    __shared__ float biases[WIDE ? FP8BLK_MAX_EXPERTS : 1];
    const int lane = threadIdx.x & 63;
    const int64_t m = WIDE ? blockIdx.x : (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const double lowest = -__builtin_inf();
    if constexpr (WIDE) {
        const int e = threadIdx.x;
        if (e < a.E) {
            float b = 0.0f;
            const double l = a.chunks > 16 ? add_chunks<32>(a, m * a.E + e, e, b) : add_chunks<16>(a, m * a.E + e, e, b);
            biases[e] = b;
            whole[e] = a.score == FP8BLK_SCORE_SOFTMAX ? l : own_score(a.score, l);
        }
        __syncthreads();
        if (threadIdx.x >= 64) return;
    }
    if (m >= a.M) return;
    double s[NE];
    uint64_t pick[NE];  // ranks; 0: not to be chosen
    float bias[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = min(lane + 64 * i, a.E - 1);
        if constexpr (WIDE) bias[i] = biases[e];
        else bias[i] = a.bias ? a.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        if constexpr (WIDE) s[i] = e < a.E ? whole[e] : lowest;
        else s[i] = e < a.E ? a.logits[m * a.E + e] : lowest;
    }
    if (a.score == FP8BLK_SCORE_SOFTMAX) {
        double top = lowest, sum = 0.0;
#pragma unroll
        for (int i = 0; i < NE; ++i) top = s[i] > top ? s[i] : top;
        top = reduce64(top, [](double p, double q) { return p > q ? p : q; });
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = exp(s[i] - top);
            sum += lane + 64 * i < a.E ? s[i] : 0.0;
        }
        sum = reduce64(sum, [](double p, double q) { return p + q; });
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] /= sum;
    } else if (!WIDE) {
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] = own_score(a.score, s[i]);
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const double c = s[i] + (double)bias[i];
        pick[i] = lane + 64 * i < a.E && c > lowest ? rank_of(c) : 0;  // NaN and -inf: never chosen
    }
    double mine = 0.0, total = 0.0;  // lane k: the k-th choice's score
    int my_id = -1;
    for (int k = 0; k < a.K; ++k) {
        uint64_t best = 0;
        double score = 0.0;
        int id = FP8BLK_MAX_EXPERTS;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (pick[i] > best) best = pick[i], score = s[i], id = lane + 64 * i;
        const uint32_t hi = (uint32_t)(best >> 32), most = most_of_wave(hi);
        if (most == 0) break;  // nothing left
        uint64_t who = __ballot(hi == most);
        if (who & (who - 1)) {  // the high halves do not tell
            const uint32_t lo = hi == most ? (uint32_t)best : 0;
            who &= __ballot(lo == most_of_wave(lo));
        }
        int at = __builtin_ctzll(who), least = __builtin_amdgcn_readlane(id, at);
        for (who &= who - 1; who; who &= who - 1) {  // a tie: the lowest index
            const int l = __builtin_ctzll(who), other = __builtin_amdgcn_readlane(id, l);
            if (other < least) least = other, at = l;
        }
        const double p = lane_value64(score, at);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (least == lane + 64 * i) pick[i] = 0;
        if (lane == k) mine = p, my_id = least;
        total += p;
    }
    if (lane < a.K) {
        if (a.normalize) mine = total > 0.0 ? mine / total : 0.0;
        a.ids[m * a.K + lane] = my_id;
        a.weights[m * a.K + lane] = (float)(mine * (double)a.scale);
    }
}

template <int NE>
void choose(const RouteArgs& a, bool wide, hipStream_t s) {
    if (wide) k_route_choose<NE, true><<<(unsigned)a.M, 64 * NE, 0, s>>>(a);
    else k_route_choose<NE, false><<<(unsigned)ceil_div(a.M, 4), 256, 0, s>>>(a);
}

// The tiles of a workgroup. Every matrix instruction waits for the conversions
// of its inputs (they share the 64-bit units), which more tiles share; fewer
// fill the compute units more evenly. So: the least of the rounds of workgroups
// over the compute units times the measured us of one round at 4096 columns.
// By 256 experts of 4096 columns, us for 4x2, 2x2, 2x1, 1x1 tiles: 2048 tokens
// 80 83 91 99, 1500 tokens 79 82 71 77, 1024 tokens 77 46 50 54, 700 tokens
// 77 45 50 43, 300 tokens 75 44 29 31.
void logits(const RouteArgs& a, int64_t te, int64_t tm, int cus, hipStream_t s) {
    const struct {
        int rx, rw;
        double us;
    } forms[] = {{4, 2, 74.5}, {2, 2, 39.0}, {2, 1, 21.5}, {1, 1, 11.8}};
    int best = 0;
    double least = 1e300;
    for (int f = 0; f < 4; ++f) {
        const double us = forms[f].us * (double)ceil_div(ceil_div(te, forms[f].rw) * ceil_div(tm, forms[f].rx), cus);
        if (us < least) least = us, best = f;
    }
    const dim3 grid((unsigned)ceil_div(tm, forms[best].rx), (unsigned)ceil_div(te, forms[best].rw));
    if (best == 0) k_route_logits<4, 2, false><<<grid, 64 * kWaves, 0, s>>>(a);
    else if (best == 1) k_route_logits<2, 2, false><<<grid, 64 * kWaves, 0, s>>>(a);
    else if (best == 2) k_route_logits<2, 1, false><<<grid, 64 * kWaves, 0, s>>>(a);
    else k_route_logits<1, 1, false><<<grid, 64 * kWaves, 0, s>>>(a);
}

bool route_shape_ok(int64_t experts, int64_t cols, int64_t M) {
    return experts >= 1 && experts <= FP8BLK_MAX_EXPERTS && M >= 1 && M <= FP8BLK_MAX_PANEL && shape_ok(experts, cols);
}

}  // namespace

size_t route_workspace_bytes(int64_t experts, int64_t cols, int64_t M) {
    if (!route_shape_ok(experts, cols, M)) return 0;
    const int64_t n = M * experts * (route_split(experts, M) ? route_chunks(cols) : 1);
    return (size_t)(ceil_div(n * (int64_t)sizeof(double), kRouteAlign) * kRouteAlign);
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
    RouteArgs a = {w_bf16, x_bf16, bias, static_cast<double*>(ws), ids, weights, (int32_t)experts, (int32_t)M, (int32_t)cols,
                   top_k, score, normalize != 0, route_chunks(cols), scale};
    const int cus = device_cus();
    if (cus < 1) return FP8BLK_ERR_HIP;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const bool split = route_split(experts, M);
    const int64_t te = ceil_div(experts, kTile), tm = ceil_div(M, kTile);
    if (split)
        k_route_logits<1, 1, true><<<dim3((unsigned)te, (unsigned)tm, (unsigned)ceil_div(a.chunks, kSplitWaves)), 64 * kSplitWaves, 0, s>>>(a);
    else
        logits(a, te, tm, cus, s);
    // As many logits a lane as there are, up to a power of two (2048 tokens, 384
    // experts of 2048 columns: 72 us with 8, 77 with 16; 1 token of 7168 13.4, 15.1).
    if (experts <= 64) choose<1>(a, split, s);
    else if (experts <= 128) choose<2>(a, split, s);
    else if (experts <= 256) choose<4>(a, split, s);
    else if (experts <= 512) choose<8>(a, split, s);
    else choose<16>(a, split, s);
    return launch_status();
}

// Rotary positions on q and k, and new keys and values into a paged cache.
//
// A pair (a, b) of a head's rotated columns is the complex number a + ib; token
// n multiplies it by mscale * exp(i p f). The angle p f of a far position has
// lost its fraction of a turn in f32 (p f = 1e6: steps of 0.06), so it is formed
// and reduced in 64 bits, and only its cosine and sine are rounded.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "fp8blk.h"
#include "fp8blk_device.hpp"
#include "fp8blk_host.hpp"

namespace fp8blk {
namespace {

struct RowsIn {  // q, k or v: [N, heads, pass | rot], and where its rows go
    const char* pass;
    const char* rot;
    int64_t pass_token, pass_head, rot_token, rot_head;  // bytes
    const uint16_t* norm;
    char* out;
    int64_t out_page, out_slot, out_head;  // bytes; q: a token is a slot
    int32_t heads, pass_units, rot_units, norm_cols;
    int32_t first;  // of the tasks that are its rows
    int32_t bf16, e4m3, rot_first;
    float scale;
};

struct RopeArgs {
    RowsIn in[3];  // q, k, v
    const double* freqs;
    const int32_t* positions;
    const int32_t* slots;
    int64_t n_slots;
    int32_t tasks, rot, page_shift, lanes_log2;
    float mscale, eps;
};

constexpr int kThreads = 256, kUnit = 8;  // a lane takes 8 columns, or 4 pairs, at a time

// cos(a) and sin(a) in 64 bits for the rounding to f32: a less its nearest
// multiple of pi/2 (taken off in two parts), then the Taylor series, whose first
// terms left out are below 2^-29 and 2^-32 for |r| <= pi/4.
__device__ __forceinline__ void cos_sin(double a, double& c, double& s) {
    const double k = __builtin_rint(a * 0.63661977236758134308);
    double r = __builtin_fma(-k, 1.57079632679489655800, a);
    r = __builtin_fma(-k, 6.12323399573676603587e-17, r);
    const double z = r * r;
    const double sr = r + r * z * (-1.0 / 6 + z * (1.0 / 120 + z * (-1.0 / 5040 + z * (1.0 / 362880))));
    const double cr = 1.0 + z * (-0.5 + z * (1.0 / 24 + z * (-1.0 / 720 + z * (1.0 / 40320 + z * (-1.0 / 3628800)))));
    const int quadrant = (int)((int64_t)k & 3);
    const double x = quadrant & 1 ? sr : cr, y = quadrant & 1 ? cr : sr;
    c = quadrant == 1 || quadrant == 2 ? -x : x;
    s = quadrant >= 2 ? -y : y;
}

typedef unsigned v2u __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load4(const char* p, bool bf16, int64_t i, float* v) {
    if (bf16) {
        const v2u d = *(__attribute__((address_space(1))) const v2u*)(p + 2 * i);
        widen2_bf16(d.x, v), widen2_bf16(d.y, v + 2);
    } else {
        const uint4 d = load_global16(p + 4 * i);
        v[0] = as_f32(d.x), v[1] = as_f32(d.y), v[2] = as_f32(d.z), v[3] = as_f32(d.w);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2bf{(__bf16)lo, (__bf16)hi});
}

// v / scale within e4m3's range; a NaN stays one.
__device__ __forceinline__ float in_e4m3(float v, float scale) {
    v = v / scale;
    return v > 448.0f ? 448.0f : v < -448.0f ? -448.0f : v;
}

__device__ __forceinline__ void store4(char* p, const RowsIn& t, int64_t i, const float* v) {
    if (t.e4m3) {
        int d = __builtin_amdgcn_cvt_pk_fp8_f32(in_e4m3(v[0], t.scale), in_e4m3(v[1], t.scale), 0, false);
        d = __builtin_amdgcn_cvt_pk_fp8_f32(in_e4m3(v[2], t.scale), in_e4m3(v[3], t.scale), d, true);
        *(__attribute__((address_space(1))) int*)(p + i) = d;
    } else {
        *(__attribute__((address_space(1))) v2u*)(p + 2 * i) = v2u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
}

// The U units of a lane in a row of t: units at, at + lanes, ... of 8 columns, the
// rotated ones 4 pairs.
template <int U, bool INTERLEAVED>
struct Units {
    float v[U][kUnit];

    // Columns of its first and last four values in the part that they come from and
    // in the written row.
    struct Place {
        bool in, turned;
        int from[2], to[2], pair;
    };
    static __device__ __forceinline__ Place place(const RowsIn& t, int u) {
        const int first = t.rot_first ? 0 : t.pass_units, j = u - first;
        Place p;
        p.in = u < t.pass_units + t.rot_units;
        p.turned = j >= 0 && j < t.rot_units;
        const int half = t.rot_units * kUnit / 2, other = t.rot_first ? u - t.rot_units : u;
        p.from[0] = !p.turned ? other * kUnit : INTERLEAVED ? kUnit * j : 4 * j;
        p.from[1] = p.turned && !INTERLEAVED ? half + 4 * j : p.from[0] + 4;
        const int start = p.turned ? first : t.rot_first ? t.rot_units : 0;
        p.to[0] = start * kUnit + p.from[0], p.to[1] = start * kUnit + p.from[1];
        p.pair = 4 * j;
        return p;
    }

    __device__ __forceinline__ void load(const RowsIn& t, int64_t n, int head, int at, int lanes) {
        if (head >= t.heads) return;
        const char* pass = t.pass + n * t.pass_token + head * t.pass_head;
        const char* rot = t.rot + n * t.rot_token + head * t.rot_head;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const Place p = place(t, at + k * lanes);
            if (!p.in) continue;
            load4(p.turned ? rot : pass, t.bf16, p.from[0], v[k]);
            load4(p.turned ? rot : pass, t.bf16, p.from[1], v[k] + 4);
        }
    }

    __device__ __forceinline__ float mean_square(const RowsIn& t, int at, int lanes, bool whole) const {
        float square = 0.0f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const Place p = place(t, at + k * lanes);
            if (p.in && (whole || !p.turned))
#pragma unroll
                for (int i = 0; i < kUnit; ++i) square = __builtin_fmaf(v[k][i], v[k][i], square);
        }
        for (int m = 1; m < lanes; m <<= 1) square += __shfl_xor(square, m);
        return square / (float)t.norm_cols;
    }

    __device__ __forceinline__ void finish(const RowsIn& t, char* out, int head, int at, int lanes, float eps, const float (*turn)[FP8BLK_MAX_ROT / 2]) {
        if (head >= t.heads) return;  // all lanes of a row
        const bool whole = t.norm_cols > t.pass_units * kUnit;
        float unit = 1.0f;
        if (t.norm) {
            float mean = mean_square(t, at, lanes, whole) + eps;
            const bool far = !(mean >= 0x1p-100f && mean <= 0x1p110f);
            if (__any(far)) {
                // Squares (and eps) that leave f32's range: once more, of such a row's
                // values times a power of two that brings those of any size back into it.
                const float by = !far ? 1.0f : mean < 1.0f ? 0x1p100f : 0x1p-70f;
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const Place p = place(t, at + k * lanes);
                    if (p.in && (whole || !p.turned))
#pragma unroll
                        for (int i = 0; i < kUnit; ++i) v[k][i] *= by;
                }
                mean = mean_square(t, at, lanes, whole) + eps * by * by;
            }
            unit = 1.0f / sqrtf(mean);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const Place p = place(t, at + k * lanes);
            if (!p.in) continue;
            if (t.norm && (whole || !p.turned)) {  // weights of the whole row by its columns, of the pass part alone by that part's
                float w[kUnit];
                load4((const char*)t.norm, true, whole ? p.to[0] : p.from[0], w);
                load4((const char*)t.norm, true, whole ? p.to[1] : p.from[1], w + 4);
#pragma unroll
                for (int i = 0; i < kUnit; ++i) v[k][i] = v[k][i] * unit * w[i];
            }
            if (p.turned) {
                const float4 c = *(const float4*)&turn[0][p.pair], s = *(const float4*)&turn[1][p.pair];
                const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& x = v[k][INTERLEAVED ? 2 * i : i];
                    float& y = v[k][INTERLEAVED ? 2 * i + 1 : i + 4];
                    const float x0 = x, y0 = y;
                    x = x0 * cs[i] - y0 * sn[i];
                    y = x0 * sn[i] + y0 * cs[i];
                }
            }
            char* const row = out + head * t.out_head;
            store4(row, t, p.to[0], v[k]);
            store4(row, t, p.to[1], v[k] + 4);
        }
    }
};

// A workgroup takes the heads of q, k and v of one token, a wave 64 / lanes of one of
// them at a time (so that all its lanes read the same description of it), a row
// `lanes` lanes. The next rows are asked for before the present ones are worked on,
// the first before the cosines and sines, which are formed once a workgroup. Bound by
// memory: 8191 tokens, 32 + 4 heads of 128, f32 to bf16 and e4m3, 50 us, 4.9 TB/s (rows
// dealt to waves whatever their kind, and loads after the previous row's stores: 78).
template <int U, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void k_rope_append(RopeArgs a) {
    __shared__ __attribute__((aligned(16))) float turn[2][FP8BLK_MAX_ROT / 2];
    const int64_t n = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lanes = 1 << a.lanes_log2, at = lane & (lanes - 1), row = lane >> a.lanes_log2, rows = 64 >> a.lanes_log2;
    const int step = 4 * gridDim.y;
    int task = 4 * blockIdx.y + wave;
    auto rows_in = [&](int t) -> const RowsIn& { return a.in[t >= a.in[2].first ? 2 : t >= a.in[1].first ? 1 : 0]; };
    Units<U, INTERLEAVED> here, next;
    if (task < a.tasks) {
        const RowsIn& t = rows_in(task);
        next.load(t, n, (task - t.first) * rows + row, at, lanes);
    }
    if ((int)threadIdx.x < a.rot / 2) {
        double c, s;
        cos_sin((double)a.positions[n] * a.freqs[threadIdx.x], c, s);
        turn[0][threadIdx.x] = (float)((double)a.mscale * c);
        turn[1][threadIdx.x] = (float)((double)a.mscale * s);
    }
    const int64_t slot = a.slots ? (int64_t)__builtin_amdgcn_readfirstlane(a.slots[n]) : -1;
    const int64_t page = slot >> a.page_shift, in_page = slot & ((1 << a.page_shift) - 1);
    const bool stored = slot >= 0 && slot < a.n_slots;
    __syncthreads();
    for (; task < a.tasks; task += step) {
        here = next;
        if (task + step < a.tasks) {
            const RowsIn& t = rows_in(task + step);
            next.load(t, n, (task + step - t.first) * rows + row, at, lanes);
        }
        const RowsIn& t = rows_in(task);
        const bool is_q = task < a.in[1].first;
        if (!is_q && !stored) continue;
        char* const out = t.out + (is_q ? n * t.out_slot : page * t.out_page + in_page * t.out_slot);
        here.finish(t, out, (task - t.first) * rows + row, at, lanes, a.eps, turn);
    }
}

template <int U>
void launch(const RopeArgs& a, bool interleaved, dim3 grid, hipStream_t s) {
    if (interleaved) k_rope_append<U, true><<<grid, kThreads, 0, s>>>(a);
    else k_rope_append<U, false><<<grid, kThreads, 0, s>>>(a);
}

// Span in bytes that [n, heads, cols] values with these strides reach.
int64_t span(int64_t n, int64_t token, int64_t heads, int64_t head, int64_t cols, int64_t size) {
    return ((n - 1) * token + (heads - 1) * head + cols) * size;
}

constexpr int64_t kMaxStride = INT64_C(1) << 40;
bool stride_ok(int64_t s, int64_t least) { return s >= least && s <= kMaxStride && s % 8 == 0; }

// q, k or v as given; false where refused.
bool rows_ok(const fp8blk_heads& h, int64_t rot, int64_t N, bool turned) {
    if (h.type != FP8BLK_F32 && h.type != FP8BLK_BF16) return false;
    if (h.heads < 1 || h.heads > FP8BLK_MAX_HEADS || h.pass_cols < 0 || h.pass_cols % 8) return false;
    if (!turned && (h.rot || h.norm || h.norm_cols)) return false;
    if (!h.pass != (h.pass_cols == 0) || !h.rot != !turned || (!h.pass && !h.rot)) return false;
    const int64_t cols = h.pass_cols + (turned ? rot : 0);
    if (cols > FP8BLK_MAX_HEAD_COLS || !aligned(h.pass, 16) || !aligned(h.rot, 16) || !aligned(h.norm, 16)) return false;
    if (h.pass && (!stride_ok(h.pass_token, 0) || !stride_ok(h.pass_head, 0))) return false;
    if (h.rot && (!stride_ok(h.rot_token, 0) || !stride_ok(h.rot_head, 0))) return false;
    return h.norm ? h.norm_cols == cols || (h.norm_cols == h.pass_cols && h.pass_cols > 0) : h.norm_cols == 0;
}

}  // namespace

bool cache_ok(const fp8blk_cache& c) {
    if (c.type != FP8BLK_BF16 && c.type != FP8BLK_E4M3) return false;
    const float lo = 0x1p-100f, hi = 0x1p100f;
    if (c.type == FP8BLK_BF16 ? c.k_scale != 1.0f || c.v_scale != 1.0f
                              : !(c.k_scale >= lo && c.k_scale <= hi && c.v_scale >= lo && c.v_scale <= hi))
        return false;
    if (c.page_size < 1 || c.page_size > FP8BLK_MAX_PAGE || (c.page_size & (c.page_size - 1)) || c.pages < 1 ||
        c.pages > ((INT64_C(1) << 31) - 1) / c.page_size || c.heads < 1 || c.heads > FP8BLK_MAX_HEADS)
        return false;
    auto cols_ok = [](int64_t n) { return n >= 16 && n <= FP8BLK_MAX_HEAD_COLS && n % 16 == 0; };
    auto strides_ok = [&](int64_t page, int64_t slot, int64_t head, int64_t cols) {
        for (int64_t s : {page, slot, head})
            if (s < cols || s > kMaxStride || s % 16) return false;
        return page <= (INT64_C(1) << 56) / c.pages;
    };
    if (!cols_ok(c.k_cols) || !cols_ok(c.v_cols) || !c.k || !aligned(c.k, 16) || !aligned(c.v, 16)) return false;
    if (!strides_ok(c.k_page, c.k_slot, c.k_head, c.k_cols)) return false;
    return c.v ? strides_ok(c.v_page, c.v_slot, c.v_head, c.v_cols) : c.v_cols <= c.k_cols;
}

int64_t cache_span(const fp8blk_cache& c, bool values) {
    const int64_t size = c.type == FP8BLK_E4M3 ? 1 : 2;
    return values ? ((c.pages - 1) * c.v_page + (c.page_size - 1) * c.v_slot + (c.heads - 1) * c.v_head + c.v_cols) * size
                  : ((c.pages - 1) * c.k_page + (c.page_size - 1) * c.k_slot + (c.heads - 1) * c.k_head + c.k_cols) * size;
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_rope_freqs(int64_t rot, double base, double factor, double original, double fast, double slow,
                                 double* freqs) {
    if (!freqs || rot < 8 || rot > FP8BLK_MAX_ROT || rot % 8) return FP8BLK_ERR_ARG;
    if (!(base > 0) || std::isinf(base) || !(factor >= 1) || std::isinf(factor)) return FP8BLK_ERR_ARG;
    if (factor > 1 && (!(original >= 1) || std::isinf(original) || !(slow >= 0) || !(fast >= slow) || std::isinf(fast)))
        return FP8BLK_ERR_ARG;
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -2.0 * (double)i / (double)rot);
        if (factor > 1) {
            const double turns = original * f / 6.283185307179586;
            const double keep = turns >= fast ? 1.0 : turns <= slow ? 0.0 : (turns - slow) / (fast - slow);
            f *= keep + (1.0 - keep) / factor;
        }
        freqs[i] = f;
    }
    return FP8BLK_OK;
}

extern "C" int fp8blk_rope_append(const fp8blk_rope* rope, const int32_t* positions, int64_t N, const fp8blk_heads* q,
                                  uint16_t* q_out, int64_t q_token, int64_t q_head, const fp8blk_heads* k,
                                  const fp8blk_heads* v, const fp8blk_cache* cache, const int32_t* slots, float eps,
                                  fp8blk_stream_t stream) {
    if (!rope || !rope->freqs || !aligned(rope->freqs, 8) || rope->rot < 8 || rope->rot > FP8BLK_MAX_ROT || rope->rot % 8 ||
        !std::isfinite(rope->mscale))
        return FP8BLK_ERR_ARG;
    if (!positions || !aligned(positions, 4) || N < 1 || N > FP8BLK_MAX_PANEL || !(eps >= 0.0f) || std::isinf(eps))
        return FP8BLK_ERR_ARG;
    if ((!q && !k) || !q != !q_out || !k != !cache || !k != !slots || (v && !k) || !aligned(slots, 4)) return FP8BLK_ERR_ARG;
    RopeArgs a = {};
    const fp8blk_heads* in[3] = {q, k, v};
    int64_t most = 0;
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        const fp8blk_heads& h = *in[i];
        if (!rows_ok(h, rope->rot, N, i < 2)) return FP8BLK_ERR_ARG;
        const int64_t size = h.type == FP8BLK_F32 ? 4 : 2;
        const int rot_units = i < 2 ? (int)(rope->rot / kUnit) : 0;
        a.in[i] = {(const char*)h.pass, (const char*)h.rot, h.pass_token * size, h.pass_head * size, h.rot_token * size,
                   h.rot_head * size, h.norm, nullptr, 0, 0, 0, (int32_t)h.heads, (int32_t)(h.pass_cols / kUnit), rot_units,
                   (int32_t)h.norm_cols, 0, h.type == FP8BLK_BF16, 0, rope->rot_first != 0, 1.0f};
        const int64_t units = h.pass_cols / kUnit + rot_units;
        most = units > most ? units : most;
    }
    struct Span {
        const void* p;
        int64_t bytes;
    } outs[3] = {};
    if (q) {
        const int64_t cols = q->pass_cols + rope->rot;
        if (!aligned(q_out, 16) || !stride_ok(q_token, cols) || !stride_ok(q_head, cols)) return FP8BLK_ERR_ARG;
        a.in[0].out = (char*)q_out;
        a.in[0].out_slot = 2 * q_token;
        a.in[0].out_head = 2 * q_head;
        outs[0] = {q_out, span(N, q_token, q->heads, q_head, cols, 2)};
    }
    if (k) {
        if (!cache_ok(*cache) || !cache->v != !v || cache->k == cache->v) return FP8BLK_ERR_ARG;
        if (k->heads != cache->heads || k->pass_cols + rope->rot != cache->k_cols) return FP8BLK_ERR_ARG;
        if (v && (v->heads != cache->heads || v->pass_cols != cache->v_cols)) return FP8BLK_ERR_ARG;
        const int64_t size = cache->type == FP8BLK_E4M3 ? 1 : 2;
        RowsIn& tk = a.in[1];
        tk.out = (char*)cache->k;
        tk.out_page = cache->k_page * size, tk.out_slot = cache->k_slot * size, tk.out_head = cache->k_head * size;
        tk.e4m3 = size == 1, tk.scale = cache->k_scale;
        outs[1] = {cache->k, cache_span(*cache, false)};
        if (v) {
            RowsIn& tv = a.in[2];
            tv.out = (char*)cache->v;
            tv.out_page = cache->v_page * size, tv.out_slot = cache->v_slot * size, tv.out_head = cache->v_head * size;
            tv.e4m3 = size == 1, tv.scale = cache->v_scale;
            outs[2] = {cache->v, cache_span(*cache, true)};
        }
        a.slots = slots;
        a.n_slots = cache->pages * cache->page_size;
        a.page_shift = __builtin_ctzll((unsigned long long)cache->page_size);
    }
    for (const Span& o : outs) {
        for (int i = 0; i < 3; ++i) {
            if (!in[i]) continue;
            const fp8blk_heads& h = *in[i];
            const int64_t size = h.type == FP8BLK_F32 ? 4 : 2;
            if (ranges_meet(o.p, o.bytes, h.pass, span(N, h.pass_token, h.heads, h.pass_head, h.pass_cols, size)) ||
                ranges_meet(o.p, o.bytes, h.rot, span(N, h.rot_token, h.heads, h.rot_head, rope->rot, size)) ||
                ranges_meet(o.p, o.bytes, h.norm, 2 * h.norm_cols))
                return FP8BLK_ERR_ARG;
        }
        if (ranges_meet(o.p, o.bytes, positions, 4 * N) || ranges_meet(o.p, o.bytes, slots, 4 * N) ||
            ranges_meet(o.p, o.bytes, rope->freqs, 4 * rope->rot))
            return FP8BLK_ERR_ARG;
    }
    if (ranges_meet(outs[0].p, outs[0].bytes, outs[1].p, outs[1].bytes) ||
        ranges_meet(outs[0].p, outs[0].bytes, outs[2].p, outs[2].bytes))
        return FP8BLK_ERR_ARG;

    a.freqs = rope->freqs;
    a.positions = positions;
    a.rot = (int32_t)rope->rot;
    a.mscale = rope->mscale;
    a.eps = eps;
    while (a.lanes_log2 < 6 && (1 << a.lanes_log2) < most) ++a.lanes_log2;
    for (RowsIn& t : a.in) {
        t.first = a.tasks;
        a.tasks += (t.heads + (64 >> a.lanes_log2) - 1) >> (6 - a.lanes_log2);
    }
    // A workgroup for 4 tasks, so that a wave reads once; of many tokens one for all of a
    // token's, which forms its angles once (256 tokens, 32 + 4 heads of 128: 4.8 us, 7.3 with
    // one; 1024: 10.4, 10.8; 2048: 15.2, 14.9).
    const dim3 grid((unsigned)N, (unsigned)(N > 1024 ? 1 : ceil_div(a.tasks, 4)));
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (most <= 64) launch<1>(a, rope->interleaved != 0, grid, s);
    else launch<2>(a, rope->interleaved != 0, grid, s);
    return launch_status();
}

// Attention of new tokens over a paged cache of keys and values.
#include "fp8blk_attn.hpp"

namespace fp8blk {
namespace {

__device__ __forceinline__ float element(const char* row, int i, bool e4m3) {
    if (e4m3) return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t*)row)[i], 0);
    return as_f32((uint32_t)((const uint16_t*)row)[i] << 16);
}

// One workgroup a row and head, wave w its keys w, w + 4, ...: running maximum and
// sum of the softmax, each lane columns lane, lane + 64, ...
__global__ __launch_bounds__(256) void k_attn_rows(AttnArgs a, int seq_of_row_steps, int k_cols, int v_cols, bool e4m3) {
    __shared__ float m_w[4], l_w[4], o_w[4][512];
    const int n = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int lo = 0, hi = a.seqs;  // the last sequence that starts at or before the row
    for (int i = 0; i < seq_of_row_steps; ++i) {
        const int mid = (lo + hi) >> 1;
        if (mid > lo) (a.starts[mid] <= n ? lo : hi) = mid;
    }
    const Seq s = sequence(a, lo);
    const int i = n - s.first;
    if (i < 0 || i >= s.rows) return;
    const int p = s.at + i, end = end_key(a, s, p);
    float q[16], o[8] = {};
    const char* q_row = a.q + n * a.q_token + h * a.q_head;
#pragma unroll
    for (int c = 0; c < 16; ++c) q[c] = c * 64 + lane < k_cols ? element(q_row, c * 64 + lane, false) : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int j = first_key(a, p) + wave; j < end; j += 4) {
        const int page = page_of(a, lo, j);
        if (page < 0) continue;
        const int64_t slot = j & ((1 << a.page_shift) - 1);
        const char* k = a.k + page * a.k_page + slot * a.k_slot + (h / a.group) * a.k_head;
        const char* v = a.v + page * a.v_page + slot * a.v_slot + (h / a.group) * a.v_head;
        float z = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c)
            if (c * 64 + lane < k_cols) z = __builtin_fmaf(q[c], element(k, c * 64 + lane, e4m3), z);
        z = tree64(z) * a.z_scale;
        const float top = z > m ? z : m, base = top == -INFINITY ? 0.0f : top;
        const float keep = exp2_fast(m - base), w = exp2_fast(z - base);
        m = top;
        l = l * keep + w;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c * 64 + lane < v_cols) o[c] = o[c] * keep + w * element(v, c * 64 + lane, e4m3);
    }
    if (lane == 0) m_w[wave] = m, l_w[wave] = l;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c * 64 + lane < v_cols) o_w[wave][c * 64 + lane] = o[c];
    __syncthreads();
    float top = fmaxf(fmaxf(m_w[0], m_w[1]), fmaxf(m_w[2], m_w[3]));
    const float base = top == -INFINITY ? 0.0f : top;
    float f[4], sum = 0.0f;
    for (int w = 0; w < 4; ++w) f[w] = exp2_fast(m_w[w] - base), sum += f[w] * l_w[w];
    const bool none = sum == 0.0f;  // the largest weight of a row that sees keys is 1
    if (a.sinks) sum += exp2_fast(a.sinks[h] * kLog2e - base);
    uint16_t* out = (uint16_t*)(a.out + n * a.out_token + h * a.out_head);
    for (int c = threadIdx.x; c < v_cols; c += 256) {
        const float v = f[0] * o_w[0][c] + f[1] * o_w[1][c] + f[2] * o_w[2][c] + f[3] * o_w[3][c];
        out[c] = __builtin_bit_cast(uint16_t, (__bf16)(none ? 0.0f : v * a.out_scale / sum));
    }
}

}  // namespace

int attn_args(AttnArgs& a, const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
              int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window, const float* sinks,
              uint16_t* out, int64_t out_token, int64_t out_head) {
    if (!cache || !batch || !q || !out || !cache_ok(*cache)) return FP8BLK_ERR_ARG;
    const fp8blk_cache& c = *cache;
    const fp8blk_batch& b = *batch;
    if (N < 1 || N > FP8BLK_MAX_PANEL || heads < 1 || heads > FP8BLK_MAX_HEADS || heads % c.heads) return FP8BLK_ERR_ARG;
    if (b.seqs < 1 || b.seqs > FP8BLK_MAX_PANEL || b.max_new < 1 || b.max_new > FP8BLK_MAX_PANEL || b.max_pages < 1 ||
        b.max_pages > (INT64_C(1) << 30) || b.max_len < 1 || b.max_len >= (INT64_C(1) << 30) || window < 0 ||
        window >= (INT64_C(1) << 30) || !std::isfinite(scale))
        return FP8BLK_ERR_ARG;
    if (!b.table || !b.lens || !b.starts) return FP8BLK_ERR_ARG;
    const void* words[] = {b.table, b.lens, b.starts, sinks};
    for (const void* p : words)
        if (!aligned(p, 4)) return FP8BLK_ERR_ARG;
    auto stride_ok = [](int64_t s, int64_t least) { return s >= least && s <= (INT64_C(1) << 40) && s % 8 == 0; };
    if (!aligned(q, 16) || !aligned(out, 16) || !stride_ok(q_token, 0) || !stride_ok(q_head, 0) ||
        !stride_ok(out_token, c.v_cols) || !stride_ok(out_head, c.v_cols))
        return FP8BLK_ERR_ARG;
    const int64_t out_bytes = 2 * ((N - 1) * out_token + (heads - 1) * out_head + c.v_cols);
    const int64_t q_bytes = 2 * ((N - 1) * q_token + (heads - 1) * q_head + c.k_cols);
    if (ranges_meet(out, out_bytes, q, q_bytes) || ranges_meet(out, out_bytes, c.k, cache_span(c, false)) ||
        (c.v && ranges_meet(out, out_bytes, c.v, cache_span(c, true))) ||
        ranges_meet(out, out_bytes, b.table, 4 * b.seqs * b.max_pages) || ranges_meet(out, out_bytes, b.lens, 4 * b.seqs) ||
        ranges_meet(out, out_bytes, b.starts, 4 * (b.seqs + 1)) || ranges_meet(out, out_bytes, sinks, 4 * heads))
        return FP8BLK_ERR_ARG;
    const int64_t size = c.type == FP8BLK_E4M3 ? 1 : 2;
    const bool latent = !c.v;
    a.k = (const char*)c.k;
    a.v = (const char*)(latent ? c.k : c.v);
    a.k_page = c.k_page * size, a.k_slot = c.k_slot * size, a.k_head = c.k_head * size;
    a.v_page = latent ? a.k_page : c.v_page * size;
    a.v_slot = latent ? a.k_slot : c.v_slot * size;
    a.v_head = latent ? a.k_head : c.v_head * size;
    a.q = (const char*)q;
    a.out = (char*)out;
    a.q_token = 2 * q_token, a.q_head = 2 * q_head, a.out_token = 2 * out_token, a.out_head = 2 * out_head;
    a.table = b.table, a.lens = b.lens, a.starts = b.starts, a.sinks = sinks;
    a.ws = nullptr;
    a.max_pages = b.max_pages;
    a.N = (int32_t)N, a.seqs = (int32_t)b.seqs, a.heads = (int32_t)heads, a.group = (int32_t)(heads / c.heads);
    a.pages = (int32_t)c.pages, a.page_shift = __builtin_ctzll((unsigned long long)c.page_size);
    a.max_new = (int32_t)b.max_new, a.window = (int32_t)window, a.causal = causal != 0;
    a.z_scale = scale * c.k_scale * kLog2e;
    a.out_scale = latent ? c.k_scale : c.v_scale;
    return FP8BLK_OK;
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_attn_bytes(const fp8blk_cache* cache, int64_t heads, int64_t seqs, int64_t max_new,
                                    int64_t max_len, int64_t window) {
    return 0;
}

static int simple(const fp8blk_cache* cache, const AttnArgs& a, hipStream_t s) {
    int steps = 0;
    while ((1 << steps) < a.seqs) ++steps;
    (void)hipGetLastError();
    k_attn_rows<<<dim3((unsigned)a.N, (unsigned)a.heads), 256, 0, s>>>(a, steps + 1, (int)cache->k_cols, (int)cache->v_cols,
                                                                       cache->type == FP8BLK_E4M3);
    return launch_status();
}

extern "C" int fp8blk_paged_attn(const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
                                 int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window,
                                 const float* sinks, uint16_t* out, int64_t out_token, int64_t out_head, void* ws,
                                 size_t ws_bytes, fp8blk_stream_t stream) {
    AttnArgs a;
    const int st = attn_args(a, cache, q, q_token, q_head, N, heads, batch, scale, causal, window, sinks, out, out_token,
                             out_head);
    if (st) return st;
    const int64_t k = cache->k_cols, v = cache->v_cols;
    if (!cache->v || !((k == v && (k == 64 || k == 128 || k == 256)) || (k == 192 && v == 128))) return FP8BLK_ERR_ARG;
    return simple(cache, a, reinterpret_cast<hipStream_t>(stream));
}

extern "C" int fp8blk_latent_attn(const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
                                  int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window,
                                  const float* sinks, uint16_t* out, int64_t out_token, int64_t out_head, void* ws,
                                  size_t ws_bytes, fp8blk_stream_t stream) {
    AttnArgs a;
    const int st = attn_args(a, cache, q, q_token, q_head, N, heads, batch, scale, causal, window, sinks, out, out_token,
                             out_head);
    if (st) return st;
    if (cache->v || cache->type != FP8BLK_BF16 || cache->heads != 1 || cache->v_cols != 512 ||
        (cache->k_cols != 512 && cache->k_cols != 576))
        return FP8BLK_ERR_ARG;
    return simple(cache, a, reinterpret_cast<hipStream_t>(stream));
}

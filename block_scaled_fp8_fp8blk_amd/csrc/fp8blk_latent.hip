// Latent attention in its absorbed form: every head reads the same row a token, as a
// key whole and as a value its first 512 columns.
//
// A row of 576 takes 2 * 576 * heads operations as keys and 2 * 512 * heads as values
// and is 1152 bytes: 128 heads stand near the card's balance of matrix cores and
// memory, 16 are bound by memory. What does not fit is registers: outputs of 512
// columns and q of 576 for 32 rows are 400 of a lane's 512. So the four waves share
// both products of a tile of 64 keys: scores by rows and keys (a wave 32 rows and 32
// keys, or 16 keys where there are only 32 rows), sums by columns (a wave 128 columns
// of every row), and the weights go from the one to the other through LDS.
#include "fp8blk_attn.hpp"

namespace fp8blk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kKeys = 64, kMine = kKeys / 4, kWaveCols = kLatent / 4;

template <int DK, int RT>
struct LatentLds {
    static constexpr int kRows = RT * kTile, kBuffer = kKeys * DK * 2;
    static constexpr int kP = 2 * kBuffer, kTop = kP + kRows * kKeys * 2, kKeep = kTop + 4 * kTile * 4, kSaid = kKeep + kRows * 4;
    static constexpr int kBytes = kSaid + 64;
};

__device__ __forceinline__ float max_groups(float v) {  // over the four lanes l % 16
    const auto r = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    return max_halves(fmaxf(as_f32(r[0]), as_f32(r[1])));
}

template <int DK, int RT>
__global__ __launch_bounds__(256, 1) void k_latent(AttnArgs a, int row_tiles, int units, int spread) {
    using L = LatentLds<DK, RT>;
    __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
    const int xcd = blockIdx.x & 7, turn = blockIdx.x >> 3, per = (row_tiles + spread - 1) / spread;
    const int unit = turn / per * (8 / spread) + xcd / spread, row_tile = row_tiles - 1 - (turn % per * spread + xcd % spread);
    if (unit >= units || row_tile < 0) return;
    const int c = unit % a.splits, s = unit / a.splits;
    const Seq seq = sequence(a, s);
    const int rows = seq.rows * a.group, r0 = row_tile * L::kRows;
    if (r0 >= rows) return;
    const Split split = split_of(a, seq, c);
    if (c > 0 && c >= split.n) return;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4;
    const int at0 = seq.at + r0 / a.group, at1 = seq.at + (min(r0 + L::kRows, rows) - 1) / a.group;
    const int lo = max(split.lo, first_key(a, at0)), hi = min(split.hi, end_key(a, seq, at1));
    const int all_lo = first_key(a, at1), all_hi = end_key(a, seq, at0);  // keys that every row sees

    // For scores: rows 32 rt + 16 ct + lane % 16, keys first .. of a tile, 16 kt + 4 g + i.
    constexpr int KT = RT;
    const int rt = RT == 2 ? wave & 1 : 0, part = RT == 2 ? wave >> 1 : wave, first = part * 16 * KT;
    v8bf q[2][DK / 32];
    int own_lo[2], own_hi[2];
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const int r = min(r0 + rt * kTile + 16 * ct + (lane & 15), rows - 1), token = r / a.group;
        own_lo[ct] = first_key(a, seq.at + token), own_hi[ct] = end_key(a, seq, seq.at + token);
        const char* p = a.q + (int64_t)(seq.first + token) * a.q_token + (r % a.group) * a.q_head + 16 * g;
#pragma unroll
        for (int t = 0; t < DK / 32; ++t) q[ct][t] = q_operand(a, p + 64 * t);
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    v16f o[kWaveCols / 32][RT] = {};

    const int mine = wave * kMine;
    constexpr uint32_t kAllMine = (1u << kMine) - 1;
    int base = split.lo + (lo - split.lo) / kKeys * kKeys;
    int page = 0;
    bool odd = false;
    TileRows next;
    const uint32_t lds_at = lds_offset(lds);
    auto rows_of = [&](int b) {
        TileRows t = tile_rows(a, page, b + mine, lo, hi, lane);
        t.held &= kAllMine;
        return t;
    };
    auto load = [&](int buffer) { load_tile<DK, kMine>(a.k, next.k, lds_at + buffer * L::kBuffer + mine * DK * 2, lane); };
    if (base < hi) {
        page = *entry(a, s, base + mine + (lane & 31));
        next = rows_of(base);
        page = *entry(a, s, base + kKeys + mine + (lane & 31));
        load(0);
    }
    char* const p_lds = lds + L::kP;
    float* const tops = (float*)(lds + L::kTop);
    float* const keeps = (float*)(lds + L::kKeep);
    uint32_t* const said = (uint32_t*)(lds + L::kSaid);  // by each wave: keys held, and whether some value is not finite
    for (int buffer = 0; base < hi; base += kKeys, buffer ^= 1) {
        char* const k_lds = lds + buffer * L::kBuffer;
        char* const own_rows = k_lds + mine * DK * 2;
        wait_loads<0>();
        if (next.held != kAllMine) clear_rows<DK, kMine>(own_rows, next.held, lane);
        if (lane == 0) said[wave] = next.held;
        __syncthreads();
        const uint4 held4 = *(const uint4*)said;
        const uint64_t held = (uint64_t)(held4.z | held4.w << 16) << 32 | (held4.x | held4.y << 16);
        if (base + kKeys < hi) {
            next = rows_of(base + kKeys);
            page = *entry(a, s, base + 2 * kKeys + mine + (lane & 31));
            load(buffer ^ 1);
        }
        const bool edge = base < all_lo || base + kKeys > all_hi;

        v4f z[2][KT] = {};
#pragma unroll
        for (int t = 0; t < DK / 32; ++t)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const int row = first + 16 * kt + (lane & 15), chunk = 4 * (t & 1) + g;
                const v8bf k = *(const v8bf*)(k_lds + row * DK * 2 + (t >> 1) * 128 + ((chunk ^ swizzle(row)) << 4));
#pragma unroll
                for (int ct = 0; ct < 2; ++ct) z[ct][kt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[ct][t], z[ct][kt], 0, 0, 0);
            }
        if (edge || held != ~(uint64_t)0) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = first + 16 * kt + 4 * g + i;
                    const bool there = held >> j & 1;
#pragma unroll
                    for (int ct = 0; ct < 2; ++ct)
                        z[ct][kt][i] = there && base + j >= own_lo[ct] && base + j < own_hi[ct] ? z[ct][kt][i] : -INFINITY;
                }
        }
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            float top = z[ct][0][0];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, z[ct][kt][i]);
            top = max_groups(top) * a.z_scale;
            if (lane < 16) tops[wave * kTile + 16 * ct + lane] = top;
        }
        __syncthreads();

        // Weights, against a maximum that all waves of these rows set alike (and lazily:
        // see tile_weights).
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
            const int r = 16 * ct + (lane & 15);
            float top = fmaxf(tops[rt * kTile + r], tops[(RT == 2 ? rt + 2 : 1) * kTile + r]);
            if constexpr (RT == 1) top = fmaxf(top, fmaxf(tops[2 * kTile + r], tops[3 * kTile + r]));
            top = top > m[ct] + 8.0f ? top : m[ct];
            const float at = top == -INFINITY ? 0.0f : top, keep = top == m[ct] ? 1.0f : exp2_fast(m[ct] - at);
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[ct][kt][i] = exp2_fast(__builtin_fmaf(z[ct][kt][i], a.z_scale, -at));
                    sum += z[ct][kt][i];
                }
                const int row = rt * kTile + r, chunk = (first + 16 * kt) / 8 + (g >> 1);
                *(uint2*)(p_lds + row * 128 + ((chunk ^ (row & 7)) << 4) + (g & 1) * 8) =
                    make_uint2(pack_bf16(z[ct][kt][0], z[ct][kt][1]), pack_bf16(z[ct][kt][2], z[ct][kt][3]));
            }
            l[ct] = __builtin_fmaf(l[ct], keep, sum);
            m[ct] = top;
            if (part == 0 && lane < 16) keeps[rt * kTile + r] = keep;
        }
        if (edge) {
            const bool some = make_finite<DK, kMine>(own_rows, lane);
            if (lane == 0) said[4 + wave] = some;
        }
        __syncthreads();
        if (edge) {
            const uint4 w = *(const uint4*)(said + 4);
            odd |= (w.x | w.y | w.z | w.w) != 0;
        }

        // Sums: columns kWaveCols * wave .. of every row.
        v8bf p[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = r * kTile + (lane & 31);
            const float keep = keeps[row];
            if (__any(keep != 1.0f))
#pragma unroll
                for (int t = 0; t < kWaveCols / 32; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[t][r][i] *= keep;
#pragma unroll
            for (int k = 0; k < 4; ++k) p[r][k] = *(const v8bf*)(p_lds + row * 128 + (((2 * k + (lane >> 5)) ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int t = 0; t < kWaveCols / 32; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // keys 16 k + 8 (lane / 32) .., their natural order, for p's is the same
                const int row = 8 * (lane >> 5) + ((lane & 15) >> 2), chunk = 4 * (t & 1) + 2 * (g & 1) + ((lane & 3) >> 1);
                const char* at = k_lds + (16 * k + row) * DK * 2 + (2 * wave + (t >> 1)) * 128 + (lane & 1) * 8;
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + ((chunk ^ swizzle(row)) << 4)));
                const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4 * DK * 2 + ((chunk ^ swizzle(row + 4)) << 4)));
                const v8bf v = __builtin_bit_cast(v8bf, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int r = 0; r < RT; ++r) o[t][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[r][k], o[t][r], 0, 0, 0);
            }
    }

    // The waves' sums of weights, and the maxima, to every wave.
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
        const float sum = bfly32(bfly16(l[ct]));
        if (lane < 16) tops[wave * kTile + 16 * ct + lane] = sum;
        if (part == 0 && lane < 16) keeps[rt * kTile + 16 * ct + lane] = m[ct];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int at = r * kTile + (lane & 31), row = r0 + at;
        if (row >= rows) continue;
        const float top = keeps[at];
        float sum = tops[at] + tops[(RT == 2 ? 2 : 1) * kTile + at];
        if constexpr (RT == 1) sum = sum + tops[2 * kTile + at] + tops[3 * kTile + at];
        const int token = row / a.group, head = row % a.group;
        const int64_t to = partial(a, s, token, head, c);
        const float factor = out_factor(a, head, top, sum);
        char* const out = a.out + (seq.first + token) * a.out_token + head * a.out_head;
#pragma unroll
        for (int t = 0; t < kWaveCols / 32; ++t)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const auto x = __builtin_amdgcn_permlane32_swap(as_u32(o[t][r][4 * j + i]), as_u32(o[t][r][4 * j + 4 + i]), false, false);
                    v[i] = as_f32(x[0]), v[4 + i] = as_f32(x[1]);
                }
                const int col = wave * kWaveCols + 32 * t + 8 * j + 8 * (lane >> 5);
                if (odd)
                    add_not_finite<kKeys>(a, s, a.v, false, col, split.lo, lo, hi, all_lo, all_hi, first_key(a, seq.at + token),
                                          end_key(a, seq, seq.at + token), v);
                if (split.n > 1) {
                    float* p = a.ws + to * kLatent + col;
                    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
                    *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    write_out(out + 2 * col, v, factor);
                }
            }
        if (split.n > 1 && wave == 0 && lane < 32) *(float2*)(partial_ml(a, kLatent) + 2 * to) = make_float2(top, sum);
    }
}

template <int DK, int RT>
void launch(const AttnArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.seqs * a.splits, tiles = ceil_div((int64_t)a.max_new * a.heads, RT * kTile);
    const Deal d = deal(units, tiles);
    k_latent<DK, RT><<<d.grid, 256, 0, s>>>(a, (int)tiles, (int)units, d.spread);
    launch_join<kLatent>(a, s);
}

}  // namespace

void launch_latent(const AttnArgs& a, int64_t k_cols, bool few, hipStream_t s) {
    if (k_cols == kLatent) few ? launch<kLatent, 1>(a, s) : launch<kLatent, 2>(a, s);
    else few ? launch<kLatent + 64, 1>(a, s) : launch<kLatent + 64, 2>(a, s);
}

}  // namespace fp8blk

// Latent attention in its absorbed form: every head reads the same row a token, as a
// key whole and as a value its first 512 columns.
//
// A row of 576 takes 2 * 576 * heads operations as keys and 2 * 512 * heads as values
// and is 1152 bytes: 128 heads stand near the card's balance of matrix cores and
// memory, 16 are bound by memory. What does not fit is registers: outputs of 512
// columns and q of 576 for 32 rows are 400 of a lane's 512, and a SIMD wants two waves.
// So eight waves share both products of a tile of 64 keys: scores by rows and keys (a
// wave 16 rows, and 16 or 32 keys of the tile), sums by columns (a wave 64 columns of
// every row), and the weights go from the one to the other through LDS; three barriers
// a tile. Two tiles in LDS are all that fits: one workgroup a compute unit.
//
// 64 rows: a tile takes 2.8 us (3.6 where all compute units read), of which the matrix
// cores work 0.9; LDS reads 420 KB of operands for it, 1.4 us. 64 sequences of 8000
// keys, 128 heads: 227 us, 630 TFLOP/s; with four waves, 32 rows and 128 columns each,
// 252. 32 rows: 16 sequences of 16384 keys, 16 heads, 68 us, 4.4 TB/s; with 16 rows, one
// tile in LDS and two workgroups a compute unit, 73.
#include "fp8blk_attn.hpp"

namespace fp8blk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kKeys = 64, kWaves = 8, kMine = kKeys / kWaves, kWaveCols = kLatent / kWaves;

template <int DK, int ROWS>
struct LatentLds {
    static constexpr int kGroups = ROWS / 16, kParts = kWaves / kGroups;  // of rows and of keys that waves take for the scores
    static constexpr int kBuffer = kKeys * DK * 2;
    static constexpr int kP = 2 * kBuffer, kTop = kP + ROWS * kKeys * 2, kKeep = kTop + kParts * ROWS * 4, kSaid = kKeep + ROWS * 4;
    static constexpr int kBytes = kSaid + 64;
    static_assert(ROWS * kLatent * 4 <= kP, "outputs take the place of the tiles");
};

__device__ __forceinline__ float max_groups(float v) {  // over the four lanes l % 16
    const auto r = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    return max_halves(fmaxf(as_f32(r[0]), as_f32(r[1])));
}

// A launch has less than 2^32 threads along x: of more workgroups than this, every
// kGridX are a row of the grid, and those past the last one have nothing to do.
constexpr unsigned kGridX = 1u << 22;

template <int DK, int ROWS, bool ONE>
__global__ __launch_bounds__(64 * kWaves, 2) void k_latent(AttnArgs a, int row_tiles, int units, int spread) {
    using L = LatentLds<DK, ROWS>;
    __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
    const unsigned block = blockIdx.x + blockIdx.y * kGridX;
    const int xcd = block & 7, turn = block >> 3, per = (row_tiles + spread - 1) / spread;
    const int unit = turn / per * (8 / spread) + xcd / spread, row_tile = row_tiles - 1 - (turn % per * spread + xcd % spread);
    if (unit >= units || row_tile < 0) return;
    const int s = unit / a.splits, c = split_at(a, unit, s);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, mine = wave * kMine;
    // Without a window the first tile is known before the sequence is: its pages are
    // asked for at once.
    int page = a.window > 0 ? 0 : page_at<ONE>(a, s, c * a.chunk + mine, lane);
    const Seq seq = sequence(a, s);
    const int rows = seq.rows * a.group, r0 = row_tile * ROWS;
    if (r0 >= rows) return;
    const Split split = split_of(a, seq, c);
    if (c > 0 && c >= split.n) return;

    const int at0 = seq.at + r0 / a.group, at1 = seq.at + (min(r0 + ROWS, rows) - 1) / a.group;
    const int lo = max(split.lo, first_key(a, at0)), hi = min(split.hi, end_key(a, seq, at1));
    const int all_lo = first_key(a, at1), all_hi = end_key(a, seq, at0);  // keys that every row sees

    // For scores: rows first_row + lane % 16, keys first + 16 kt + 4 g + i of a tile.
    constexpr int RT = ROWS / kTile, KT = kKeys / 16 / L::kParts;
    const int first_row = wave % L::kGroups * 16, part = wave / L::kGroups, first = part * 16 * KT, own_row = first_row + (lane & 15);
    const int own_token = min(r0 + own_row, rows - 1) / a.group;
    const int own_lo = first_key(a, seq.at + own_token), own_hi = end_key(a, seq, seq.at + own_token);
    float m = -INFINITY, l = 0.0f;
    v16f o[kWaveCols / 32][RT] = {};

    constexpr uint32_t kAllMine = (1u << kMine) - 1;
    int base = split.lo + (lo - split.lo) / kKeys * kKeys;
    bool odd = false;
    TileRows<ONE> next;
    const uint32_t lds_at = lds_offset(lds), off = load_offset(a.k_slot, lane);
    auto find = [&](int b) {  // the tile at b, whose pages `page` has; and the next one's pages
        next = tile_rows<ONE, kMine>(a, page, b + mine, lo, hi, lane);
        page = page_at<ONE>(a, s, b + kKeys + mine, lane);
    };
    auto load = [&](int buffer) {
        load_tile<DK, kMine, ONE>(a.k, next.k, a.k_slot, off, lds_at + buffer * L::kBuffer + mine * DK * 2, lane);
    };
    if (base < hi) {
        if (a.window > 0) page = page_at<ONE>(a, s, base + mine, lane);
        find(base);
        load(0);
    }
    // q's rows come through the other buffer, each once (a wave for itself would read
    // rows that two or four of them need: 147 KB a workgroup).
    v8bf q[DK / 32];
    {
        const int r = min(r0 + wave * 8 + (lane & 7), rows - 1), token = r / a.group;
        if (wave * 8 < ROWS)
            load_tile<DK, 8, false>(a.q, (seq.first + token) * a.q_token + (r - token * a.group) * a.q_head, 0, 0,
                                    lds_at + L::kBuffer + wave * 8 * DK * 2, lane);
        wait_loads<0>();
        __syncthreads();
#pragma unroll
        for (int t = 0; t < DK / 32; ++t)
            q[t] = *(const v8bf*)(lds + L::kBuffer + row_at<DK>(own_row) + (t >> 1) * 1024 + chunk_at(4 * (t & 1) + g, own_row));
    }
    char* const p_lds = lds + L::kP;
    float* const tops = (float*)(lds + L::kTop);
    float* const keeps = (float*)(lds + L::kKeep);
    uint32_t* const said = (uint32_t*)(lds + L::kSaid);  // by each wave: keys held, and whether some value is not finite
    as_operands(a, q);
    for (int buffer = 0; base < hi; base += kKeys, buffer ^= 1) {
        char* const k_lds = lds + buffer * L::kBuffer;
        char* const own_rows = k_lds + mine * DK * 2;
        wait_loads<0>();
        if (next.held != kAllMine) clear_rows<DK, kMine>(own_rows, next.held, lane);
        if (lane == 0) said[wave] = next.held;
        __syncthreads();
        uint64_t held = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) held |= (uint64_t)said[w] << (kMine * w);
        if (base + kKeys < hi) {
            find(base + kKeys);
            load(buffer ^ 1);
        }
        const bool edge = base < all_lo || base + kKeys > all_hi;

        v4f z[KT] = {};
        {
            constexpr int kSteps = DK / 32, kAhead = kSteps % 3 ? 4 : 6 / KT;
            v8bf x[2][kAhead][KT];
            auto read = [&](int b) {
#pragma unroll
                for (int t = 0; t < kAhead; ++t)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const int step = b * kAhead + t, row = first + 16 * kt + (lane & 15);
                        x[b & 1][t][kt] = *(const v8bf*)(k_lds + row_at<DK>(row) + (step >> 1) * 1024 + chunk_at(4 * (step & 1) + g, row));
                    }
            };
            read(0);
#pragma unroll
            for (int b = 0; b < kSteps / kAhead; ++b) {
                if (b + 1 < kSteps / kAhead) read(b + 1);
                keep_order();
#pragma unroll
                for (int t = 0; t < kAhead; ++t)
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
                        z[kt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[b & 1][t][kt], q[b * kAhead + t], z[kt], 0, 0, 0);
                keep_order();
            }
        }
        if (edge || held != ~(uint64_t)0) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = first + 16 * kt + 4 * g + i;
                    z[kt][i] = (held >> j & 1) && base + j >= own_lo && base + j < own_hi ? z[kt][i] : -INFINITY;
                }
        }
        {
            float top = z[0][0];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, z[kt][i]);
            top = max_groups(top) * a.z_scale;
            if (lane < 16) tops[part * ROWS + own_row] = top;
        }
        __syncthreads();

        // Weights, against a maximum that all waves of these rows set alike (and lazily:
        // see tile_weights).
        {
            float top = tops[own_row];
#pragma unroll
            for (int p = 1; p < L::kParts; ++p) top = fmaxf(top, tops[p * ROWS + own_row]);
            top = top > m + 8.0f ? top : m;
            const float at = top == -INFINITY ? 0.0f : top, keep = top == m ? 1.0f : exp2_fast(m - at);
            const float less = less_coarse(a, z, at);
            float sum = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[kt][i] = exp2_fast(__builtin_fmaf(z[kt][i], a.z_scale, -less));
                const v2bf w[2] = {{(__bf16)z[kt][0], (__bf16)z[kt][1]}, {(__bf16)z[kt][2], (__bf16)z[kt][3]}};
                sum = add2(w[1], add2(w[0], sum));
                const int chunk = (first + 16 * kt) / 8 + (g >> 1);
                *(uint2*)(p_lds + own_row * 128 + ((chunk ^ (own_row & 7)) << 4) + (g & 1) * 8) =
                    make_uint2(__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1]));
            }
            l = __builtin_fmaf(l, keep, sum);
            m = top;
            if (part == 0 && lane < 16) keeps[own_row] = keep;
        }
        if (edge) {
            const bool some = make_finite<DK, kMine>(own_rows, lane);
            if (lane == 0) said[kWaves + wave] = some;
        }
        __syncthreads();
        if (edge) {
#pragma unroll
            for (int w = 0; w < kWaves; ++w) odd |= said[kWaves + w] != 0;
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
        v8bf x[2][4];
        auto read = [&](int t) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // keys 16 k + 8 (lane / 32) .., their natural order, for p's is the same
                const int row = (lane & 15) >> 2, chunk = 4 * (t & 1) + 2 * (g & 1) + ((lane & 3) >> 1);
                const char* at = k_lds + row_at<DK>(16 * k) + row_at<DK>(8 * (lane >> 5) + row) + (kWaveCols / 64 * wave + (t >> 1)) * 1024 + (lane & 1) * 8;
                typedef __attribute__((address_space(3))) v4s lds_v4s;
                const v4s lo4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + chunk_at(chunk, row)));
                const v4s hi4 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4 * 128 + chunk_at(chunk, row + 4)));
                x[t & 1][k] = __builtin_bit_cast(v8bf, __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        };
        read(0);
#pragma unroll
        for (int t = 0; t < kWaveCols / 32; ++t) {
            if (t + 1 < kWaveCols / 32) read(t + 1);
            keep_order();
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int r = 0; r < RT; ++r) o[t][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[t & 1][k], p[r][k], o[t][r], 0, 0, 0);
            keep_order();
        }
    }

    // Outputs through LDS, in place of the tiles, so that a row is written in one piece:
    // rows of 512 floats, 16 bytes at chunk ^ (row % 8). The waves' sums of weights and
    // the maxima go the same way.
    __syncthreads();
    const float mine_sum = bfly32(bfly16(l));
    if (lane < 16) tops[part * ROWS + own_row] = mine_sum;
    if (part == 0 && lane < 16) keeps[own_row] = m;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int at = r * kTile + (lane & 31);
#pragma unroll
        for (int t = 0; t < kWaveCols / 32; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int chunk = (kWaveCols / 4 * wave + 8 * t + 2 * j + (lane >> 5)) ^ (at & 7);
                *(float4*)(lds + at * kLatent * 4 + chunk * 16) =
                    make_float4(o[t][r][4 * j], o[t][r][4 * j + 1], o[t][r][4 * j + 2], o[t][r][4 * j + 3]);
            }
    }
    __syncthreads();
    // Wave w writes rows w, w + kWaves, ...; lane i knows where the ith of them goes.
    constexpr int kOwn = ROWS / kWaves;
    const int own = wave + kWaves * (lane & (kOwn - 1)), token = min(r0 + own, rows - 1) / a.group;
    const int head = min(r0 + own, rows - 1) - token * a.group;
    const float top = keeps[own];
    float sum = tops[own], factor = 1.0f;
#pragma unroll
    for (int p = 1; p < L::kParts; ++p) sum += tops[p * ROWS + own];
    char* to;
    if (split.n > 1) {
        const int64_t at = partial(a, s, token, head, c);
        to = (char*)(a.ws + at * kLatent);
        if (lane < kOwn && r0 + own < rows) *(float2*)(partial_ml(a, kLatent) + 2 * at) = make_float2(top, sum);
    } else {
        to = a.out + (seq.first + token) * a.out_token + head * a.out_head;
        factor = out_factor(a, head, top, sum);
    }
#pragma unroll 4
    for (int k = 0; k < kOwn; ++k) {
        const int at = wave + kWaves * k;
        if (r0 + at >= rows) break;
        const char* p = lds + at * kLatent * 4;
        const float4 x = *(const float4*)(p + ((2 * lane) ^ (at & 7)) * 16), y = *(const float4*)(p + ((2 * lane + 1) ^ (at & 7)) * 16);
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (odd) {
            const int i = (r0 + at) / a.group;
            add_not_finite<kKeys>(a, s, a.v, false, 8 * lane, split.lo, lo, hi, all_lo, all_hi, first_key(a, seq.at + i),
                                  end_key(a, seq, seq.at + i), v);
        }
        char* const row = (char*)of_row((int64_t)to, k);
        if (split.n > 1) {
            *(float4*)(row + 32 * lane) = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(row + 32 * lane + 16) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            write_out(row + 16 * lane, v, lane_value(factor, k));
        }
    }
}

template <int DK, int ROWS>
void launch(const AttnArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.seqs * a.splits, tiles = ceil_div((int64_t)a.max_new * a.heads, ROWS);
    const Deal d = deal(units, tiles);
    const dim3 grid(d.grid < kGridX ? d.grid : kGridX, (unsigned)ceil_div(d.grid, kGridX));
    if (one_page(a, kMine)) k_latent<DK, ROWS, true><<<grid, 64 * kWaves, 0, s>>>(a, (int)tiles, (int)units, d.spread);
    else k_latent<DK, ROWS, false><<<grid, 64 * kWaves, 0, s>>>(a, (int)tiles, (int)units, d.spread);
    launch_join<kLatent>(a, s);
}

}  // namespace

void launch_latent(const AttnArgs& a, int64_t k_cols, bool few, hipStream_t s) {
    if (k_cols == kLatent) few ? launch<kLatent, 32>(a, s) : launch<kLatent, 64>(a, s);
    else few ? launch<kLatent + 64, 32>(a, s) : launch<kLatent + 64, 64>(a, s);
}

}  // namespace fp8blk

// Attention of new tokens over a paged cache of keys and values.
#include "fp8blk_attn.hpp"

#include <algorithm>

namespace fp8blk {
namespace {

// --- few rows: decode and verify ----------------------------------------------------
//
// Rows of one sequence whose heads share a key head are 32 columns of a tile (row r:
// token r / group, head r % group), which few rows leave partly empty: bound by the
// cache's bytes, the matrix cores wait. A workgroup takes a split of the keys, its
// four waves tiles 0, 4, ...; 1, 5, ...; each with buffers, maximum, sum and outputs
// of its own, so that nothing waits for another wave before the end, where the four
// are joined in order. While a wave forms scores its values are on their way, and
// while it sums values the next tile's keys are. 32 sequences of up to 16384 keys, 32
// heads of 128 over 4: 109 us and 6 for the join, 5.1 TB/s, what a copy reaches. e4m3 goes
// through registers, where it is widened, to the same tiles: 70 and 6 us, 3.9 TB/s.
// All key heads of a page on one XCD, one after the other: their rows are neighbours.
template <int DK, int DV>
struct FewLds {
    static constexpr int kK = kTile * DK * 2, kV = kTile * DV * 2, kPages = 256;
    static constexpr int kWave = kK + kV + kPages, kBytes = 4 * kWave;
    static_assert(kK + kV >= kTile * DV * 4, "a wave's outputs take the place of its tile");
};

// ROWS rows of COLS e4m3 into registers, and from there widened to LDS.
template <int COLS, int ROWS = kTile>
struct Codes {
    static constexpr int kAll = COLS / 16 * ROWS, kN = (kAll + 63) / 64;  // 16-byte loads
    uint4 d[kN];
};
template <bool ONE, int COLS, int ROWS>
__device__ __forceinline__ void load_codes(const char* base, int64_t rows, int64_t slot, Codes<COLS, ROWS>& r, int lane) {
    constexpr int kChunks = COLS / 16;
#pragma unroll
    for (int n = 0; n < Codes<COLS, ROWS>::kN; ++n) {
        const int at = min(64 * n + lane, Codes<COLS, ROWS>::kAll - 1);
        if constexpr (ONE && 64 % kChunks == 0)
            r.d[n] = load_global16(base + rows + n * (64 / kChunks) * slot + ((uint32_t)(lane / kChunks) * (uint32_t)slot + lane % kChunks * 16));
        else if constexpr (ONE) r.d[n] = load_global16(base + rows + ((uint32_t)(at / kChunks) * (uint32_t)slot + at % kChunks * 16));
        else r.d[n] = load_global16(base + of_row(rows, at / kChunks) + at % kChunks * 16);
    }
}
__device__ __forceinline__ uint2 widen4_e4m3(uint32_t d) {
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true)));
}
template <int COLS, int ROWS>
__device__ __forceinline__ void store_codes(char* lds, const Codes<COLS, ROWS>& r, int lane) {
    constexpr int kChunks = COLS / 16;
#pragma unroll
    for (int n = 0; n < Codes<COLS, ROWS>::kN; ++n) {
        // lanes past the last load have taken it too and store it once more
        const int at = min(64 * n + lane, Codes<COLS, ROWS>::kAll - 1), row = at / kChunks, c = 2 * (at % kChunks);
        char* p = lds + row_at<COLS>(row);
        const uint2 x = widen4_e4m3(r.d[n].x), y = widen4_e4m3(r.d[n].y), z = widen4_e4m3(r.d[n].z), w = widen4_e4m3(r.d[n].w);
        *(uint4*)(p + chunk_at(c, row)) = make_uint4(x.x, x.y, y.x, y.y);
        *(uint4*)(p + chunk_at(c + 1, row)) = make_uint4(z.x, z.y, w.x, w.y);
    }
}

template <int DK, int DV, bool E4M3, bool ONE>
__global__ __launch_bounds__(256, (FewLds<DK, DV>::kBytes <= 80 * 1024 ? 2 : 1)) void k_attn_few(AttnArgs a, int row_tiles, int units) {
    using L = FewLds<DK, DV>;
    __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
    __shared__ int odd_waves[4];
    // Workgroup b runs on XCD b % 8: all key heads and row tiles of a split, which read
    // the same keys or their neighbours in memory, on one XCD, one after the other.
    const int kv_heads = a.heads / a.group, parts = row_tiles * kv_heads;
    const int xcd = blockIdx.x & 7, turn = blockIdx.x >> 3;
    const int part = turn % parts, unit = turn / parts * 8 + xcd;
    if (unit >= units) return;
    const int row_tile = part / kv_heads, kv = part % kv_heads, s = unit / a.splits, c = split_at(a, unit, s);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Without a window the wave's first tile is known before the sequence is: its pages
    // are asked for at once.
    const int early = c * a.chunk + wave * kTile;
    int page = a.window > 0 ? 0 : page_at<ONE>(a, s, early, lane);
    const Seq seq = sequence(a, s);
    const int rows = seq.rows * a.group, r0 = row_tile * kTile;
    if (r0 >= rows) return;
    const Split split = split_of(a, seq, c);
    if (c > 0 && c >= split.n) return;

    const int q_row = r0 + (lane & 31);
    const int t0 = r0 / a.group, t1 = min(r0 + kTile, rows) - 1;  // first token, last row
    const int token = min(q_row, rows - 1) / a.group, head = kv * a.group + min(q_row, rows - 1) % a.group;
    const int at0 = seq.at + t0, at1 = seq.at + t1 / a.group;     // positions of the tile's first and last row
    const int lo = max(split.lo, first_key(a, at0)), hi = min(split.hi, end_key(a, seq, at1));
    const int own_lo = first_key(a, seq.at + token), own_hi = end_key(a, seq, seq.at + token);
    const int all_lo = first_key(a, at1), all_hi = end_key(a, seq, at0);  // keys that every row sees

    char* const k_lds = lds + wave * L::kWave;
    char* const v_lds = k_lds + L::kK;
    int32_t* const pages = (int32_t*)(v_lds + L::kV);
    const uint32_t k_at = lds_offset(k_lds), v_at = lds_offset(v_lds), pages_at = lds_offset(pages);
    const char* const k_base = a.k + kv * a.k_head;
    const char* const v_base = a.v + kv * a.v_head;

    v8bf q[DK / 16];
    load_q(a.q + (int64_t)(seq.first + token) * a.q_token + head * a.q_head + 16 * (lane >> 5), 32, q);
    v16f o[DV / 32] = {};
    Running run = {-INFINITY, 0.0f};

    // The wave's tiles: those of the split whose number is `wave` modulo 4.
    int tile = (lo - split.lo) / kTile;
    tile += (wave - tile) & 3;
    int base = split.lo + tile * kTile;
    TileRows<ONE> next, here;
    Codes<E4M3 ? DK : 32> k_codes;
    Codes<E4M3 ? DV : 32> v_codes;
    bool odd = false;
    const uint32_t k_off = load_offset(a.k_slot, lane), v_off = load_offset(a.v_slot, lane);
    auto load_k = [&](int b) {  // of the tile at b, whose pages `page` has; and the pages of the wave's next
        next = tile_rows<ONE>(a, page, b, lo, hi, lane);
        if constexpr (E4M3 || ONE) page = page_at<ONE>(a, s, b + 4 * kTile, lane);
        else load_lds4((const char*)entry(a, s, b + 4 * kTile + (lane & 31)), pages_at);
        if constexpr (E4M3) load_codes<ONE>(k_base, next.k, a.k_slot, k_codes, lane);
        else load_tile<DK, kTile, ONE>(k_base, next.k, a.k_slot, k_off, k_at, lane);
    };
    auto load_v = [&] {
        if constexpr (E4M3) load_codes<ONE>(v_base, next.v, a.v_slot, v_codes, lane);
        else load_tile<DV, kTile, ONE>(v_base, next.v, a.v_slot, v_off, v_at, lane);
    };
    if (base < hi) {
        if (a.window > 0) page = page_at<ONE>(a, s, base, lane);
        load_k(base);
        load_v();
    }
    as_operands(a, q);
    for (; base < hi; base += 4 * kTile) {
        const bool more = base + 4 * kTile < hi;
        here = next;
        if constexpr (E4M3) store_codes(k_lds, k_codes, lane);
        else wait_loads<L::kV / 1024>();
        v16f z[1] = {tile_scores<DK>(k_lds, q, lane)};
        if (more) {
            if constexpr (!E4M3 && !ONE) page = pages[lane & 31];
            wait_reads();
            load_k(base + 4 * kTile);
        }
        const bool edge = base < all_lo || base + kTile > all_hi;
        if (edge || here.held != ~0u) hide(z[0], here.held & keys_between(base, own_lo, own_hi), lane);
        v8bf p[1][2];
        rescale(o, tile_weights(a, z, run, p));
        if constexpr (E4M3) store_codes(v_lds, v_codes, lane);
        else if (more) wait_loads<DK / 16 + (ONE ? 0 : 1)>();
        else wait_loads<0>();
        if (here.held != ~0u) clear_rows<DV>(v_lds, here.held, lane);
        if (edge) odd |= make_finite<DV, kTile>(v_lds, lane);
        tile_sums<DV>(v_lds, p[0], o, lane);
        if (more) {
            wait_reads();
            load_v();
        }
    }

    // Join the four waves, in order; a wave's outputs lie as rows of DV floats, 16 bytes
    // at chunk ^ (row % 8).
    wait_reads();
    float* const ml = (float*)pages;
    run.l = bfly32(run.l);
    if (lane < 32) ml[lane] = run.m;
    else ml[lane] = run.l;
    if (lane == 0) odd_waves[wave] = odd;
    {
        char* p = k_lds + (lane & 31) * DV * 4;
#pragma unroll
        for (int t = 0; t < DV / 32; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const v16f& x = o[t];
                const int chunk = (8 * t + 2 * j + (lane >> 5)) ^ (lane & 7);
                *(float4*)(p + chunk * 16) = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            }
    }
    constexpr int kOnes = DV / 8;  // threads a row
    __syncthreads();
#pragma unroll 1
    for (int r = threadIdx.x / kOnes; r < kTile && r0 + r < rows; r += 256 / kOnes) {
        const int d = threadIdx.x % kOnes, col = 8 * d;
        float m[4], l[4], top = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float* of = (const float*)(lds + w * L::kWave + L::kK + L::kV);
            m[w] = of[r], l[w] = of[32 + r];
            top = fmaxf(top, m[w]);
        }
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f, v[8] = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float f = exp2_fast(m[w] - base);
            sum = __builtin_fmaf(f, l[w], sum);
            const char* p = lds + w * L::kWave + r * DV * 4;
            const float4 x = *(const float4*)(p + ((2 * d) ^ (r & 7)) * 16), y = *(const float4*)(p + ((2 * d + 1) ^ (r & 7)) * 16);
            const float e[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(f, e[i], v[i]);
        }
        const int row = r0 + r, i = row / a.group, h = kv * a.group + row % a.group;
        if (odd_waves[0] | odd_waves[1] | odd_waves[2] | odd_waves[3])
            add_not_finite<kTile>(a, s, v_base, E4M3, col, split.lo, lo, hi, all_lo, all_hi, first_key(a, seq.at + i),
                                  end_key(a, seq, seq.at + i), v);
        if (split.n > 1) {
            const int64_t at = partial(a, s, i, h, c);
            float* p = a.ws + at * DV + col;
            *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (col == 0) *(float2*)(partial_ml(a, DV) + 2 * at) = make_float2(top, sum);
        } else {
            write_out(a.out + (seq.first + i) * a.out_token + h * a.out_head + 2 * col, v, out_factor(a, h, top, sum));
        }
    }
}

// --- many rows: a prompt's chunk ------------------------------------------------------
//
// GROUPS of 32 rows share tiles of 64 keys, which their waves load together, the next
// one while this one is worked on; one barrier a tile. With HALVES 2 two waves share 32
// rows, each 32 keys of a tile with maximum, sum and outputs of its own, joined at the
// end. Bound by the matrix cores, their operands from LDS (a quarter of a tile's 4800
// cycles each), the softmax between them and the barrier; only another wave on the SIMD
// hides one behind the other. 2048 new tokens of 8192, 32 heads of 128 over 4: 257 us,
// 940 TFLOP/s of the 1290 that a large matrix product reaches. Tiles of 64 keys, not
// 32: half the barriers (heads of 192 and 128, 73 -> 59 us). A third buffer gave nothing.
template <int DK, int DV, bool ONE, int GROUPS, int HALVES>
struct ChunkLds {
    static constexpr int kKeys = 64, kTiles = kKeys / kTile / HALVES, kWaves = GROUPS * HALVES, kRows = kKeys / kWaves;
    static constexpr int kK = kKeys * DK * 2, kV = kKeys * DV * 2;
    // ONE leaves nothing to say to other waves: with heads of 192 and 128 two workgroups
    // take all 160 KB
    static constexpr int kOut = GROUPS * kTile * DV * 4;  // outputs, where the tiles were
    static constexpr int kSaid = 2 * (kK + kV), kEnd = kSaid + (ONE ? 0 : 8 * kWaves), kStates = HALVES == 2 ? GROUPS * 64 * 8 : 0;
    static constexpr int kJoin = kOut + kStates <= kSaid ? kOut : kEnd;
    static constexpr int kBytes = kJoin == kEnd ? kEnd + kStates : kEnd;
};
constexpr int kChunkRows = 4 * kTile;

template <int DK, int DV, bool E4M3, bool ONE, int GROUPS, int HALVES>
__global__ __launch_bounds__(64 * GROUPS * HALVES, (GROUPS * HALVES == 8 || ChunkLds<DK, DV, ONE, GROUPS, HALVES>::kBytes <= 80 * 1024 ? 2 : 1)) void k_attn_chunk(AttnArgs a, int row_tiles, int units, int spread, bool pairs) {
    using L = ChunkLds<DK, DV, ONE, GROUPS, HALVES>;
    constexpr int kMost = GROUPS * kTile;
    __shared__ __attribute__((aligned(16))) char lds[L::kBytes];
    // Workgroup b runs on XCD b % 8: a unit's row tiles, which read the same keys, on
    // `spread` XCDs, those with the most keys first. pairs: all units' longest tiles
    // first, on all of an XCD's 32 compute units, then from the shortest up, beside them.
    const int xcd = blockIdx.x & 7, per = (row_tiles + spread - 1) / spread;
    int turn = blockIdx.x >> 3;
    if (pairs) {
        const int side = (units + 8 / spread - 1) / (8 / spread);
        if (turn >= 32) turn = 32 + gridDim.x / 8 - 1 - turn;
        turn = (turn + turn / side) % side * per + turn / side;
    }
    const int unit = turn / per * (8 / spread) + xcd / spread, row_tile = row_tiles - 1 - (turn % per * spread + xcd % spread);
    if (unit >= units || row_tile < 0) return;
    const int kv_heads = a.heads / a.group;
    const int of = unit / a.splits, c = split_at(a, unit, of), kv = of % kv_heads, s = of / kv_heads;
    const Seq seq = sequence(a, s);
    const int rows = seq.rows * a.group, r0 = row_tile * kMost;
    if (r0 >= rows) return;
    const Split split = split_of(a, seq, c);
    if (c > 0 && c >= split.n) return;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = wave / GROUPS, w0 = r0 + wave % GROUPS * kTile, q_row = min(w0 + (lane & 31), rows - 1);
    const int token = q_row / a.group, head = kv * a.group + q_row % a.group;
    // positions of the first and last row of the workgroup and of the wave
    const int at0 = seq.at + r0 / a.group, at1 = seq.at + (min(r0 + kMost, rows) - 1) / a.group;
    const int wave0 = seq.at + min(w0, rows - 1) / a.group, wave1 = seq.at + min(w0 + kTile - 1, rows - 1) / a.group;
    const int lo = max(split.lo, first_key(a, at0)), hi = min(split.hi, end_key(a, seq, at1));
    const int all_lo = first_key(a, at1), all_hi = end_key(a, seq, at0);
    const int wave_lo = first_key(a, wave0), wave_hi = w0 < rows ? end_key(a, seq, wave1) : 0;
    const int own_lo = first_key(a, seq.at + token), own_hi = end_key(a, seq, seq.at + token);

    const char* const k_base = a.k + kv * a.k_head;
    const char* const v_base = a.v + kv * a.v_head;
    v8bf q[DK / 16];
    load_q(a.q + (int64_t)(seq.first + token) * a.q_token + head * a.q_head + 16 * (lane >> 5), 32, q);
    v16f o[DV / 32] = {};
    Running run = {-INFINITY, 0.0f};

    // The wave loads rows kRows * wave .. of every tile; its lanes hold their offsets.
    const int mine = wave * L::kRows;
    constexpr uint32_t kMine = (uint32_t)(((uint64_t)1 << L::kRows) - 1);
    int base = split.lo + (lo - split.lo) / L::kKeys * L::kKeys;
    TileRows<ONE> next;
    uint32_t held[2], held_next[2] = {};  // the tile's keys that a page holds (else: what other waves say)
    int page = 0, parts[4] = {};         // the next tile's pages: the wave's (or its lanes'); ONE: of each 16 keys
    bool odd = false;
    Codes<E4M3 ? DK : 64, E4M3 ? L::kRows : 16> k_codes;
    Codes<E4M3 ? DV : 64, E4M3 ? L::kRows : 16> v_codes;
    const int own_part = mine / 16;
    const uint32_t lds_at = lds_offset(lds), k_off = load_offset(a.k_slot, lane), v_off = load_offset(a.v_slot, lane);
    auto find = [&](int b) {
        if constexpr (ONE)
#pragma unroll
            for (int w = 0; w < 4; ++w) parts[w] = page_at<true>(a, s, b + 16 * w, lane);
        else page = page_at<ONE>(a, s, b + mine, lane);
    };
    auto load = [&](int b, int buffer) {  // the tile at b
        if constexpr (ONE) {
            page = own_part < 2 ? own_part < 1 ? parts[0] : parts[1] : own_part < 3 ? parts[2] : parts[3];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t there = ((uint32_t)parts[2 * t] < (uint32_t)a.pages ? 0xffffu : 0u) |
                                       ((uint32_t)parts[2 * t + 1] < (uint32_t)a.pages ? 0xffff0000u : 0u);
                held_next[t] = there & keys_between(b + t * kTile, lo, hi);
            }
        }
        next = tile_rows<ONE, L::kRows>(a, page, b + mine, lo, hi, lane);
        find(b + L::kKeys);
        if constexpr (E4M3) {
            load_codes<ONE>(k_base, next.k, a.k_slot, k_codes, lane);
            load_codes<ONE>(v_base, next.v, a.v_slot, v_codes, lane);
        } else {
            const uint32_t to = lds_at + buffer * (L::kK + L::kV);
            load_tile<DK, L::kRows, ONE>(k_base, next.k, a.k_slot, k_off, to + mine * DK * 2, lane);
            load_tile<DV, L::kRows, ONE>(v_base, next.v, a.v_slot, v_off, to + L::kK + mine * DV * 2, lane);
        }
    };
    if (base < hi) {
        find(base);
        load(base, 0);
    }
    as_operands(a, q);
    for (int buffer = 0; base < hi; base += L::kKeys, buffer ^= 1) {
        char* const k_lds = lds + buffer * (L::kK + L::kV);
        char* const v_lds = k_lds + L::kK;
        if constexpr (E4M3) {
            store_codes(k_lds + mine * DK * 2, k_codes, lane);
            store_codes(v_lds + mine * DV * 2, v_codes, lane);
        } else {
            wait_loads<0>();
        }
        char* const own_v = v_lds + mine * DV * 2;
        if (next.held != kMine) clear_rows<DV, L::kRows>(own_v, next.held, lane);
        if (base < all_lo || base + L::kKeys > all_hi) odd |= make_finite<DV, L::kRows>(own_v, lane);
        uint32_t* const said = (uint32_t*)(lds + L::kSaid) + L::kWaves * buffer;
        if (!ONE && lane == 0) said[wave] = next.held;
        __syncthreads();
        if constexpr (ONE) {
#pragma unroll
            for (int t = 0; t < 2; ++t) held[t] = held_next[t];
        } else {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                held[t] = 0;
#pragma unroll
                for (int w = 0; w < L::kWaves / 2; ++w) held[t] |= said[t * (L::kWaves / 2) + w] << (w * L::kRows);
            }
        }
        if (base + L::kKeys < hi) load(base + L::kKeys, buffer ^ 1);
        const bool active = base < wave_hi && base + L::kKeys > wave_lo;
        if (!active) continue;
        v16f z[L::kTiles];
        uint32_t seen[L::kTiles];
        bool all = true;
#pragma unroll
        for (int t = 0; t < L::kTiles; ++t) {
            const int sub = HALVES == 2 ? half : t;
            z[t] = tile_scores<DK>(k_lds + sub * kTile * DK * 2, q, lane);
            seen[t] = (sub ? held[1] : held[0]) & keys_between(base + sub * kTile, own_lo, own_hi);
            all = all && seen[t] == ~0u;
        }
        if (!__all(all))
#pragma unroll
            for (int t = 0; t < L::kTiles; ++t) hide(z[t], seen[t], lane);
        v8bf p[L::kTiles][2];
        rescale(o, tile_weights(a, z, run, p));
#pragma unroll
        for (int t = 0; t < L::kTiles; ++t) tile_sums<DV>(v_lds + (HALVES == 2 ? half : t) * kTile * DV * 2, p[t], o, lane);
    }

    // Whether any wave has made a value finite.
    __syncthreads();
    if (lane == 0) ((int*)lds)[wave] = odd;
    __syncthreads();
    odd = false;
#pragma unroll
    for (int w = 0; w < L::kWaves; ++w) odd |= ((const int*)lds)[w] != 0;
    __syncthreads();
    // Outputs through LDS, so that a row is written in one piece: a wave's lie as rows of
    // DV floats, 16 bytes at chunk ^ (row % 8). Lane r knows where row r % 32 goes.
    static_assert(L::kOut <= 2 * (L::kK + L::kV), "outputs take the place of the tiles");
    char* const o_lds = lds + wave % GROUPS * kTile * DV * 4;
    if constexpr (HALVES == 2) {
        float2* const ml = (float2*)(lds + L::kJoin) + 64 * (wave % GROUPS) + lane;
        if (half) {
            *ml = make_float2(run.m, run.l);
#pragma unroll
            for (int t = 0; t < DV / 32; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(float4*)(o_lds + (4 * t + j) * 1024 + lane * 16) = make_float4(o[t][4 * j], o[t][4 * j + 1], o[t][4 * j + 2], o[t][4 * j + 3]);
        }
        __syncthreads();
        if (half) return;
        const float2 other = *ml;
        const float top = fmaxf(run.m, other.x), at = top == -INFINITY ? 0.0f : top;
        const float f = exp2_fast(run.m - at), g = exp2_fast(other.x - at);
        run.m = top;
        run.l = __builtin_fmaf(g, other.y, f * run.l);
#pragma unroll
        for (int t = 0; t < DV / 32; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = *(const float4*)(o_lds + (4 * t + j) * 1024 + lane * 16);
                const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][4 * j + i] = __builtin_fmaf(g, e[i], f * o[t][4 * j + i]);
            }
        wait_reads();
    }
#pragma unroll
    for (int t = 0; t < DV / 32; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *(float4*)(o_lds + (lane & 31) * DV * 4 + (((8 * t + 2 * j + (lane >> 5)) ^ (lane & 7)) << 4)) =
                make_float4(o[t][4 * j], o[t][4 * j + 1], o[t][4 * j + 2], o[t][4 * j + 3]);
    run.l = bfly32(run.l);
    float factor = 1.0f;
    char* to;
    if (split.n > 1) {
        const int64_t part = partial(a, s, token, head, c);
        to = (char*)(a.ws + part * DV);
        if (lane < 32 && w0 + lane < rows) *(float2*)(partial_ml(a, DV) + 2 * part) = make_float2(run.m, run.l);
    } else {
        to = a.out + (seq.first + token) * a.out_token + head * a.out_head;
        factor = out_factor(a, head, run.m, run.l);
    }
    constexpr int kOnes = DV / 8;  // lanes a row
#pragma unroll 4
    for (int k = 0; k < kTile; k += 64 / kOnes) {
        const int r = k + lane / kOnes, d = lane % kOnes;
        char* const row = (char*)of_row((int64_t)to, r);
        const float f = __shfl(factor, r);
        const int row_lo = __shfl(own_lo, r), row_hi = __shfl(own_hi, r);
        if (w0 + r >= rows) continue;
        const char* const p = o_lds + r * DV * 4;
        const float4 x = *(const float4*)(p + (((2 * d) ^ (r & 7)) << 4)), y = *(const float4*)(p + (((2 * d + 1) ^ (r & 7)) << 4));
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (odd)
            add_not_finite<L::kKeys>(a, s, v_base, E4M3, 8 * d, split.lo, lo, hi, all_lo, all_hi, row_lo, row_hi, v);
        if (split.n > 1) {
            *(float4*)(row + 32 * d) = make_float4(v[0], v[1], v[2], v[3]);
            *(float4*)(row + 32 * d + 16) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            write_out(row + 16 * d, v, f);
        }
    }
}

bool attn_ranges_ok(const fp8blk_cache& c, int64_t heads, int64_t seqs, int64_t max_new, int64_t max_len, int64_t window) {
    constexpr int64_t kMost = INT64_C(1) << 30;
    return heads >= 1 && heads <= FP8BLK_MAX_HEADS && heads % c.heads == 0 && seqs >= 1 && seqs <= FP8BLK_MAX_PANEL &&
           max_new >= 1 && max_new <= FP8BLK_MAX_PANEL && max_len >= 1 && max_len < kMost && window >= 0 && window < kMost;
}
bool attn_sizes_ok(const fp8blk_cache& c, int64_t heads, int64_t seqs, int64_t max_new, int64_t max_len, int64_t window) {
    return attn_ranges_ok(c, heads, seqs, max_new, max_len, window) &&
           seqs * heads * ceil_div(max_new, 128) <= INT64_C(1) << 22;  // below 2^32 threads along x (latent rows: see kGridX)
}

}  // namespace

int attn_args(AttnArgs& a, const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
              int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window, const float* sinks,
              uint16_t* out, int64_t out_token, int64_t out_head) {
    if (!cache || !batch || !q || !out || !cache_ok(*cache)) return FP8BLK_ERR_ARG;
    const fp8blk_cache& c = *cache;
    const fp8blk_batch& b = *batch;
    if (N < 1 || N > FP8BLK_MAX_PANEL || b.max_pages < 1 || b.max_pages > (INT64_C(1) << 30) || !std::isfinite(scale) ||
        !attn_sizes_ok(c, heads, b.seqs, b.max_new, b.max_len, window))
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
    a.z_scale = std::fabs(scale) * c.k_scale * kLog2e;
    if (std::isinf(a.z_scale)) return FP8BLK_ERR_ARG;
    a.q_and = a.z_scale > 0.0f ? ~0u : 0u;
    a.q_xor = a.z_scale > 0.0f && scale < 0.0f ? 0x80008000u : 0u;
    if (!(a.z_scale > 0.0f)) a.z_scale = 1.0f;
    a.z_back = 1.0f / a.z_scale;
    a.splits = 1;
    a.chunk = 1 << 30;
    a.out_scale = latent ? c.k_scale : c.v_scale;
    return FP8BLK_OK;
}

}  // namespace fp8blk

using namespace fp8blk;

namespace {

struct Plan {
    bool few;  // rows of a panel beside each other in one tile, the keys dealt to the waves
    int32_t splits, chunk;
    size_t bytes;
};

// Keys that a call's rows see at most of a sequence.
int64_t seen_of(bool panel, int64_t max_new, int64_t max_len, int64_t window) {
    return window > 0 ? std::min(max_len, window + (panel ? FP8BLK_MAX_M : max_new)) : max_len;
}

// Splits of a sequence's `seen` keys, from the workgroups that a call has without them.
//
// Latent: one workgroup a compute unit, with keys enough that the sums' way through memory
// does not take longer than they do (8192 keys, 128 heads: 64 splits 21 us, 32 22,
// 128 30). A chunk's sequences are of unequal length: twice as many where they are
// long (8 of 100 tokens of up to 9000, 16 heads 382 -> 217, 4 of 877 of up to 14367,
// one head 172 -> 112, 3 of 64 of up to 16000 166 -> 170; where all are as long as
// that 5 to 16% more).
int64_t latent_splits(int64_t units, int64_t seen, bool few, bool several_chunks) {
    int64_t n = std::min(256 / units, ceil_div(seen, few ? 128 : 256));
    if (several_chunks && n > 0 && seen >= 3000 * n) n *= 2;
    return n;
}

// A workgroup streams 768 keys a split or more, as many splits as fill the card at
// least: 4096 keys, 4 key heads: 32 splits 10.8 us, 8 13.8, one 41; 32 sequences of
// up to 16384: 22 splits 115, 4 136 (all of 16384: 212 and 205, one 233). From 512
// units on none (128 sequences of up to 4096: 116, in 2 splits 140), nor below 512 keys.
constexpr int64_t kFewStep = 4 * kTile, kFewUnits = 512;
int64_t few_splits(int64_t units, int64_t seen) {
    return seen <= 512 ? 1 : std::min(std::max(256 / units, units < kFewUnits ? std::min(ceil_div(seen, 768), 16384 / units) : 1), ceil_div(seen, kFewStep));
}

// A tile of 64 keys takes a workgroup 1.1 us, each split of a row writes and reads
// 8 bytes a column: n^2 splits are best where n^2 * rows * columns is some
// thousand times the keys (causal rows see max_new / 2 less; of sequences of
// different lengths fewer splits hold keys). Up to `fill` they only use idle
// compute units; more have to be twice as many, at least 4 and not past `most`.
// 500 new tokens of 3000, 32 heads over 4: 49 us in 4 splits, 53 in 2, 58 in one;
// 3 sequences of 500 of up to 6000, 16 heads: 68 in 4, 107 in one (alike long ones:
// 118, 128); 1000 of 1000, 16 heads: 25 in one, 33 in 2.
struct ChunkSplits {
    int64_t fill, most, best;
};
constexpr int64_t kChunkUnits = 384;
ChunkSplits chunk_splits(int64_t units, int64_t seen, int64_t seqs, int64_t max_new, int64_t heads, int64_t cols) {
    ChunkSplits c;
    c.fill = std::max<int64_t>(256 / units, 1);
    c.most = units <= (seqs > 1 ? kChunkUnits : 255) ? std::max<int64_t>((seqs > 1 ? 1024 : 512) / units, 4) : 1;
    const double best = (seqs > 1 ? 18000.0 : 7500.0) * (double)std::max<int64_t>(seen - max_new / 2, 1) / ((double)seqs * max_new * heads * cols);
    for (c.best = 1; 2 * c.best * c.best <= best; c.best *= 2) {
    }
    c.best = std::min(c.best, ceil_div(seen, 128));
    return c;
}

// 32 rows of a latent panel a workgroup where there are few tiles, 64 where that many rows
// read the keys more than once, or write more splits (128 heads, one sequence of 4000 keys:
// 18 us, with 64 rows 25, two tokens 21 and 27; of 16000: 25, 30, two tokens 41 and 34;
// 64 of 8000: 266, 226).
constexpr int64_t kFewLatentTiles = 256;
int64_t latent_tiles(int64_t seqs, int64_t heads, int64_t seen) { return seqs * ceil_div(heads, kLatentRows) * ceil_div(seen, 64); }

size_t bytes_of(int64_t rows, int64_t splits, int64_t cols) { return splits > 1 ? (size_t)(rows * splits * (cols + 2)) * sizeof(float) : 0; }

// Which kernel a call takes and how its keys are split. Up to FP8BLK_MAX_M new tokens
// the number of them has no say, so that a row's bits do not depend on it.
Plan plan(const fp8blk_cache& c, int64_t heads, int64_t seqs, int64_t max_new, int64_t max_len, int64_t window) {
    const int64_t group = heads / c.heads;
    const bool panel = max_new <= FP8BLK_MAX_M, latent = !c.v;
    const int64_t seen = seen_of(panel, max_new, max_len, window);
    Plan p;
    p.few = panel && (!latent || group <= kTile || latent_tiles(seqs, group, seen) <= kFewLatentTiles);
    const int64_t tile = latent ? (p.few ? kTile : kLatentRows) : kChunkRows;
    const int64_t units = seqs * c.heads * (p.few && !latent ? 1 : ceil_div(panel ? group : max_new * group, tile));
    const int64_t step = p.few && !latent ? kFewStep : 64;
    int64_t n;
    if (latent) {
        n = latent_splits(units, seen, p.few, !panel && seqs > 1);
    } else if (p.few) {
        n = few_splits(units, seen);
    } else {
        const ChunkSplits r = chunk_splits(units, seen, seqs, max_new, heads, c.v_cols);
        n = r.best;
        while (n > r.fill && (n > r.most || n < 4 || n < 2 * r.fill)) n = std::max(n / 2, r.fill);
    }
    n = std::max<int64_t>(n, 1);
    p.chunk = (int32_t)(ceil_div(ceil_div(seen, n), step) * step);
    p.splits = (int32_t)(ceil_div(seen, p.chunk) + (window > 0 ? 1 : 0));
    if (n == 1) p.splits = 1, p.chunk = 1 << 30;
    p.bytes = bytes_of(seqs * max_new * heads, p.splits, c.v_cols);
    return p;
}

// The most bytes that plan asks for with up to so many sequences, new tokens and keys
// (which is not what it asks for with just as many: more rows leave less room for splits).
// All rules above give no fewer splits for more keys, a chunk's before it halves them; so the
// largest max_len counts, for each number of sequences and of row tiles that leaves room
// for splits; of the new tokens that make up such a number of tiles the fewest for
// the splits, the most for the rows.
size_t most_bytes(const fp8blk_cache& c, int64_t heads, int64_t seqs, int64_t max_new, int64_t max_len, int64_t window) {
    const int64_t group = heads / c.heads, edge = window > 0 ? 1 : 0;
    const bool latent = !c.v;
    size_t most = 0;
    auto take = [&](int64_t rows, int64_t n) { most = std::max(most, n > 1 ? bytes_of(rows, n + edge, c.v_cols) : 0); };
    const int64_t panel = std::min<int64_t>(max_new, FP8BLK_MAX_M), seen = seen_of(true, panel, max_len, window);
    for (int64_t s = 1; s <= seqs && s * c.heads < kFewUnits; ++s) {
        const int64_t rows = s * panel * heads;
        if (!latent) {
            take(rows, few_splits(s * c.heads, seen));
            continue;
        }
        const int64_t few_seen = group <= kTile ? seen : std::min(seen, 64 * (kFewLatentTiles / latent_tiles(s, group, 1)));
        if (few_seen > 0) take(rows, latent_splits(s * ceil_div(group, kTile), few_seen, true, false));
        if (few_seen < seen) take(rows, latent_splits(s * ceil_div(group, kLatentRows), seen, false, false));
    }
    const int64_t tile = latent ? kLatentRows : kChunkRows, units = latent ? 256 : kChunkUnits;
    for (int64_t s = 1; s <= seqs && s * c.heads <= units; ++s)
        for (int64_t tiles = 1; s * c.heads * tiles <= units; ++tiles) {
            const int64_t from = std::max<int64_t>((tiles - 1) * tile / group + 1, FP8BLK_MAX_M + 1), to = std::min(tiles * tile / group, max_new);
            if (from > max_new) break;
            if (from > to) continue;
            const int64_t u = s * c.heads * tiles, all = seen_of(false, to, max_len, window);
            if (latent) {
                take(s * to * heads, latent_splits(u, all, false, s > 1));
            } else {
                const ChunkSplits r = chunk_splits(u, all, s, from, heads, c.v_cols);
                take(s * to * heads, r.best <= r.fill ? r.best : std::max(r.fill, std::min(r.best, r.most)));
            }
        }
    return most;
}

template <int DK, int DV, bool E4M3, bool ONE>
void launch_few(const AttnArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.seqs * a.splits, tiles = ceil_div((int64_t)a.max_new * a.group, kTile);
    k_attn_few<DK, DV, E4M3, ONE><<<(unsigned)(ceil_div(units, 8) * 8 * tiles * (a.heads / a.group)), 256, 0, s>>>(a, (int)tiles, (int)units);
}

template <int DK, int DV, bool E4M3, bool ONE>
void launch_chunk(const AttnArgs& a, hipStream_t s) {
    const int64_t units = (int64_t)a.seqs * (a.heads / a.group) * a.splits;
    const int64_t tiles = ceil_div((int64_t)a.max_new * a.group, kChunkRows);
    const Deal d = deal(units, tiles);
    // A wave waits for its own products and powers, so a SIMD wants two. Heads of 256,
    // of which LDS holds one workgroup a compute unit: eight waves (3 sequences of 777
    // tokens: 106 us, four waves some 25 more; e4m3 or in small pages the registers do not allow
    // for them). Up to 256 workgroups: 64 rows for four waves, twice as many workgroups
    // (2000 tokens of 16 heads of 192 and 128: 49 us; 128 rows for four waves 60, for
    // eight 55). More: 128 rows for four, which read a tile for twice as many rows (2048
    // of 8192 tokens: 257 us, 64 rows 317).
    if constexpr (DV == 256 && ONE && !E4M3) {
        k_attn_chunk<DK, DV, E4M3, ONE, 4, 2><<<d.grid, 512, 0, s>>>(a, (int)tiles, (int)units, d.spread, false);
    } else {
        if constexpr (DV <= 128)
            if (units * tiles <= 256) {
                const int64_t fine = ceil_div((int64_t)a.max_new * a.group, 2 * kTile);
                const Deal d = deal(units, fine);
                k_attn_chunk<DK, DV, E4M3, ONE, 2, 2><<<d.grid, 256, 0, s>>>(a, (int)fine, (int)units, d.spread, d.grid <= 512);
                return;
            }
        // Of two workgroups a compute unit that all run at once, the long ones with short
        // ones (4 sequences of 1000 tokens, 16 heads: 34 us, else 41; 2048 of 8192 tokens, 256,
        // 262). Where there are more, the next one goes to whichever is free, and units one
        // after the other read their keys from L2 (6 of 1500 of 6000: 189 us, as above 243).
        k_attn_chunk<DK, DV, E4M3, ONE, 4, 1><<<d.grid, 256, 0, s>>>(a, (int)tiles, (int)units, d.spread, d.grid <= 512);
    }
}

template <int DK, int DV, bool E4M3>
void launch(const AttnArgs& a, bool few, hipStream_t s) {
    if (few) one_page(a, kTile) ? launch_few<DK, DV, E4M3, true>(a, s) : launch_few<DK, DV, E4M3, false>(a, s);
    else one_page(a, 16) ? launch_chunk<DK, DV, E4M3, true>(a, s) : launch_chunk<DK, DV, E4M3, false>(a, s);
    launch_join<DV>(a, s);
}

}  // namespace

extern "C" size_t fp8blk_attn_bytes(const fp8blk_cache* cache, int64_t heads, int64_t seqs, int64_t max_new,
                                    int64_t max_len, int64_t window) {
    if (!cache || !cache_ok(*cache) || !attn_sizes_ok(*cache, heads, seqs, max_new, max_len, window)) return 0;
    return plan(*cache, heads, seqs, max_new, max_len, window).bytes;
}

extern "C" size_t fp8blk_attn_most_bytes(const fp8blk_cache* cache, int64_t heads, int64_t seqs, int64_t max_new,
                                         int64_t max_len, int64_t window) {
    if (!cache || !cache_ok(*cache) || !attn_ranges_ok(*cache, heads, seqs, max_new, max_len, window)) return 0;
    return most_bytes(*cache, heads, seqs, max_new, max_len, window);
}

namespace {

// The rest of a call whose arguments have been checked.
int attend(AttnArgs& a, const fp8blk_cache& c, const fp8blk_batch& b, int64_t heads, int64_t window, void* ws, size_t ws_bytes,
           fp8blk_stream_t stream) {
    const Plan p = plan(c, heads, b.seqs, b.max_new, b.max_len, window);
    if (p.bytes && (!ws || ws_bytes < p.bytes || !aligned(ws, 256))) return FP8BLK_ERR_WORKSPACE;
    a.ws = (float*)ws;
    a.splits = p.splits, a.chunk = p.chunk;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const bool e4m3 = c.type == FP8BLK_E4M3;
    switch (c.k_cols) {
        case 64: e4m3 ? launch<64, 64, true>(a, p.few, s) : launch<64, 64, false>(a, p.few, s); break;
        case 128: e4m3 ? launch<128, 128, true>(a, p.few, s) : launch<128, 128, false>(a, p.few, s); break;
        case 192: e4m3 ? launch<192, 128, true>(a, p.few, s) : launch<192, 128, false>(a, p.few, s); break;
        case 256: e4m3 ? launch<256, 256, true>(a, p.few, s) : launch<256, 256, false>(a, p.few, s); break;
        default: launch_latent(a, c.k_cols, p.few, s); break;
    }
    return launch_status();
}

}  // namespace

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
    return attend(a, *cache, *batch, heads, window, ws, ws_bytes, stream);
}

extern "C" int fp8blk_latent_attn(const fp8blk_cache* cache, const uint16_t* q, int64_t q_token, int64_t q_head, int64_t N,
                                  int64_t heads, const fp8blk_batch* batch, float scale, int causal, int64_t window,
                                  const float* sinks, uint16_t* out, int64_t out_token, int64_t out_head, void* ws,
                                  size_t ws_bytes, fp8blk_stream_t stream) {
    AttnArgs a;
    const int st = attn_args(a, cache, q, q_token, q_head, N, heads, batch, scale, causal, window, sinks, out, out_token,
                             out_head);
    if (st) return st;
    if (cache->v || cache->type != FP8BLK_BF16 || cache->heads != 1 || cache->v_cols != kLatent ||
        (cache->k_cols != kLatent && cache->k_cols != kLatent + 64))
        return FP8BLK_ERR_ARG;
    return attend(a, *cache, *batch, heads, window, ws, ws_bytes, stream);
}

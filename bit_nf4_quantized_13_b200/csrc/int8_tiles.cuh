// int8_tiles.cuh -- what the Int8 linear's two tensor-core products share: the
// tiles of ragged row ranges (dense: one range), and the bf16 store of a
// transposed accumulator.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qlora {

constexpr int kTileRows = 256;  // weight-side rows of a tile: 128 in each CTA of a pair

// The experts' row ranges and tiles, in shared memory.
struct RowTable {
    int* off;    // E + 1: expert e's rows are [off[e], off[e + 1]), ascending in [0, T]
    int* tile0;  // E + 1: tiles of the experts before e; tile0[E]: all tiles
};
constexpr int kRowTableBytes = 2 * 4 * (QLORA_MAX_EXPERTS + 1);

__device__ __forceinline__ RowTable row_table(void* smem) {
    return RowTable{static_cast<int*>(smem), static_cast<int*>(smem) + QLORA_MAX_EXPERTS + 1};
}

// An expert's m token rows are cut into the fewest tiles of at most `cap`
// tokens, all of the same width (a multiple of 32): 257 rows are two tiles of
// 160, not one of 256 and one of 32, whose stages cost nearly as much.
__host__ __device__ inline int token_tiles(int m, int cap) { return (m + cap - 1) / cap; }
__host__ __device__ inline int token_width(int m, int cap) {
    const int t = token_tiles(m, cap);
    return t > 0 ? ((m + t - 1) / t + 31) & ~31 : 0;
}

// Filled by one warp.  An offset counts as no less than the one before it and
// at most T, so the ranges are disjoint and inside the rows whatever it holds.
// num_w: weight-side tiles of one expert.
__device__ __forceinline__ void build_table(const RowRanges& rr, int E, int num_w, int cap, const RowTable& tb,
                                            int lane) {
    const int T = static_cast<int>(rr.T);
    int top = 0, tiles = 0;  // the last offset and the tiles so far
    if (rr.offsets) top = min(max(rr.offsets[0], 0), T);
    if (lane == 0) {
        tb.off[0] = top;
        tb.tile0[0] = 0;
    }
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        int hi = T;
        if (rr.offsets) hi = e < E ? min(rr.offsets[e + 1], T) : 0;
        hi = max(hi, top);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) hi = max(hi, __shfl_up_sync(0xffffffffu, hi, o));  // lanes < o: their own
        int lo = __shfl_up_sync(0xffffffffu, hi, 1);
        if (lane == 0) lo = top;
        int n = e < E ? token_tiles(hi - lo, cap) * num_w : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += up;
        }
        if (e < E) {
            tb.off[e + 1] = hi;
            tb.tile0[e + 1] = tiles + n;
        }
        tiles += __shfl_sync(0xffffffffu, n, 31);
        top = __shfl_sync(0xffffffffu, hi, 31);
    }
}

struct Tile {
    int expert, row0;  // expert, first weight-side row
    int tok0, toks;    // first token row (of all T), tokens
};

// Tile `unit`: experts in order; inside an expert bands of kBand weight tiles
// with the token tiles slowest in a band, so that the pairs at work at the
// same time cover a compact block of tokens and weights (kept in L2).
__device__ __forceinline__ Tile tile_of(const RowTable& tb, int E, int num_w, int cap, int unit) {
    constexpr int kBand = 8;
    int e = 0, above = E;  // tile0[e] <= unit < tile0[above]
    while (above - e > 1) {
        const int c = (e + above) >> 1;
        if (tb.tile0[c] <= unit)
            e = c;
        else
            above = c;
    }
    const int lo = tb.off[e], hi = tb.off[e + 1];
    const int u = unit - tb.tile0[e];
    const int num_t = token_tiles(hi - lo, cap), width = token_width(hi - lo, cap);
    const int band_tiles = kBand * num_t;
    const int band = u / band_tiles, in = u % band_tiles;
    const int rows_in_band = min(kBand, num_w - band * kBand);
    const int t = in / rows_in_band;
    Tile s;
    s.expert = e;
    s.row0 = (band * kBand + in % rows_in_band) * kTileRows;
    s.tok0 = lo + t * width;
    s.toks = min(width, hi - s.tok0);
    return s;
}

// A schedule: every tile, or (where the tiles leave most pairs of SMs idle: few
// of them, with a long contraction) each tile's stages cut into `parts` runs
// for as many pairs.  A part leaves its sums in a workspace slot of its own and
// a second kernel adds them in order, so no pair waits for another and the
// result does not depend on the order of arrival.
struct Schedule {
    RowRanges rr;
    int E;
    int num_w;           // weight-side tiles of one expert
    int kbt;             // stages of a tile
    int parts;           // parts of a tile
    uint32_t* slots;     // parts > 1: a slot for each part
    int64_t slot_words;  // 256 rows of the widest tile's tokens
};

// One part of a tile.
struct Item {
    Tile tl;
    int kb0, stages;
};

__device__ __forceinline__ Item item_of(const Schedule& q, const RowTable& tb, int cap, int it) {
    Item x;
    int tile = it;
    x.kb0 = 0;
    x.stages = q.kbt;
    if (q.parts > 1) {
        tile = it / q.parts;
        const int part = it - tile * q.parts;
        x.kb0 = part * q.kbt / q.parts;
        x.stages = (part + 1) * q.kbt / q.parts - x.kb0;
    }
    x.tl = tile_of(tb, q.E, q.num_w, cap, tile);
    return x;
}

// A slot holds [CTA][chunk of 32 tokens][group of 4 tokens][row][4], so that
// each lane's 16 bytes of a group are part of 512 contiguous ones.
__device__ __forceinline__ uint4* slot_at(const Schedule& q, int slot, uint32_t rank, int chunk, int group, int row) {
    return reinterpret_cast<uint4*>(q.slots + slot * q.slot_words + rank * (q.slot_words / 2) +
                                    (static_cast<int64_t>(chunk * 8 + group) * (kTileRows / 2) + row) * 4);
}

__device__ __forceinline__ void slot_store(const Schedule& q, int slot, uint32_t rank, int chunk, int row,
                                           const uint32_t (&v)[32]) {
#pragma unroll
    for (int g = 0; g < 8; ++g)
        *slot_at(q, slot, rank, chunk, g, row) = make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
}

// The adding kernel's block (tile, chunk of 32 tokens, CTA) of kAddThreads, a
// row each: the tile and the row's sums over the parts (kInt: integers, else
// fp32); false where the tile has no such chunk.
constexpr int kAddThreads = kTileRows / 2;
template <bool kInt>
__device__ __forceinline__ bool add_parts(const Schedule& q, int cap, Tile* tl, uint32_t (&v)[32]) {
    __shared__ int s_table[kRowTableBytes / 4];
    const RowTable tb = row_table(s_table);
    if (threadIdx.x < 32) build_table(q.rr, q.E, q.num_w, cap, tb, static_cast<int>(threadIdx.x));
    __syncthreads();
    const int tile = static_cast<int>(blockIdx.x), chunk = static_cast<int>(blockIdx.y);
    sm100::grid_dependency_wait();  // the parts' sums
    if (tile >= tb.tile0[q.E]) return false;
    *tl = tile_of(tb, q.E, q.num_w, cap, tile);
    if (chunk * 32 >= tl->toks) return false;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0u;  // the bits of 0.0f too
#pragma unroll 2
    for (int j = 0; j < q.parts; ++j) {
        uint4 x[8];
#pragma unroll
        for (int g = 0; g < 8; ++g)
            x[g] = __ldcg(slot_at(q, tile * q.parts + j, blockIdx.z, chunk, g, static_cast<int>(threadIdx.x)));
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const uint32_t y[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t& a = v[4 * g + i];
                a = kInt ? a + y[i] : __float_as_uint(__uint_as_float(a) + __uint_as_float(y[i]));
            }
        }
    }
    return true;
}

// The most tiles of a problem, and the parts each is cut into: as many as give
// every pair of SMs one, of at least kMinStages stages, if that takes
// `min_saved` stages off a pair's work.  Adding them costs about 5 us and 0.4
// us a part, so they end at kMaxParts.
constexpr int kMinStages = 8, kMaxParts = 16;
inline Schedule schedule_of(const RowRanges& rr, int E, int64_t w_rows, int64_t kbt, int cap, int min_saved,
                            int64_t* tiles) {
    Schedule q{};
    q.rr = rr;
    q.E = E;
    q.num_w = static_cast<int>(ceil_div(w_rows, kTileRows));
    q.kbt = static_cast<int>(kbt);
    q.slot_words = static_cast<int64_t>(kTileRows) * (rr.T < cap ? round_up(rr.T, 32) : cap);
    *tiles = E == 1 ? static_cast<int64_t>(token_tiles(static_cast<int>(rr.T), cap)) * q.num_w
                    : int8_tiles(rr.T, E, w_rows, cap);
    const int64_t pairs = num_sms() / 2 > 0 ? num_sms() / 2 : 1;
    int64_t parts = pairs / (*tiles > 0 ? *tiles : 1);
    if (parts > kbt / kMinStages) parts = kbt / kMinStages;
    if (parts > kMaxParts) parts = kMaxParts;
    q.parts = parts > 1 && kbt - kbt / parts >= min_saved ? static_cast<int>(parts) : 1;
    return q;
}
inline size_t slots_bytes(const Schedule& q, int64_t tiles) {
    return q.parts == 1 ? 0 : static_cast<size_t>(tiles * q.parts * q.slot_words) * 4;
}

// The adding kernel's launch, dependent on the product's.
inline cudaLaunchConfig_t add_config(cudaLaunchAttribute (&attr)[1], const Schedule& q, int64_t tiles,
                                     cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(q.slot_words / kTileRows / 32), 2);
    cfg.blockDim = dim3(kAddThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// The MMA's width for a tile's tokens, and the token rows each CTA of the
// pair copies for it (half of them, in a box of 32, 64 or 128 rows).
__device__ __forceinline__ int mma_tokens(int toks) { return (toks + 31) & ~31; }
__device__ __forceinline__ int box_index(int half) { return half > 64 ? 2 : half > 32 ? 1 : 0; }
constexpr int kBoxes = 3;
__host__ __device__ constexpr int box_rows(int i) { return 32 << i; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// Four codes -> two bf16 pairs of RN32(code * sc); ms = {sc, sc}.  The fp32
// steps are done two at a time (each half is the ordinary IEEE operation).
__device__ __forceinline__ void convert4(uint32_t codes, uint64_t ms, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;  // code + 128
    uint32_t f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = prmt(u, 0x4B000000u, 0x7540u + i);  // 2^23 + 128 + code
    asm("{\n\t.reg .b64 a, b, m;\n\t"
        "mov.b64 a, {%2, %3};\n\t"
        "mov.b64 b, {%4, %5};\n\t"
        "mov.b64 m, {%7, %7};\n\t"
        "add.rn.f32x2 a, a, m;\n\t"
        "add.rn.f32x2 b, b, m;\n\t"
        "mul.rn.f32x2 a, a, %6;\n\t"
        "mul.rn.f32x2 b, b, %6;\n\t"
        ".reg .f32 a0, a1, b0, b1;\n\t"
        "mov.b64 {a0, a1}, a;\n\t"
        "mov.b64 {b0, b1}, b;\n\t"
        "cvt.rn.bf16x2.f32 %0, a1, a0;\n\t"
        "cvt.rn.bf16x2.f32 %1, b1, b0;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]), "l"(ms), "r"(0xCB000080u /* -(2^23 + 128) */));
}

// Stores 32 tokens x 32 columns of a row-major bf16 matrix: lane `lane` holds
// column `col` (= col0 + lane, col0 a multiple of 32) of the tokens 0 .. 31 as
// v[]; `left` of the tokens exist.  Rows whose length is a multiple of 4 are
// stored 8 bytes a lane: two exchanges between neighbouring lanes turn 4
// tokens x 1 column into 1 token x 4 columns, a quarter of the stores.
__device__ __forceinline__ void store_bf16_chunk(uint16_t* out, int ncols, int col, int left, const float (&v)[32],
                                                 int lane) {
    const bool ok = col < ncols;
    uint32_t w[16];  // tokens 2 i (low half) and 2 i + 1
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (ncols % 4 == 0) {
        const bool odd = lane & 1, upper = lane & 2;
        out += col & ~3;  // this lane's 4 columns (all of them exist or none)
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // tokens 4 i .. 4 i + 3
            // even lanes: tokens 4 i and 4 i + 2 of columns (col, col + 1); odd lanes: 4 i + 1 and 4 i + 3
            const uint32_t sel = odd ? 0x3276u : 0x5410u;
            const uint32_t a = prmt(w[2 * i], __shfl_xor_sync(0xffffffffu, w[2 * i], 1), sel);
            const uint32_t b = prmt(w[2 * i + 1], __shfl_xor_sync(0xffffffffu, w[2 * i + 1], 1), sel);
            // lanes with bit 1 clear keep the first token's 4 columns, the others the second's
            const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? a : b, 2);
            const int j = 4 * i + (odd ? 1 : 0) + (upper ? 2 : 0);
            if (ok && j < left)
                *reinterpret_cast<uint2*>(out + static_cast<int64_t>(j) * ncols) =
                    upper ? make_uint2(got, b) : make_uint2(a, got);
        }
    } else {
        out += col;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (ok && j < left)
                out[static_cast<int64_t>(j) * ncols] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
    }
}

}  // namespace qlora

// int8_tiles.cuh -- what the Int8 linear's two tensor-core products share: the
// tiles of ragged row ranges (dense: one range), and the bf16 store of a
// transposed accumulator.
#pragma once

#include "common.cuh"
#include "kernels.h"

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

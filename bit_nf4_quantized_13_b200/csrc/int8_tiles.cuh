// int8_tiles.cuh -- what the Int8 linear's two tensor-core products share: the
// tiles of ragged row ranges (dense: one range) and their schedule, the parts of
// tiles cut along the contraction, the conversion of codes and the bf16 store of
// a transposed accumulator.
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
constexpr int kRowTableBytes = (2 * 4 * (QLORA_MAX_EXPERTS + 1) + 15) / 16 * 16;

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

// The schedule of a product.  Tiles go round-robin to the pairs of SMs, whole
// but in the last round: where its tiles leave most pairs idle, each one's
// stages are cut into `parts` runs for as many pairs.  A part leaves its sums in
// a workspace slot of its own and a second kernel adds them in order, so no pair
// waits for another and the result does not depend on the order of arrival.
struct Schedule {
    RowRanges rr;
    int E;
    int num_w;           // weight-side tiles of one expert
    int cap;             // most tokens of a tile
    int kbt;             // stages of a tile
    int min_saved;       // stages that parts must take off a pair's work
    int pairs;           // of the launch
    uint32_t* slots;     // a slot for each part (at most `pairs`); nullptr: whole tiles only
    int64_t slot_words;  // 256 rows of the widest tile's tokens
};

// Filled by one warp.  An offset counts as no less than the one before it and
// at most T, so the ranges are disjoint and inside the rows whatever it holds.
__device__ __forceinline__ void build_table(const Schedule& q, const RowTable& tb, int lane) {
    const RowRanges& rr = q.rr;
    const int E = q.E;
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
        int n = e < E ? token_tiles(hi - lo, q.cap) * q.num_w : 0;
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
__device__ __forceinline__ Tile tile_of(const Schedule& q, const RowTable& tb, int unit) {
    constexpr int kBand = 8;
    int e = 0, above = q.E;  // tile0[e] <= unit < tile0[above]
    while (above - e > 1) {
        const int c = (e + above) >> 1;
        if (tb.tile0[c] <= unit)
            e = c;
        else
            above = c;
    }
    const int lo = tb.off[e], hi = tb.off[e + 1];
    const int u = unit - tb.tile0[e];
    const int num_t = token_tiles(hi - lo, q.cap), width = token_width(hi - lo, q.cap);
    const int band_tiles = kBand * num_t;
    const int band = u / band_tiles, in = u % band_tiles;
    const int rows_in_band = min(kBand, q.num_w - band * kBand);
    const int t = in / rows_in_band;
    Tile s;
    s.expert = e;
    s.row0 = (band * kBand + in % rows_in_band) * kTileRows;
    s.tok0 = lo + t * width;
    s.toks = min(width, hi - s.tok0);
    return s;
}

// The last round of `tiles` tiles: its first tile and their parts, as many as
// give every pair one, of at least kMinStages stages.  Adding them costs about 5
// us and 0.4 us a part, so they end at kMaxParts.
constexpr int kMinStages = 8, kMaxParts = 16;
struct Tail {
    int first, parts;
};
__host__ __device__ inline Tail tail_of(const Schedule& q, int tiles, int pairs) {
    Tail t;
    t.first = tiles / pairs * pairs;
    const int left = tiles - t.first;
    int parts = left > 0 ? pairs / left : 1;
    if (parts > q.kbt / kMinStages) parts = q.kbt / kMinStages;
    if (parts > kMaxParts) parts = kMaxParts;
    t.parts = parts > 1 && q.kbt - q.kbt / parts >= q.min_saved ? parts : 1;
    return t;
}

// What the pairs work on: the items of one launch, in shared memory.
struct Items {
    int count;
    Tail tail;
};
__device__ __forceinline__ Items items_of(const Schedule& q, const RowTable& tb) {
    Items x;
    const int tiles = tb.tile0[q.E];
    x.tail = q.slots ? tail_of(q, tiles, q.pairs) : Tail{tiles, 1};
    x.count = x.tail.first + (tiles - x.tail.first) * x.tail.parts;
    return x;
}

// One item: a tile, or a part of one.
struct alignas(16) Item {
    Tile tl;
    int kb0, stages;
    int slot;  // -1: the whole tile
};

__device__ __forceinline__ Item item_of(const Schedule& q, const RowTable& tb, const Items& items, int it) {
    Item x;
    int tile = it;
    x.kb0 = 0;
    x.stages = q.kbt;
    x.slot = -1;
    const int parts = items.tail.parts;
    if (parts > 1 && it >= items.tail.first) {
        x.slot = it - items.tail.first;
        const int t = x.slot / parts, part = x.slot - t * parts;
        tile = items.tail.first + t;
        x.kb0 = part * q.kbt / parts;
        x.stages = (part + 1) * q.kbt / parts - x.kb0;
    }
    x.tl = tile_of(q, tb, tile);
    return x;
}

// A pair's first items, worked out once by a thread each: every warp asks for
// every item, and the search and divisions of item_of would cost each of them
// some 400 cycles a tile, against 4000 to 9000 of a tile of 16 stages.
constexpr int kListed = 64;
constexpr int kItemListBytes = kListed * static_cast<int>(sizeof(Item));
__device__ __forceinline__ void list_items(const Schedule& q, const RowTable& tb, const Items& items, int pair, int pairs,
                                           Item* list) {
    for (int i = threadIdx.x; i < kListed && pair + i * pairs < items.count; i += blockDim.x)
        list[i] = item_of(q, tb, items, pair + i * pairs);
}
// The pair's i-th item, `it` of all.
__device__ __forceinline__ Item listed_item(const Schedule& q, const RowTable& tb, const Items& items, const Item* list,
                                            int i, int it) {
    return i < kListed ? list[i] : item_of(q, tb, items, it);
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

// The adding kernel's block (tile of the last round, chunk of 32 tokens, CTA)
// of kAddThreads, a row each: the tile and the row's sums over the parts (kInt:
// integers, else fp32); false where there is no such tile or chunk.
constexpr int kAddThreads = kTileRows / 2;
template <bool kInt>
__device__ __forceinline__ bool add_parts(const Schedule& q, Tile* tl, uint32_t (&v)[32]) {
    __shared__ int s_table[kRowTableBytes / 4];
    const RowTable tb = row_table(s_table);
    if (threadIdx.x < 32) build_table(q, tb, static_cast<int>(threadIdx.x));
    __syncthreads();
    const int tiles = tb.tile0[q.E], t = static_cast<int>(blockIdx.x), chunk = static_cast<int>(blockIdx.y);
    const Tail tail = tail_of(q, tiles, q.pairs);
    sm100::grid_dependency_wait();  // the parts' sums
    if (tail.parts == 1 || tail.first + t >= tiles) return false;
    *tl = tile_of(q, tb, tail.first + t);
    if (chunk * 32 >= tl->toks) return false;
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0u;  // the bits of 0.0f too
#pragma unroll 2
    for (int j = 0; j < tail.parts; ++j) {
        uint4 x[8];
#pragma unroll
        for (int g = 0; g < 8; ++g)
            x[g] = __ldcg(slot_at(q, t * tail.parts + j, blockIdx.z, chunk, g, static_cast<int>(threadIdx.x)));
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

// The schedule for `most` pairs at most, without its slots.
inline Schedule schedule_of(const RowRanges& rr, int E, int64_t w_rows, int64_t kbt, int cap, int min_saved,
                            int64_t most) {
    Schedule q{};
    q.rr = rr;
    q.E = E;
    q.num_w = static_cast<int>(ceil_div(w_rows, kTileRows));
    q.cap = cap;
    q.kbt = static_cast<int>(kbt);
    q.min_saved = min_saved;
    q.slot_words = static_cast<int64_t>(kTileRows) * (rr.T < cap ? round_up(rr.T, 32) : cap);
    // no more pairs than there can be items
    int64_t parts = kbt / kMinStages < kMaxParts ? kbt / kMinStages : kMaxParts;
    if (parts < 1) parts = 1;
    const int64_t tiles = E == 1 ? static_cast<int64_t>(token_tiles(static_cast<int>(rr.T), cap)) * q.num_w
                                 : int8_tiles(rr.T, E, w_rows, cap);
    q.pairs = static_cast<int>(tiles * parts < most ? tiles * parts : most);
    return q;
}

// Bytes of its slots: none where no tile will be cut, which for a dense product
// (every row, one weight) is known here; for experts only the device knows.
inline size_t slots_bytes(const Schedule& q) {
    const int parts = q.kbt / kMinStages < kMaxParts ? q.kbt / kMinStages : kMaxParts;
    if (parts < 2 || q.pairs < 2 || q.kbt - q.kbt / parts < q.min_saved) return 0;
    if (q.E == 1 && tail_of(q, token_tiles(static_cast<int>(q.rr.T), q.cap) * q.num_w, q.pairs).parts == 1) return 0;
    return static_cast<size_t>(q.pairs * q.slot_words) * 4;
}

inline int sm_pairs() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }

// The adding kernel's launch, dependent on the product's: a tile of the last
// round is cut only if there are two pairs for it.
inline cudaLaunchConfig_t add_config(cudaLaunchAttribute (&attr)[1], const Schedule& q, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(q.pairs / 2), static_cast<unsigned>(q.slot_words / kTileRows / 32), 2);
    cfg.blockDim = dim3(kAddThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// The MMA's width for a tile's tokens, and the token rows each CTA of the
// pair copies for it (half of them, in a box of 32, 64 or 128 rows).
__host__ __device__ constexpr int mma_tokens(int toks) { return (toks + 31) & ~31; }
__host__ __device__ constexpr int box_index(int half) { return half > 64 ? 2 : half > 32 ? 1 : 0; }
constexpr int kBoxes = 3;
__host__ __device__ constexpr int box_rows(int i) { return 32 << i; }
// The boxes that a schedule's tiles can need: the first ones.  The others' maps
// are not made (each takes the host part of a microsecond).
inline int boxes_of(const Schedule& q) {
    return box_index(mma_tokens(q.rr.T < q.cap ? static_cast<int>(q.rr.T) : q.cap) / 2) + 1;
}

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

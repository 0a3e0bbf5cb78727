// int8_pair_sm100.cu -- the Int8 linear's forward on the tensor cores, on
// pairs of SMs, dense or grouped by expert:
//
//   Y[m][n] = (sum_k xq[m][k] wq[n][k]) * sx[m] * sw[n]
//
// tcgen05.mma.kind::i8 (8-bit operands, exact 32-bit integer sums, twice the
// rate of bf16) computes the product transposed, D[n][m], with the weight as
// the MMA's A operand: a tile is 256 output channels (128 in each CTA of the
// pair) x up to 256 tokens.  The weight's side is never ragged but at its
// end, so the MMA's N follows the tokens instead: a tile with m tokens issues
// N = round_up(m, 32) and copies only those token rows.  That is what makes
// one kernel serve experts with any number of rows, and short batches.
//
// Warp roles (320 threads per CTA, persistent over the pair's tiles):
//   warp 0     TMA producer (both CTAs, into their own shared memory; the
//              bytes count on the even CTA's barrier): 128 bytes of
//              contraction per stage, a ring of kStages
//   warp 1     MMA issuer (one thread of the even CTA)
//   warps 2-9  epilogue: TMEM lane quarter w % 4 (32 output channels), every
//              second 32-token column chunk; scales, rounding, stores
//              coalesced along the channels
// Two accumulators of 256 columns alternate, so a tile's epilogue runs under
// the next tile's MMAs.
//
// Tiles go round-robin to the pairs.  When the last round would leave at
// least half of the pairs idle (short batches, narrow weights), the stages of
// its tiles are shared out evenly and a tile may be split along the
// contraction: every part adds up in its own workspace slot, and the warp
// that arrives last at a region's counter sums the slots.  No one waits for
// another pair (two such kernels may share the GPU), and integer sums make
// the result independent of the order.
//
// Every mbarrier wait is bounded; a timeout records QLORA_ERR_TIMEOUT in a
// sticky device word and ends the role.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace qlora {

__device__ int g_int8_error = 0;  // sticky: QLORA_ERR_TIMEOUT if a wait gave up

namespace {

using namespace sm100;

constexpr int kRowsCta = 128;                  // output channels per CTA
constexpr int kRowsPair = 2 * kRowsCta;        // MMA M
constexpr int kTileTok = 256;                  // largest MMA N
constexpr int kBK = 128;                       // contraction bytes per stage
constexpr int kStages = 6;
constexpr int kABytes = kRowsCta * kBK;        // 16 KiB
constexpr int kBBytes = kTileTok / 2 * kBK;    // 16 KiB: half of the tokens in each CTA
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kSmallBox = 16;                  // token rows of the ragged tiles' copies
constexpr uint32_t kTmemCols = 512;
constexpr int kBarOff = kStages * kStageBytes;
constexpr int kTableOff = kBarOff + 256;
constexpr int kSmemBytes = 1024 /* alignment slack */ + kTableOff + 2 * 4 * (QLORA_MAX_EXPERTS + 1);
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;
constexpr int kMinStagesPerPair = 4;
constexpr int kCounters = 2 * kEpiWarps;       // regions of a tile: the epilogue warps of both CTAs

struct Params {
    const float* xs;   // T token scales
    const float* ws;   // E x N channel scales
    RowRanges rr;
    int E, N, K;
    int num_w;         // weight tiles of one expert
    int kbt;           // stages of a tile
    void* out;
    int* counters;     // split tiles: kCounters per tail tile, zero at the start
    int* partial;      // split tiles: two slots per pair
    int slot_cols;     // tokens a slot holds (a multiple of 32)
};

struct Pipe {
    uint32_t smem, bar0, tmem, rank;
    int pair, num_pairs;
    __device__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ uint32_t empty(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ uint32_t acc_full(int b) const { return bar0 + 8u * (2 * kStages + b); }
    __device__ uint32_t acc_empty(int b) const { return bar0 + 8u * (2 * kStages + 2 + b); }
    __device__ uint32_t drain() const { return bar0 + 8u * (2 * kStages + 4); }
    __device__ uint32_t sA(int s) const { return smem + static_cast<uint32_t>(s * kStageBytes); }
    __device__ uint32_t sB(int s) const { return sA(s) + kABytes; }
};

// The experts' row ranges and tiles, in shared memory.
struct Table {
    int* off;    // E + 1: expert e's rows are [off[e], off[e + 1]), ascending in [0, T]
    int* tile0;  // E + 1: tiles of the experts before e; tile0[E]: all tiles
};

// A pair's share: `rounds` whole tiles pair + r * pairs, then (the first
// `tpairs` pairs) the iterations [lo, hi) of the tail (tile * kbt + stage,
// relative to tile `tail0`).  A range is at least kMinStagesPerPair and at
// most half a tile (+ 1 stage) long, so it touches at most two tail tiles.
struct Plan {
    int pairs;    // pairs that take part
    int rounds, tail0, tail_it, tpairs;
    int lo, hi, t_first, nseg;
};

__device__ __forceinline__ int tail_lo(int pair, int tail_it, int tpairs) {
    return static_cast<int>(static_cast<int64_t>(pair) * tail_it / tpairs);
}

__device__ __forceinline__ Plan make_plan(int units, int kbt, int pair, int num_pairs) {
    Plan r{};
    const int by_work = units * kbt / kMinStagesPerPair;  // < 2^31: checked by the host
    r.pairs = max(1, min(num_pairs, by_work));
    const int rem = units % r.pairs;
    const int tpairs = min(r.pairs, rem * kbt / kMinStagesPerPair);
    if (rem != 0 && 2 * rem <= tpairs) {
        r.rounds = units / r.pairs;
        r.tail0 = r.rounds * r.pairs;
        r.tail_it = rem * kbt;
        r.tpairs = tpairs;
    } else {
        r.rounds = pair < units ? (units - pair + r.pairs - 1) / r.pairs : 0;
        r.tail0 = units;
    }
    if (pair >= r.pairs) {
        r.rounds = 0;
        return r;
    }
    if (pair < r.tpairs) {
        r.lo = tail_lo(pair, r.tail_it, r.tpairs);
        r.hi = tail_lo(pair + 1, r.tail_it, r.tpairs);
        r.t_first = r.lo / kbt;
    }
    r.nseg = r.rounds + (r.hi > r.lo ? (r.hi - 1) / kbt - r.t_first + 1 : 0);
    return r;
}

// One tile's part of the pair's work.
struct Seg {
    int expert, row0;          // expert, first output channel of the tile
    int tok0, toks;            // first token row (of all T), tokens of the tile
    int kb_begin, kb_end;
    int tail_tile;             // split rounds: index of the tile in the tail, else -1
};

constexpr int kBand = 8;

// Tile `unit`: experts in order; inside an expert bands of kBand weight
// tiles with the token tiles slowest in a band, so the pairs at work at the
// same time cover a compact block of tokens and channels (kept in L2).
__device__ __forceinline__ void tile_of(const Params& p, const Table& tb, int unit, Seg& sg) {
    int e = 0, above = p.E;  // tile0[e] <= unit < tile0[above]
    while (above - e > 1) {
        const int c = (e + above) >> 1;
        if (tb.tile0[c] <= unit)
            e = c;
        else
            above = c;
    }
    const int lo = tb.off[e], hi = tb.off[e + 1];
    const int u = unit - tb.tile0[e];
    const int num_t = (hi - lo + kTileTok - 1) / kTileTok;
    const int band_tiles = kBand * num_t;
    const int band = u / band_tiles, in = u % band_tiles;
    const int rows_in_band = min(kBand, p.num_w - band * kBand);
    const int t = in / rows_in_band;
    sg.expert = e;
    sg.row0 = (band * kBand + in % rows_in_band) * kRowsPair;
    sg.tok0 = lo + t * kTileTok;
    sg.toks = min(kTileTok, hi - sg.tok0);
}

__device__ __forceinline__ void seg_of(const Params& p, const Table& tb, const Plan& R, int pair, int i, Seg& sg) {
    if (i < R.rounds) {
        sg.kb_begin = 0;
        sg.kb_end = p.kbt;
        sg.tail_tile = -1;
        tile_of(p, tb, pair + i * R.pairs, sg);
    } else {
        sg.tail_tile = R.t_first + (i - R.rounds);
        const int base = sg.tail_tile * p.kbt;
        sg.kb_begin = max(R.lo - base, 0);
        sg.kb_end = min(R.hi - base, p.kbt);
        tile_of(p, tb, R.tail0 + sg.tail_tile, sg);
    }
}

__device__ __forceinline__ int mma_tokens(const Seg& sg) { return (sg.toks + 31) & ~31; }

__device__ void role_tma(const Pipe& P, const Params& p, const Table& tb, const Plan& R, const CUtensorMap* tm_w,
                         const CUtensorMap* tm_x, const CUtensorMap* tm_x16) {
    int local = 0;
    for (int i = 0; i < R.nseg; ++i) {
        Seg sg;
        seg_of(p, tb, R, P.pair, i, sg);
        const int half = mma_tokens(sg) / 2;
        const int wrow = sg.expert * p.N + sg.row0 + static_cast<int>(P.rank) * kRowsCta;
        const int xrow = sg.tok0 + static_cast<int>(P.rank) * half;
        const uint32_t tx = 2u * static_cast<uint32_t>(kABytes + half * kBK);
        for (int kb = sg.kb_begin; kb < sg.kb_end; ++kb, ++local) {
            const int s = local % kStages;
            const uint32_t ph = static_cast<uint32_t>(local / kStages) & 1u;
            if (!mbar_wait(P.empty(s), ph ^ 1u, &g_int8_error)) return;
            const uint32_t bar = cluster_map(P.full(s), 0);
            if (P.rank == 0) mbar_arrive_expect_tx(P.full(s), tx);
            tma_load_2d_pair(P.sA(s), tm_w, bar, kb * kBK, wrow);
            if (half == kTileTok / 2) {
                tma_load_2d_pair(P.sB(s), tm_x, bar, kb * kBK, xrow);
            } else {
                for (int r = 0; r < half; r += kSmallBox)
                    tma_load_2d_pair(P.sB(s) + static_cast<uint32_t>(r * kBK), tm_x16, bar, kb * kBK, xrow + r);
            }
        }
    }
}

__device__ void role_mma(const Pipe& P, const Params& p, const Table& tb, const Plan& R) {
    int local = 0;
    for (int i = 0; i < R.nseg; ++i) {
        Seg sg;
        seg_of(p, tb, R, P.pair, i, sg);
        const int b = i & 1;
        const uint32_t idesc = idesc_i8(kRowsPair, mma_tokens(sg));
        if (!mbar_wait(P.acc_empty(b), (static_cast<uint32_t>(i >> 1) & 1u) ^ 1u, &g_int8_error)) return;
        tc_fence_after();
        for (int kb = sg.kb_begin; kb < sg.kb_end; ++kb, ++local) {
            const int s = local % kStages;
            const uint32_t ph = static_cast<uint32_t>(local / kStages) & 1u;
            if (!mbar_wait(P.full(s), ph, &g_int8_error)) return;
            tc_fence_after();
            const uint64_t ad = sdesc_kmajor_sw128(P.sA(s)), bd = sdesc_kmajor_sw128(P.sB(s));
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes along a row: 2 descriptor units
                mma_i8_ss_pair(P.tmem + b * kTileTok, ad + static_cast<uint64_t>(2 * kk),
                               bd + static_cast<uint64_t>(2 * kk), idesc, (kb > sg.kb_begin || kk > 0) ? 1u : 0u);
            tc_commit_pair_mc(P.empty(s), kPairMask);
        }
        tc_commit_pair_mc(P.acc_full(b), kPairMask);
    }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int lane) {
    int ok = 1;
    if (lane == 0) ok = mbar_wait(bar, parity, &g_int8_error) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

// Parts of tail tile t: the pairs whose ranges meet its kbt iterations.
__device__ __forceinline__ int pair_of(const Plan& R, int it) {
    return static_cast<int>((static_cast<int64_t>(it + 1) * R.tpairs - 1) / R.tail_it);
}

// Scales a chunk of 32 tokens (one column a token, one lane a channel),
// rounds and stores it.  (RN32(sum) * sx) * sw, in that order: the first
// product cannot leave the fp32 range for tokens whose scale is normal.
template <bool kF32>
__device__ __forceinline__ void store_chunk(const Params& p, const uint32_t (&acc)[32], const Seg& sg, int col,
                                            int chan, bool chan_ok, float sw, int lane) {
    const int left = sg.toks - col;  // tokens of the chunk that exist
    const float sx_lane = lane < left ? __ldg(p.xs + sg.tok0 + col + lane) : 0.0f;
    const int64_t o = static_cast<int64_t>(sg.tok0 + col) * p.N + chan;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float sx = __shfl_sync(0xffffffffu, sx_lane, j);
        const float v = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc[j])), sx), sw);
        if (chan_ok && j < left) {
            if (kF32)
                static_cast<float*>(p.out)[o + static_cast<int64_t>(j) * p.N] = v;
            else
                static_cast<uint16_t*>(p.out)[o + static_cast<int64_t>(j) * p.N] = f32_to_bf16_bits(v);
        }
    }
}

__device__ __forceinline__ int4 ld_cg_i4(const int* p) {
    int4 v;
    asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <bool kF32>
__device__ void role_epilogue(const Pipe& P, const Params& p, const Table& tb, const Plan& R, int warp, int lane) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const int lrow = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int64_t slot_ints = static_cast<int64_t>(kRowsPair) * p.slot_cols;
    // this lane's 32 sums of column chunk c in slot `slot`: eight groups of
    // four, one group 512 contiguous bytes a warp
    auto slot_at = [&](int slot, int c, int g) {
        return p.partial + slot * slot_ints + static_cast<int64_t>(P.rank) * (slot_ints / 2) +
               (static_cast<int64_t>(c * 8 + g) * kRowsCta + lrow) * 4;
    };
    for (int i = 0; i < R.nseg; ++i) {
        Seg sg;
        seg_of(p, tb, R, P.pair, i, sg);
        const int b = i & 1;
        const int chunks = mma_tokens(sg) / 32;
        const bool whole = sg.kb_begin == 0 && sg.kb_end == p.kbt;
        const int chan = sg.row0 + static_cast<int>(P.rank) * kRowsCta + lrow;
        const bool chan_ok = chan < p.N;
        const float sw = chan_ok ? __ldg(p.ws + static_cast<int64_t>(sg.expert) * p.N + chan) : 0.0f;
        const int my_slot = whole ? 0 : 2 * P.pair + (sg.tail_tile - R.t_first);
        if (!warp_wait(P.acc_full(b), static_cast<uint32_t>(i >> 1) & 1u, lane)) return;
        tc_fence_after();
#pragma unroll 1
        for (int c = half; c < chunks; c += 2) {
            uint32_t acc[32];
            tmem_ld_32x32b_x32(P.tmem + lane_base + static_cast<uint32_t>(b * kTileTok + c * 32), acc);
            tmem_wait_ld();
            if (whole) {
                store_chunk<kF32>(p, acc, sg, c * 32, chan, chan_ok, sw, lane);
            } else {
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    *reinterpret_cast<int4*>(slot_at(my_slot, c, g)) =
                        make_int4(static_cast<int>(acc[4 * g]), static_cast<int>(acc[4 * g + 1]),
                                  static_cast<int>(acc[4 * g + 2]), static_cast<int>(acc[4 * g + 3]));
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_map(P.acc_empty(b), 0));
        if (whole) continue;
        // the region (this warp's channels and chunks) is complete once every
        // part has counted itself; the last one to do so adds the slots
        const int base = sg.tail_tile * p.kbt;
        const int j0 = pair_of(R, base), j1 = pair_of(R, base + p.kbt - 1);
        __threadfence();
        __syncwarp();
        int old = 0;
        if (lane == 0)
            old = atomicAdd(p.counters + sg.tail_tile * kCounters + static_cast<int>(P.rank) * kEpiWarps + (warp - 2), 1);
        old = __shfl_sync(0xffffffffu, old, 0);
        if (old != j1 - j0) continue;
        __threadfence();
#pragma unroll 1
        for (int c = half; c < chunks; c += 2) {
            uint32_t acc[32] = {};
#pragma unroll 1
            for (int j = j0; j <= j1; ++j) {
                const int slot = 2 * j + (sg.tail_tile - tail_lo(j, R.tail_it, R.tpairs) / p.kbt);
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const int4 v = ld_cg_i4(slot_at(slot, c, g));
                    acc[4 * g] += static_cast<uint32_t>(v.x);
                    acc[4 * g + 1] += static_cast<uint32_t>(v.y);
                    acc[4 * g + 2] += static_cast<uint32_t>(v.z);
                    acc[4 * g + 3] += static_cast<uint32_t>(v.w);
                }
            }
            store_chunk<kF32>(p, acc, sg, c * 32, chan, chan_ok, sw, lane);
        }
    }
}

// One warp.  An offset counts as no less than the one before it and at most
// T, so the ranges are disjoint and inside the rows whatever it holds.
__device__ __forceinline__ void build_table(const Params& p, const Table& tb, int lane) {
    const int T = static_cast<int>(p.rr.T);
    int top = 0, tiles = 0;  // the last offset and the tiles so far
    if (lane == 0) {
        top = p.rr.offsets ? min(max(p.rr.offsets[0], 0), T) : 0;
        tb.off[0] = top;
        tb.tile0[0] = 0;
    }
    top = __shfl_sync(0xffffffffu, top, 0);
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + lane;
        int hi = T;
        if (p.rr.offsets) hi = e < p.E ? min(p.rr.offsets[e + 1], T) : 0;
        hi = max(hi, top);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) hi = max(hi, __shfl_up_sync(0xffffffffu, hi, o));  // lanes < o: their own
        int lo = __shfl_up_sync(0xffffffffu, hi, 1);
        if (lane == 0) lo = top;
        int n = e < p.E ? (hi - lo + kTileTok - 1) / kTileTok * p.num_w : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += up;
        }
        if (e < p.E) {
            tb.off[e + 1] = hi;
            tb.tile0[e + 1] = tiles + n;
        }
        tiles += __shfl_sync(0xffffffffu, n, 31);
        top = __shfl_sync(0xffffffffu, hi, 31);
    }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
k_int8_gemm_pair(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_x16, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
    const Table tb{reinterpret_cast<int*>(smem + kTableOff),
                   reinterpret_cast<int*>(smem + kTableOff) + QLORA_MAX_EXPERTS + 1};
    __shared__ Plan s_plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Pipe P;
    P.smem = smem_u32(smem);
    P.bar0 = smem_u32(bars);
    P.rank = cluster_ctarank();
    P.pair = static_cast<int>(blockIdx.x >> 1);
    P.num_pairs = static_cast<int>(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(P.full(s), 1);   // the even CTA's expect_tx arrival (+ both CTAs' bytes)
            mbar_init(P.empty(s), 1);  // the pair MMA's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(P.acc_full(b), 1);
            mbar_init(P.acc_empty(b), 2 * kEpiWarps);
        }
        mbar_init(P.drain(), 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    if (warp == 1 && lane == 0) {
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_x16);
    }
    if (warp == 2) {
        build_table(p, tb, lane);
        __syncwarp();
        if (lane == 0) s_plan = make_plan(tb.tile0[p.E], p.kbt, P.pair, P.num_pairs);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // both CTAs' barriers are initialised before any remote arrive
    cluster_wait();
    tc_fence_after();
    P.tmem = *tmem_slot;
    const Plan& R = s_plan;
    grid_dependency_wait();  // the quantized tokens, and the zeroed counters
    if (warp == 0) {
        if (lane == 0) role_tma(P, p, tb, R, &tm_w, &tm_x, &tm_x16);
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && P.rank == 0) {
            role_mma(P, p, tb, R);
            // every pair MMA issued (also on an early exit) has completed
            // before the tensor memory can be freed
            tc_commit_pair_mc(P.drain(), 1);
            mbar_wait(P.drain(), 0u, &g_int8_error);
        }
        __syncwarp();
    } else {
        role_epilogue<kF32>(P, p, tb, R, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // neither CTA frees its tensor memory or leaves while the pair may still use it
    cluster_wait();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(P.tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ host
// `rows` rows of K codes, ld bytes apart; 128-byte swizzled boxes of kBK
// codes x box_rows rows, zero fill outside.
bool make_map_i8(CUtensorMap* m, const void* base, int64_t K, int64_t rows, int64_t ld, uint32_t box_rows) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    cuuint32_t box[2] = {kBK, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute (&attr)[2], int pairs, cudaStream_t st, bool dependent) {
    cudaLaunchConfig_t cfg{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cfg;
}

template <bool kF32>
int max_pairs() {
    static ContextMemo<int> memo;
    uint64_t ctx = 0;
    if (!current_context_id(&ctx)) return 0;
    int n = 0;
    memo.get(ctx, &n, [](int* v) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = pair_config(attr, num_sms(), nullptr, false);
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, k_int8_gemm_pair<kF32>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            c = 0;
        }
        *v = c;
        return true;
    });
    return n;
}

int ws_pairs() { return num_sms() / 2 > 0 ? num_sms() / 2 : 1; }
size_t counter_bytes() { return static_cast<size_t>(round_up(static_cast<int64_t>(ws_pairs()) * kCounters * 4, 256)); }
int64_t slot_cols(int64_t T) { return T < kTileTok ? round_up(T, 32) : kTileTok; }

template <bool kF32>
cudaError_t launch_pair(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& mx16, const Params& p,
                        int64_t tiles, cudaStream_t st, bool dependent) {
    static ContextMemo<int> attr_memo;
    cudaError_t e = ensure_smem_limit(attr_memo, k_int8_gemm_pair<kF32>, kSmemBytes);
    if (e != cudaSuccess) return e;
    int pairs = max_pairs<kF32>();
    if (pairs > ws_pairs()) pairs = ws_pairs();
    const int64_t by_work = tiles * p.kbt / kMinStagesPerPair;
    if (by_work < pairs) pairs = static_cast<int>(by_work > 1 ? by_work : 1);
    if (pairs <= 0) return cudaErrorNotSupported;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(attr, pairs, st, dependent);
    e = cudaLaunchKernelEx(&cfg, k_int8_gemm_pair<kF32>, mw, mx, mx16, p);
    note_launches(1);
    return e;
}

}  // namespace

// The largest number of tiles that T rows in E ranges can need.
int64_t int8_pair_tiles(int64_t T, const Int8Weight& w) {
    return (T / kTileTok + (T < w.E ? T : w.E)) * ceil_div(w.N, kRowsPair);
}

bool int8_pair_supported(int64_t T, const Int8Weight& w) {
    return int8_pair_tiles(T, w) * ceil_div(w.K, kBK) < (int64_t(1) << 31);
}

// Workspace: the counters (zeroed before every launch), then two slots per
// pair of SMs.
size_t int8_pair_counter_bytes() { return counter_bytes(); }
size_t int8_pair_workspace(int64_t T) {
    return counter_bytes() + static_cast<size_t>(ws_pairs()) * 2 * kRowsPair * static_cast<size_t>(slot_cols(T)) * 4;
}

cudaError_t launch_int8_fwd_pair(const int8_t* x_codes, const float* x_scale, const Int8Weight& w,
                                 const RowRanges& rr, void* out, int out_dtype, void* ws, cudaStream_t st,
                                 bool dependent) {
    Params p{};
    p.xs = x_scale;
    p.ws = w.scale;
    p.rr = rr;
    p.E = w.E;
    p.N = static_cast<int>(w.N);
    p.K = static_cast<int>(w.K);
    p.num_w = static_cast<int>(ceil_div(w.N, kRowsPair));
    p.kbt = static_cast<int>(ceil_div(w.K, kBK));
    p.out = out;
    p.counters = static_cast<int*>(ws);
    p.partial = reinterpret_cast<int*>(static_cast<char*>(ws) + counter_bytes());
    p.slot_cols = static_cast<int>(slot_cols(rr.T));
    CUtensorMap mw, mx, mx16;
    if (!make_map_i8(&mw, w.codes, w.K, w.E * w.N, w.ld, kRowsCta) ||
        !make_map_i8(&mx, x_codes, w.K, rr.T, w.ld, kTileTok / 2) ||
        !make_map_i8(&mx16, x_codes, w.K, rr.T, w.ld, kSmallBox))
        return cudaErrorInvalidValue;
    const int64_t tiles = int8_pair_tiles(rr.T, w);
    return out_dtype == 0 ? launch_pair<true>(mw, mx, mx16, p, tiles, st, dependent)
                          : launch_pair<false>(mw, mx, mx16, p, tiles, st, dependent);
}

int int8_device_error(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_int8_error, sizeof(int)) != cudaSuccess) return QLORA_ERR_CUDA;
    if (reset && v) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_int8_error, &zero, sizeof(int)) != cudaSuccess) return QLORA_ERR_CUDA;
    }
    return v;
}

}  // namespace qlora

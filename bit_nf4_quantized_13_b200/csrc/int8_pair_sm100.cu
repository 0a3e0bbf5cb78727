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
//              contraction per stage, a ring of six to nine
//   warp 1     MMA issuer (one thread of the even CTA)
//   warps 2-9  epilogue: TMEM lane quarter w % 4 (32 output channels), every
//              second 32-token column chunk; scales, rounding, stores
//              coalesced along the channels
// Two accumulators of 256 columns alternate, so a tile's epilogue runs under
// the next tile's MMAs.
//
// Large products are bound by the tensor pipe: 4096 x 11008 x 4096 takes 111 us
// (3330 TOP/s, the pipe 80 to 91% active), 8192 x 8192 x 8192 303 us.  Few tokens
// are bound by the weight stream: 1500 rows over 64 experts of 1024 x 2048 take
// 32 us (142 MB).
//
// Every mbarrier wait is bounded; a timeout records QLORA_ERR_TIMEOUT in a
// sticky device word and ends the role.
#include <cudaTypedefs.h>

#include "common.cuh"
#include "int8_tiles.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace qlora {

__device__ int g_int8_error = 0;  // sticky: QLORA_ERR_TIMEOUT if a wait gave up

namespace {

using namespace sm100;

constexpr int kRowsCta = 128;                  // output channels per CTA
constexpr int kRowsPair = kTileRows;           // MMA M: 128 in each CTA
static_assert(kRowsPair == 2 * kRowsCta, "a tile's rows are halved between the CTAs");
constexpr int kTileTok = 256;                  // largest MMA N
constexpr int kBK = 128;                       // contraction bytes per stage
constexpr int kABytes = kRowsCta * kBK;        // 16 KiB
constexpr int kRingBytes = 192 * 1024;
constexpr int kMaxStages = 9;
constexpr int kEpiWarps = 8;
constexpr int kWarpChunks = kTileTok / 32 / 2;   // 32-token chunks of an epilogue warp
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kBarOff = kRingBytes;
constexpr int kTableOff = kBarOff + 256;
constexpr int kSmemBytes = 1024 /* alignment slack */ + kTableOff + kRowTableBytes + kItemListBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;

struct Params {
    const float* xs;   // T token scales
    const float* ws;   // E x N channel scales
    Schedule q;        // weight tiles: ceil(N / 256); stages: ceil(K / 128)
    int N;
    int boxes;         // token maps made
    int stages;        // of the ring
    int stage_bytes;   // the weight's 16 KiB, then half of the tokens
    void* out;
};

// The ring for tiles of up to `cap` tokens: the smaller the tokens' part of a
// stage (boxes for 64, 128 or 256), the more stages are in flight, which is
// what the weight stream of small tiles needs.
__host__ __device__ constexpr int stage_bytes(int cap) {
    return kABytes + (cap > 128 ? kTileTok : cap > 64 ? 128 : 64) / 2 * kBK;
}
__host__ __device__ constexpr int ring_stages(int cap) { return kRingBytes / stage_bytes(cap); }
static_assert(ring_stages(64) == kMaxStages && ring_stages(128) == 8 && ring_stages(kTileTok) == 6, "rings");
static_assert(8 * (2 * kMaxStages + 5) + 4 <= kTableOff - kBarOff, "barriers and the TMEM address");

struct Maps {
    CUtensorMap w;          // weight rows: boxes of kRowsCta
    CUtensorMap x[kBoxes];  // token rows: boxes of box_rows(i)
};

struct Pipe {
    uint32_t smem, bar0, tmem, rank;
    int pair, num_pairs;
    Item* list;
    __device__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ uint32_t empty(int s) const { return bar0 + 8u * (kMaxStages + s); }
    __device__ uint32_t acc_full(int b) const { return bar0 + 8u * (2 * kMaxStages + b); }
    __device__ uint32_t acc_empty(int b) const { return bar0 + 8u * (2 * kMaxStages + 2 + b); }
    __device__ uint32_t drain() const { return bar0 + 8u * (2 * kMaxStages + 4); }
};

__device__ void role_tma(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, const Maps& maps) {
    int s = 0;
    uint32_t ph = 1;
    for (int i = 0, it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const Tile& tl = x.tl;
        const int half = mma_tokens(tl.toks) / 2;
        const int box = box_index(half);
        const int wrow = tl.expert * p.N + tl.row0 + static_cast<int>(P.rank) * kRowsCta;
        const int xrow = tl.tok0 + static_cast<int>(P.rank) * half;
        const uint32_t tx = 2u * static_cast<uint32_t>(kABytes + box_rows(box) * kBK);
        for (int kb = x.kb0; kb < x.kb0 + x.stages; ++kb) {
            if (!mbar_wait(P.empty(s), ph, &g_int8_error)) return;
            const uint32_t bar = cluster_map(P.full(s), 0);
            if (P.rank == 0) mbar_arrive_expect_tx(P.full(s), tx);
            const uint32_t stage = P.smem + static_cast<uint32_t>(s * p.stage_bytes);
            tma_load_2d_pair(stage, &maps.w, bar, kb * kBK, wrow);
            tma_load_2d_pair(stage + kABytes, &maps.x[box], bar, kb * kBK, xrow);
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
    }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int lane) {
    int ok = 1;
    if (lane == 0) ok = mbar_wait(bar, parity, &g_int8_error) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    return ok != 0;
}

__device__ void role_mma(const Pipe& P, const Params& p, const RowTable& tb, const Items& items) {
    const uint64_t a0 = sdesc_kmajor_sw128(P.smem), b0 = sdesc_kmajor_sw128(P.smem + kABytes);
    int s = 0, i = 0;
    uint32_t ph = 0;
    for (int it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const int b = i & 1;
        const uint32_t idesc = idesc_i8(kRowsPair, mma_tokens(x.tl.toks));
        if (!mbar_wait(P.acc_empty(b), (static_cast<uint32_t>(i >> 1) & 1u) ^ 1u, &g_int8_error)) return;
        tc_fence_after();
        for (int kb = 0; kb < x.stages; ++kb) {
            if (!mbar_wait(P.full(s), ph, &g_int8_error)) return;
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(s) * static_cast<uint64_t>(p.stage_bytes / 16);
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk)  // 32 bytes along a row: 2 descriptor units
                mma_i8_ss_pair(P.tmem + b * kTileTok, a0 + off + 2 * kk, b0 + off + 2 * kk, idesc,
                                    (kb > 0 || kk > 0) ? 1u : 0u);
            tc_commit_pair_mc(P.empty(s), kPairMask);
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        tc_commit_pair_mc(P.acc_full(b), kPairMask);
    }
}

// Scales a chunk of 32 tokens (a column each; a lane is a channel), rounds
// and stores it: (RN32(sum) * sx) * sw, in that order.  The first product is no
// smaller than sx, so it loses nothing at the lower end of fp32; it is at most
// 127 K max|x|, beyond the upper end only for tokens above FLT_MAX / (127 K).
// All 32 values are formed before the first store: with a branch between them
// each one exposed its own latency.
template <bool kF32>
__device__ __forceinline__ void store_chunk(const Params& p, const uint32_t (&acc)[32], const float* sx,
                                            const Tile& tl, int col, int chan, float sw, int lane) {
    const int left = tl.toks - col;  // tokens of the chunk that exist
    float v[32];
#pragma unroll
    for (int j4 = 0; j4 < 8; ++j4) {
        const float4 s4 = *reinterpret_cast<const float4*>(sx + 4 * j4);
        v[4 * j4] = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc[4 * j4])), s4.x), sw);
        v[4 * j4 + 1] = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc[4 * j4 + 1])), s4.y), sw);
        v[4 * j4 + 2] = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc[4 * j4 + 2])), s4.z), sw);
        v[4 * j4 + 3] = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(acc[4 * j4 + 3])), s4.w), sw);
    }
    const int64_t row0 = static_cast<int64_t>(tl.tok0 + col) * p.N;
    if constexpr (kF32) {
        float* o = static_cast<float*>(p.out) + row0 + chan;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (chan < p.N && j < left) o[static_cast<int64_t>(j) * p.N] = v[j];
    } else {
        store_bf16_chunk(static_cast<uint16_t*>(p.out) + row0, p.N, chan, left, v, lane);
    }
}

template <bool kF32>
__device__ void role_epilogue(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, int warp, int lane) {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    __shared__ __align__(16) float s_sx[kEpiWarps][kWarpChunks * 32];
    float* sx = s_sx[warp - 2];
    int i = 0;
    for (int it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const Tile& tl = x.tl;
        const int b = i & 1;
        const int chunks = mma_tokens(tl.toks) / 32;
        const int chan = tl.row0 + static_cast<int>(P.rank) * kRowsCta + quarter * 32 + lane;
        const float sw = chan < p.N ? __ldg(p.ws + static_cast<int64_t>(tl.expert) * p.N + chan) : 0.0f;
        // the token scales of this warp's chunks, on their way before the sums are ready
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kWarpChunks; ++q) {
            const int tok = (half + 2 * q) * 32 + lane;
            sx[q * 32 + lane] = tok < tl.toks ? p.xs[tl.tok0 + tok] : 0.0f;
        }
        __syncwarp();
        if (!warp_wait(P.acc_full(b), static_cast<uint32_t>(i >> 1) & 1u, lane)) return;
        tc_fence_after();
#pragma unroll 1  // the code of one chunk: a tile's first pass over it is fetched cold
        for (int c = half; c < chunks; c += 2) {
            uint32_t acc[32];
            tmem_ld_32x32b_x32(P.tmem + lane_base + static_cast<uint32_t>(b * kTileTok + c * 32), acc);
            tmem_wait_ld();
            if (x.slot < 0)
                store_chunk<kF32>(p, acc, sx + (c / 2) * 32, tl, c * 32, chan, sw, lane);
            else
                slot_store(p.q, x.slot, P.rank, c, quarter * 32 + lane, acc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_map(P.acc_empty(b), 0));
    }
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
k_int8_gemm_pair(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);
    const RowTable tb = row_table(smem + kTableOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Pipe P;
    P.smem = smem_u32(smem);
    P.bar0 = smem_u32(bars);
    P.rank = cluster_ctarank();
    P.pair = static_cast<int>(blockIdx.x >> 1);
    P.num_pairs = static_cast<int>(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
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
        tma_prefetch_desc(&maps.w);
        for (int i = 0; i < p.boxes; ++i) tma_prefetch_desc(&maps.x[i]);
    }
    if (warp == 2) build_table(p.q, tb, lane);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // both CTAs' barriers are initialised before any remote arrive
    cluster_wait();
    tc_fence_after();
    P.tmem = *tmem_slot;
    const Items items = items_of(p.q, tb);
    P.list = reinterpret_cast<Item*>(smem + kTableOff + kRowTableBytes);
    list_items(p.q, tb, items, P.pair, P.num_pairs, P.list);
    __syncthreads();
    grid_dependency_wait();  // the quantized tokens
    if (warp == 0) {
        if (elect_one()) role_tma(P, p, tb, items, maps);
        __syncwarp();
    } else if (warp == 1) {
        if (P.rank == 0 && elect_one()) {
            role_mma(P, p, tb, items);
            // every pair MMA issued (also on an early exit) has completed
            // before the tensor memory can be freed
            tc_commit_pair_mc(P.drain(), 1);
            mbar_wait(P.drain(), 0u, &g_int8_error);
        }
        __syncwarp();
    } else {
        role_epilogue<kF32>(P, p, tb, items, warp, lane);
    }
    grid_launch_dependents();  // the kernel that adds the parts
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // neither CTA frees its tensor memory or leaves while the pair may still use it
    cluster_wait();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(P.tmem, kTmemCols);
    }
}

template <bool kF32>
__global__ void __launch_bounds__(kAddThreads) k_int8_gemm_add(const __grid_constant__ Params p) {
    __shared__ __align__(16) float s_sx[32];
    const int tok = static_cast<int>(blockIdx.y) * 32, lane = threadIdx.x & 31;
    Tile tl;
    uint32_t sums[32];
    if (!add_parts<true>(p.q, &tl, sums)) return;
    if (threadIdx.x < 32) s_sx[lane] = tok + lane < tl.toks ? p.xs[tl.tok0 + tok + lane] : 0.0f;
    __syncthreads();
    const int chan = tl.row0 + static_cast<int>(blockIdx.z) * kRowsCta + static_cast<int>(threadIdx.x);
    const float sw = chan < p.N ? __ldg(p.ws + static_cast<int64_t>(tl.expert) * p.N + chan) : 0.0f;
    store_chunk<kF32>(p, sums, s_sx, tl, tok, chan, sw, lane);
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

template <bool kF32>
cudaError_t launch_pair(const Maps& maps, const Params& p, cudaStream_t st, bool dependent) {
    static ContextMemo<int> attr_memo;
    cudaError_t e = ensure_smem_limit(attr_memo, k_int8_gemm_pair<kF32>, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (max_pairs<kF32>() < 1) return cudaErrorNotSupported;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(attr, p.q.pairs, st, dependent);
    e = cudaLaunchKernelEx(&cfg, k_int8_gemm_pair<kF32>, maps, p);
    note_launches(1);
    if (e != cudaSuccess || !p.q.slots) return e;
    cudaLaunchAttribute dep[1];
    const cudaLaunchConfig_t add = add_config(dep, p.q, st);
    e = cudaLaunchKernelEx(&add, k_int8_gemm_add<kF32>, p);
    note_launches(1);
    return e;
}

Schedule schedule_with(const RowRanges& rr, const Int8Weight& w, int cap) {
    // in a captured graph 500 x 512 x 11008 takes 20.6 us in whole tiles and 17.7 in parts
    return schedule_of(rr, w.E, w.N, ceil_div(w.K, kBK), cap, 48, sm_pairs());
}

// Cycles of the pairs' rounds over T rows of one weight.  Measured on 72 tiles
// (one round): a stage of m tokens takes 270 cycles for m = 64, 317 for 128, 470
// for 192, 590 for 256; a tile begins and ends in about 1500; adding parts takes
// 5 us and 0.4 us a part.
int64_t cycles(const Schedule& q) {
    const int T = static_cast<int>(q.rr.T), tiles = token_tiles(T, q.cap) * q.num_w;
    const Tail tail = tail_of(q, tiles, q.pairs);
    const int64_t stage = 180 + token_width(T, q.cap) * 8 / 5;
    int64_t c = tail.first / q.pairs * (q.kbt * stage + 1500);
    if (tail.first < tiles) c += (q.kbt + tail.parts - 1) / tail.parts * stage + 1500;
    return tail.parts > 1 ? c + 9500 + 760 * tail.parts : c;
}

// The most tokens of a tile.  Dense: the width whose rounds take the fewest
// cycles (with tiles of 256 only, 512 x 4096 x 11008 takes 39 us in place of 29,
// 777 x 5120 x 5120 33 in place of 27; 39 of 40 shapes of 200 to 3000 tokens are
// within 10% of the best width).  Experts: their average rows decide (an expert
// with more takes its weight through the L2 once a tile).
int tile_cap(int64_t T, const Int8Weight& w) {
    const int64_t m = ceil_div(T, T < w.E ? T : w.E);
    if (m <= 64) return 64;
    if (w.E > 1) return m <= 128 ? 128 : kTileTok;
    // the last answer, because a call asks several times (2 us of its host time)
    struct Asked {
        int64_t T, N, K;
        int pairs, cap;
    };
    static thread_local Asked last{};
    const Asked now{T, w.N, w.K, sm_pairs(), 0};
    if (last.T == now.T && last.N == now.N && last.K == now.K && last.pairs == now.pairs) return last.cap;
    int best = 0;
    int64_t least = 0;
    for (int cap = kTileTok; cap >= 64; cap -= 32) {
        const int64_t c = cycles(schedule_with(RowRanges{nullptr, T}, w, cap));
        if (best == 0 || c < least) {
            best = cap;
            least = c;
        }
    }
    last = now;
    last.cap = token_width(static_cast<int>(T), best);
    return last.cap;
}

Schedule schedule(const RowRanges& rr, const Int8Weight& w) { return schedule_with(rr, w, tile_cap(rr.T, w)); }

}  // namespace

// The largest number of tiles that T rows in E ranges can need.
int64_t int8_tiles(int64_t T, int E, int64_t w_rows, int tile_tok) {
    return (T / tile_tok + (T < E ? T : E)) * ceil_div(w_rows, kTileRows);
}

bool int8_pair_supported(int64_t T, const Int8Weight& w) {
    return int8_tiles(T, w.E, w.N, tile_cap(T, w)) * ceil_div(w.K, kBK) < (int64_t(1) << 31);
}

// Workspace: the parts' slots.
size_t int8_pair_workspace(int64_t T, const Int8Weight& w) {
    return slots_bytes(schedule(RowRanges{nullptr, T}, w));
}

cudaError_t launch_int8_fwd_pair(const int8_t* x_codes, const float* x_scale, const Int8Weight& w,
                                 const RowRanges& rr, void* out, int out_dtype, void* ws, cudaStream_t st,
                                 bool dependent) {
    Params p{};
    p.xs = x_scale;
    p.ws = w.scale;
    p.q = schedule(rr, w);
    if (int8_pair_workspace(rr.T, w) > 0) p.q.slots = static_cast<uint32_t*>(ws);
    p.boxes = boxes_of(p.q);
    p.stages = ring_stages(p.q.cap);
    p.stage_bytes = stage_bytes(p.q.cap);
    p.N = static_cast<int>(w.N);
    p.out = out;
    Maps maps;
    bool ok = make_map_i8(&maps.w, w.codes, w.K, w.E * w.N, w.ld, kRowsCta);
    for (int i = 0; i < p.boxes; ++i) ok = ok && make_map_i8(&maps.x[i], x_codes, w.K, rr.T, w.ld, box_rows(i));
    if (!ok) return cudaErrorInvalidValue;
    return out_dtype == 0 ? launch_pair<true>(maps, p, st, dependent)
                          : launch_pair<false>(maps, p, st, dependent);
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

// int8_dx_sm100.cu -- the Int8 linear's input gradient on the tensor cores, on
// pairs of SMs, dense or grouped by expert:
//
//   dX[m][k] = sum_n dY[m][n] * W'[n][k],   W' = bf16(RN32(wq[n][k] * sw[n]))
//
// computed transposed, D[k][m] += W'^T[k][n] * dY[m][n], with the weight as
// the MMA's A operand (MN-major: a row of the staged tile holds consecutive k
// of one n), so the codes are read in their natural row-major layout.  A tile
// is 256 columns k (128 in each CTA of the pair) x up to 256 tokens; as in the
// forward, the MMA's N follows the tokens of a ragged tile.
//
// The conversion of the weights is the other half of the work, and of a tile
// of few tokens nearly all of it: 64 x 128 codes per CTA for 4 MMAs.  Its warps
// do nothing else (when they also loaded the codes through registers and wrote
// the outputs, a stage of few tokens took 700 to 900 cycles):
//
//   warp 0       copies dY's token halves (TMA, bytes on the even CTA's barrier)
//   warp 1       issues the MMAs (one thread of the even CTA)
//   warp 2       copies the codes (TMA) into a ring of kRaw stages of 8 KiB
//   warps 4-19   converters: warp w takes the stages i with i % 4 == (w - 4) / 4,
//                a quarter of the stage's 64 x 128 codes, from shared memory
//                into the swizzled bf16 tile
//   warps 20-23  epilogue of the TMEM lane quarter w % 4, under the next tile's
//                stages (two accumulators)
//
// A stage takes 530 to 590 cycles with up to 128 tokens and 670 with 160 to 256
// (74 tiles, by the contraction's length), where its MMAs take 156 at 32 and 512
// at 256: 4096 x 11008 x 4096 takes 238 us (tensor pipe 86% active), 1500 rows
// over 64 experts of 1024 x 2048 47 us (137 MB, 22 us at the copy rate).  Cycle
// counters in a large product (752 a stage): of a converter warp's 2450 a turn
// (one stage in four) loading and converting takes 800, storing and the proxy
// fence 550, waiting for the slot 600.  The shared memory's traffic (codes and
// bf16 tile in and out, dY in and out: 80 KiB a stage of 256 tokens) is 640 cycles
// at 128 bytes each.  Without the arithmetic 706 of 752 remain.  Tried and slower: the
// weights through tensor memory (no shared-memory operand, but 500 to 600 cycles
// a stage of 128 to 192 tokens), tiles of 512 tokens with codes loaded through
// registers, polling by one lane of a warp (+20%).  One barrier a stage for both
// operands saves the issuing thread a wait (1500 rows: 3 us of 52).
//
// Conversion: a code, offset by 128, is placed in the mantissa of 2^23 by a
// byte permute; one subtraction gives the exact value, one multiplication
// RN32(code * scale), one packing conversion two bf16 (convert4).
//
// The copied codes are swizzled too (16-byte piece ^ row % 8).  A lane's row in
// a group of 8 is chosen so that the two rows of each 8 lanes differ in bit 2
// (the load of 4 neighbouring pieces) and in bit 0 (the store of every second
// piece): neither has bank conflicts.
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

__device__ int g_int8_dx_error = 0;  // sticky: QLORA_ERR_TIMEOUT if a wait gave up

namespace {

using namespace sm100;

constexpr int kRowsCta = kTileRows / 2;   // columns k per CTA
constexpr int kTileTok = 256;             // largest MMA N
constexpr int kBK = 64;                   // contraction (n) per stage
constexpr int kStages = 4;
constexpr int kPanelBytes = kBK * 128;    // 64 n x 64 k bf16
constexpr int kABytes = 2 * kPanelBytes;  // 16 KiB
constexpr int kBBytes = kTileTok / 2 * kBK * 2;  // 16 KiB: half of the tokens
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kRaw = 10;
constexpr int kRawBytes = kBK * kRowsCta;  // 8 KiB of codes
constexpr int kConvWarp0 = 4, kConvWarps = 16, kEpiWarp0 = kConvWarp0 + kConvWarps;
constexpr int kParts = kConvWarps / 4;
static_assert(kParts == kStages, "a part's stages must always use the same ring slot");
// A part waits for the codes of stage i + kParts once it has stored stage i, that
// is when the MMAs of stage i - kStages are done.  By then the use of the slot
// before, stage i + kParts - kRaw, must be over: else its predecessor's parity
// would be taken for the one waited for.
static_assert(kRaw >= kStages + kParts, "the codes' ring");
constexpr int kThreads = 32 * (kEpiWarp0 + 4);
constexpr uint32_t kTmemCols = 512;
constexpr int kRawOff = kStages * kStageBytes;
constexpr int kBarOff = kRawOff + kRaw * kRawBytes;
constexpr int kTableOff = kBarOff + 512;
constexpr int kSmemBytes = 1024 /* alignment slack */ + kTableOff + kRowTableBytes + kItemListBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;

struct Params {
    const float* scale;  // E x N
    Schedule q;          // column tiles: ceil(K / 256); stages: ceil(N / 64)
    int N, K;
    int boxes;           // token maps made
    uint16_t* dX;
};

struct Maps {
    CUtensorMap w;          // codes: boxes of 64 n x 128 k
    CUtensorMap y[kBoxes];  // dY rows: boxes of box_rows(i) x 64 columns
};

struct Pipe {
    uint32_t smem, bar0, tmem, rank;
    int pair, num_pairs;
    Item* list;
    __device__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ uint32_t empty(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ uint32_t raw_full(int s) const { return bar0 + 8u * (2 * kStages + s); }
    __device__ uint32_t raw_empty(int s) const { return bar0 + 8u * (2 * kStages + kRaw + s); }
    __device__ uint32_t acc_full(int b) const { return bar0 + 8u * (2 * kStages + 2 * kRaw + b); }
    __device__ uint32_t acc_empty(int b) const { return bar0 + 8u * (2 * kStages + 2 * kRaw + 2 + b); }
    __device__ uint32_t drain() const { return bar0 + 8u * (2 * kStages + 2 * kRaw + 4); }
    __device__ uint32_t sA(int s) const { return smem + static_cast<uint32_t>(s * kStageBytes); }
    __device__ uint32_t sRaw(int s) const { return smem + static_cast<uint32_t>(kRawOff + s * kRawBytes); }
};
constexpr int kBars = 2 * kStages + 2 * kRaw + 5;
static_assert(8 * kBars + 8 <= kTableOff - kBarOff, "barriers and the TMEM address");

// A position in a ring of kSlots, with the parity of its turn.
template <int kSlots>
struct Ring {
    int slot;
    uint32_t turn;
    __device__ void step(int n) {
        slot += n;
        if (slot >= kSlots) {
            slot -= kSlots;
            turn ^= 1u;
        }
    }
};

__device__ void role_tokens(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, const Maps& maps) {
    Ring<kStages> ring{0, 1};
    for (int i = 0, it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const Tile& tl = x.tl;
        const int half = mma_tokens(tl.toks) / 2, box = box_index(half);
        const int row = tl.tok0 + static_cast<int>(P.rank) * half;
        const uint32_t tx = 2u * static_cast<uint32_t>(box_rows(box) * kBK * 2);
        for (int kb = x.kb0; kb < x.kb0 + x.stages; ++kb, ring.step(1)) {
            if (!mbar_wait(P.empty(ring.slot), ring.turn, &g_int8_dx_error)) return;
            if (P.rank == 0) mbar_arrive_expect_tx(P.full(ring.slot), tx);
            tma_load_2d_pair(P.sA(ring.slot) + kABytes, &maps.y[box], cluster_map(P.full(ring.slot), 0), kb * kBK, row);
        }
    }
}

__device__ void role_codes(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, const Maps& maps) {
    Ring<kRaw> ring{0, 1};
    for (int i = 0, it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const int col = x.tl.row0 + static_cast<int>(P.rank) * kRowsCta, n0 = x.tl.expert * p.N;
        for (int kb = x.kb0; kb < x.kb0 + x.stages; ++kb, ring.step(1)) {
            if (!mbar_wait(P.raw_empty(ring.slot), ring.turn, &g_int8_dx_error)) return;
            mbar_arrive_expect_tx(P.raw_full(ring.slot), kRawBytes);
            tma_load_2d(P.sRaw(ring.slot), &maps.w, P.raw_full(ring.slot), col, n0 + kb * kBK);
        }
    }
}

// Every lane waits; the warp proceeds (or gives up) together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_int8_dx_error));
}

// The pair's i-th item uses accumulator i & 1 (columns (i & 1) * 256).
__device__ void role_mma(const Pipe& P, const Params& p, const RowTable& tb, const Items& items) {
    const uint64_t a0 = sdesc_mnmajor_sw128(P.sA(0), kPanelBytes), b0 = sdesc_kmajor_sw128(P.sA(0) + kABytes);
    Ring<kStages> ring{0, 0};
    int i = 0;
    for (int it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const uint32_t idesc = idesc_bf16(kTileRows, mma_tokens(x.tl.toks), 1, 0);
        const int b = i & 1;
        if (!mbar_wait(P.acc_empty(b), (static_cast<uint32_t>(i >> 1) & 1u) ^ 1u, &g_int8_dx_error)) return;
        tc_fence_after();
        for (int kb = 0; kb < x.stages; ++kb, ring.step(1)) {
            if (!mbar_wait(P.full(ring.slot), ring.turn, &g_int8_dx_error)) return;
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(ring.slot) * (kStageBytes / 16);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)  // A: 16 rows of 128 bytes; B: 32 bytes along a row
                mma_bf16_ss_pair(P.tmem + b * kTileTok, a0 + off + kk * (2048 / 16), b0 + off + kk * 2, idesc,
                                 (kb > 0 || kk > 0) ? 1u : 0u);
            tc_commit_pair_mc(P.empty(ring.slot), kPairMask);
        }
        tc_commit_pair_mc(P.acc_full(b), kPairMask);
    }
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ void role_convert(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, int cwarp, int lane) {
    const int quarter = cwarp & 3, part = cwarp >> 2;
    const int panel = quarter >> 1;                 // which 64 of this CTA's 128 columns
    const int c = lane & 3;                         // 16-code piece of the 64
    const int q = lane >> 3;
    const int r = (lane & 4) ? q ^ 5 : q;           // row within 8
    const int row0 = (quarter & 1) * 32 + r;        // + 8 j: this lane's rows of the stage
    const uint32_t full0 = cluster_map(P.full(part), 0);
    const uint32_t src0 = static_cast<uint32_t>(row0 * 128 + (((panel * 4 + c) ^ r) << 4));
    const uint32_t dst = P.sA(part) + static_cast<uint32_t>(panel * kPanelBytes + row0 * 128);
    const uint32_t dst0 = dst + (((2 * c) ^ r) << 4), dst1 = dst + (((2 * c + 1) ^ r) << 4);
    Ring<kRaw> raw{part, 0};
    uint32_t turn = 1;
    int kb = part;  // this part's next stage, counted from the item's first
    for (int i = 0, it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const float* scale = p.scale + static_cast<int64_t>(x.tl.expert) * p.N;
        // rows past N hold other codes or zeros: scale 0 makes them 0
        int n = (x.kb0 + kb) * kBK + (quarter & 1) * 32 + lane;
        float next = n < p.N ? __ldg(scale + n) : 0.0f;
        for (; kb < x.stages; kb += kParts) {
            const float mine = next;
            n += kParts * kBK;  // the scales of this part's next stage, on their way meanwhile
            next = n < p.N ? __ldg(scale + n) : 0.0f;
            if (!warp_wait(P.raw_full(raw.slot), raw.turn)) return;
            const uint32_t src = P.sRaw(raw.slot) + src0;
            uint4 cb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) cb[j] = lds_v4(src + j * 1024);
            uint32_t v[32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float sc = __shfl_sync(0xffffffffu, mine, 8 * j + r);
                const uint64_t ms = (static_cast<uint64_t>(__float_as_uint(sc)) << 32) | __float_as_uint(sc);
                const uint32_t w4[4] = {cb[j].x, cb[j].y, cb[j].z, cb[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) convert4(w4[i], ms, v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
            }
            __syncwarp();  // every lane has its codes
            if (lane == 0) mbar_arrive(P.raw_empty(raw.slot));
            raw.step(kParts);
            if (!warp_wait(P.empty(part), turn)) return;
            turn ^= 1u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + j * 1024), "r"(v[8 * j]),
                             "r"(v[8 * j + 1]), "r"(v[8 * j + 2]), "r"(v[8 * j + 3])
                             : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst1 + j * 1024), "r"(v[8 * j + 4]),
                             "r"(v[8 * j + 5]), "r"(v[8 * j + 6]), "r"(v[8 * j + 7])
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(full0);
        }
        kb -= x.stages;
    }
}

// This thread's 32 sums (tokens tok .. of column `col`) to dX.
__device__ __forceinline__ void store_sums(const Params& p, const uint32_t (&sums)[32], const Tile& tl, int tok,
                                           int col, int lane) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(sums[j]);
    store_bf16_chunk(p.dX + static_cast<int64_t>(tl.tok0 + tok) * p.K, p.K, col, tl.toks - tok, v, lane);
}

__device__ void role_epilogue(const Pipe& P, const Params& p, const RowTable& tb, const Items& items, int quarter, int lane) {
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    int i = 0;
    for (int it = P.pair; it < items.count; it += P.num_pairs, ++i) {
        const Item x = listed_item(p.q, tb, items, P.list, i, it);
        const int b = i & 1, row = quarter * 32 + lane;
        if (!warp_wait(P.acc_full(b), static_cast<uint32_t>(i >> 1) & 1u)) return;
        tc_fence_after();
#pragma unroll 1
        for (int tok = 0; tok < x.tl.toks; tok += 32) {
            uint32_t acc[32];
            tmem_ld_32x32b_x32(P.tmem + lane_base + static_cast<uint32_t>(b * kTileTok + tok), acc);
            tmem_wait_ld();
            if (x.slot < 0)
                store_sums(p, acc, x.tl, tok, x.tl.row0 + static_cast<int>(P.rank) * kRowsCta + row, lane);
            else
                slot_store(p.q, x.slot, P.rank, tok / 32, row, acc);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_map(P.acc_empty(b), 0));
    }
}

__global__ void __launch_bounds__(kThreads, 1)
k_int8_dx_pair(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
    const RowTable tb = row_table(smem + kTableOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    Pipe P;
    P.smem = smem_u32(smem);
    P.bar0 = smem_u32(bars);
    P.rank = cluster_ctarank();
    P.pair = static_cast<int>(blockIdx.x >> 1);
    P.num_pairs = static_cast<int>(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(P.full(s), 1 + 2 * 4);  // the even CTA's expect_tx (+ both CTAs' bytes), the part's warps in each CTA
            mbar_init(P.empty(s), 1);         // the pair MMA's commit
        }
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(P.raw_full(s), 1);    // this CTA's expect_tx arrival (+ its bytes)
            mbar_init(P.raw_empty(s), 4);   // the part's four warps
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(P.acc_full(b), 1);
            mbar_init(P.acc_empty(b), 2 * 4);
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
        for (int i = 0; i < p.boxes; ++i) tma_prefetch_desc(&maps.y[i]);
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
    grid_dependency_wait();  // dY's padded rows
    if (warp == 0) {
        if (elect_one()) role_tokens(P, p, tb, items, maps);
    } else if (warp == 1) {
        if (P.rank == 0 && elect_one()) {
            role_mma(P, p, tb, items);
            // every pair MMA issued (also on an early exit) has completed
            // before the tensor memory can be freed
            tc_commit_pair_mc(P.drain(), 1);
            mbar_wait(P.drain(), 0u, &g_int8_dx_error);
        }
    } else if (warp == 2) {
        if (elect_one()) role_codes(P, p, tb, items, maps);
    } else if (warp >= kEpiWarp0) {
        role_epilogue(P, p, tb, items, warp & 3, lane);
    } else if (warp >= kConvWarp0) {
        role_convert(P, p, tb, items, warp - kConvWarp0, lane);
    }
    __syncwarp();
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

__global__ void __launch_bounds__(kAddThreads) k_int8_dx_add(const __grid_constant__ Params p) {
    Tile tl;
    uint32_t sums[32];
    if (add_parts<false>(p.q, &tl, sums))
        store_sums(p, sums, tl, static_cast<int>(blockIdx.y) * 32,
                   tl.row0 + static_cast<int>(blockIdx.z) * kRowsCta + static_cast<int>(threadIdx.x), threadIdx.x & 31);
}

// Rows of dY whose length is not a multiple of 8 (a copy's row stride is a
// multiple of 16 bytes), into rows of `ld` elements.
__global__ void __launch_bounds__(256) k_pad_rows(const uint16_t* __restrict__ src, int64_t rows, int n, int ld,
                                                  uint16_t* __restrict__ dst) {
    grid_launch_dependents();
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x)
        for (int i = threadIdx.x; i < n; i += 256) dst[m * ld + i] = src[m * n + i];
}

// ------------------------------------------------------------------ host
// A row-major matrix of `rows` rows, `stride` bytes apart, of `inner`
// elements; 128-byte swizzled boxes of box_inner x box_rows, zero fill outside.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t inner, int64_t rows, int64_t stride,
              uint32_t box_inner, uint32_t box_outer) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

int max_pairs() {
    static ContextMemo<int> memo;
    uint64_t ctx = 0;
    if (!current_context_id(&ctx)) return 0;
    int n = 0;
    memo.get(ctx, &n, [](int* v) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = pair_config(attr, num_sms(), nullptr, false);
        int c = 0;
        if (cudaOccupancyMaxActiveClusters(&c, k_int8_dx_pair, &cfg) != cudaSuccess) {
            cudaGetLastError();
            c = 0;
        }
        *v = c;
        return true;
    });
    return n;
}

// In a captured graph 256 x 5120 x 5120 takes 34.5 us in whole tiles and 23.6 in
// three parts, 500 x 10000 x 128 54 and 25, 16 x 5120 x 5120 26 and 18.
Schedule schedule(const RowRanges& rr, const Int8Weight& w) {
    return schedule_of(rr, w.E, w.K, ceil_div(w.N, kBK), kTileTok, 32, sm_pairs());
}

// Workspace: dY's rows padded to 16 bytes, where N is not a multiple of 8, then
// the parts' slots.
size_t padded_bytes(int64_t T, const Int8Weight& w) {
    return w.N % 8 == 0 ? 0 : static_cast<size_t>(round_up(T * round_up(w.N, 8) * 2, 256));
}
size_t parts_bytes(int64_t T, const Int8Weight& w) {
    return slots_bytes(schedule(RowRanges{nullptr, T}, w));
}

}  // namespace

bool int8_dx_supported(int64_t T, const Int8Weight& w) {
    return int8_tiles(T, w.E, w.K, kTileTok) * ceil_div(w.N, kBK) < (int64_t(1) << 31);
}

size_t int8_dx_workspace(int64_t T, const Int8Weight& w) { return padded_bytes(T, w) + parts_bytes(T, w); }

cudaError_t launch_int8_dx(const uint16_t* dY, const Int8Weight& w, const RowRanges& rr, uint16_t* dX, void* ws,
                           cudaStream_t st) {
    static ContextMemo<int> attr_memo;
    cudaError_t e = ensure_smem_limit(attr_memo, k_int8_dx_pair, kSmemBytes);
    if (e != cudaSuccess) return e;
    if (max_pairs() < 1) return cudaErrorNotSupported;
    const int64_t ldy = round_up(w.N, 8);
    if (ldy != w.N) {
        const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
        k_pad_rows<<<static_cast<unsigned>(rr.T < cap ? rr.T : cap), 256, 0, st>>>(
            dY, rr.T, static_cast<int>(w.N), static_cast<int>(ldy), static_cast<uint16_t*>(ws));
        note_launches(1);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        dY = static_cast<const uint16_t*>(ws);
    }
    Params p{};
    p.scale = w.scale;
    p.q = schedule(rr, w);
    if (parts_bytes(rr.T, w) > 0) p.q.slots = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + padded_bytes(rr.T, w));
    p.N = static_cast<int>(w.N);
    p.K = static_cast<int>(w.K);
    p.boxes = boxes_of(p.q);
    p.dX = dX;
    Maps maps;
    bool ok = make_map(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K, w.E * w.N, w.ld, kRowsCta, kBK);
    for (int i = 0; i < p.boxes; ++i)
        ok = ok && make_map(&maps.y[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dY, w.N, rr.T, ldy * 2, kBK,
                            static_cast<uint32_t>(box_rows(i)));
    if (!ok) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config(attr, p.q.pairs, st, ldy != w.N);
    e = cudaLaunchKernelEx(&cfg, k_int8_dx_pair, maps, p);
    note_launches(1);
    if (e != cudaSuccess || !p.q.slots) return e;
    cudaLaunchAttribute dep[1];
    const cudaLaunchConfig_t add = add_config(dep, p.q, st);
    e = cudaLaunchKernelEx(&add, k_int8_dx_add, p);
    note_launches(1);
    return e;
}

int int8_dx_device_error(int reset) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_int8_dx_error, sizeof(int)) != cudaSuccess) return QLORA_ERR_CUDA;
    if (reset && v) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_int8_dx_error, &zero, sizeof(int)) != cudaSuccess) return QLORA_ERR_CUDA;
    }
    return v;
}

}  // namespace qlora

// int8_dx_sm100.cu -- the Int8 linear's input gradient on the tensor cores, on
// pairs of SMs, dense or grouped by expert:
//
//   dX[m][k] = sum_n dY[m][n] * W'[n][k],   W' = bf16(RN32(wq[n][k] * sw[n]))
//
// computed transposed, D[k][m] += W'^T[k][n] * dY[m][n], with the weight as
// the MMA's A operand (MN-major: a row of the staged tile holds consecutive k
// of one n), so the codes are read in their natural row-major layout.  A tile
// is 256 columns k (128 in each CTA of the pair) x up to 512 tokens, held as
// one or two accumulators of 256: a converted weight tile then feeds 512
// tokens, which keeps the shared-memory traffic (16 KiB converted, 32 KiB of
// dY copied, 64 KiB read by the MMAs per 1024 MMA cycles) under its 128 bytes
// a cycle.  As in the forward, the MMA's N follows the tokens of a ragged
// tile, and a tile of up to 256 tokens uses one accumulator and leaves the
// other to the next tile.
//
// Warp roles (576 threads per CTA, persistent over the pair's tiles):
//   warp 0      TMA producer of dY (both CTAs, into their own shared memory;
//               the bytes count on the even CTA's barrier)
//   warp 1      MMA issuer (one thread of the even CTA)
//   warps 2-17  converters: warp w takes the stages i with i % 4 ==
//               (w - 2) / 4 (always ring slot i % 4), a quarter of the stage's
//               64 x 128 codes; then the epilogue of its TMEM lane quarter
// A warp's load instruction covers 64 consecutive codes of 8 rows; a lane
// turns 16 codes of a row into two 16-byte pieces of the swizzled tile
// without bank conflicts.  Conversion: a code, offset by 128, is placed in the
// mantissa of 2^23 by a byte permute; one subtraction gives the exact value,
// one multiplication RN32(code * scale), one packing conversion two bf16.
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

constexpr int kRowsCta = kTileRows / 2;             // columns k per CTA
constexpr int kSubTok = 256;                        // largest MMA N: tokens of an accumulator
constexpr int kSubs = 2;
constexpr int kTileTok = kSubs * kSubTok;
constexpr int kBK = 64;                             // contraction (n) per stage
constexpr int kStages = 4;
constexpr int kPanelBytes = kBK * 128;              // 64 n x 64 k bf16
constexpr int kABytes = 2 * kPanelBytes;            // 16 KiB
constexpr int kBHalfBytes = kSubTok / 2 * kBK * 2;  // 16 KiB: half of an accumulator's tokens
constexpr int kStageBytes = kABytes + kSubs * kBHalfBytes;
constexpr int kConvWarps = 16;
constexpr int kParts = kConvWarps / 4;
static_assert(kParts == kStages, "a part's stages must always use the same ring slot");
constexpr int kThreads = 32 * (2 + kConvWarps);
constexpr uint32_t kTmemCols = 512;
constexpr int kBarOff = kStages * kStageBytes;
constexpr int kTableOff = kBarOff + 256;
constexpr int kSmemBytes = 1024 /* alignment slack */ + kTableOff + kRowTableBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
constexpr uint16_t kPairMask = 0x3;

struct Params {
    Int8Weight w;
    RowRanges rr;
    int num_w;      // column tiles: ceil(K / 256)
    int kbt;        // stages of a tile: ceil(N / 64)
    uint16_t* dX;
};

struct Maps {
    CUtensorMap y[kBoxes];  // dY rows: boxes of box_rows(i) x 64 columns
};

struct Pipe {
    uint32_t smem, bar0, tmem, rank;
    int pair, num_pairs;
    __device__ uint32_t full_b(int s) const { return bar0 + 8u * s; }
    __device__ uint32_t full_a(int s) const { return bar0 + 8u * (kStages + s); }
    __device__ uint32_t empty(int s) const { return bar0 + 8u * (2 * kStages + s); }
    __device__ uint32_t acc_full(int b) const { return bar0 + 8u * (3 * kStages + b); }
    __device__ uint32_t acc_empty(int b) const { return bar0 + 8u * (3 * kStages + 2 + b); }
    __device__ uint32_t drain() const { return bar0 + 8u * (3 * kStages + 4); }
    __device__ uint32_t sA(int s) const { return smem + static_cast<uint32_t>(s * kStageBytes); }
    __device__ uint32_t sB(int s, int sub) const { return sA(s) + kABytes + sub * kBHalfBytes; }
};

// Tokens of accumulator `sub` of a tile.
__device__ __forceinline__ int sub_tokens(const Tile& tl, int sub) {
    return min(max(tl.toks - sub * kSubTok, 0), kSubTok);
}

__device__ void role_tma(const Pipe& P, const Params& p, const RowTable& tb, int units, const Maps& maps) {
    int local = 0;
    for (int u = P.pair; u < units; u += P.num_pairs) {
        const Tile tl = tile_of(tb, p.w.E, p.num_w, kTileTok, u);
        int box[kSubs], row[kSubs];
        uint32_t tx = 0;
        int subs = 0;
        for (int sub = 0; sub < kSubs; ++sub) {
            const int n = sub_tokens(tl, sub);
            if (n == 0) break;
            const int half = mma_tokens(n) / 2;
            box[sub] = box_index(half);
            row[sub] = tl.tok0 + sub * kSubTok + static_cast<int>(P.rank) * half;
            tx += 2u * static_cast<uint32_t>(box_rows(box[sub]) * kBK * 2);
            ++subs;
        }
        for (int kb = 0; kb < p.kbt; ++kb, ++local) {
            const int s = local % kStages;
            const uint32_t ph = static_cast<uint32_t>(local / kStages) & 1u;
            if (!mbar_wait(P.empty(s), ph ^ 1u, &g_int8_dx_error)) return;
            const uint32_t bar = cluster_map(P.full_b(s), 0);
            if (P.rank == 0) mbar_arrive_expect_tx(P.full_b(s), tx);
            for (int sub = 0; sub < subs; ++sub)
                tma_load_2d_pair(P.sB(s, sub), &maps.y[box[sub]], bar, kb * kBK, row[sub]);
        }
    }
}

// Every lane waits; the warp proceeds (or gives up) together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_int8_dx_error));
}

// Accumulators are taken in turn: the g-th one used is columns (g & 1) * 256,
// for the (g >> 1)-th time.
__device__ void role_mma(const Pipe& P, const Params& p, const RowTable& tb, int units) {
    const uint64_t a0 = sdesc_mnmajor_sw128(P.sA(0), kPanelBytes), b0 = sdesc_kmajor_sw128(P.sB(0, 0));
    int s = 0, g = 0;
    uint32_t ph = 0;
    for (int u = P.pair; u < units; u += P.num_pairs) {
        const Tile tl = tile_of(tb, p.w.E, p.num_w, kTileTok, u);
        const int subs = tl.toks > kSubTok ? 2 : 1;
        const uint32_t idesc0 = idesc_bf16(kTileRows, mma_tokens(sub_tokens(tl, 0)), 1, 0);
        const uint32_t idesc1 = idesc_bf16(kTileRows, mma_tokens(sub_tokens(tl, 1)), 1, 0);
        for (int a = g; a < g + subs; ++a)
            if (!mbar_wait(P.acc_empty(a & 1), (static_cast<uint32_t>(a >> 1) & 1u) ^ 1u, &g_int8_dx_error)) return;
        tc_fence_after();
        const uint32_t d0 = P.tmem + (g & 1) * kSubTok, d1 = P.tmem + ((g + 1) & 1) * kSubTok;
        for (int kb = 0; kb < p.kbt; ++kb) {
            if (!mbar_wait(P.full_b(s), ph, &g_int8_dx_error)) return;
            if (!mbar_wait(P.full_a(s), ph, &g_int8_dx_error)) return;
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(s) * (kStageBytes / 16);
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk) {
                const uint64_t ad = a0 + off + kk * (2048 / 16);  // 16 rows of 128 bytes
                const uint64_t bd = b0 + off + kk * 2;            // 32 bytes along a row
                const uint32_t more = (kb > 0 || kk > 0) ? 1u : 0u;
                mma_bf16_ss_pair(d0, ad, bd, idesc0, more);
                if (subs == 2) mma_bf16_ss_pair(d1, ad, bd + kBHalfBytes / 16, idesc1, more);
            }
            tc_commit_pair_mc(P.empty(s), kPairMask);
            if (++s == kStages) {
                s = 0;
                ph ^= 1u;
            }
        }
        for (int sub = 0; sub < subs; ++sub, ++g) tc_commit_pair_mc(P.acc_full(g & 1), kPairMask);
    }
}

__device__ __forceinline__ uint4 ldg_codes(const int8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Outputs of the tile `tl`, whose accumulators are the g-th and following:
// this warp's TMEM lane quarter, every fourth 32-token chunk.
__device__ __forceinline__ bool tile_epilogue(const Pipe& P, const Params& p, const Tile& tl, int& g, int part,
                                              int quarter, int lane) {
    const int subs = tl.toks > kSubTok ? 2 : 1;
    const int col = tl.row0 + static_cast<int>(P.rank) * kRowsCta + quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int K = static_cast<int>(p.w.K);
    for (int sub = 0; sub < subs; ++sub, ++g) {
        const int b = g & 1;
        const int toks = sub_tokens(tl, sub);
        if (!warp_wait(P.acc_full(b), static_cast<uint32_t>(g >> 1) & 1u)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = part; c * 32 < toks; c += kParts) {
            uint32_t acc[32];
            tmem_ld_32x32b_x32(P.tmem + lane_base + static_cast<uint32_t>(b * kSubTok + c * 32), acc);
            tmem_wait_ld();
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(acc[j]);
            const int tok = sub * kSubTok + c * 32;
            store_bf16_chunk(p.dX + static_cast<int64_t>(tl.tok0 + tok) * K, K, col, tl.toks - tok, v, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(cluster_map(P.acc_empty(b), 0));
    }
    return true;
}

__device__ void role_convert(const Pipe& P, const Params& p, const RowTable& tb, int units, int warp, int lane) {
    const int quarter = warp & 3;
    const int part = (warp - 2) >> 2;
    const int panel = quarter >> 1;                // which 64 of this CTA's 128 columns
    const int r = lane >> 2, c = lane & 3;         // row within 8, 16-code piece of the 64
    const uint32_t full_a0 = cluster_map(P.full_a(part), 0);
    const int tiles = P.pair < units ? (units - P.pair + P.num_pairs - 1) / P.num_pairs : 0;
    const int ld = static_cast<int>(p.w.ld), N = static_cast<int>(p.w.N);
    const uint32_t dst = P.sA(part) + static_cast<uint32_t>(panel * kPanelBytes);

    // the cursor of the code loads: stage l_kb of this pair's tile l_tile
    int l_tile = 0, l_kb = part;
    const int8_t* l_codes = nullptr;  // row 0 of the tile's expert, this lane's first column
    const float* l_scale = nullptr;
    bool l_in = false;                // the column is inside the padded row
    auto open_tile = [&]() {          // moves l_kb into its tile
        while (l_kb >= p.kbt) {
            l_kb -= p.kbt;
            ++l_tile;
        }
        if (l_tile >= tiles) return;
        const Tile tl = tile_of(tb, p.w.E, p.num_w, kTileTok, P.pair + l_tile * P.num_pairs);
        const int k = tl.row0 + static_cast<int>(P.rank) * kRowsCta + panel * 64 + c * 16;
        l_codes = p.w.codes + static_cast<int64_t>(tl.expert) * N * ld + k;
        l_scale = p.w.scale + static_cast<int64_t>(tl.expert) * N;
        l_in = k < ld;
    };
    uint4 cb[4];
    float sc[4];
    const int64_t ld8 = static_cast<int64_t>(8) * ld;
    auto issue = [&]() {  // loads the cursor's stage and moves the cursor to this part's next one
        if (l_tile >= tiles) return;
        const int n0 = l_kb * kBK + (quarter & 1) * 32;  // the quarter's first row
        const int8_t* src = l_codes + static_cast<int64_t>(n0 + r) * ld;
        const float* scale = l_scale + n0 + r;
        if (l_in && n0 + 32 <= N) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                cb[j] = ldg_codes(src + j * ld8);
                sc[j] = __ldg(scale + 8 * j);
            }
            // this part's next stage but one of the same tile, towards L2: the
            // loads above are only one of this part's stages ahead
            if (c == 0 && n0 + 2 * kStages * kBK + 32 <= N) {
                const int8_t* far = src + static_cast<int64_t>(2 * kStages * kBK) * ld;
#pragma unroll
                for (int j = 0; j < 4; ++j) prefetch_l2(far + j * ld8);
            }
        } else {  // rows past N are zero (they are part of the contraction)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool ok = l_in && n0 + r + 8 * j < N;
                cb[j] = ok ? ldg_codes(src + j * ld8) : make_uint4(0u, 0u, 0u, 0u);
                sc[j] = ok ? __ldg(scale + 8 * j) : 0.0f;
            }
        }
        l_kb += kStages;
        if (l_kb >= p.kbt) open_tile();
    };

    int next_epi = 0, g = 0;  // the next tile whose outputs this warp writes
    open_tile();
    issue();
    uint32_t ph = 1;
    int tile = 0, kb = part;  // the stage being converted
    for (;; kb += kStages) {
        for (; kb >= p.kbt; kb -= p.kbt) ++tile;
        if (tile >= tiles) break;
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w4[4] = {cb[j].x, cb[j].y, cb[j].z, cb[j].w};
            const uint64_t ms = (static_cast<uint64_t>(__float_as_uint(sc[j])) << 32) | __float_as_uint(sc[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) convert4(w4[i], ms, v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
        }
        if (!warp_wait(P.empty(part), ph)) return;
        ph ^= 1u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = (quarter & 1) * 32 + 8 * j + r;  // row & 7 == r
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 dst + static_cast<uint32_t>(row * 128 + (((2 * c + h) ^ r) << 4))),
                             "r"(v[8 * j + 4 * h]), "r"(v[8 * j + 4 * h + 1]), "r"(v[8 * j + 4 * h + 2]),
                             "r"(v[8 * j + 4 * h + 3])
                             : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(full_a0);
        // the tiles before this stage's are complete or about to be: write
        // them now, with the next tile's first stages already converted
        while (next_epi < tile) {
            const Tile tl = tile_of(tb, p.w.E, p.num_w, kTileTok, P.pair + next_epi * P.num_pairs);
            if (!tile_epilogue(P, p, tl, g, part, quarter, lane)) return;
            ++next_epi;
        }
        issue();
    }
    while (next_epi < tiles) {
        const Tile tl = tile_of(tb, p.w.E, p.num_w, kTileTok, P.pair + next_epi * P.num_pairs);
        if (!tile_epilogue(P, p, tl, g, part, quarter, lane)) return;
        ++next_epi;
    }
}

__global__ void __launch_bounds__(kThreads, 1)
k_int8_dx_pair(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kStages + 5);
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
            mbar_init(P.full_b(s), 1);      // the even CTA's expect_tx arrival (+ both CTAs' bytes)
            mbar_init(P.full_a(s), 2 * 4);  // the part's four warps in each CTA
            mbar_init(P.empty(s), 1);       // the pair MMA's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(P.acc_full(b), 1);
            mbar_init(P.acc_empty(b), 2 * kConvWarps);
        }
        mbar_init(P.drain(), 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    if (warp == 1 && lane == 0)
        for (int i = 0; i < kBoxes; ++i) tma_prefetch_desc(&maps.y[i]);
    if (warp == 2) build_table(p.rr, p.w.E, p.num_w, kTileTok, tb, lane);
    tc_fence_before();
    __syncthreads();
    cluster_arrive();  // both CTAs' barriers are initialised before any remote arrive
    cluster_wait();
    tc_fence_after();
    P.tmem = *tmem_slot;
    const int units = tb.tile0[p.w.E];
    if (warp == 0) {
        if (elect_one()) role_tma(P, p, tb, units, maps);
        __syncwarp();
    } else if (warp == 1) {
        if (P.rank == 0 && elect_one()) {
            role_mma(P, p, tb, units);
            // every pair MMA issued (also on an early exit) has completed
            // before the tensor memory can be freed
            tc_commit_pair_mc(P.drain(), 1);
            mbar_wait(P.drain(), 0u, &g_int8_dx_error);
        }
        __syncwarp();
    } else {
        role_convert(P, p, tb, units, warp, lane);
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

// Rows of dY whose length is not a multiple of 8 (a copy's row stride is a
// multiple of 16 bytes), into rows of `ld` elements.
__global__ void __launch_bounds__(256) k_pad_rows(const uint16_t* __restrict__ src, int64_t rows, int n, int ld,
                                                  uint16_t* __restrict__ dst) {
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x)
        for (int i = threadIdx.x; i < n; i += 256) dst[m * ld + i] = src[m * n + i];
}

// ------------------------------------------------------------------ host
bool make_map_dy(CUtensorMap* m, const void* base, int64_t N, int64_t rows, int64_t ld, uint32_t box) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t boxes[2] = {kBK, box};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute (&attr)[1], int pairs, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

int max_pairs() {
    static ContextMemo<int> memo;
    uint64_t ctx = 0;
    if (!current_context_id(&ctx)) return 0;
    int n = 0;
    memo.get(ctx, &n, [](int* v) {
        cudaLaunchAttribute attr[1];
        const cudaLaunchConfig_t cfg = pair_config(attr, num_sms(), nullptr);
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

// The most tokens of a tile: kTileTok (this kernel) or kSubTok (the narrow
// one).  Dense: the fewer cycles, by the measured cost of 64 n of a tile (this
// kernel 2.1 a token, 800 at least; the narrow one 2.8, 475 at least) times
// the rounds of tiles.  512 x 5120 x 5120 takes 61 us here and 41 there, 4096 x
// 11008 x 4096 246 and 266.  Experts: ragged rows fill wide tiles badly and
// level out better in small ones (eight experts of 11008 x 4096 with 57 to 1540
// of 4096 rows: 334 and 309 us), so wide tiles are left to experts of 1024 rows
// and more on average.
int tile_cap(int64_t T, const Int8Weight& w) {
    if (w.E > 1) return T < 1024 * static_cast<int64_t>(w.E) ? kSubTok : kTileTok;
    const int64_t pairs = num_sms() / 2 > 0 ? num_sms() / 2 : 1;
    const int m = static_cast<int>(T);
    auto rounds = [&](int cap) { return ceil_div(token_tiles(m, cap) * ceil_div(w.K, kTileRows), pairs); };
    auto cost = [&](int cap, int tenths, int least) {
        const int c = token_width(m, cap) * tenths / 10;
        return c > least ? c : least;
    };
    const int64_t narrow = rounds(kSubTok) * cost(kSubTok, 28, 475) / int8_dx_narrow_parts(T, w);
    return narrow <= rounds(kTileTok) * cost(kTileTok, 21, 800) ? kSubTok : kTileTok;
}

}  // namespace

bool int8_dx_supported(int64_t T, const Int8Weight& w) {
    return int8_tiles(T, w.E, w.K, kSubTok) * ceil_div(w.N, kBK) < (int64_t(1) << 31);
}

// Workspace: dY's rows padded to 16 bytes, where N is not a multiple of 8, then
// the narrow kernel's.
size_t dx_padded_bytes(int64_t T, const Int8Weight& w) {
    return w.N % 8 == 0 ? 0 : static_cast<size_t>(round_up(T * round_up(w.N, 8) * 2, 256));
}

size_t int8_dx_workspace(int64_t T, const Int8Weight& w) {
    return dx_padded_bytes(T, w) + (tile_cap(T, w) == kSubTok ? int8_dx_narrow_workspace(T, w) : 0);
}

cudaError_t launch_int8_dx(const uint16_t* dY, const Int8Weight& w, const RowRanges& rr, uint16_t* dX, void* ws,
                           cudaStream_t st) {
    cudaError_t e;
    const int64_t ld = round_up(w.N, 8);
    if (ld != w.N) {
        const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
        k_pad_rows<<<static_cast<unsigned>(rr.T < cap ? rr.T : cap), 256, 0, st>>>(
            dY, rr.T, static_cast<int>(w.N), static_cast<int>(ld), static_cast<uint16_t*>(ws));
        note_launches(1);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        dY = static_cast<const uint16_t*>(ws);
    }
    if (tile_cap(rr.T, w) == kSubTok)
        return launch_int8_dx_narrow(dY, ld, w, rr, dX, static_cast<char*>(ws) + dx_padded_bytes(rr.T, w), st);
    static ContextMemo<int> attr_memo;
    e = ensure_smem_limit(attr_memo, k_int8_dx_pair, kSmemBytes);
    if (e != cudaSuccess) return e;
    const int most = max_pairs();
    if (most <= 0) return cudaErrorNotSupported;
    Params p{};
    p.w = w;
    p.rr = rr;
    p.num_w = static_cast<int>(ceil_div(w.K, kTileRows));
    p.kbt = static_cast<int>(ceil_div(w.N, kBK));
    p.dX = dX;
    Maps maps;
    bool ok = true;
    for (int i = 0; i < kBoxes; ++i) ok = ok && make_map_dy(&maps.y[i], dY, w.N, rr.T, ld, box_rows(i));
    if (!ok) return cudaErrorInvalidValue;
    const int64_t tiles = int8_tiles(rr.T, w.E, w.K, kTileTok);
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pair_config(attr, static_cast<int>(tiles < most ? tiles : most), st);
    e = cudaLaunchKernelEx(&cfg, k_int8_dx_pair, maps, p);
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

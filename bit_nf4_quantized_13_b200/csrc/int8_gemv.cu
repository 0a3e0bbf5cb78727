// int8_gemv.cu -- the Int8 linear's forward for a few tokens, dense or grouped
// by expert: one pass over the weights that have tokens,
//
//   Y[m][n] = (sum_k xq[m][k] wq[n][k]) * sx[m] * sw[n]
//
// HBM-bound on the weight stream, so everything serves the loads: no shared
// memory in their way, no tensor maps or cluster launch, one launch (the
// tokens are quantized in the kernel while its first weights are on the way)
// where the tokens are few enough for every block to do so.
//
// A block of 8 warps takes 16 output channels at a time; its warps share out
// the contraction in units of 256 codes a channel.  Lane 4 g + t holds 16
// consecutive codes of channels g and g + 8, which are the A fragments of two
// mma.m16n8k32 (the contraction index is permuted the same way in both
// operands, so no code moves between lanes); a warp reads 64 bytes of each of
// 16 rows per two instructions and keeps eight such loads in flight, across
// steps too (sixteen were no faster).  Integer sums are exact, so the warps' partial
// sums may be added in any order: through shared memory, once a step.  Two
// blocks an SM (up to 128 registers, no spills) stream as fast as three or four and
// leave room for the token fragments; giving each warp whole steps, to have
// fewer barriers, was slower (16 tokens, six experts of 11008 x 4096: 62
// against 57 us).  8 x 22016 x 8192: 38 us, 181 MB read (4.8 TB/s).
#include <limits.h>

#include "int8_rows.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;               // output channels of a block's step
constexpr int kUnit = 256;              // codes of a row in a warp's unit
constexpr int kHalf = kUnit / 2;
constexpr int kXPad = 64;               // bytes between token rows in shared memory, against bank conflicts
constexpr int kBlocksPerSm = 2;
// Tokens that every block quantizes itself: their bf16 values and their codes
// stay in shared memory.  One kernel then does what two would, which saves 3
// us on the host; its blocks repeat the work, which is why it ends here (5120
// values: 1 us of the kernel).
constexpr int kMaxFusedValues = 10240;
constexpr int kMaxFused = 4;
constexpr int kMaxTokens = 16;

struct GemvParams {
    const uint16_t* X;   // fused: T x K bf16
    const int8_t* xc;    // else: T x ld codes
    const float* xs;     //       T scales
    Int8Weight w;
    RowRanges rr;
    int groups;          // ceil(N / kRows)
    void* out;
};

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream(const int8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Four vectors of a half unit: rows g and g + 8, codes 16 t .. and 64 + 16 t ..
struct HalfUnit {
    uint4 v[4];
};

// Eight values of token m from element e on.
__device__ __forceinline__ RowVec<uint16_t> load_token(const GemvParams& p, int m, int e) {
    const uint16_t* row = p.X + static_cast<int64_t>(m) * p.w.K;
    RowVec<uint16_t> v;
    if (p.w.K % 8 == 0)
        v.load<true>(row, e, p.w.K, nullptr);
    else
        v.load<false>(row, e, p.w.K, p.X + p.rr.T * p.w.K);
    return v;
}

// Expert e's two offsets; behind the last expert, ones that start no range.
__device__ __forceinline__ int2 expert_offsets(const GemvParams& p, int e) {
    return e < p.w.E ? make_int2(p.rr.offsets[e], p.rr.offsets[e + 1]) : make_int2(INT_MAX, INT_MAX);
}

// T <= 8 NT tokens.  kDense: one weight, every row; as a variable of the same
// kernel it cost 16 x 4096 x 4096 7.5 us in place of 7.3.
template <int NT, bool kFused, bool kF32, bool kDense>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
k_int8_gemv(const GemvParams p) {
    extern __shared__ __align__(16) int8_t s_x[];  // fused: T rows of ld + kXPad bytes
    __shared__ int s_sum[kWarps][kRows][8 * NT];
    __shared__ int4 s_range[8 * NT];  // (expert, first row, end): disjoint ranges of T rows, at most T that have any
    __shared__ float s_scale[kMaxFused];
    __shared__ uint32_t s_max[kMaxFused][kWarps];
    __shared__ int s_count;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ld = static_cast<int>(p.w.ld);  // T * ld < 2^31: checked by the host
    const int T = static_cast<int>(p.rr.T);

    uint16_t* s_raw = reinterpret_cast<uint16_t*>(s_x + (kFused ? T * (ld + kXPad) : 0));  // fused: T rows of ld values
    if (kFused) {
        // the tokens' values first, before the weights' loads fill the memory system
        for (int m = 0; m < T; ++m) {
            uint32_t a = 0u;
            for (int e = static_cast<int>(threadIdx.x) * 8; e < ld; e += kThreads * 8) {
                const RowVec<uint16_t> v = load_token(p, m, e);
                *reinterpret_cast<uint4*>(s_raw + m * ld + e) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
                a = abs_max(v, a);
            }
            a = __reduce_max_sync(0xffffffffu, a);
            if (lane == 0) s_max[m][warp] = a;
        }
    }

    // the experts that have tokens, in order
    int active = 1;
    if (!kDense) {
        if (warp == 0) {
            int n = 0, top = 0;
            bool ascending = true;  // so far: no offset lies below the one before it
            int2 next = expert_offsets(p, lane);
            for (int e0 = 0; e0 < p.w.E; e0 += 32) {
                const int e = e0 + lane;
                int lo = min(max(next.x, 0), T), hi = min(max(next.y, 0), T);
                next = expert_offsets(p, e + 32);  // on their way meanwhile: 1024 experts 10.8 -> 8.6 us
                if (!ascending || !__all_sync(0xffffffffu, hi >= lo)) {  // each counts as no less than the one before
                    top = ascending ? __shfl_sync(0xffffffffu, lo, 0) : top;
                    ascending = false;
                    hi = max(hi, top);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) hi = max(hi, __shfl_up_sync(0xffffffffu, hi, o));
                    lo = __shfl_up_sync(0xffffffffu, hi, 1);
                    if (lane == 0) lo = top;
                    top = __shfl_sync(0xffffffffu, hi, 31);
                }
                const bool any = e < p.w.E && hi > lo;
                const uint32_t has = __ballot_sync(0xffffffffu, any);
                if (any) {
                    const int i = n + __popc(has & ((1u << lane) - 1u));
                    s_range[i] = make_int4(e, lo, hi, 0);
                }
                n += __popc(has);
            }
            if (lane == 0) s_count = n;
        }
        __syncthreads();
        active = s_count;
    }
    const int steps = active * p.groups;
    const int nunits = (ld + kUnit - 1) / kUnit;

    // the cursor of this warp's weight loads
    int l_step = static_cast<int>(blockIdx.x), l_unit = warp;
    const int8_t* l_row = nullptr;  // channel g of the step, code 16 t
    bool l_ok0 = false, l_ok1 = false;
    auto open_step = [&]() {
        if (l_step >= steps) return;
        const int e = kDense ? 0 : s_range[l_step / p.groups].x;
        const int n = (kDense ? l_step : l_step % p.groups) * kRows + g;
        l_ok0 = n < p.w.N;
        l_ok1 = n + 8 < p.w.N;
        l_row = p.w.codes + (static_cast<int64_t>(e) * p.w.N + n) * ld + 16 * t;
    };
    auto load_half = [&](HalfUnit& h, int half) {
        const int k = l_unit * kUnit + half * kHalf;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool in = l_step < steps && k + 64 * i + 16 * t < ld;
            const int8_t* src = l_row + k + 64 * i;
            h.v[2 * i] = in && l_ok0 ? ld_stream(src) : make_uint4(0u, 0u, 0u, 0u);
            h.v[2 * i + 1] = in && l_ok1 ? ld_stream(src + static_cast<int64_t>(8) * ld) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto advance = [&]() {
        l_unit += kWarps;
        if (l_unit >= nunits) {
            l_unit = warp;
            l_step += static_cast<int>(gridDim.x);
            open_step();
        }
    };
    HalfUnit h0, h1;  // the next unit
    if (warp < nunits) {
        open_step();
        load_half(h0, 0);
        load_half(h1, 1);
        advance();
    }

    if (kFused) {  // quantize them; a thread encodes the values that it staged
        __syncthreads();
        for (int m = 0; m < T; ++m) {
            uint32_t a = 0u;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) a = max(a, s_max[m][i]);
            float sc;
            const float c = row_constant(a, &sc);
            if (threadIdx.x == 0) s_scale[m] = sc;
            for (int e = static_cast<int>(threadIdx.x) * 8; e < ld; e += kThreads * 8) {
                const uint4 w = *reinterpret_cast<const uint4*>(s_raw + m * ld + e);
                RowVec<uint16_t> v;
                v.w[0] = w.x;
                v.w[1] = w.y;
                v.w[2] = w.z;
                v.w[3] = w.w;
                encode(v, c, s_x + m * (ld + kXPad) + e);
            }
        }
        __syncthreads();
    } else {
        sm100::grid_dependency_wait();  // the quantized tokens
    }

    for (int step = static_cast<int>(blockIdx.x); step < steps; step += static_cast<int>(gridDim.x)) {
        int e = 0, lo = 0, hi = T, n0 = step * kRows;  // at most T <= 8 NT rows
        if (!kDense) {
            const int at = step / p.groups;
            const int4 r = s_range[at];
            e = r.x;
            lo = r.y;
            hi = r.z;
            n0 = (step - at * p.groups) * kRows;
        }
        int acc[NT][4] = {};
        auto multiply = [&](const HalfUnit& half, int k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int kk = k + 64 * i + 16 * t;
                const uint4 a = half.v[2 * i], b = half.v[2 * i + 1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int m = lo + 8 * nt + g;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (m < hi && kk < ld)
                        x = *reinterpret_cast<const uint4*>(kFused ? s_x + m * (ld + kXPad) + kk : p.xc + m * ld + kk);
                    mma_s8(acc[nt], a.x, b.x, a.y, b.y, x.x, x.y);
                    mma_s8(acc[nt], a.z, b.z, a.w, b.w, x.z, x.w);
                }
            }
        };
        for (int u = warp; u < nunits; u += kWarps) {
            multiply(h0, u * kUnit);
            load_half(h0, 0);
            multiply(h1, u * kUnit + kHalf);
            load_half(h1, 1);
            advance();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            *reinterpret_cast<int2*>(&s_sum[warp][g][8 * nt + 2 * t]) = make_int2(acc[nt][0], acc[nt][1]);
            *reinterpret_cast<int2*>(&s_sum[warp][g + 8][8 * nt + 2 * t]) = make_int2(acc[nt][2], acc[nt][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * 8 * NT; i += kThreads) {
            const int r = i % kRows, m = lo + i / kRows, n = n0 + r;
            if (m < hi && n < p.w.N) {
                int sum = 0;
#pragma unroll
                for (int wv = 0; wv < kWarps; ++wv) sum += s_sum[wv][r][i / kRows];
                const float sx = kFused ? s_scale[m] : p.xs[m];
                const float sw = __ldg(p.w.scale + static_cast<int64_t>(e) * p.w.N + n);
                const float v = __fmul_rn(__fmul_rn(__int2float_rn(sum), sx), sw);
                const int64_t o = static_cast<int64_t>(m) * p.w.N + n;
                if (kF32)
                    static_cast<float*>(p.out)[o] = v;
                else
                    static_cast<uint16_t*>(p.out)[o] = f32_to_bf16_bits(v);
            }
        }
        __syncthreads();
    }
}

template <int NT, bool kFused, bool kDense>
cudaError_t gemv_launch(const GemvParams& p, int out_dtype, cudaStream_t st, bool dependent) {
    const int64_t steps = static_cast<int64_t>(p.groups) * (p.rr.T < p.w.E ? p.rr.T : p.w.E);
    const int64_t cap = static_cast<int64_t>(num_sms()) * kBlocksPerSm;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(steps < cap ? steps : cap));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kFused ? static_cast<size_t>(p.rr.T) * (3 * p.w.ld + kXPad) : 0;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = out_dtype == 0 ? cudaLaunchKernelEx(&cfg, k_int8_gemv<NT, kFused, true, kDense>, p)
                                         : cudaLaunchKernelEx(&cfg, k_int8_gemv<NT, kFused, false, kDense>, p);
    note_launches(1);
    return e;
}

template <bool kDense>
cudaError_t gemv_any(const GemvParams& p, int out_dtype, cudaStream_t st, bool dependent) {
    if (p.X) return gemv_launch<1, true, kDense>(p, out_dtype, st, false);
    if (p.rr.T <= 8) return gemv_launch<1, false, kDense>(p, out_dtype, st, dependent);
    return gemv_launch<2, false, kDense>(p, out_dtype, st, dependent);
}

}  // namespace

// Up to 8 tokens always.  Up to 16, unless the tensor-core kernel's tiles (256
// channels each) fill half of the SM pairs: in a captured graph 16 x 13824 x 5120
// takes 19.6 us here and 17.1 there, 16 x 4096 x 4096 7.2 and 11.3.
bool int8_gemv_pays(int64_t T, const Int8Weight& w) {
    if (T <= 8) return true;
    return T <= kMaxTokens && int8_tiles(T, w.E, w.N, 256) * 4 < num_sms();
}

bool int8_gemv_fused(int64_t T, const Int8Weight& w) { return T <= kMaxFused && T * w.ld <= kMaxFusedValues; }

cudaError_t launch_int8_fwd_gemv(const uint16_t* X, const int8_t* x_codes, const float* x_scale, const Int8Weight& w,
                                 const RowRanges& rr, void* out, int out_dtype, cudaStream_t st, bool dependent) {
    const GemvParams p{X, x_codes, x_scale, w, rr, static_cast<int>(ceil_div(w.N, kRows)), out};
    return rr.offsets ? gemv_any<false>(p, out_dtype, st, dependent) : gemv_any<true>(p, out_dtype, st, dependent);
}

}  // namespace qlora

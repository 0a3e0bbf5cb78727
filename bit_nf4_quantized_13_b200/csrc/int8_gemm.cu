// int8_gemm.cu -- the Int8 linear's input gradient on the CUDA cores, dense
// or grouped by expert (rows [offsets[e], offsets[e + 1]) of dY use weight e):
//
//   dX[m][k] = sum_n dY[m][n] * bf16(RN32(wq[n][k] * sw[n]))  fp32 sums
#include "common.cuh"
#include "kernels.h"

namespace qlora {
namespace {

constexpr int kTile = 64;   // outputs of a block: 64 x 64, 4 x 4 a thread
constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
k_int8_dx(const uint16_t* __restrict__ dY, const Int8Weight w, const RowRanges rr, uint16_t* __restrict__ dX) {
    __shared__ float sy[kTile][33], sw[32][kTile + 1];
    int lo, hi;
    expert_rows(rr, blockIdx.z, &lo, &hi);
    const int64_t m0 = lo + static_cast<int64_t>(blockIdx.y) * kTile;
    if (m0 >= hi) return;
    const int64_t k0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int8_t* wc = w.codes + static_cast<int64_t>(blockIdx.z) * w.N * w.ld;
    const float* ws = w.scale + static_cast<int64_t>(blockIdx.z) * w.N;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t n0 = 0; n0 < w.N; n0 += 32) {
        for (int i = threadIdx.x; i < kTile * 32; i += kThreads) {
            const int r = i / 32;
            const int64_t n = n0 + i % 32;
            sy[r][i % 32] = (m0 + r < hi && n < w.N) ? bf16_bits_to_f32(dY[(m0 + r) * w.N + n]) : 0.0f;
            const int64_t nw = n0 + i / kTile, k = k0 + i % kTile;
            float v = 0.0f;
            if (nw < w.N && k < w.K)
                v = bf16_bits_to_f32(f32_to_bf16_bits(__fmul_rn(static_cast<float>(wc[nw * w.ld + k]), ws[nw])));
            sw[i / kTile][i % kTile] = v;
        }
        __syncthreads();
        for (int nn = 0; nn < 32; ++nn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sy[ty + 16 * i][nn], sw[nn][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, k = k0 + tx + 16 * j;
            if (m < hi && k < w.K) dX[m * w.K + k] = f32_to_bf16_bits(acc[i][j]);
        }
}

dim3 grid_for(int64_t cols, const RowRanges& rr, int E) {
    return dim3(static_cast<unsigned>(ceil_div(cols, kTile)), static_cast<unsigned>(ceil_div(rr.T, kTile)),
                static_cast<unsigned>(E));
}

}  // namespace

cudaError_t launch_int8_dx(const uint16_t* dY, const Int8Weight& w, const RowRanges& rr, uint16_t* dX,
                           cudaStream_t st) {
    k_int8_dx<<<grid_for(w.K, rr, w.E), kThreads, 0, st>>>(dY, w, rr, dX);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace qlora

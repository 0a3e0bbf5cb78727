// int8_rows.cu -- Int8 absmax quantization of matrix rows: the study notes'
// (gitcode.csdn.net) section 3.1, eq. (1) with one block per row, which gives
// a scale to each token of an activation and to each output channel of a
// weight:
//
//   a = max |x| over the row,  c = RN32(127 / a),
//   code = round_half_away(RN32(c x)),  scale = RN32(a / 127)
//
// c = scale = 0 and codes 0 where a is 0 or so small that c overflows; a row
// holding a NaN or Inf gets codes 0 and scale NaN.  Rows of codes are padded
// with zero codes to a multiple of 16 bytes.
//
// HBM-bound: 2 (bf16) or 4 (fp32) bytes read and one written per element.  A
// row is read once into registers (up to kVecs 16-byte vectors per thread),
// reduced, and encoded from there; only longer rows are read a second time,
// for the part that did not fit.  A warp takes a row of up to kVecs * 32
// vectors, so its reduction needs no barrier; a 256-thread block takes a
// longer one.
#include "int8_rows.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // vectors of a row held by one thread (32 registers)

// kGroup threads (32 or kThreads) per row.
template <typename T, bool kAligned, int kGroup>
__global__ void __launch_bounds__(kThreads)
k_int8_rows(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld, int8_t* __restrict__ codes,
            float* __restrict__ scale, int* __restrict__ status) {
    sm100::grid_launch_dependents();
    using V = RowVec<T, kAligned>;
    constexpr int kRows = kThreads / kGroup;
    const int tid = threadIdx.x % kGroup, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup;
    if (row >= rows) return;  // a whole group (a warp where kGroup is 32)
    const T* xr = x + row * K;
    int8_t* cr = codes + row * ld;
    V v[kVecs];
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t e = static_cast<int64_t>(i * kGroup + tid) * V::kPer;
        if (e < ld) v[i].load(xr, e, K);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (static_cast<int64_t>(i * kGroup + tid) * V::kPer < ld) a = abs_max(v[i], a);
    for (int64_t e = static_cast<int64_t>(kVecs * kGroup + tid) * V::kPer; e < ld; e += kGroup * V::kPer) {
        V t;
        t.load(xr, e, K);
        a = abs_max(t, a);
    }
    a = __reduce_max_sync(0xffffffffu, a);
    if (kGroup > 32) {
        __shared__ uint32_t s_max[kThreads / 32];
        if (lane == 0) s_max[threadIdx.x >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) a = max(a, s_max[i]);
    }
    float sc;
    const float c = row_constant(a, &sc);
    if (tid == 0) {
        scale[row] = sc;
        if (isnan(sc) && status) atomicExch(status, QLORA_ERR_NONFINITE);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t e = static_cast<int64_t>(i * kGroup + tid) * V::kPer;
        if (e < ld) encode(v[i], c, cr + e);
    }
    for (int64_t e = static_cast<int64_t>(kVecs * kGroup + tid) * V::kPer; e < ld; e += kGroup * V::kPer) {
        V t;
        t.load(xr, e, K);
        encode(t, c, cr + e);
    }
}

template <typename T, bool kAligned>
cudaError_t rows_launch(const T* x, int64_t rows, int64_t K, int64_t ld, int8_t* codes, float* scale, int* status,
                        cudaStream_t st) {
    constexpr int kPer = RowVec<T, kAligned>::kPer;
    if (ld <= 32 * kVecs * kPer) {
        const int64_t grid = ceil_div(rows, kThreads / 32);
        k_int8_rows<T, kAligned, 32><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(x, rows, K, ld, codes, scale, status);
    } else {
        k_int8_rows<T, kAligned, kThreads><<<static_cast<unsigned>(rows), kThreads, 0, st>>>(x, rows, K, ld, codes, scale,
                                                                                          status);
    }
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int8_rows(const void* x, int x_dtype, int64_t rows, int64_t K, int8_t* codes, float* scale,
                             int32_t* status, cudaStream_t st) {
    int* flag = reinterpret_cast<int*>(status);
    if (flag) {
        const cudaError_t e = cudaMemsetAsync(flag, 0, sizeof(int), st);
        if (e != cudaSuccess) return e;
    }
    const int64_t ld = int8_row_bytes(K);
    if (x_dtype == 0) {
        const float* p = static_cast<const float*>(x);
        return K % 4 == 0 ? rows_launch<float, true>(p, rows, K, ld, codes, scale, flag, st)
                          : rows_launch<float, false>(p, rows, K, ld, codes, scale, flag, st);
    }
    const uint16_t* p = static_cast<const uint16_t*>(x);
    return K % 8 == 0 ? rows_launch<uint16_t, true>(p, rows, K, ld, codes, scale, flag, st)
                      : rows_launch<uint16_t, false>(p, rows, K, ld, codes, scale, flag, st);
}

}  // namespace qlora

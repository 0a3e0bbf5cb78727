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
// reduced, and encoded from there; only rows of more than 256 such threads are
// read a second time, for the part that did not fit.  8, 32, 64, 128 or 256
// threads take a row; within a warp there is no barrier at all.  8192 x 8192
// bf16: 37 us (201 MB).
#include "int8_rows.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qlora {
namespace {

constexpr int kVecs = 8;  // vectors of a row held by one thread (32 registers)

constexpr int block_threads(int group) { return group < 128 ? 128 : group; }

// kGroup threads per row.
template <typename T, bool kAligned, int kGroup>
__global__ void __launch_bounds__(block_threads(kGroup))
k_int8_rows(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld, int8_t* __restrict__ codes,
            float* __restrict__ scale, int* __restrict__ status) {
    sm100::grid_launch_dependents();
    using V = RowVec<T>;
    constexpr int kRows = block_threads(kGroup) / kGroup, kWarps = kGroup / 32;
    const int tid = threadIdx.x % kGroup, group = threadIdx.x / kGroup, lane = threadIdx.x & 31;
    const uint32_t lanes = kGroup >= 32 ? 0xffffffffu : ((1u << (kGroup & 31)) - 1u) << (lane - tid % 32);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
    if (row >= rows) return;  // a whole group
    const T* xr = x + row * K;
    const T* end = x + rows * K;
    int8_t* cr = codes + row * ld;
    V v[kVecs];
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int64_t e = static_cast<int64_t>(i * kGroup + tid) * V::kPer;
        if (e < ld) v[i].template load<kAligned>(xr, e, K, end);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (static_cast<int64_t>(i * kGroup + tid) * V::kPer < ld) a = abs_max(v[i], a);
    for (int64_t e = static_cast<int64_t>(kVecs * kGroup + tid) * V::kPer; e < ld; e += kGroup * V::kPer) {
        V t;
        t.template load<kAligned>(xr, e, K, end);
        a = abs_max(t, a);
    }
    a = __reduce_max_sync(lanes, a);
    if (kWarps > 1) {
        __shared__ uint32_t s_max[kRows][kWarps > 0 ? kWarps : 1];
        if (lane == 0) s_max[group][tid >> 5] = a;
        sm100::named_bar_sync(1 + group, kGroup);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) a = max(a, s_max[group][i]);
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
        t.template load<kAligned>(xr, e, K, end);
        encode(t, c, cr + e);
    }
}

template <typename T, bool kAligned, int kGroup>
cudaError_t rows_launch(const T* x, int64_t rows, int64_t K, int64_t ld, int8_t* codes, float* scale, int* status,
                        cudaStream_t st) {
    constexpr int kBlock = block_threads(kGroup);
    const int64_t grid = ceil_div(rows, kBlock / kGroup);
    k_int8_rows<T, kAligned, kGroup><<<static_cast<unsigned>(grid), kBlock, 0, st>>>(x, rows, K, ld, codes, scale, status);
    note_launches(1);
    return cudaGetLastError();
}

template <typename T, bool kAligned>
cudaError_t rows_any(const T* x, int64_t rows, int64_t K, int64_t ld, int8_t* codes, float* scale, int* status,
                     cudaStream_t st) {
    // vectors per thread: many where rows abound (bytes in flight: 8192 x 8192
    // bf16 took 47 us with four, 37 with eight), few where they do not (one
    // row's latency); a shifted vector takes two loads
    const int per_thread = rows < 1024 ? 2 : kAligned ? kVecs : kVecs / 2;
    const int64_t threads = ceil_div(ld, RowVec<T>::kPer * per_thread);
    if (threads <= 8) return rows_launch<T, kAligned, 8>(x, rows, K, ld, codes, scale, status, st);
    if (threads <= 32) return rows_launch<T, kAligned, 32>(x, rows, K, ld, codes, scale, status, st);
    if (threads <= 64) return rows_launch<T, kAligned, 64>(x, rows, K, ld, codes, scale, status, st);
    if (threads <= 128) return rows_launch<T, kAligned, 128>(x, rows, K, ld, codes, scale, status, st);
    return rows_launch<T, kAligned, 256>(x, rows, K, ld, codes, scale, status, st);
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
        return K % 4 == 0 ? rows_any<float, true>(p, rows, K, ld, codes, scale, flag, st)
                          : rows_any<float, false>(p, rows, K, ld, codes, scale, flag, st);
    }
    const uint16_t* p = static_cast<const uint16_t*>(x);
    return K % 8 == 0 ? rows_any<uint16_t, true>(p, rows, K, ld, codes, scale, flag, st)
                      : rows_any<uint16_t, false>(p, rows, K, ld, codes, scale, flag, st);
}

}  // namespace qlora

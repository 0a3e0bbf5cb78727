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
#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;  // vectors of a row held by one thread (32 registers)

// kPer values of a row from element e on, 16 bytes; elements past K read 0.
template <typename T, bool kAligned>
struct RowVec;

template <bool kAligned>
struct RowVec<float, kAligned> {
    static constexpr int kPer = 4;
    uint32_t w[4];
    __device__ __forceinline__ void load(const float* row, int64_t e, int64_t K) {
        if (kAligned && e + 4 <= K) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + e));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = e + i < K ? __float_as_uint(row[e + i]) : 0u;
        }
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
};

template <bool kAligned>
struct RowVec<uint16_t, kAligned> {
    static constexpr int kPer = 8;
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t* row, int64_t e, int64_t K) {
        if (kAligned && e + 8 <= K) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + e));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = e + 2 * i < K ? row[e + 2 * i] : 0u;
                const uint32_t hi = e + 2 * i + 1 < K ? row[e + 2 * i + 1] : 0u;
                w[i] = lo | (hi << 16);
            }
        }
    }
    __device__ __forceinline__ float at(int i) const {
        return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
};

// The largest |value| as bit patterns: non-negative fp32 patterns sort like
// the values, with Inf and NaN above every finite one.
template <typename V>
__device__ __forceinline__ uint32_t abs_max(const V& v, uint32_t a) {
#pragma unroll
    for (int i = 0; i < V::kPer; ++i) a = max(a, __float_as_uint(v.at(i)) & 0x7fffffffu);
    return a;
}

template <typename V>
__device__ __forceinline__ void encode(const V& v, float c, int8_t* out) {
    uint32_t o[V::kPer / 4];
#pragma unroll
    for (int j = 0; j < V::kPer / 4; ++j) {
        o[j] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[j] |= (static_cast<uint32_t>(static_cast<int>(roundf(__fmul_rn(c, v.at(4 * j + i))))) & 0xffu) << (8 * i);
    }
    if (V::kPer == 8)
        *reinterpret_cast<uint2*>(out) = make_uint2(o[0], o[V::kPer / 4 - 1]);
    else
        *reinterpret_cast<uint32_t*>(out) = o[0];
}

// kGroup threads (32 or kThreads) per row.
template <typename T, bool kAligned, int kGroup>
__global__ void __launch_bounds__(kThreads)
k_int8_rows(const T* __restrict__ x, int64_t rows, int64_t K, int64_t ld, int8_t* __restrict__ codes,
            float* __restrict__ scale, int* __restrict__ status, int* __restrict__ zero, int n_zero) {
    sm100::grid_launch_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n_zero; i += kThreads) zero[i] = 0;
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
    const bool finite = a < 0x7f800000u;
    const float top = __uint_as_float(a);
    float c = finite && a != 0u ? __fdiv_rn(127.0f, top) : 0.0f;
    if (!isfinite(c)) c = 0.0f;
    if (tid == 0) {
        scale[row] = finite ? (c > 0.0f ? __fdiv_rn(top, 127.0f) : 0.0f) : __uint_as_float(0x7fc00000u);
        if (!finite && status) atomicExch(status, QLORA_ERR_NONFINITE);
    }
    // 0 * Inf is NaN, which the conversion to an integer turns into 0
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
                        int* zero, int n_zero, cudaStream_t st) {
    constexpr int kPer = RowVec<T, kAligned>::kPer;
    if (ld <= 32 * kVecs * kPer) {
        const int64_t grid = ceil_div(rows, kThreads / 32);
        k_int8_rows<T, kAligned, 32><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(x, rows, K, ld, codes, scale, status,
                                                                                      zero, n_zero);
    } else {
        k_int8_rows<T, kAligned, kThreads><<<static_cast<unsigned>(rows), kThreads, 0, st>>>(x, rows, K, ld, codes, scale,
                                                                                          status, zero, n_zero);
    }
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int8_rows(const void* x, int x_dtype, int64_t rows, int64_t K, int8_t* codes, float* scale,
                             int32_t* status, cudaStream_t st, int* zero, int n_zero) {
    int* flag = reinterpret_cast<int*>(status);
    if (flag) {
        const cudaError_t e = cudaMemsetAsync(flag, 0, sizeof(int), st);
        if (e != cudaSuccess) return e;
    }
    const int64_t ld = int8_row_bytes(K);
    if (x_dtype == 0) {
        const float* p = static_cast<const float*>(x);
        return K % 4 == 0 ? rows_launch<float, true>(p, rows, K, ld, codes, scale, flag, zero, n_zero, st)
                          : rows_launch<float, false>(p, rows, K, ld, codes, scale, flag, zero, n_zero, st);
    }
    const uint16_t* p = static_cast<const uint16_t*>(x);
    return K % 8 == 0 ? rows_launch<uint16_t, true>(p, rows, K, ld, codes, scale, flag, zero, n_zero, st)
                      : rows_launch<uint16_t, false>(p, rows, K, ld, codes, scale, flag, zero, n_zero, st);
}

}  // namespace qlora

// int8_rows.cuh -- the Int8 row quantization's per-element steps (eq. 1 with
// one block per row), shared by the row quantizer and by the small-batch
// product that quantizes its tokens itself: both give the same bytes.
#pragma once

#include "common.cuh"

namespace qlora {

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

// Codes of one vector.  Where c is 0, c * x is 0, or NaN for a non-finite x,
// which the conversion to an integer also turns into 0.
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

// c and scale of a row whose largest |x| has the bit pattern `a`; a row that
// holds a NaN or Inf has c = 0 and scale NaN.
__device__ __forceinline__ float row_constant(uint32_t a, float* scale) {
    if (a >= 0x7f800000u) {
        *scale = __uint_as_float(0x7fc00000u);
        return 0.0f;
    }
    const float top = __uint_as_float(a);
    float c = a != 0u ? __fdiv_rn(127.0f, top) : 0.0f;
    if (!isfinite(c)) c = 0.0f;
    *scale = c > 0.0f ? __fdiv_rn(top, 127.0f) : 0.0f;
    return c;
}

}  // namespace qlora

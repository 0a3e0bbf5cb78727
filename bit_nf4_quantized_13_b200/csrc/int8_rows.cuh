// int8_rows.cuh -- the Int8 row quantization's per-element steps (eq. 1 with
// one block per row), shared by the row quantizer and by the small-batch
// product that quantizes its tokens itself: both give the same bytes.
#pragma once

#include "common.cuh"

namespace qlora {

// kPer values of a row from element e on (e a multiple of kPer), 16 bytes;
// elements past K read 0.  kAligned: rows start at multiples of 16 bytes.
// Else (the row length is no multiple of 16 bytes) a vector lies across two
// aligned ones, which are both loaded and shifted together: one value at a
// time took twice as long.  `end` is the end of the whole matrix, which starts
// at a multiple of 16 bytes: nothing behind it is read.
template <typename T>
struct RowVec {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    uint32_t w[4];

    __device__ __forceinline__ void one_by_one(const T* row, int64_t e, int64_t K) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = e + i < K ? __float_as_uint(row[e + i]) : 0u;
            } else {
                const uint32_t lo = e + 2 * i < K ? row[e + 2 * i] : 0u;
                const uint32_t hi = e + 2 * i + 1 < K ? row[e + 2 * i + 1] : 0u;
                w[i] = lo | (hi << 16);
            }
        }
    }

    template <bool kAligned>
    __device__ __forceinline__ void load(const T* row, int64_t e, int64_t K, const T* end) {
        const T* p = row + e;
        if constexpr (kAligned) {
            if (e + kPer <= K) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
                w[0] = v.x;
                w[1] = v.y;
                w[2] = v.z;
                w[3] = v.w;
                return;
            }
        } else {
            const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
            const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - mis);
            if (e + kPer <= K && reinterpret_cast<const char*>(q) + 32 <= reinterpret_cast<const char*>(end)) {
                const uint4 a = __ldg(q), b = __ldg(q + 1);
                uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                if (mis & 8u) {
#pragma unroll
                    for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
                }
                if (mis & 4u) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = (mis & 2u) ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
                return;
            }
        }
        one_by_one(row, e, K);
    }

    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
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

// round_half_away(v) for |v| < 2^22: |v| + 1/2 rounded towards zero cannot
// reach an integer that the exact sum does not reach, so its integer part is
// that of the exact sum.
__device__ __forceinline__ int round_half_away(float v) {
    return __float2int_rz(__fadd_rz(v, copysignf(0.5f, v)));
}

// Codes of one vector.  Where c is 0, c * x is 0, or NaN for a non-finite x,
// which the conversion to an integer also turns into 0.
template <typename V>
__device__ __forceinline__ void encode(const V& v, float c, int8_t* out) {
    uint32_t o[V::kPer / 4];
#pragma unroll
    for (int j = 0; j < V::kPer / 4; ++j) {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = static_cast<uint32_t>(round_half_away(__fmul_rn(c, v.at(4 * j + i))));
        o[j] = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
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

// int8_zero.cu -- zeroes the rows of an expert product's output that belong to
// no expert: the rows before the first offset and from the last one on.  The
// products leave those as they were, so an output that the caller has just
// allocated needs them cleared.
//
// Bound by the writes of those rows, and by the launch where there are none:
// 8192 x 4096 bf16 over 16 experts takes 1.5 us with no such row and 6 us with
// half of the rows, where clearing the whole output (67 MB) takes 17.5 us.  In a
// loop of calls it adds 3.5 us to a forward of 16 rows and 5 to one of 8192.
#include "common.cuh"
#include "kernels.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

// Zeroes bytes [a, b) of out (16-byte aligned; a and b even), the grid's threads in turn.
__device__ __forceinline__ void zero_bytes(char* out, int64_t a, int64_t b) {
    if (a >= b) return;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t a16 = min((a + 15) / 16 * 16, b), b16 = max(b / 16 * 16, a16);
    for (int64_t i = a16 + first * 16; i < b16; i += stride * 16)
        *reinterpret_cast<uint4*>(out + i) = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t i = a + first * 2; i < a16; i += stride * 2) *reinterpret_cast<uint16_t*>(out + i) = 0;
    for (int64_t i = b16 + first * 2; i < b; i += stride * 2) *reinterpret_cast<uint16_t*>(out + i) = 0;
}

// An offset counts as no less than the one before it and as in [0, T], as in
// the products: the rows of the experts are [first offset, largest offset).
__global__ void __launch_bounds__(kThreads) k_int8_zero_rows(const RowRanges rr, int E, int64_t row_bytes, char* out) {
    __shared__ int s_top[kThreads / 32];
    const int T = static_cast<int>(rr.T);
    int top = 0;
    for (int e = static_cast<int>(threadIdx.x); e <= E; e += kThreads) top = max(top, min(rr.offsets[e], T));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) top = max(top, s_top[i]);
    const int first = min(max(rr.offsets[0], 0), T);
    zero_bytes(out, 0, first * row_bytes);
    zero_bytes(out, top * row_bytes, T * row_bytes);
}

}  // namespace

cudaError_t launch_int8_zero_rows(const RowRanges& rr, int E, int64_t row_bytes, void* out, cudaStream_t st) {
    const int64_t blocks = ceil_div(rr.T * row_bytes, 16 * kThreads), cap = static_cast<int64_t>(num_sms()) * 4;
    k_int8_zero_rows<<<static_cast<unsigned>(blocks < cap ? blocks : cap), kThreads, 0, st>>>(
        rr, E, row_bytes, static_cast<char*>(out));
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace qlora

// outer_rows.cu -- zeros in the token rows that no sequence of a packed call holds.  The recurrence
// leaves them as they were, and memory that was only allocated must not reach the sums over all
// rows that follow (a projection's weight gradient).  The host does not know where the
// sequences end, so the rows are found here; without any the launch is all that it costs (2 us).
#include <algorithm>

#include "gdr_internal.h"

namespace gdr {

namespace {

struct Tensors {
    char* p[3];
};

// A block takes every gridDim.x-th outer row, 16 bytes per thread and step.
__global__ void __launch_bounds__(256)
outer_rows_kernel(Tensors t, const int32_t* cu, int B, long long T, long long row_bytes,
                  long long pitch_bytes) {
    const long long lo = min(max((long long)cu[0], 0LL), T);
    const long long hi = min(max((long long)cu[B], lo), T);
    for (long long i = blockIdx.x; i < lo + T - hi; i += gridDim.x) {
        const long long row = i < lo ? i : i - lo + hi;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (!t.p[k]) continue;
            char* at = t.p[k] + row * pitch_bytes;
            for (long long b = 16LL * threadIdx.x; b < row_bytes; b += 16LL * blockDim.x)
                *reinterpret_cast<uint4*>(at + b) = make_uint4(0, 0, 0, 0);
        }
    }
}

}  // namespace

cudaError_t launch_zero_outer_rows(void* x, void* y, void* z, const int32_t* cu_seqlens, int B, int T,
                                   long long row_bytes, long long pitch_bytes, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    const Tensors t = {{static_cast<char*>(x), static_cast<char*>(y), static_cast<char*>(z)}};
    outer_rows_kernel<<<(unsigned)std::min(T, 4 * device_sms()), 256, 0, stream>>>(
        t, cu_seqlens, B, T, row_bytes, pitch_bytes);
    return cudaGetLastError();
}

}  // namespace gdr

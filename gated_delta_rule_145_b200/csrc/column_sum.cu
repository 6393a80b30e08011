// column_sum.cu -- the last step of every parameter gradient: the sums of the per-CTA
// partial rows that a backward kernel left in the workspace.
//
// part [P][N] fp32 -> out0 [n0] (columns 0 .. n0 - 1) and out1 [N - n0] (the others).
// The rows are added in a fixed order (thread row y takes rows y, y + 32, ...; then a tree
// over y), so a call's result does not depend on which CTA finished first, as it would with
// atomic adds.  With P = 0 the sums are zero.
#include "gdr_internal.h"
#include "tcgen05.cuh"

namespace gdr {

namespace {

constexpr int kSumX = 32, kSumY = 32;

__global__ void __launch_bounds__(kSumX * kSumY)
column_sum_kernel(const float* __restrict__ part, long long P, int N, float* __restrict__ out0,
                  int n0, float* __restrict__ out1) {
    __shared__ float sm[kSumY][kSumX + 1];
    // launched while the kernel before it in the stream, which wrote part, may still run
    tc::grid_dep_wait();
    const int x = threadIdx.x % kSumX, y = threadIdx.x / kSumX;
    const int n = blockIdx.x * kSumX + x;
    float s = 0.f;
    if (n < N) {
#pragma unroll 8
        for (long long p = y; p < P; p += kSumY) s += part[p * N + n];
    }
    sm[y][x] = s;
    __syncthreads();
#pragma unroll
    for (int h = kSumY / 2; h > 0; h /= 2) {
        if (y < h) sm[y][x] += sm[y + h][x];
        __syncthreads();
    }
    if (y == 0 && n < N) {
        float* out = n < n0 ? out0 : out1;
        if (out) out[n < n0 ? n : n - n0] = sm[0][x];
    }
}

}  // namespace

cudaError_t launch_column_sum(const float* part, long long P, int N, float* out0, int n0,
                              float* out1, cudaStream_t stream) {
    if (N <= 0) return cudaSuccess;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((N + kSumX - 1) / kSumX));
    cfg.blockDim = dim3(kSumX * kSumY);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, column_sum_kernel, part, P, N, out0, n0, out1);
}

}  // namespace gdr

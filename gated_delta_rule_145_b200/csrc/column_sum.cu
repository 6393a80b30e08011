// column_sum.cu -- the last step of every parameter gradient: the sums of the per-CTA
// partial rows that a backward kernel left in the workspace.
//
// part [P][N] fp32 -> out0 [n0] (columns 0 .. n0 - 1) and out1 [N - n0] (the others).
// The rows are added in a fixed order (thread row y takes rows y, y + Y, ...; then a tree
// over y), so a call's result does not depend on which CTA finished first, as it would with
// atomic adds.  With P = 0 the sums are zero.  A thread takes four columns; few blocks of
// many rows (a norm's 128 columns) need all their loads in flight at once, many blocks of few rows
// (a convolution's taps) need small blocks: Y = 16 up to 128 rows, above 128, or 32 where 256
// blocks and more share the SMs.  Of 1184 rows of 128 columns it takes 7.5 us, of 148 of 12288 7.7
// (two more with Y = 128; one thread per column and 32 rows of threads: four more).
#include "gdr_internal.h"
#include "tcgen05.cuh"

namespace gdr {

namespace {

constexpr int kSumX = 8;  // threads across: 32 columns

template <int Y>
__global__ void __launch_bounds__(kSumX * Y)
column_sum_kernel(const float* __restrict__ part, long long P, int N, float* __restrict__ out0,
                  int n0, float* __restrict__ out1) {
    __shared__ float4 sm[Y][kSumX];
    const int x = threadIdx.x % kSumX, y = threadIdx.x / kSumX;
    const int n = 4 * (blockIdx.x * kSumX + x);
    // launched while the kernel before it in the stream, which wrote part, may still run
    tc::grid_dep_wait();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < N) {
#pragma unroll 8
        for (long long p = y; p < P; p += Y) {
            const float4 v = *reinterpret_cast<const float4*>(part + p * N + n);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
    }
    sm[y][x] = s;
    __syncthreads();
#pragma unroll
    for (int h = Y / 2; h > 0; h /= 2) {
        if (y < h) {
            const float4 v = sm[y + h][x];
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            sm[y][x] = s;
        }
        __syncthreads();
    }
    if (y == 0 && n < N) {
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float* out = n + e < n0 ? out0 : out1;
            if (out) out[n + e < n0 ? n + e : n + e - n0] = v[e];
        }
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
    cfg.gridDim = dim3((unsigned)((N + 4 * kSumX - 1) / (4 * kSumX)));
    const int Y = P <= 128 ? 16 : cfg.gridDim.x < 256 ? 128 : 32;
    cfg.blockDim = dim3(kSumX * Y);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, Y == 128  ? column_sum_kernel<128>
                                    : Y == 32 ? column_sum_kernel<32>
                                              : column_sum_kernel<16>,
                              part, P, N, out0, n0, out1);
}

}  // namespace gdr

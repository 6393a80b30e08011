// mixer_grad.cu -- the backward passes of the steps on either side of the rule
// (mixer_io.cu holds the forward ones):
//   conv   s_t = bias + sum_{i<4} w_i x_{t-3+i},  y = SiLU(s):
//              ds_t = dy_t sig(s_t) (1 + s_t (1 - sig(s_t)))
//              dx_t = sum_i w_i ds_{t+3-i},  dw_i = sum_t ds_t x_{t-3+i},  dbias = sum_t ds_t;
//          the three inputs before the call (the state) get the same sum, and the gradient of
//          the state after the call goes to the inputs it copies.
//   norm   y = o r w SiLU(z),  r = 1 / sqrt(mean(o^2) + eps),  q = dy w SiLU(z):
//              do = r q - o r^3 mean(q o),  dz = dy o r w SiLU'(z),  dw = sum_rows dy o r SiLU(z).
// Both are bound by memory: every input is read once, s and r are computed again instead of
// being kept by the forward pass.  Parameter gradients leave each CTA as one row of partial
// sums, which column_sum.cu adds in a fixed order.
#include <algorithm>

#include "gdr_common.cuh"
#include "gdr_internal.h"

namespace gdr {

namespace {

__device__ __forceinline__ float ex2g(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpg(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sigmoid(v) by 1 / (1 + 2^(-v log2 e)): relative error ~1e-6, 0 where the power is +inf
__device__ __forceinline__ float sigmoid_fast(float v) {
    return rcpg(1.0f + ex2g(v * -1.4426950408889634f));
}

__device__ __forceinline__ void unpack4(const uint2 u, float (&f)[4]) {
    const float2 l = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 h = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    f[0] = l.x; f[1] = l.y; f[2] = h.x; f[3] = h.y;
}
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
    const __nv_bfloat162 l = __floats2bfloat162_rn(f[0], f[1]), h = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
}

// ------------------------------------------------------------------------ conv + SiLU

constexpr int kW = 4;
constexpr int kGSeg = 64;     // tokens per warp
constexpr int kGWarps = 8;    // segments per CTA
constexpr int kGCh = 128;     // channels per CTA: four per lane

// CTA -> (channel tile, group of 8 segments of the B * nseg segments); warp -> segment.
// part [groups][5 C]: the taps' sums as [C][4], then the bias's.
__global__ void __launch_bounds__(32 * kGWarps)
conv_backward_kernel(ConvGrads p, int nct, int nseg, float* part) {
    __shared__ float sm[kGWarps][5][kGCh];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int ct = blockIdx.x % nct, group = blockIdx.x / nct;
    const int c = ct * kGCh + 4 * lane;
    const long long sid = (long long)group * kGWarps + warp;
    const bool live = c < p.C && sid < (long long)p.B * nseg;
    float aw[kW][4] = {}, ab[4] = {};
    if (live) {
        const int b = (int)(sid / nseg);
        const int T = p.T, C = p.C;
        const int t0 = (int)(sid % nseg) * kGSeg, t1 = min(T, t0 + kGSeg);
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + ((size_t)b * T) * C + c;
        const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(p.grad_y) + ((size_t)b * T) * C + c;
        __nv_bfloat16* dx = static_cast<__nv_bfloat16*>(p.grad_x) + ((size_t)b * T) * C + c;
        float w[4][kW], bs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int i = 0; i < kW; ++i) w[e][i] = p.weight[(size_t)(c + e) * kW + i];
            bs[e] = p.bias ? p.bias[c + e] : 0.f;
        }
        const size_t st = ((size_t)b * C + c) * 3;
        float h[3][4], ds[3][4] = {};  // x at t - 3 .. t - 1; ds at t - 3 .. t - 1
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int t = t0 - 3 + j;
            if (t >= 0) {
                unpack4(*reinterpret_cast<const uint2*>(x + (size_t)t * C), h[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) h[j][e] = p.state_in ? p.state_in[st + 3 * e + t + 3] : 0.f;
            }
        }
        for (int t = t0; t < t1 + 3; ++t) {
            float v[4] = {}, d[4] = {};
            if (t < T) {
                float g[4];
                unpack4(__ldcs(reinterpret_cast<const uint2*>(x + (size_t)t * C)), v);
                unpack4(__ldcs(reinterpret_cast<const uint2*>(dy + (size_t)t * C)), g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float s = bs[e] + w[e][0] * h[0][e] + w[e][1] * h[1][e] +
                                    w[e][2] * h[2][e] + w[e][3] * v[e];
                    const float sg = sigmoid_fast(s);
                    d[e] = g[e] * sg * (1.f + s * (1.f - sg));
                    if (t < t1) {
                        aw[0][e] += d[e] * h[0][e];
                        aw[1][e] += d[e] * h[1][e];
                        aw[2][e] += d[e] * h[2][e];
                        aw[3][e] += d[e] * v[e];
                        ab[e] += d[e];
                    }
                }
            }
            // the input three tokens back has all four of its terms
            const int u = t - 3;
            if (u >= t0 || t0 == 0) {
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = w[e][3] * ds[0][e] + w[e][2] * ds[1][e] + w[e][1] * ds[2][e] + w[e][0] * d[e];
                    // the state after the call holds the inputs T - 3 .. T - 1
                    if (p.grad_state_out && u >= T - 3) o[e] += p.grad_state_out[st + 3 * e + u - (T - 3)];
                }
                if (u >= 0) {
                    __stcs(reinterpret_cast<uint2*>(dx + (size_t)u * C), pack4(o));
                } else if (p.grad_state_in) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) p.grad_state_in[st + 3 * e + u + 3] = o[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[0][e] = h[1][e]; h[1][e] = h[2][e]; h[2][e] = v[e];
                ds[0][e] = ds[1][e]; ds[1][e] = ds[2][e]; ds[2][e] = d[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int i = 0; i < kW; ++i) sm[warp][i][4 * lane + e] = aw[i][e];
        sm[warp][4][4 * lane + e] = ab[e];
    }
    __syncthreads();
    float* row = part + (size_t)group * 5 * p.C;
    for (int k = threadIdx.x; k < 5 * kGCh; k += blockDim.x) {
        const int i = k / kGCh, ch = k % kGCh, cc = ct * kGCh + ch;
        if (cc >= p.C) continue;
        float s = 0.f;
#pragma unroll
        for (int wi = 0; wi < kGWarps; ++wi) s += sm[wi][i][ch];
        row[i < kW ? (size_t)cc * kW + i : (size_t)kW * p.C + cc] = s;
    }
}

// ---------------------------------------------------------------------- gated RMSNorm

constexpr int kNThreads = 256;

__device__ __forceinline__ void load_z4(const float* p, float (&z)[4]) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    z[0] = v.x; z[1] = v.y; z[2] = v.z; z[3] = v.w;
}
__device__ __forceinline__ void load_z4(const __nv_bfloat16* p, float (&z)[4]) {
    unpack4(__ldcs(reinterpret_cast<const uint2*>(p)), z);
}
__device__ __forceinline__ void store_z4(float* p, const float (&z)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(z[0], z[1], z[2], z[3]));
}
__device__ __forceinline__ void store_z4(__nv_bfloat16* p, const float (&z)[4]) {
    __stcs(reinterpret_cast<uint2*>(p), pack4(z));
}

// L = d / 4 adjacent lanes share a row, four values each; a warp takes 32 / L rows at a
// time, grid-stride.  part [gridDim.x][d].
template <typename Tz, int D>
__global__ void __launch_bounds__(kNThreads)
gated_rmsnorm_backward_kernel(NormGrads p, float* part) {
    constexpr int L = D / 4, R = kNThreads / L;  // lanes per row, rows per block
    __shared__ float sm[R][D];
    const int sub = threadIdx.x / L, lane = threadIdx.x % L;
    const float4 w4 = *reinterpret_cast<const float4*>(p.weight + 4 * lane);
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
    const Tz* z = static_cast<const Tz*>(p.z);
    Tz* dz = static_cast<Tz*>(p.grad_z);
    float acc[4] = {};
    for (long long base = (long long)blockIdx.x * R; base < p.rows; base += (long long)gridDim.x * R) {
        const long long row = base + sub;
        const bool live = row < p.rows;
        const size_t at = (size_t)row * D + 4 * lane;
        float o[4] = {}, g[4] = {}, zv[4] = {}, q[4], ss = 0.f, qo = 0.f;
        if (live) {
            load_z4(p.o + at, o);
            load_z4(p.grad_y + at, g);
            load_z4(z + at, zv);
        }
        float silu[4], dsilu[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float sg = sigmoid_fast(zv[e]);
            silu[e] = zv[e] * sg;
            dsilu[e] = sg * (1.f + zv[e] * (1.f - sg));
            q[e] = g[e] * w[e] * silu[e];
            ss += o[e] * o[e];
            qo += q[e] * o[e];
        }
#pragma unroll
        for (int k = L / 2; k > 0; k /= 2) {
            ss += __shfl_xor_sync(0xffffffffu, ss, k);
            qo += __shfl_xor_sync(0xffffffffu, qo, k);
        }
        const float r = 1.0f / sqrtf(ss / (float)D + p.eps);
        const float m = r * r * r * (qo / (float)D);
        float go[4], gz[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            go[e] = r * q[e] - o[e] * m;
            const float gor = g[e] * o[e] * r;
            gz[e] = gor * w[e] * dsilu[e];
            if (live) acc[e] += gor * silu[e];
        }
        if (live) {
            store_z4(p.grad_o + at, go);
            store_z4(dz + at, gz);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sm[sub][4 * lane + e] = acc[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kNThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) s += sm[k][c];
        part[(size_t)blockIdx.x * D + c] = s;
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    return n;
}

template <typename Tz>
cudaError_t norm_backward(const NormGrads& p, unsigned grid, float* part, cudaStream_t stream) {
    switch (p.d) {
        case 32: gated_rmsnorm_backward_kernel<Tz, 32><<<grid, kNThreads, 0, stream>>>(p, part); break;
        case 64: gated_rmsnorm_backward_kernel<Tz, 64><<<grid, kNThreads, 0, stream>>>(p, part); break;
        case 128: gated_rmsnorm_backward_kernel<Tz, 128><<<grid, kNThreads, 0, stream>>>(p, part); break;
        default: return cudaErrorNotSupported;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_short_conv_silu_backward(const ConvGrads& p, cudaStream_t stream) {
    const size_t state_bytes = sizeof(float) * p.B * p.C * 3;
    if (p.T == 0) {  // nothing was convolved: the state passed through
        if (p.grad_state_in && p.grad_state_in != p.grad_state_out) {
            const cudaError_t e =
                p.grad_state_out ? cudaMemcpyAsync(p.grad_state_in, p.grad_state_out, state_bytes,
                                                   cudaMemcpyDeviceToDevice, stream)
                                 : cudaMemsetAsync(p.grad_state_in, 0, state_bytes, stream);
            if (e != cudaSuccess) return e;
        }
        return launch_column_sum(nullptr, 0, 5 * p.C, p.grad_weight, 4 * p.C, p.grad_bias, stream);
    }
    const int nseg = (p.T + kGSeg - 1) / kGSeg;
    const long long groups = ((long long)p.B * nseg + kGWarps - 1) / kGWarps;
    const int nct = (p.C + kGCh - 1) / kGCh;
    if (groups * nct > 0x7fffffffLL) return cudaErrorNotSupported;
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * groups * 5 * p.C, stream);
    if (e != cudaSuccess) return e;
    conv_backward_kernel<<<(unsigned)(groups * nct), 32 * kGWarps, 0, stream>>>(p, nct, nseg, part);
    e = cudaGetLastError();
    if (e == cudaSuccess)
        e = launch_column_sum(part, groups, 5 * p.C, p.grad_weight, 4 * p.C, p.grad_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

cudaError_t launch_gated_rmsnorm_backward(const NormGrads& p, cudaStream_t stream) {
    if (p.rows == 0) return launch_column_sum(nullptr, 0, p.d, p.grad_weight, p.d, nullptr, stream);
    const long long rpb = kNThreads / (p.d / 4);
    const unsigned grid = (unsigned)std::min<long long>((p.rows + rpb - 1) / rpb, (long long)sm_count() * 8);
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * grid * p.d, stream);
    if (e != cudaSuccess) return e;
    e = p.z_f32 ? norm_backward<float>(p, grid, part, stream)
                : norm_backward<__nv_bfloat16>(p, grid, part, stream);
    if (e == cudaSuccess)
        e = launch_column_sum(part, grid, p.d, p.grad_weight, p.d, nullptr, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace gdr

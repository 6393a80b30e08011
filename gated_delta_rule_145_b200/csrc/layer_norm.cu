// layer_norm.cu -- layer normalisation of rows of d values in front of the mixer, and its
// backward pass with the reduction of the weight's and bias's gradients over the rows:
//     y  = xh * weight + bias,  xh = (x - mean) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//     dx = rstd * (dyw - mean(dyw) - xh * mean(dyw * xh)),  dyw = dy * weight
//     dweight = sum_rows dy * xh,  dbias = sum_rows dy.
// Both are bound by memory (forward: x in, y out; backward: x, dy in, dx out).  A row lives in
// the registers of the threads that loaded it, eight adjacent values each, so it is read
// once; the variance is taken from the centred values (two passes over registers), which
// keeps its accuracy where the mean is far from zero.
#include <algorithm>

#include "gdr_common.cuh"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr int kVec = 8;           // adjacent values per thread
constexpr int kSubThreads = 256;  // block of the narrow form
constexpr int kSubMaxD = 256;     // widest row of the narrow form: one warp's lanes

__device__ __forceinline__ void load_vec(const float* p, float (&v)[kVec]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[kVec]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[kVec]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[kVec]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void load_param(const float* p, float (&v)[kVec]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum over the threads that share a row.  Sub: `tpr` adjacent lanes (a power of two).
// Otherwise the whole block, through `sm` (one float2 per warp; the caller alternates
// between two buffers, so one barrier per sum is enough).
template <bool Sub>
__device__ __forceinline__ float2 row_sum(float2 v, int tpr, float2* sm) {
    if constexpr (Sub) {
        for (int o = tpr / 2; o > 0; o /= 2) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        return v;
    } else {
        v.x = warp_sum(v.x);
        v.y = warp_sum(v.y);
        const int lane = threadIdx.x % 32, nw = blockDim.x / 32;
        if (lane == 0) sm[threadIdx.x / 32] = v;
        __syncthreads();
        v = lane < nw ? sm[lane] : make_float2(0.f, 0.f);
        return make_float2(warp_sum(v.x), warp_sum(v.y));
    }
}

// A block takes `rpb` rows at a time (Sub: one per group of `tpr` lanes; otherwise one),
// grid-stride.  NV vectors per thread, `tpr` vectors apart.
template <typename Tin, int NV, bool Sub>
__global__ void __launch_bounds__(Sub ? kSubThreads : 1024)
layer_norm_kernel(const Tin* x, const float* __restrict__ weight, const float* __restrict__ bias,
                  Tin* y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
                  long long rows, int d, int tpr, float eps) {
    __shared__ float2 sm[2][32];
    const int rpb = Sub ? kSubThreads / tpr : 1;
    const int sub = Sub ? threadIdx.x / tpr : 0, lane = Sub ? threadIdx.x % tpr : threadIdx.x;
    for (long long base = (long long)blockIdx.x * rpb; base < rows;
         base += (long long)gridDim.x * rpb) {
        const long long row = base + sub;
        const bool live = row < rows;
        float v[NV][kVec];
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (lane + n * tpr);
            if (live && c < d) {
                load_vec(x + row * d + c, v[n]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[n][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += v[n][e];
        }
        const float mean = row_sum<Sub>(make_float2(s, 0.f), tpr, sm[0]).x / (float)d;
        float ss = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const bool in = kVec * (lane + n * tpr) < d;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                v[n][e] -= mean;
                if (in) ss += v[n][e] * v[n][e];
            }
        }
        const float var = row_sum<Sub>(make_float2(ss, 0.f), tpr, sm[1]).x / (float)d;
        const float rstd = 1.0f / sqrtf(var + eps);
        if (live && lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (lane + n * tpr);
            if (!live || c >= d) continue;
            float w[kVec], bs[kVec], o[kVec];
            load_param(weight + c, w);
            if (bias) load_param(bias + c, bs);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                o[e] = v[n][e] * rstd * w[e] + (bias ? bs[e] : 0.f);
            store_vec(y + row * d + c, o);
        }
    }
}

// As above; the columns' sums stay in registers over all rows of a block and leave as one
// row of part [gridDim.x][2 d] (dweight, then dbias).
template <typename Tin, int NV, bool Sub>
__global__ void __launch_bounds__(Sub ? kSubThreads : 1024)
layer_norm_backward_kernel(const Tin* __restrict__ x, const float* __restrict__ weight,
                           const float* __restrict__ mean, const float* __restrict__ rstd,
                           const Tin* dy, Tin* dx, float* __restrict__ part, long long rows,
                           int d, int tpr) {
    __shared__ float2 sm[2][32];
    __shared__ float acc_sm[Sub ? kSubThreads * kVec : 1];
    const int rpb = Sub ? kSubThreads / tpr : 1;
    const int sub = Sub ? threadIdx.x / tpr : 0, lane = Sub ? threadIdx.x % tpr : threadIdx.x;
    float w[NV][kVec], dw[NV][kVec], db[NV][kVec];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = kVec * (lane + n * tpr);
#pragma unroll
        for (int e = 0; e < kVec; ++e) w[n][e] = dw[n][e] = db[n][e] = 0.f;
        if (c < d) load_param(weight + c, w[n]);
    }
    int buf = 0;
    const float inv = 1.0f / (float)d;
    for (long long base = (long long)blockIdx.x * rpb; base < rows;
         base += (long long)gridDim.x * rpb, buf ^= 1) {
        const long long row = base + sub;
        const bool live = row < rows;
        const float mu = live ? mean[row] : 0.f, rs = live ? rstd[row] : 0.f;
        float xh[NV][kVec], g[NV][kVec];
        float2 m = make_float2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (lane + n * tpr);
            if (live && c < d) {
                load_vec(x + row * d + c, xh[n]);
                load_vec(dy + row * d + c, g[n]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) xh[n][e] = mu, g[n][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                xh[n][e] = (xh[n][e] - mu) * rs;
                dw[n][e] += g[n][e] * xh[n][e];
                db[n][e] += g[n][e];
                g[n][e] *= w[n][e];
                m.x += g[n][e];
                m.y += g[n][e] * xh[n][e];
            }
        }
        m = row_sum<Sub>(m, tpr, sm[buf]);
        m.x *= inv;
        m.y *= inv;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (lane + n * tpr);
            if (!live || c >= d) continue;
            float o[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) o[e] = rs * (g[n][e] - m.x - xh[n][e] * m.y);
            store_vec(dx + row * d + c, o);
        }
    }
    float* out = part + (size_t)blockIdx.x * 2 * d;
    if constexpr (Sub) {
        // the groups of lanes that took other rows hold the same columns
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kVec; ++e) acc_sm[e * kSubThreads + threadIdx.x] = k ? db[0][e] : dw[0][e];
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += kSubThreads) {
                float s = 0.f;
                for (int q = 0; q < rpb; ++q) s += acc_sm[(c % kVec) * kSubThreads + q * tpr + c / kVec];
                out[k * d + c] = s;
            }
        }
    } else {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (lane + n * tpr);
            if (c >= d) continue;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                out[c + e] = dw[n][e];
                out[d + c + e] = db[n][e];
            }
        }
    }
}

// How rows of d values are laid out over threads.
struct Shape {
    int threads, tpr, nv, rpb;
    bool sub;
};
Shape shape_of(int d) {
    Shape s;
    const int vecs = (d + kVec - 1) / kVec;
    s.sub = d <= kSubMaxD;
    if (s.sub) {
        s.tpr = 1;
        while (s.tpr < vecs) s.tpr *= 2;
        s.threads = kSubThreads;
        s.nv = 1;
        s.rpb = kSubThreads / s.tpr;
    } else {
        s.nv = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
        s.threads = ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
        s.tpr = s.threads;
        s.rpb = 1;
    }
    return s;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    return n;
}

// Blocks of a grid-stride pass: 1024 threads' worth per SM, at most one row group each.
unsigned grid_of(const Shape& s, long long rows) {
    const long long need = (rows + s.rpb - 1) / s.rpb;
    const long long fit = (long long)sm_count() * std::max(1, 1024 / s.threads);
    return (unsigned)std::min(need, fit);
}

template <typename Tin>
cudaError_t forward(const LayerNormParams& p, cudaStream_t stream) {
    const Shape s = shape_of(p.d);
    const unsigned grid = grid_of(s, p.rows);
    const Tin* x = static_cast<const Tin*>(p.x);
    Tin* y = static_cast<Tin*>(p.y);
    auto go = [&](auto kernel) {
        kernel<<<grid, s.threads, 0, stream>>>(x, p.weight, p.bias, y, p.mean, p.rstd, p.rows,
                                               p.d, s.tpr, p.eps);
    };
    if (s.sub) go(layer_norm_kernel<Tin, 1, true>);
    else if (s.nv == 1) go(layer_norm_kernel<Tin, 1, false>);
    else if (s.nv == 2) go(layer_norm_kernel<Tin, 2, false>);
    else go(layer_norm_kernel<Tin, 4, false>);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t backward(const LayerNormGrads& p, const Shape& s, unsigned grid, float* part,
                     cudaStream_t stream) {
    const Tin* x = static_cast<const Tin*>(p.x);
    const Tin* dy = static_cast<const Tin*>(p.grad_y);
    Tin* dx = static_cast<Tin*>(p.grad_x);
    auto go = [&](auto kernel) {
        kernel<<<grid, s.threads, 0, stream>>>(x, p.weight, p.mean, p.rstd, dy, dx, part, p.rows,
                                               p.d, s.tpr);
    };
    if (s.sub) go(layer_norm_backward_kernel<Tin, 1, true>);
    else if (s.nv == 1) go(layer_norm_backward_kernel<Tin, 1, false>);
    else if (s.nv == 2) go(layer_norm_backward_kernel<Tin, 2, false>);
    else go(layer_norm_backward_kernel<Tin, 4, false>);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& p, cudaStream_t stream) {
    if (p.rows == 0) return cudaSuccess;
    return p.in == InType::BF16 ? forward<__nv_bfloat16>(p, stream) : forward<float>(p, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormGrads& p, cudaStream_t stream) {
    if (p.rows == 0)  // the sums over no rows
        return launch_column_sum(nullptr, 0, 2 * p.d, p.grad_weight, p.d, p.grad_bias, stream);
    const Shape s = shape_of(p.d);
    const unsigned grid = grid_of(s, p.rows);
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * grid * 2 * p.d, stream);
    if (e != cudaSuccess) return e;
    e = p.in == InType::BF16 ? backward<__nv_bfloat16>(p, s, grid, part, stream)
                             : backward<float>(p, s, grid, part, stream);
    if (e == cudaSuccess)
        e = launch_column_sum(part, grid, 2 * p.d, p.grad_weight, p.d, p.grad_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace gdr

// mixer_grad.cu -- the backward passes of the steps on either side of the rule
// (mixer_io.cu holds the forward ones):
//   conv   s_t = bias + sum_{i<4} w_i x_{t-3+i},  y = SiLU(s):
//              ds_t = dy_t sig(s_t) (1 + s_t (1 - sig(s_t)))
//              dx_t = sum_i w_i ds_{t+3-i},  dw_i = sum_t ds_t x_{t-3+i},  dbias = sum_t ds_t;
//          the three inputs before the call (the state) get the same sum, and the gradient of
//          the state after the call goes to the inputs it copies.
//   norm   y = o r w SiLU(z),  r = 1 / sqrt(mean(o^2) + eps),  q = dy w SiLU(z):
//              do = r (q - n mean(q n)),  dz = dy n w SiLU'(z),  dw = sum_rows dy n SiLU(z),  n = o r.
// Both are bound by memory: every input is read once, s and r are computed again instead of
// being kept by the forward pass.  Parameter gradients leave each CTA as one row of partial
// sums, which column_sum.cu adds in a fixed order.
#include <algorithm>

#include "gdr_common.cuh"
#include "gdr_internal.h"
#include "tcgen05.cuh"
#include "tma_map.h"

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

// For fp32 gradients: 2^(-v log2 e) from the special-function unit would carry the rounding of the
// product, 2e-6 of the value for far gates; its reciprocal is good to an ulp.  ([393216, 128] with a
// bf16 gate stays at 150 us with a cold L2; with a division 158.)
__device__ __forceinline__ float sigmoid(float v) { return rcpg(1.0f + expf(-v)); }

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
constexpr int kGWarps = 8;    // segments of tokens per CTA, one per warp
constexpr int kGCh = 128;     // channels per CTA: four per lane
constexpr int kGBatch = 8;    // tokens per batch of loads
constexpr int kGRing = 3;     // batches in shared memory: one in use, two in flight
constexpr int kGMinSeg = 32;  // tokens of a segment; three more on each side are read again

__device__ __forceinline__ float2 bf2(uint32_t u) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Two adjacent channels walking along time: the taps, the three inputs and the three ds before
// the current token, and the sums of the parameters' gradients.  Taps and bias are held times
// -log2 e, so that they give the exponent m = -s log2 e of the sigmoid; ds times -ln 2, so
// that dx, of products of a tap and a ds, needs no scale, and the sums one at the end.
struct ConvLane {
    float2 w[kW], bias;
    float2 h0, h1, h2;  // x at t - 3, t - 2, t - 1
    float2 d0, d1, d2;  // ds likewise
    float2 sum_w[kW], sum_b;

    // ds of the token with input v and output gradient g, times -ln 2
    __device__ __forceinline__ float2 slope(float2 v, float2 g) const {
        float2 m = __ffma2_rn(w[0], h0, bias);
        m = __ffma2_rn(w[1], h1, m);
        m = __ffma2_rn(w[2], h2, m);
        m = __ffma2_rn(w[3], v, m);
        // SiLU'(s) = r (1 + s (1 - r)), r = sigmoid(s) = 1 / (1 + 2^m)
        const float2 den = __fadd2_rn(make_float2(ex2g(m.x), ex2g(m.y)), splat(1.f));
        const float2 r = make_float2(rcpg(den.x), rcpg(den.y));
        const float2 q = __ffma2_rn(m, __ffma2_rn(r, splat(-kLn2 * kLn2), splat(kLn2 * kLn2)),
                                    splat(-kLn2));
        return __fmul2_rn(g, __fmul2_rn(r, q));
    }
    __device__ __forceinline__ void add(float2 v, float2 d) {
        sum_w[0] = __ffma2_rn(d, h0, sum_w[0]);
        sum_w[1] = __ffma2_rn(d, h1, sum_w[1]);
        sum_w[2] = __ffma2_rn(d, h2, sum_w[2]);
        sum_w[3] = __ffma2_rn(d, v, sum_w[3]);
        sum_b = __fadd2_rn(sum_b, d);
    }
    // the gradient of the input three tokens back, which has all its terms with this token's d
    __device__ __forceinline__ float2 out(float2 d) const {
        float2 o = __fmul2_rn(w[3], d0);
        o = __ffma2_rn(w[2], d1, o);
        o = __ffma2_rn(w[1], d2, o);
        return __ffma2_rn(w[0], d, o);
    }
    __device__ __forceinline__ void shift(float2 v, float2 d) {
        h0 = h1; h1 = h2; h2 = v;
        d0 = d1; d1 = d2; d2 = d;
    }
};

// Set by a kernel that gave up a bounded wait; gdr_device_status reads it.
__device__ int g_mixer_grad_status;

// x and dy of kGBatch tokens of a warp's 128 channels, each by one TMA copy.
struct alignas(128) ConvBatch {
    uint2 x[kGBatch][32], g[kGBatch][32];
};
struct ConvMaps {
    CUtensorMap x, g;
};
union ConvBackwardSmem {
    ConvBatch ring[kGWarps][kGRing];
    float sums[kGWarps][5][kGCh];
};

// CTA -> (channel tile, group of 8 segments of the B * nseg segments); warp -> segments of
// `seg` tokens, lane -> four channels, one token after the other, its loads two batches
// ahead (held in registers, one batch at a time, the loads' latency showed: 0.6 of HBM; by
// asynchronous copies of eight bytes per lane they cost a tenth of the instructions).
// [1, 8192, 18432] takes 177 us with a cold L2 and 184 among other passes (0.78 and 0.75 of a
// copy's rate), [8, 2048, 4096] 89 us (0.69): 89 instructions per token and four channels use 53 %
// of the issue slots and 53 % of the fp32 pipe ([1, 2048, 18432]).  With four warps per scheduler
// the largest stall is the wait for a dependent result, and registers allow no more warps.  (Two channels per
// lane and twice the warps: 228 us; one reciprocal for two channels, with the minima that keep
// the product finite: 189.)
// part [groups][5 C]: the taps' sums as [C][4], then the bias's.
template <bool Loop>
__global__ void __launch_bounds__(32 * kGWarps, 2)
conv_backward_kernel(const __grid_constant__ ConvMaps maps, ConvGrads p, int nct, int nseg, int seg,
                     int groups, float* part) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ uint64_t bars[kGWarps][kGRing];
    ConvBackwardSmem& smem = *reinterpret_cast<ConvBackwardSmem*>(smem_raw);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint64_t* full = bars[warp];  // a warp's own: its ring needs no barrier of the block
    if (lane == 0) {
        for (int i = 0; i < kGRing; ++i) tc::mbar_init(&full[i], 1);
        tc::mbar_init_fence();
    }
    __syncwarp();
    bool dead = false;
    int issued = 0, taken = 0;  // batches copied (lane 0's), batches waited for
    const int ct = blockIdx.x % nct, group = blockIdx.x / nct;
    // lanes behind the last channel go along on the tile's first ones and store nothing
    const bool in_c = ct * kGCh + 4 * lane < p.C;
    const int c = ct * kGCh + (in_c ? 4 * lane : 0);
    const long long segments = (long long)p.B * nseg;
    const float2 zero = splat(0.f);
    ConvLane a[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        a[k].sum_b = a[k].d0 = a[k].d1 = a[k].d2 = zero;
#pragma unroll
        for (int i = 0; i < kW; ++i) a[k].sum_w[i] = zero;
    }
    // this warp's segments: one, unless (Loop) there are more than the grid's groups take
    for (long long sid = (long long)group * kGWarps + warp; sid < segments;
         sid = Loop ? sid + (long long)groups * kGWarps : segments) {
        const int b = (int)(sid / nseg), T = p.T, C = p.C;
        const int t0 = (int)(sid % nseg) * seg, t1 = min(T, t0 + seg);
        const size_t base = (size_t)b * T * C + c;
        const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(p.x) + base;
        __nv_bfloat16* dx = static_cast<__nv_bfloat16*>(p.grad_x) + base;
        const size_t st = ((size_t)b * C + c) * 3;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 u = *reinterpret_cast<const float4*>(p.weight + (size_t)(c + 2 * k) * kW);
            const float4 v = *reinterpret_cast<const float4*>(p.weight + (size_t)(c + 2 * k + 1) * kW);
            a[k].w[0] = __fmul2_rn(make_float2(u.x, v.x), splat(-kLog2e));
            a[k].w[1] = __fmul2_rn(make_float2(u.y, v.y), splat(-kLog2e));
            a[k].w[2] = __fmul2_rn(make_float2(u.z, v.z), splat(-kLog2e));
            a[k].w[3] = __fmul2_rn(make_float2(u.w, v.w), splat(-kLog2e));
            a[k].d0 = a[k].d1 = a[k].d2 = zero;
            a[k].bias = p.bias ? __fmul2_rn(make_float2(p.bias[c + 2 * k], p.bias[c + 2 * k + 1]),
                                            splat(-kLog2e))
                               : zero;
        }
        // the three inputs before the segment: x, or the state (oldest first)
        float2 h[3][2];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int t = t0 - 3 + j;
            h[j][0] = h[j][1] = zero;
            if (t >= 0) {
                const uint2 u = *reinterpret_cast<const uint2*>(x + (size_t)t * C);
                h[j][0] = bf2(u.x);
                h[j][1] = bf2(u.y);
            } else if (p.state_in) {
                const float* s = p.state_in + st + t + 3;
                h[j][0] = make_float2(s[0], s[3]);
                h[j][1] = make_float2(s[6], s[9]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) a[k].h0 = h[0][k], a[k].h1 = h[1][k], a[k].h2 = h[2][k];

        // one token: ds, the sums (`sum`), the input three tokens back
        auto token = [&](uint2 ux, uint2 ug, bool sum) {
            const float2 v[2] = {bf2(ux.x), bf2(ux.y)};
            const float2 d[2] = {a[0].slope(v[0], bf2(ug.x)), a[1].slope(v[1], bf2(ug.y))};
            if (sum) {
                a[0].add(v[0], d[0]);
                a[1].add(v[1], d[1]);
            }
            const float4 o = make_float4(a[0].out(d[0]).x, a[0].out(d[0]).y, a[1].out(d[1]).x,
                                         a[1].out(d[1]).y);
            a[0].shift(v[0], d[0]);
            a[1].shift(v[1], d[1]);
            return o;
        };
        ConvBatch* ring = smem.ring[warp];
        const int end = min(T, t1 + 3);  // tokens read: three past the segment
        auto fetch = [&](int t) {  // lane 0; rows behind `end` come too, and are not used
            if (t >= end || dead) return;
            ConvBatch& to = ring[issued % kGRing];
            uint64_t* bar = &full[issued % kGRing];
            tc::mbar_arrive_expect_tx(bar, (uint32_t)sizeof(ConvBatch));
            tc::tma_load_2d(&to.x[0][0], &maps.x, ct * kGCh, b * T + t, bar);
            tc::tma_load_2d(&to.g[0][0], &maps.g, ct * kGCh, b * T + t, bar);
            ++issued;
        };
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < kGRing - 1; ++k) fetch(t0 + k * kGBatch);
        }
#pragma unroll 1
        for (int t = t0; t < t1 + 3; t += kGBatch) {
            __syncwarp();  // every lane has read the batch before: its slot takes the one two ahead
            if (lane == 0) fetch(t + (kGRing - 1) * kGBatch);
            const int slot = taken % kGRing;
            if (t < end) {
                if (!dead && !tc::mbar_wait(&full[slot], (uint32_t)(taken / kGRing) & 1u)) {
                    dead = true;
                    if (lane == 0) atomicExch(&g_mixer_grad_status, 1);
                }
                ++taken;
            }
            __syncwarp();
            const ConvBatch& now = ring[slot];
            __nv_bfloat16* op = dx + ((ptrdiff_t)t - 3) * C;
            if (t > t0 && t + kGBatch <= t1) {
#pragma unroll
                for (int i = 0; i < kGBatch; ++i) {
                    const float4 o = token(now.x[i][lane], now.g[i][lane], true);
                    const float f[4] = {o.x, o.y, o.z, o.w};
                    if (in_c) __stcs(reinterpret_cast<uint2*>(op + (size_t)i * C), pack4(f));
                }
                continue;
            }
            // the first batch, and those that reach the segment's end (past T: zeros)
#pragma unroll 1
            for (int i = 0; i < kGBatch; ++i) {
                const int u = t + i - 3;
                if (u >= t1) break;
                uint2 ux = make_uint2(0, 0), ug = ux;
                if (t + i < end) {
                    ux = now.x[i][lane];
                    ug = now.g[i][lane];
                }
                const float4 o = token(ux, ug, t + i < t1);
                if ((u < t0 && t0 > 0) || !in_c) continue;  // another segment's, or nobody's
                float f[4] = {o.x, o.y, o.z, o.w};
                // the state after the call holds the inputs T - 3 .. T - 1
                if (p.grad_state_out && u >= T - 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] += p.grad_state_out[st + 3 * e + u - (T - 3)];
                }
                if (u >= 0) {
                    __stcs(reinterpret_cast<uint2*>(op + (size_t)i * C), pack4(f));
                } else if (p.grad_state_in) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) p.grad_state_in[st + 3 * e + u + 3] = f[e];
                }
            }
        }
    }
    if (dead && lane == 0)  // copies may still be in flight: the CTA stays for them
        for (int k = max(0, issued - kGRing); k < issued; ++k)
            tc::mbar_wait(&full[k % kGRing], (uint32_t)(k / kGRing) & 1u);
    __syncthreads();  // the ring is done with: its memory takes the sums
    float(*sm)[5][kGCh] = smem.sums;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int ch = 4 * lane + 2 * k;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            sm[warp][i][ch] = a[k].sum_w[i].x;
            sm[warp][i][ch + 1] = a[k].sum_w[i].y;
        }
        sm[warp][4][ch] = a[k].sum_b.x;
        sm[warp][4][ch + 1] = a[k].sum_b.y;
    }
    __syncthreads();
    float* row = part + (size_t)group * 5 * p.C;
    for (int k = threadIdx.x; k < 5 * kGCh; k += blockDim.x) {
        const int i = k / kGCh, ch = k % kGCh, cc = ct * kGCh + ch;
        if (cc >= p.C) continue;
        float s = 0.f;
#pragma unroll
        for (int wi = 0; wi < kGWarps; ++wi) s += sm[wi][i][ch];
        row[i < kW ? (size_t)cc * kW + i : (size_t)kW * p.C + cc] = s * -kLog2e;
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
// time, grid-stride.  part [gridDim.x][d].  [393216, 128] with a bf16 gate takes 142 us with its
// column sums (0.86 of a copy's rate), the kernel alone 0.90: memory bounds it.
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
            const float sg = sigmoid(zv[e]);
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
        // n = o r before it meets anything else: powers of r leave fp32's range (r^3 is zero for
        // rows of 1e15, infinite for rows of 1e-13) where the gradient does not
        const float r = 1.0f / sqrtf(ss / (float)D + p.eps);
        const float m = r * (qo / (float)D);
        float go[4], gz[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float n = o[e] * r, gn = g[e] * n;
            go[e] = r * (q[e] - n * m);
            gz[e] = gn * w[e] * dsilu[e];
            if (live) acc[e] += gn * silu[e];
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
    // Segments: for one to eight waves of CTAs, the most segments that they hold, and of these
    // the number that takes the fewest token steps (a segment costs some 24 beside its own).
    const int nct = (p.C + kGCh - 1) / kGCh;
    const long long slots = 2LL * device_sms();
    int seg = 0, nseg = 0;
    long long best = 0;
    for (int waves = 1; waves <= 8; ++waves) {
        const long long most = std::max<long long>(1, waves * slots / nct * kGWarps / p.B);
        const long long len = std::max<long long>(
            kGMinSeg, ((p.T + most - 1) / most + kGBatch - 1) / kGBatch * kGBatch);
        const long long n = (p.T + len - 1) / len;
        const long long ctas = (p.B * n + kGWarps - 1) / kGWarps * nct;
        const long long cost = (ctas + slots - 1) / slots * (std::min<long long>(len, p.T) + 24);
        if (!seg || cost < best) seg = (int)len, nseg = (int)n, best = cost;
    }
    // at most eight waves of CTAs, which bounds the partial sums too
    const long long all = ((long long)p.B * nseg + kGWarps - 1) / kGWarps;
    const long long groups = std::min(all, std::max<long long>(1, 8 * slots / nct));
    if (groups * nct > 0x7fffffffLL) return cudaErrorNotSupported;
    ConvMaps maps;
    const uint64_t rows = (uint64_t)p.B * p.T;
    if (!make_map_pitched(&maps.x, p.x, false, p.C, rows, p.C, kGCh, kGBatch) ||
        !make_map_pitched(&maps.g, p.grad_y, false, p.C, rows, p.C, kGCh, kGBatch))
        return cudaErrorNotSupported;
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * groups * 5 * p.C, stream);
    if (e != cudaSuccess) return e;
    auto kernel = groups < all ? conv_backward_kernel<true> : conv_backward_kernel<false>;
    e = allow_smem((const void*)kernel, sizeof(ConvBackwardSmem));
    if (e == cudaSuccess) {
        kernel<<<(unsigned)(groups * nct), 32 * kGWarps, sizeof(ConvBackwardSmem), stream>>>(
            maps, p, nct, nseg, seg, (int)groups, part);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess)
        e = launch_column_sum(part, groups, 5 * p.C, p.grad_weight, 4 * p.C, p.grad_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

cudaError_t launch_gated_rmsnorm_backward(const NormGrads& p, cudaStream_t stream) {
    if (p.rows == 0) return launch_column_sum(nullptr, 0, p.d, p.grad_weight, p.d, nullptr, stream);
    const long long rpb = kNThreads / (p.d / 4);
    const unsigned grid = (unsigned)std::min<long long>((p.rows + rpb - 1) / rpb, (long long)device_sms() * 8);
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

int read_and_clear_mixer_grad_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_mixer_grad_status, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_mixer_grad_status, &zero, sizeof(int));
    }
    return v;
}

}  // namespace gdr

// layer_norm.cu -- layer normalisation of rows of d values in front of the mixer, and its
// backward pass with the reduction of the weight's and bias's gradients over the rows:
//     y  = xh * weight + bias,  xh = (x - mean) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//     dx = rstd * (dyw - mean(dyw) - xh * mean(dyw * xh)),  dyw = dy * weight
//     dweight = sum_rows dy * xh,  dbias = sum_rows dy.
// Both are bound by memory (forward: x in, y out; backward: x, dy in, dx out), and a row is
// read once.  The variance is taken from the centred values (a second pass over registers),
// which keeps its accuracy where the mean is far from zero.
#include <algorithm>

#include "gdr_common.cuh"
#include "gdr_internal.h"
#include "tcgen05.cuh"

namespace gdr {

namespace {

// Set by a backward kernel that gave up a bounded wait; gdr_device_status reads it.
__device__ int g_layer_norm_status;

constexpr int kVec = 8;  // adjacent values per thread and vector

// Eight values as loaded: four registers of bf16 pairs, or eight of fp32.
template <typename Tin>
struct Raw;
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void lds(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void pin() {}
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        v[0] = make_float2(a.x, a.y);
        v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y);
        v[3] = make_float2(b.z, b.w);
    }
};
template <>
struct Raw<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        u = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void lds(const __nv_bfloat16* p) {
        u = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    // What follows expands the packed values anew; the compiler would otherwise keep the
    // expanded ones from one pass over them to the next, in twice the registers.
    __device__ __forceinline__ void pin() {
        asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
    }
    __device__ __forceinline__ void get(float2 (&v)[4]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    }
};
__device__ __forceinline__ void store_vec(float* p, const float2 (&v)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(v[i].x, v[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void load_param(const float* p, float2 (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ float2 bcast2(float v) { return make_float2(v, v); }

// s / d from inv = 1 / d rounded: the product and one correction by its remainder (a row of one
// value keeps that value as its mean), a third of a division's instructions.
__device__ __forceinline__ float mean_of(float s, float d, float inv) {
    const float q = s * inv;
    return fabsf(q) < INFINITY ? fmaf(fmaf(-q, d, s), inv, q) : q;
}
// 1 / sqrt(v): the special-function unit's estimate and one Newton step (not where they meet 0
// or infinity).
__device__ __forceinline__ float inv_sqrt(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v < INFINITY ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;
}

// Sum over `lanes` adjacent lanes (a power of two).
template <int lanes>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------------------------- forward
// A row belongs to L adjacent lanes, NV vectors each, L vectors apart, and stays in their
// registers as loaded (bf16 in pairs): no barrier, and a whole row of loads in flight per
// warp; U rows at a time where rows are short.  (One block per row, eight values per thread and
// two barriers, ran [8192, 6144] bf16 at 0.25 of HBM.)  Statistics, then y, re-expand the
// registers.  [65536, 768] bf16 45 us (0.68 of a copy's rate), [393216, 128] 51 us (0.60):
// bound by the shuffles and the scalar work of a row beside its few values.
template <typename Tin, int NV>
constexpr int kRawRegs = NV * (sizeof(Tin) == 2 ? 4 : 8);
template <typename Tin, int NV>
constexpr int kRowsAtOnce = kRawRegs<Tin, NV> <= 8 ? 4 : kRawRegs<Tin, NV> <= 16 ? 2 : 1;

// blocks of 128 threads per SM whose registers hold the raw values and ~32 more
template <typename Tin, int NV>
constexpr int kForwardBlocks = 512 / (kRawRegs<Tin, NV> * kRowsAtOnce<Tin, NV> + 32);

template <typename Tin, int NV, int L>
__global__ void __launch_bounds__(128, kForwardBlocks<Tin, NV>)
layer_norm_kernel(const Tin* x, const float* __restrict__ weight, const float* __restrict__ bias,
                  Tin* y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
                  long long rows, int d, float eps) {
    constexpr int U = kRowsAtOnce<Tin, NV>;
    const int lane = threadIdx.x % L, per = blockDim.x / L;
    const float inv = 1.0f / (float)d;
    extern __shared__ __align__(128) float params[];  // weight, then bias (zeros without one)
    for (int i = 4 * threadIdx.x; i < d; i += 4 * blockDim.x) {
        *reinterpret_cast<float4*>(params + i) = *reinterpret_cast<const float4*>(weight + i);
        *reinterpret_cast<float4*>(params + d + i) =
            bias ? *reinterpret_cast<const float4*>(bias + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    for (long long base = (long long)blockIdx.x * per * U; base < rows;
         base += (long long)gridDim.x * per * U) {
        const long long row0 = base + threadIdx.x / L;  // then per rows apart
        Raw<Tin> raw[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = row0 + u * per;
            const Tin* xp = x + row * d + kVec * lane;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                if (row < rows && kVec * (lane + n * L) < d)
                    raw[u][n].load(xp + n * L * kVec);
                else
                    raw[u][n].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = row0 + u * per;
            float2 s2 = bcast2(0.f), q2 = s2;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float2 v[4];
                raw[u][n].get(v);
                s2 = __fadd2_rn(s2, __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3])));
            }
            const float mean = mean_of(lane_sum<L>(s2.x + s2.y), (float)d, inv);
            const float2 neg = bcast2(-mean);
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float2 v[4];
                raw[u][n].pin();
                raw[u][n].get(v);
                if (kVec * (lane + n * L) < d) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = __fadd2_rn(v[e], neg);
                        q2 = __ffma2_rn(v[e], v[e], q2);
                    }
                }
            }
            const float rstd = inv_sqrt(fmaf(lane_sum<L>(q2.x + q2.y), inv, eps));
            if (row < rows && lane == 0) {
                if (mean_out) mean_out[row] = mean;
                if (rstd_out) rstd_out[row] = rstd;
            }
            Tin* yp = y + row * d + kVec * lane;
            const float2 r2 = bcast2(rstd);
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c = kVec * (lane + n * L);
                if (row < rows && c < d) {
                    float2 v[4], w[4], b[4];
                    raw[u][n].pin();
                    raw[u][n].get(v);
                    load_param(params + c, w);
                    load_param(params + d + c, b);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[e], neg), r2), w[e], b[e]);
                    store_vec(yp + n * L * kVec, v);
                }
            }
        }
    }
}

// Wide rows: a team of one to six warps (the block) per U rows, NV vectors per thread and row, so
// that a thread's share stays small enough for many teams per SM and each load of the
// parameters serves U rows.  [8192, 6144] bf16 takes 39 us (5.2 TB/s, 0.79 of a copy's rate;
// two thirds of the issue slots are used), [8192, 4096] fp32 51 us (0.80).  (A warp per row:
// 64 us at [8192, 6144] bf16, with 12 warps per SM and the parameters' loads twice the row's;
// its next row staged in shared memory: 72.)
template <typename Tin>
constexpr int kTeamRows = sizeof(Tin) == 2 ? 2 : 1;

template <int U>
__device__ __forceinline__ void team_sum(float (&v)[U], float (*sm)[U]) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, nw = blockDim.x / 32;
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = warp_sum(v[u]);
    if (nw == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) sm[warp][u] = v[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[u] = 0.f;
        for (int w = 0; w < nw; ++w) v[u] += sm[w][u];
    }
}

template <typename Tin, int NV>
__global__ void __launch_bounds__(192, 4)
layer_norm_team_kernel(const Tin* x, const float* __restrict__ weight,
                       const float* __restrict__ bias, Tin* y, float* __restrict__ mean_out,
                       float* __restrict__ rstd_out, long long rows, int d, float eps) {
    constexpr int U = kTeamRows<Tin>;
    __shared__ float sm[2][6][U];  // each sum has its own: one barrier per sum
    const int tid = threadIdx.x, T = blockDim.x;
    const float inv = 1.0f / (float)d;
    for (long long row0 = (long long)blockIdx.x * U; row0 < rows; row0 += (long long)gridDim.x * U) {
        Raw<Tin> raw[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int c = kVec * (tid + n * T);
                if (row0 + u < rows && c < d)
                    raw[u][n].load(x + (row0 + u) * d + c);
                else
                    raw[u][n].zero();
            }
        }
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 s2 = bcast2(0.f);
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float2 v[4];
                raw[u][n].get(v);
                s2 = __fadd2_rn(s2, __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3])));
            }
            mean[u] = s2.x + s2.y;
        }
        team_sum<U>(mean, sm[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] = mean_of(mean[u], (float)d, inv);
            const float2 neg = bcast2(-mean[u]);
            float2 q2 = bcast2(0.f);
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float2 v[4];
                raw[u][n].pin();
                raw[u][n].get(v);
                if (kVec * (tid + n * T) < d) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = __fadd2_rn(v[e], neg);
                        q2 = __ffma2_rn(v[e], v[e], q2);
                    }
                }
            }
            rstd[u] = q2.x + q2.y;
        }
        team_sum<U>(rstd, sm[1]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rstd[u] = inv_sqrt(fmaf(rstd[u], inv, eps));
            if (tid == u && row0 + u < rows) {
                if (mean_out) mean_out[row0 + u] = mean[u];
                if (rstd_out) rstd_out[row0 + u] = rstd[u];
            }
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * (tid + n * T);
            if (c < d) {
                float2 w[4], b[4];
                load_param(weight + c, w);
                if (bias) {
                    load_param(bias + c, b);
                } else {
                    b[0] = b[1] = b[2] = b[3] = bcast2(0.f);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float2 v[4];
                    raw[u][n].pin();
                    raw[u][n].get(v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = __fmul2_rn(__fadd2_rn(v[e], bcast2(-mean[u])), bcast2(rstd[u]));
                        v[e] = __ffma2_rn(v[e], w[e], b[e]);
                    }
                    if (row0 + u < rows) store_vec(y + (row0 + u) * d + c, v);
                }
            }
        }
    }
}

// Few rows: a block per row, NV vectors per thread.
__device__ __forceinline__ float block_sum(float v, float* sm) {
    v = warp_sum(v);
    const int lane = threadIdx.x % 32, nw = blockDim.x / 32;
    if (lane == 0) sm[threadIdx.x / 32] = v;
    __syncthreads();
    return warp_sum(lane < nw ? sm[lane] : 0.f);
}

template <typename Tin, int NV>
__global__ void __launch_bounds__(1024)
layer_norm_block_kernel(const Tin* x, const float* __restrict__ weight,
                        const float* __restrict__ bias, Tin* y, float* __restrict__ mean_out,
                        float* __restrict__ rstd_out, long long rows, int d, float eps) {
    __shared__ float sm[2][32];  // each sum has its own: one barrier per sum
    const int tpr = blockDim.x;
    const float inv = 1.0f / (float)d;
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        Raw<Tin> raw[NV];
        float2 s2 = bcast2(0.f), q2 = s2;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * ((int)threadIdx.x + n * tpr);
            if (c < d) raw[n].load(x + row * d + c); else raw[n].zero();
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float2 v[4];
            raw[n].get(v);
            s2 = __fadd2_rn(s2, __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3])));
        }
        const float mean = mean_of(block_sum(s2.x + s2.y, sm[0]), (float)d, inv);
        const float2 neg = bcast2(-mean);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float2 v[4];
            raw[n].pin();
            raw[n].get(v);
            if (kVec * ((int)threadIdx.x + n * tpr) < d) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = __fadd2_rn(v[e], neg);
                    q2 = __ffma2_rn(v[e], v[e], q2);
                }
            }
        }
        const float rstd = inv_sqrt(fmaf(block_sum(q2.x + q2.y, sm[1]), inv, eps));
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = kVec * ((int)threadIdx.x + n * tpr);
            if (c < d) {
                float2 v[4], w[4], b[4];
                raw[n].pin();
                raw[n].get(v);
                load_param(weight + c, w);
                if (bias) {
                    load_param(bias + c, b);
                } else {
                    b[0] = b[1] = b[2] = b[3] = bcast2(0.f);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[e], neg), bcast2(rstd)), w[e], b[e]);
                store_vec(y + row * d + c, v);
            }
        }
    }
}

// Backward, wide rows: thread -> kVec columns (NV times) of all its block's rows, so that the
// weight and the columns' sums stay in registers.  The block takes groups of up to kRingRows
// rows from a ring in shared memory (bulk copies: rows are contiguous), so the bytes in flight
// depend neither on registers nor on barriers; the values are expanded again after the
// barrier behind the two sums of each row instead of being held.  [8192, 6144] bf16 takes
// 67 us (0.69 of a copy's rate), [8192, 4096] fp32 80 us (0.77): the two barriers of a group
// and the sums between them, which one block per SM cannot overlap.  (Both phases of two
// groups per barrier: 98 us; one barrier per group, a slot refilled behind the next one: 74;
// a column's sums over a warp's rows by shared-memory atomics would add in no fixed order.)
constexpr int kRingRows = 4;

// Adds v[0 .. 7] over the warp: lane l ends with the sum of v[l % 8].  Each exchange halves
// the values a lane still carries: 9 shuffles instead of 40.
__device__ __forceinline__ float sum8(float (&v)[8], int lane) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float keep = lane & 4 ? v[k + 4] : v[k], send = lane & 4 ? v[k] : v[k + 4];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float keep = lane & 2 ? v[k + 2] : v[k], send = lane & 2 ? v[k] : v[k + 2];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, 2);
    }
    const float keep = lane & 1 ? v[1] : v[0], send = lane & 1 ? v[0] : v[1];
    float s = keep + __shfl_xor_sync(0xffffffffu, send, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 8);
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    return s;
}
// The block's eight sums, over its warps' rows of sm: lane l gets value l % 8.
__device__ __forceinline__ float total8(const float (*sm)[8], int nw, int lane) {
    float t = 0.f;
    for (int i = lane / 8; i < nw; i += 4) t += sm[i][lane % 8];
    t += __shfl_xor_sync(0xffffffffu, t, 8);
    t += __shfl_xor_sync(0xffffffffu, t, 16);
    return t;
}

// A block's groups of rows and their ring; T tensors per slot.  Slots are counted along
// instead of taken modulo their number: a 64-bit remainder costs as much as a row's work.
template <typename Tin, int T>
struct Ring {
    Tin* base;
    uint64_t* full;
    int stages, group_rows, d, mine, slot_elems;
    long long rows;
    int issued = 0, issue_slot = 0;
    __device__ __forceinline__ Ring(uint8_t* smem, uint64_t* bars, int stages_, int group_rows_,
                                    long long rows_, int d_)
        : base(reinterpret_cast<Tin*>(smem)), full(bars), stages(stages_), group_rows(group_rows_),
          d(d_), slot_elems(T * d_ * group_rows_), rows(rows_) {
        const long long groups = (rows + group_rows - 1) / group_rows;
        mine = (int)((groups - blockIdx.x + gridDim.x - 1) / gridDim.x);
    }
    __device__ __forceinline__ long long row0(int k) const {
        return (blockIdx.x + (long long)k * gridDim.x) * group_rows;
    }
    __device__ __forceinline__ int count(int k) const {  // 0 outside [0, mine)
        return k < 0 || k >= mine ? 0 : (int)min((long long)group_rows, rows - row0(k));
    }
    __device__ __forceinline__ int next(int slot) const { return slot + 1 == stages ? 0 : slot + 1; }
    // one thread: the next group's copies, if there is one
    __device__ __forceinline__ void issue(const Tin* a, const Tin* b) {
        if (issued >= mine) return;
        const uint32_t bytes = (uint32_t)count(issued) * (uint32_t)(d * sizeof(Tin));
        uint64_t* bar = &full[issue_slot];
        Tin* to = base + (size_t)issue_slot * slot_elems;
        const long long from = row0(issued) * d;
        tc::mbar_arrive_expect_tx(bar, T * bytes);
        tc::bulk_load(to, a + from, bytes, bar);
        if (T > 1) tc::bulk_load(to + d * group_rows, b + from, bytes, bar);
        ++issued;
        issue_slot = next(issue_slot);
    }
    // after a wait that gave up, copies may still be in flight: the block stays for them
    __device__ __forceinline__ void drain() const {
        for (int k = max(0, issued - stages); k < issued; ++k)
            tc::mbar_wait(&full[k % stages], (uint32_t)(k / stages) & 1u);
    }
};

// ------------------------------------------------------------------------------ backward
// part [gridDim.x][2 d]: each block's sums over its rows, dweight, then dbias.
template <typename Tin, int NV, int Threads>
__global__ void __launch_bounds__(Threads, Threads == 512 ? 1 : 2)
layer_norm_backward_kernel(const Tin* __restrict__ x, const float* __restrict__ weight,
                           const float* __restrict__ mean, const float* __restrict__ rstd,
                           const Tin* dy, Tin* dx, float* __restrict__ part, long long rows, int d,
                           int stages, int group_rows) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ float sums[2][Threads / 32][8];
    __shared__ uint64_t full[8];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, nw = blockDim.x / 32;
    Ring<Tin, 2> ring(smem_raw, full, stages, group_rows, rows, d);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
        tc::mbar_init_fence();
        for (int i = 0; i < stages; ++i) ring.issue(x, dy);
    }
    float2 w[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = kVec * (tid + n * (int)blockDim.x);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[n][e] = dw[n][e] = db[n][e] = bcast2(0.f);
        if (c < d) load_param(weight + c, w[n]);
    }
    __syncthreads();
    // statistics of group k + 1, loaded while group k is worked on: lane r those of row r
    float mu_next = 0.f, rs_next = 0.f;
    auto load_stats = [&](int k) {
        if (lane < ring.count(k)) {
            mu_next = -mean[ring.row0(k) + lane];
            rs_next = rstd[ring.row0(k) + lane];
        }
    };
    load_stats(0);
    bool dead = false;
    int slot = 0;
    uint32_t parity = 0;
    const float inv = 1.0f / (float)d;
    for (int k = 0; k < ring.mine; ++k) {
        const int n_rows = ring.count(k);
        float m[8], mu[kRingRows], rs[kRingRows];
#pragma unroll
        for (int r = 0; r < kRingRows; ++r) {
            mu[r] = __shfl_sync(0xffffffffu, mu_next, r);
            rs[r] = __shfl_sync(0xffffffffu, rs_next, r);
            m[2 * r] = m[2 * r + 1] = 0.f;
        }
        load_stats(k + 1);
        if (!dead && !tc::mbar_wait(&full[slot], parity)) {
            dead = true;
            if (lane == 0) atomicExch(&g_layer_norm_status, 1);
        }
        __syncwarp();
        const Tin *xs = ring.base + (size_t)slot * ring.slot_elems, *gs = xs + d * group_rows;
#pragma unroll
        for (int r = 0; r < kRingRows; ++r) {
            if (r < n_rows) {
                // xh = (x - mean) rstd, as in the forward pass: x rstd - mean rstd would leave the
                // rounding of mean rstd, which a row of one value (xh = 0) has nowhere else
                const float2 r2 = bcast2(rs[r]), shift = bcast2(mu[r]);
                float2 m1 = bcast2(0.f), m2 = m1;
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = kVec * (tid + n * (int)blockDim.x);
                    if (c < d) {
                        Raw<Tin> a, b;
                        a.lds(xs + r * d + c);
                        b.lds(gs + r * d + c);
                        float2 xv[4], g[4];
                        a.get(xv);
                        b.get(g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 xh = __fmul2_rn(__fadd2_rn(xv[e], shift), r2);
                            dw[n][e] = __ffma2_rn(g[e], xh, dw[n][e]);
                            db[n][e] = __fadd2_rn(db[n][e], g[e]);
                            const float2 q = __fmul2_rn(g[e], w[n][e]);
                            m1 = __fadd2_rn(m1, q);
                            m2 = __ffma2_rn(q, xh, m2);
                        }
                    }
                }
                m[2 * r] = m1.x + m1.y;
                m[2 * r + 1] = m2.x + m2.y;
            }
        }
        const float s = sum8(m, lane);
        if (lane < 8) sums[k & 1][warp][lane] = s;
        __syncthreads();
        const float t = total8(sums[k & 1], nw, lane) * -inv;
        Tin* dxp = dx + ring.row0(k) * d;
#pragma unroll
        for (int r = 0; r < kRingRows; ++r) {
            // dx = rstd (q - m1 - xh m2) as rstd (g w + (x - mean) k1 + n1); rstd^2 could overflow
            const float n1 = __shfl_sync(0xffffffffu, t, 2 * r);
            const float n2 = __shfl_sync(0xffffffffu, t, 2 * r + 1);
            if (r < n_rows) {
                const float2 r2 = bcast2(rs[r]), k1 = bcast2(n2 * rs[r]), k0 = bcast2(n1);
                const float2 shift = bcast2(mu[r]);
#pragma unroll
                for (int n = 0; n < NV; ++n) {
                    const int c = kVec * (tid + n * (int)blockDim.x);
                    if (c < d) {
                        Raw<Tin> a, b;
                        a.lds(xs + r * d + c);
                        b.lds(gs + r * d + c);
                        float2 xv[4], g[4];
                        a.get(xv);
                        b.get(g);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            g[e] = __fmul2_rn(__ffma2_rn(g[e], w[n][e], __ffma2_rn(__fadd2_rn(xv[e], shift), k1, k0)), r2);
                        store_vec(dxp + (long long)r * d + c, g);
                    }
                }
            }
        }
        __syncthreads();
        // every warp is done with the group: its slot takes the next one
        if (tid == 0 && !dead) ring.issue(x, dy);
        slot = ring.next(slot);
        if (slot == 0) parity ^= 1;
    }
    float* out = part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = kVec * (tid + n * (int)blockDim.x);
        if (c < d) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                *reinterpret_cast<float2*>(out + c + 2 * e) = dw[n][e];
                *reinterpret_cast<float2*>(out + d + c + 2 * e) = db[n][e];
            }
        }
    }
    if (dead && tid == 0) ring.drain();
}

// Narrow rows (d <= 256): L adjacent lanes per row, one vector each, U rows of loads in flight.
// [393216, 128] bf16 64 us (0.72 of a copy's rate).
constexpr int kNarrowThreads = 256, kNarrowRows = 4;

template <typename Tin, int L>
__global__ void __launch_bounds__(kNarrowThreads)
layer_norm_backward_narrow_kernel(const Tin* __restrict__ x, const float* __restrict__ weight,
                                  const float* __restrict__ mean, const float* __restrict__ rstd,
                                  const Tin* dy, Tin* dx, float* __restrict__ part, long long rows,
                                  int d) {
    constexpr int per = kNarrowThreads / L, U = kNarrowRows;
    __shared__ float acc[kVec][kNarrowThreads];
    const int lane = threadIdx.x % L, c = kVec * lane;
    const bool in = c < d;
    float2 w[4], dw[4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = dw[e] = db[e] = bcast2(0.f);
    if (in) load_param(weight + c, w);
    const float inv = 1.0f / (float)d;
    for (long long base = (long long)blockIdx.x * per * U; base < rows;
         base += (long long)gridDim.x * per * U) {
        Raw<Tin> a[U], b[U];
        float mu[U], rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * per + threadIdx.x / L;
            const bool live = row < rows;
            mu[u] = live ? mean[row] : 0.f;
            rs[u] = live ? rstd[row] : 0.f;
            a[u].zero();
            b[u].zero();
            if (live && in) {
                a[u].load(x + row * d + c);
                b[u].load(dy + row * d + c);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * per + threadIdx.x / L;
            const float2 r2 = bcast2(rs[u]), shift = bcast2(-mu[u]);
            float2 xh[4], g[4], m1 = bcast2(0.f), m2 = m1;
            a[u].get(xh);
            b[u].get(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xh[e] = __fmul2_rn(__fadd2_rn(xh[e], shift), r2);
                dw[e] = __ffma2_rn(g[e], xh[e], dw[e]);
                db[e] = __fadd2_rn(db[e], g[e]);
                g[e] = __fmul2_rn(g[e], w[e]);
                m1 = __fadd2_rn(m1, g[e]);
                m2 = __ffma2_rn(g[e], xh[e], m2);
            }
            const float2 n1 = bcast2(lane_sum<L>(m1.x + m1.y) * -inv);
            const float2 n2 = bcast2(lane_sum<L>(m2.x + m2.y) * -inv);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                g[e] = __fmul2_rn(__ffma2_rn(xh[e], n2, __fadd2_rn(g[e], n1)), r2);
            if (row < rows && in) store_vec(dx + row * d + c, g);
        }
    }
    // the groups of lanes that took other rows hold the same columns
    float* out = part + (size_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[2 * e][threadIdx.x] = k ? db[e].x : dw[e].x;
            acc[2 * e + 1][threadIdx.x] = k ? db[e].y : dw[e].y;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < d; i += kNarrowThreads) {
            float s = 0.f;
            for (int q = 0; q < per; ++q) s += acc[i % kVec][q * L + i / kVec];
            out[k * d + i] = s;
        }
    }
}

// Rows too wide for the ring (two slots, or 32 columns for each of 512 threads): the columns' sums by threads that keep eight columns
// over a slice of the rows, then dx by a block per row that reads it twice.
constexpr int kRingMaxD = 16384;

template <typename Tin>
__global__ void __launch_bounds__(128)
layer_norm_columns_kernel(const Tin* __restrict__ x, const float* __restrict__ mean,
                          const float* __restrict__ rstd, const Tin* __restrict__ dy,
                          float* __restrict__ part, long long rows, int d) {
    const int c = kVec * (blockIdx.x * 128 + threadIdx.x);
    if (c >= d) return;
    float2 dw[4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[e] = db[e] = bcast2(0.f);
    for (long long row = blockIdx.y; row < rows; row += gridDim.y) {
        Raw<Tin> a, b;
        a.load(x + row * d + c);
        b.load(dy + row * d + c);
        float2 xv[4], g[4];
        a.get(xv);
        b.get(g);
        const float2 r2 = bcast2(rstd[row]), shift = bcast2(-mean[row]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dw[e] = __ffma2_rn(g[e], __fmul2_rn(__fadd2_rn(xv[e], shift), r2), dw[e]);
            db[e] = __fadd2_rn(db[e], g[e]);
        }
    }
    float* out = part + (size_t)blockIdx.y * 2 * d + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2*>(out + 2 * e) = dw[e];
        *reinterpret_cast<float2*>(out + d + 2 * e) = db[e];
    }
}

template <typename Tin>
__global__ void __launch_bounds__(1024)
layer_norm_backward_wide_kernel(const Tin* __restrict__ x, const float* __restrict__ weight,
                                const float* __restrict__ mean, const float* __restrict__ rstd,
                                const Tin* dy, Tin* dx, long long rows, int d) {
    __shared__ float sm[2][32];
    for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
        const float2 r2 = bcast2(rstd[row]), shift = bcast2(-mean[row]);
        float2 m1 = bcast2(0.f), m2 = m1;
        for (int c = kVec * threadIdx.x; c < d; c += kVec * blockDim.x) {
            Raw<Tin> a, b;
            a.load(x + row * d + c);
            b.load(dy + row * d + c);
            float2 xv[4], g[4], w[4];
            a.get(xv);
            b.get(g);
            load_param(weight + c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 q = __fmul2_rn(g[e], w[e]);
                m1 = __fadd2_rn(m1, q);
                m2 = __ffma2_rn(q, __fmul2_rn(__fadd2_rn(xv[e], shift), r2), m2);
            }
        }
        const float2 n1 = bcast2(block_sum(m1.x + m1.y, sm[0]) / -(float)d);
        const float2 n2 = bcast2(block_sum(m2.x + m2.y, sm[1]) / -(float)d);
        for (int c = kVec * threadIdx.x; c < d; c += kVec * blockDim.x) {
            Raw<Tin> a, b;
            a.load(x + row * d + c);
            b.load(dy + row * d + c);
            float2 xv[4], g[4], w[4];
            a.get(xv);
            b.get(g);
            load_param(weight + c, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 xh = __fmul2_rn(__fadd2_rn(xv[e], shift), r2);
                g[e] = __fmul2_rn(__ffma2_rn(xh, n2, __ffma2_rn(g[e], w[e], n1)), r2);
            }
            store_vec(dx + row * d + c, g);
        }
    }
}

// Shared memory for rings, per SM; beside it each block needs its sums and barriers.
constexpr size_t kRoom = 212 * 1024;

// Rows per group and slots of a ring whose rows take `row` bytes per slot, for `blocks` blocks per
// SM: the most rows per group that leave `want` slots (a group's phases and one to fill).
struct RingShape {
    int group_rows, stages;
    RingShape(size_t row, int blocks, int want) {
        const size_t room = kRoom / blocks;
        group_rows = kRingRows;
        while (group_rows > 1 && want * group_rows * row > room) group_rows /= 2;
        stages = (int)std::min<size_t>(want, room / (group_rows * row));
    }
};

template <typename Tin>
cudaError_t forward(const LayerNormParams& p, cudaStream_t stream) {
    const Tin* x = static_cast<const Tin*>(p.x);
    Tin* y = static_cast<Tin*>(p.y);
    const int vecs = (p.d + kVec - 1) / kVec, sms = device_sms();
    // up to four rows per SM, and rows above 9216 columns: a block of up to 512 threads per row
    if (vecs > 1152 || (vecs > 128 && p.rows <= 4LL * sms)) {
        const int nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;  // at most 512 threads, to d = 16384
        const int threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
        const unsigned grid = (unsigned)std::min<long long>(p.rows, sms * 2LL);
        auto kernel = nv == 1   ? layer_norm_block_kernel<Tin, 1>
                      : nv == 2 ? layer_norm_block_kernel<Tin, 2>
                                : layer_norm_block_kernel<Tin, 4>;
        kernel<<<grid, threads, 0, stream>>>(x, p.weight, p.bias, y, p.mean, p.rstd, p.rows, p.d,
                                             p.eps);
        return cudaGetLastError();
    }
    auto go = [&](auto kernel, int L, int U, int blocks) {
        // few rows: one warp per block, to use more SMs
        const int threads = p.rows * L <= 128LL * sms * U ? 32 : 128;
        const long long per = (long long)threads / L * U, need = (p.rows + per - 1) / per;
        const size_t smem = 2 * sizeof(float) * p.d;  // 8 KB at most
        const unsigned grid =  // as many blocks as the SMs' registers hold, grid-stride
            (unsigned)std::min<long long>(need, (long long)sms * std::min(32, blocks * 128 / threads));
        kernel<<<grid, threads, smem, stream>>>(x, p.weight, p.bias, y, p.mean, p.rstd, p.rows, p.d,
                                                p.eps);
        return cudaGetLastError();
    };
    if (vecs <= 1) return go(layer_norm_kernel<Tin, 1, 1>, 1, kRowsAtOnce<Tin, 1>, kForwardBlocks<Tin, 1>);
    if (vecs <= 4) return go(layer_norm_kernel<Tin, 1, 4>, 4, kRowsAtOnce<Tin, 1>, kForwardBlocks<Tin, 1>);
    if (vecs <= 8) return go(layer_norm_kernel<Tin, 1, 8>, 8, kRowsAtOnce<Tin, 1>, kForwardBlocks<Tin, 1>);
    if (vecs <= 16) return go(layer_norm_kernel<Tin, 1, 16>, 16, kRowsAtOnce<Tin, 1>, kForwardBlocks<Tin, 1>);
    if (vecs <= 32) return go(layer_norm_kernel<Tin, 1, 32>, 32, kRowsAtOnce<Tin, 1>, kForwardBlocks<Tin, 1>);
    if (vecs <= 64) return go(layer_norm_kernel<Tin, 2, 32>, 32, kRowsAtOnce<Tin, 2>, kForwardBlocks<Tin, 2>);
    if (vecs <= 128) return go(layer_norm_kernel<Tin, 4, 32>, 32, kRowsAtOnce<Tin, 4>, kForwardBlocks<Tin, 4>);
    // teams of up to six warps, four to six vectors per thread
    const int warps = (vecs + 191) / 192, nv = (vecs + 32 * warps - 1) / (32 * warps);
    constexpr int U = kTeamRows<Tin>;
    auto kernel = nv <= 4   ? layer_norm_team_kernel<Tin, 4>
                  : nv == 5 ? layer_norm_team_kernel<Tin, 5>
                            : layer_norm_team_kernel<Tin, 6>;
    const unsigned grid =  // at most 85 registers a thread: 768 threads per SM, grid-stride
        (unsigned)std::min<long long>((p.rows + U - 1) / U, (long long)sms * (768 / (32 * warps)));
    kernel<<<grid, 32 * warps, 0, stream>>>(x, p.weight, p.bias, y, p.mean, p.rstd, p.rows, p.d, p.eps);
    return cudaGetLastError();
}

// Launches of the backward pass: how many blocks (= rows of partial sums) and on what.
template <typename Tin>
struct BackwardPlan {
    bool narrow, wide;
    int L, nv, threads, group_rows, stages;
    size_t smem;
    unsigned grid;
    explicit BackwardPlan(const LayerNormGrads& p) {
        const int vecs = (p.d + kVec - 1) / kVec;
        narrow = vecs <= 32;
        if (narrow) {
            L = vecs <= 1 ? 1 : vecs <= 4 ? 4 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32;
            const long long per = (long long)kNarrowThreads / L * kNarrowRows;
            grid = (unsigned)std::min<long long>((p.rows + per - 1) / per, (long long)device_sms() * 4);
            return;
        }
        wide = p.d > kRingMaxD || RingShape(2 * sizeof(Tin) * p.d, 1, 2).stages < 2;
        if (wide) {  // slices of rows, for two blocks per SM
            const long long across = (vecs + 127) / 128;
            grid = (unsigned)std::min<long long>(p.rows, std::max<long long>(1, 2 * device_sms() / across));
            return;
        }
        // 8 columns per thread up to 384 threads, several blocks per SM; above, 16 columns, two
        // blocks up to 256 threads and one above; then up to 32 columns in 512 threads.  A thread's
        // work per row (the shuffles, the scalars) is shared by its columns (6144 columns: 66 us;
        // 71 in 768 threads of 8 columns, 75 in two blocks and two rows per group; 4096 columns: 56
        // in two blocks, 62 in one).  Fewer blocks where they would leave each a single row per
        // group.
        nv = vecs <= 384 ? 1 : vecs <= 1024 ? 2 : 4;
        threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;
        const size_t row = 2 * sizeof(Tin) * p.d;  // x and dy
        int blocks = nv == 1 ? std::max(1, std::min(8, 768 / threads)) : threads <= 256 ? 2 : 1;
        while (blocks > 1 && RingShape(row, blocks, 2).group_rows < 2) --blocks;
        const RingShape ring(row, blocks, 2);
        group_rows = ring.group_rows;
        stages = ring.stages;
        smem = (size_t)stages * group_rows * row;
        const long long groups = (p.rows + group_rows - 1) / group_rows;
        grid = (unsigned)std::min<long long>(groups, (long long)blocks * device_sms());
    }
};

template <typename Tin>
cudaError_t backward(const LayerNormGrads& p, const BackwardPlan<Tin>& plan, float* part,
                     cudaStream_t stream) {
    const Tin* x = static_cast<const Tin*>(p.x);
    const Tin* dy = static_cast<const Tin*>(p.grad_y);
    Tin* dx = static_cast<Tin*>(p.grad_x);
    if (plan.narrow) {
        auto go = [&](auto kernel) {
            kernel<<<plan.grid, kNarrowThreads, 0, stream>>>(x, p.weight, p.mean, p.rstd, dy, dx,
                                                             part, p.rows, p.d);
        };
        switch (plan.L) {
            case 1: go(layer_norm_backward_narrow_kernel<Tin, 1>); break;
            case 4: go(layer_norm_backward_narrow_kernel<Tin, 4>); break;
            case 8: go(layer_norm_backward_narrow_kernel<Tin, 8>); break;
            case 16: go(layer_norm_backward_narrow_kernel<Tin, 16>); break;
            default: go(layer_norm_backward_narrow_kernel<Tin, 32>); break;
        }
        return cudaGetLastError();
    }
    if (plan.wide) {
        const dim3 grid((unsigned)((p.d + 128 * kVec - 1) / (128 * kVec)), plan.grid);
        layer_norm_columns_kernel<Tin><<<grid, 128, 0, stream>>>(x, p.mean, p.rstd, dy, part, p.rows, p.d);
        layer_norm_backward_wide_kernel<Tin><<<(unsigned)std::min<long long>(p.rows, 2LL * device_sms()),
                                               1024, 0, stream>>>(x, p.weight, p.mean, p.rstd, dy, dx,
                                                                  p.rows, p.d);
        return cudaGetLastError();
    }
    auto kernel = plan.nv == 4          ? layer_norm_backward_kernel<Tin, 4, 512>
                  : plan.nv == 1        ? layer_norm_backward_kernel<Tin, 1, 384>
                  : plan.threads <= 256 ? layer_norm_backward_kernel<Tin, 2, 256>
                                        : layer_norm_backward_kernel<Tin, 2, 512>;
    const cudaError_t e = allow_smem((const void*)kernel, plan.smem);
    if (e != cudaSuccess) return e;
    kernel<<<plan.grid, plan.threads, plan.smem, stream>>>(x, p.weight, p.mean, p.rstd, dy, dx, part,
                                                           p.rows, p.d, plan.stages, plan.group_rows);
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t backward(const LayerNormGrads& p, cudaStream_t stream) {
    const BackwardPlan<Tin> plan(p);
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * plan.grid * 2 * p.d, stream);
    if (e != cudaSuccess) return e;
    e = backward<Tin>(p, plan, part, stream);
    if (e == cudaSuccess)
        e = launch_column_sum(part, plan.grid, 2 * p.d, p.grad_weight, p.d, p.grad_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormParams& p, cudaStream_t stream) {
    if (p.rows == 0) return cudaSuccess;
    return p.in == InType::BF16 ? forward<__nv_bfloat16>(p, stream) : forward<float>(p, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormGrads& p, cudaStream_t stream) {
    if (p.rows == 0)  // the sums over no rows
        return launch_column_sum(nullptr, 0, 2 * p.d, p.grad_weight, p.d, p.grad_bias, stream);
    return p.in == InType::BF16 ? backward<__nv_bfloat16>(p, stream) : backward<float>(p, stream);
}

int read_and_clear_layer_norm_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_layer_norm_status, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_layer_norm_status, &zero, sizeof(int));
    }
    return v;
}

}  // namespace gdr

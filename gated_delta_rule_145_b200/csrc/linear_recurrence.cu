// linear_recurrence.cu -- the gated linear recurrence with a vector state: every channel c
// of every sequence keeps one fp32 value h and each token t does
//     h <- h * exp(g_t) + sigmoid(b_t) * x_t,     out_t = h,
//     g_t = -exp(A_log[c]) * softplus(a_t + dt_bias[c]),
// the gates of the gated delta rule on a diagonal state, and its backward pass:
//     D_t  = dout_t + exp(g_{t+1}) D_{t+1}     (the last token adds the final state's gradient)
//     dx_t = i_t D_t,   db_t = x_t D_t i_t (1 - i_t)         with i_t = sigmoid(b_t)
//     dg_t = exp(g_t) h_{t-1} D_t,   da_t = -exp(A_log) sigmoid(a_t + dt_bias) dg_t
//     dA_log = sum_t dg_t g_t,   ddt_bias = sum_t da_t,   dinit = exp(g_0) D_0.
// Both are bound by memory: forward reads x, a, b and writes h, backward reads x, a, b, h
// and dout and writes dx, da, db, each once.
#include <algorithm>

#include "gdr_common.cuh"
#include "gdr_internal.h"

namespace gdr {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 ex2f2(float2 v) { return make_float2(ex2f(v.x), ex2f(v.y)); }
__device__ __forceinline__ float2 rcpf2(float2 v) { return make_float2(rcpf(v.x), rcpf(v.y)); }
__device__ __forceinline__ float2 bcast2(float v) { return make_float2(v, v); }

// Two adjacent channels of one token, widened to fp32.
__device__ __forceinline__ float2 load_pair(const float* p) {
    return __ldcs(reinterpret_cast<const float2*>(p));
}
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* p) {
    const uint32_t u = __ldcs(reinterpret_cast<const unsigned int*>(p));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
__device__ __forceinline__ void store_pair(float* p, float2 v) {
    __stcs(reinterpret_cast<float2*>(p), v);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
    __stcs(reinterpret_cast<unsigned int*>(p), *reinterpret_cast<const uint32_t*>(&r));
}

// The gates of two channels.  A = -exp(A_log), A2 = A log2(e): the log-decay is kept in
// base 2, y = log2(e) g, as the special-function unit's exponential takes it.
struct Channels {
    float2 A, A2, bias;
};

// softplus(z) = max(z, 0) + log1p(t) with t = e^{-|z|} in (0, 1], and log1p(t) = t Q(t),
// Q the degree-8 polynomial whose largest relative error on [0, 1] is smallest (3e-8; a
// weighted least-squares fit).  Small values of softplus are slow channels, whose state
// sums over many tokens: there the relative error of g, not the absolute one, is what the
// result sees, so log(1 + t) from the special-function unit (absolute error) will not do.
__device__ __forceinline__ float2 log1p_poly2(float2 t) {
    float2 q = bcast2(5.232629366e-03f);
    q = __ffma2_rn(q, t, bcast2(-2.950498648e-02f));
    q = __ffma2_rn(q, t, bcast2(7.822556049e-02f));
    q = __ffma2_rn(q, t, bcast2(-1.366321445e-01f));
    q = __ffma2_rn(q, t, bcast2(1.910599321e-01f));
    q = __ffma2_rn(q, t, bcast2(-2.484297901e-01f));
    q = __ffma2_rn(q, t, bcast2(3.331909776e-01f));
    q = __ffma2_rn(q, t, bcast2(-4.999949336e-01f));
    q = __ffma2_rn(q, t, bcast2(9.999999404e-01f));
    return __fmul2_rn(q, t);
}

struct Gate {
    float2 z, t, p;  // a + dt_bias, e^{-|z|}, softplus(z)
};
__device__ __forceinline__ Gate decay_gate(float2 a, const Channels& ch) {
    Gate g;
    g.z = __fadd2_rn(a, ch.bias);
    g.t = ex2f2(make_float2(-fabsf(g.z.x) * kLog2e, -fabsf(g.z.y) * kLog2e));
    g.p = __fadd2_rn(make_float2(fmaxf(g.z.x, 0.f), fmaxf(g.z.y, 0.f)), log1p_poly2(g.t));
    return g;
}

__device__ __forceinline__ float2 sigmoid2(float2 b) {
    const float2 e = ex2f2(__fmul2_rn(b, bcast2(-kLog2e)));
    return rcpf2(__fadd2_rn(e, bcast2(1.f)));
}

// sigmoid(v) and 1 - sigmoid(v), both to full relative accuracy, from t = e^{-|v|}
__device__ __forceinline__ void sigmoid_both(float v, float t, float& s, float& c) {
    const float r = rcpf(1.f + t), tr = t * r;
    s = v >= 0.f ? r : tr;
    c = v >= 0.f ? tr : r;
}

__device__ __forceinline__ Channels load_channels(const float* A_log, const float* dt_bias,
                                                  int c) {
    Channels ch;
    ch.A = make_float2(-expf(A_log[c]), -expf(A_log[c + 1]));
    ch.A2 = __fmul2_rn(ch.A, bcast2(kLog2e));
    ch.bias = make_float2(dt_bias[c], dt_bias[c + 1]);
    return ch;
}

// Token range of sequence s, held within the T tokens of the call.
__device__ __forceinline__ void seq_bounds(const int32_t* cu, int s, int T, long long& t0,
                                           long long& t1) {
    seq_range(cu, s, T, t0, t1);
    if (cu) {
        t0 = min(max(t0, 0LL), (long long)T);
        t1 = min(max(t1, t0), (long long)T);
    }
}

// The gradients of one token's two channels, given D (the gradient of its h), the state
// before it and its inputs; acc_A and acc_bias take the parameters' gradients, and D becomes
// the gradient of the state before the token.
template <typename Tin>
__device__ __forceinline__ void grad_token(float2 x, float2 a, float2 b, float2 prev, float2& D,
                                           const Channels& ch, Tin* dx, Tin* da, Tin* db,
                                           float2& acc_A, float2& acc_bias) {
    const Gate g = decay_gate(a, ch);
    const float2 lam = ex2f2(__fmul2_rn(ch.A2, g.p));
    float2 sz, i, ci;
    float unused;
    sigmoid_both(g.z.x, g.t.x, sz.x, unused);
    sigmoid_both(g.z.y, g.t.y, sz.y, unused);
    sigmoid_both(b.x, ex2f(-fabsf(b.x) * kLog2e), i.x, ci.x);
    sigmoid_both(b.y, ex2f(-fabsf(b.y) * kLog2e), i.y, ci.y);
    const float2 vx = __fmul2_rn(i, D);
    const float2 vb = __fmul2_rn(__fmul2_rn(vx, x), ci);
    const float2 Dn = __fmul2_rn(lam, D);
    const float2 dg = __fmul2_rn(Dn, prev);
    const float2 dgA = __fmul2_rn(dg, ch.A);
    const float2 va = __fmul2_rn(dgA, sz);
    store_pair(dx, vx);
    store_pair(da, va);
    store_pair(db, vb);
    acc_A = __ffma2_rn(dgA, g.p, acc_A);
    acc_bias = __fadd2_rn(acc_bias, va);
    D = Dn;
}

// ------------------------------------------------------------- sequential form
// Thread -> two channels of the sequences s = blockIdx.y, + gridDim.y, ...; one token after
// the other, the state in registers.  For single tokens and short sequences, where there is
// nothing to split.
constexpr int kSeqThreads = 128;

template <typename Tin>
__global__ void __launch_bounds__(kSeqThreads)
recurrence_seq_kernel(RecurrenceParams p) {
    const int c = 2 * (blockIdx.x * kSeqThreads + threadIdx.x);
    if (c >= p.C) return;
    const Channels ch = load_channels(p.A_log, p.dt_bias, c);
    const Tin* x = static_cast<const Tin*>(p.x) + c;
    const Tin* a = static_cast<const Tin*>(p.a) + c;
    const Tin* b = static_cast<const Tin*>(p.b) + c;
    for (int s = blockIdx.y; s < p.nseq; s += gridDim.y) {
        long long t0, t1;
        seq_bounds(p.cu_seqlens, s, p.T, t0, t1);
        const size_t at = (size_t)s * p.C + c;
        float2 h = p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                : make_float2(0.f, 0.f);
#pragma unroll 4
        for (long long t = t0; t < t1; ++t) {
            const float2 xv = load_pair(x + t * p.ld), av = load_pair(a + t * p.ld),
                         bv = load_pair(b + t * p.ld);
            const Gate g = decay_gate(av, ch);
            const float2 lam = ex2f2(__fmul2_rn(ch.A2, g.p));
            h = __ffma2_rn(lam, h, __fmul2_rn(sigmoid2(bv), xv));
            store_pair(p.out + t * p.C + c, h);
        }
        if (p.final_state) *reinterpret_cast<float2*>(p.final_state + at) = h;
    }
}

// part [gridDim.y][2 C]: this row of CTAs' sums for A_log, then for dt_bias.
template <typename Tin>
__global__ void __launch_bounds__(kSeqThreads)
recurrence_seq_backward_kernel(RecurrenceParams p, RecurrenceGrads r, float* part) {
    const int c = 2 * (blockIdx.x * kSeqThreads + threadIdx.x);
    if (c >= p.C) return;
    const Channels ch = load_channels(p.A_log, p.dt_bias, c);
    const Tin* x = static_cast<const Tin*>(p.x) + c;
    const Tin* a = static_cast<const Tin*>(p.a) + c;
    const Tin* b = static_cast<const Tin*>(p.b) + c;
    Tin* dx = static_cast<Tin*>(r.grad_x) + c;
    Tin* da = static_cast<Tin*>(r.grad_a) + c;
    Tin* db = static_cast<Tin*>(r.grad_b) + c;
    float2 acc_A = make_float2(0.f, 0.f), acc_bias = make_float2(0.f, 0.f);
    for (int s = blockIdx.y; s < p.nseq; s += gridDim.y) {
        long long t0, t1;
        seq_bounds(p.cu_seqlens, s, p.T, t0, t1);
        const size_t at = (size_t)s * p.C + c;
        float2 D = r.grad_final ? *reinterpret_cast<const float2*>(r.grad_final + at)
                                : make_float2(0.f, 0.f);
        const float2 init = p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                         : make_float2(0.f, 0.f);
#pragma unroll 2
        for (long long t = t1 - 1; t >= t0; --t) {
            const float2 prev = t > t0 ? load_pair(p.out + (t - 1) * p.C + c) : init;
            D = __fadd2_rn(D, load_pair(r.grad_out + t * p.C + c));
            grad_token(load_pair(x + t * p.ld), load_pair(a + t * p.ld), load_pair(b + t * p.ld),
                       prev, D, ch, dx + t * r.ld_grad, da + t * r.ld_grad, db + t * r.ld_grad,
                       acc_A, acc_bias);
        }
        if (r.grad_init) *reinterpret_cast<float2*>(r.grad_init + at) = D;
    }
    float* row = part + (size_t)blockIdx.y * 2 * p.C;
    *reinterpret_cast<float2*>(row + c) = acc_A;
    *reinterpret_cast<float2*>(row + p.C + c) = acc_bias;
}

// Rows of CTAs of the sequential form: the partial sums have one row each.
int seq_rows(int nseq) { return std::min(nseq, 64); }

}  // namespace

cudaError_t launch_recurrence(const RecurrenceParams& p, cudaStream_t stream) {
    const dim3 grid((unsigned)((p.C / 2 + kSeqThreads - 1) / kSeqThreads),
                    (unsigned)std::min(p.nseq, 65535));
    if (p.in == InType::BF16)
        recurrence_seq_kernel<__nv_bfloat16><<<grid, kSeqThreads, 0, stream>>>(p);
    else
        recurrence_seq_kernel<float><<<grid, kSeqThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_recurrence_backward(const RecurrenceParams& p, const RecurrenceGrads& r,
                                       cudaStream_t stream) {
    const int rows = seq_rows(p.nseq);
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * rows * 2 * p.C, stream);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)((p.C / 2 + kSeqThreads - 1) / kSeqThreads), (unsigned)rows);
    if (p.in == InType::BF16)
        recurrence_seq_backward_kernel<__nv_bfloat16><<<grid, kSeqThreads, 0, stream>>>(p, r, part);
    else
        recurrence_seq_backward_kernel<float><<<grid, kSeqThreads, 0, stream>>>(p, r, part);
    e = cudaGetLastError();
    if (e == cudaSuccess)
        e = launch_column_sum(part, rows, 2 * p.C, r.grad_A_log, p.C, r.grad_dt_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace gdr

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
#include <atomic>

#include "gdr_common.cuh"
#include "gdr_internal.h"
#include "tcgen05.cuh"
#include "tma_map.h"

namespace gdr {

namespace {

// Set by a tiled kernel that gave up a bounded wait; gdr_device_status reads it.
__device__ int g_recurrence_status;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);

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
// The larger and the smaller of two; a NaN stays one (fmaxf and fminf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float m;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
// The decay 2^y of a token or of several: never zero, so that an infinite state stays infinite in
// every form and not only where no product of decays underflows (0 inf).  Times a finite state
// the floor, the smallest float, is nothing.
__device__ __forceinline__ float decay(float y) { return max_nan(ex2f(y), 1.4e-45f); }
__device__ __forceinline__ float2 decay(float2 y) { return make_float2(decay(y.x), decay(y.y)); }
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

// The gates of two channels in base 2, as the special-function unit's exponential takes them:
// A = -exp(A_log), bias = dt_bias log2(e).
struct Channels {
    float2 A, bias;
};

// zl = log2(e) z for z = a + dt_bias; t = e^{-|z|} in (0, 1]; y = A log2(e) softplus(z), the
// base-2 log-decay.  softplus(z) = max(z, 0) + log1p(t) and log2(e) log1p(t) = t Q(t), Q the
// degree-8 polynomial whose largest relative error on [0, 1] is smallest (3.2e-8; a linear program,
// each coefficient rounded to fp32 before the next ones are fitted).  Small values of softplus are slow channels, whose state sums over
// many tokens: there the relative error of the log-decay, not the absolute one, is what the
// result sees, so log(1 + t) from the special-function unit (absolute error) will not do.
struct Gate {
    float2 zl, t, y;
};
__device__ __forceinline__ Gate decay_gate(float2 a, const Channels& ch) {
    Gate g;
    g.zl = __ffma2_rn(a, bcast2(kLog2e), ch.bias);
    g.t = ex2f2(make_float2(-fabsf(g.zl.x), -fabsf(g.zl.y)));
    float2 q = bcast2(7.650659885e-03f);
    q = __ffma2_rn(q, g.t, bcast2(-4.299838841e-02f));
    q = __ffma2_rn(q, g.t, bcast2(1.136108041e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-1.978190541e-01f));
    q = __ffma2_rn(q, g.t, bcast2(2.760109305e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-3.585188985e-01f));
    q = __ffma2_rn(q, g.t, bcast2(4.807103872e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-7.213414311e-01f));
    q = __ffma2_rn(q, g.t, bcast2(1.442695022e+00f));
    q = __ffma2_rn(q, g.t, make_float2(fmaxf(g.zl.x, 0.f), fmaxf(g.zl.y, 0.f)));
    g.y = __fmul2_rn(ch.A, q);
    return g;
}

// e^{-v}.  The product v log2(e) is rounded, which the power turns into a relative error of |v| 2^-24,
// 2e-6 for far gates: nothing beside the 2^-9 that a bf16 b carries, so bf16 calls take it as it
// is.  fp32 ones give the power what the product lost (kLog2eLow: what kLog2e lost), of a v that is
// bounded where the power is 0 or infinite anyway, and stay near an ulp.
template <typename Tin>
__device__ __forceinline__ float2 neg_exp(float2 v) {
    if constexpr (sizeof(Tin) == 2) {
        return ex2f2(__fmul2_rn(v, bcast2(-kLog2e)));
    } else {
        v = make_float2(max_nan(min_nan(v.x, 1000.f), -1000.f), max_nan(min_nan(v.y, 1000.f), -1000.f));
        const float2 p = __fmul2_rn(v, bcast2(-kLog2e));
        float2 low = __ffma2_rn(v, bcast2(-kLog2e), make_float2(-p.x, -p.y));
        low = __ffma2_rn(v, bcast2(-kLog2eLow), low);
        return __fmul2_rn(ex2f2(p), __ffma2_rn(low, bcast2(kLn2), bcast2(1.f)));
    }
}
// x sigmoid(b)
template <typename Tin>
__device__ __forceinline__ float2 gated_input(float2 x, float2 b) {
    return __fmul2_rn(x, rcpf2(__fadd2_rn(neg_exp<Tin>(b), bcast2(1.f))));
}

__device__ __forceinline__ Channels load_channels(const float* A_log, const float* dt_bias,
                                                  int c) {
    Channels ch;
    ch.A = make_float2(-expf(A_log[c]), -expf(A_log[c + 1]));
    ch.bias = __fmul2_rn(make_float2(dt_bias[c], dt_bias[c + 1]), bcast2(kLog2e));
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

// One token's backward step on two channels.  The factors of D, the gradient of its h, in da and
// (times log2 e) dA_log, from the token's decay lam and the state before it; returns the decay's
// base-2 logarithm.  sigmoid(v) is r = 1 / (1 + t) for v >= 0 and t r below, t = e^{-|v|}, so that
// small values keep their relative accuracy; sigmoid(v) (1 - sigmoid(v)) is t r^2 for both signs.
// Both forms of the backward pass use these, so they agree bit for bit where they add in the
// same order.
__device__ __forceinline__ float2 decay_factors(float2 a, float2 prev, const Channels& ch, float2& lam,
                                                float2& fa, float2& fA) {
    const Gate g = decay_gate(a, ch);
    lam = decay(g.y);
    const float2 rz = rcpf2(__fadd2_rn(g.t, bcast2(1.f))), tz = __fmul2_rn(g.t, rz);
    const float2 slope = make_float2(g.zl.x >= 0.f ? rz.x : tz.x, g.zl.y >= 0.f ? rz.y : tz.y);
    const float2 lp = __fmul2_rn(lam, prev);
    fa = __fmul2_rn(__fmul2_rn(lp, ch.A), slope);
    // (a at its type's highest value makes the log-decay infinite: lam times it would be NaN, not 0)
    fA = __fmul2_rn(lp, make_float2(max_nan(g.y.x, -1024.f), max_nan(g.y.y, -1024.f)));
    return g.y;
}
// Those in dx and db.
template <typename Tin>
__device__ __forceinline__ void input_factors(float2 x, float2 b, float2& fx, float2& fb) {
    const float2 tb = neg_exp<Tin>(make_float2(fabsf(b.x), fabsf(b.y)));
    const float2 rb = rcpf2(__fadd2_rn(tb, bcast2(1.f))), tr = __fmul2_rn(tb, rb);
    fx = make_float2(b.x >= 0.f ? rb.x : tr.x, b.y >= 0.f ? rb.y : tr.y);
    fb = __fmul2_rn(x, __fmul2_rn(rb, tr));
}
template <typename Tin>
__device__ __forceinline__ void store_grads(float2 fx, float2 fb, float2 fa, float2 fA, float2 D, Tin* dx,
                                            Tin* da, Tin* db, float2& acc_A, float2& acc_bias) {
    const float2 va = __fmul2_rn(fa, D);
    store_pair(dx, __fmul2_rn(fx, D));
    store_pair(da, va);
    store_pair(db, __fmul2_rn(fb, D));
    acc_A = __ffma2_rn(fA, D, acc_A);
    acc_bias = __fadd2_rn(acc_bias, va);
}

// ------------------------------------------------------------- sequential form
// Thread -> two channels of the sequences s = blockIdx.y, + gridDim.y, ...; one token after
// the other, the state in registers.  For single tokens and short sequences, where there is
// nothing to split.  One token of 64 sequences x 6144 channels takes 4 us: a launch, one round of
// loads and the stores; 32 tokens 31 us (0.62 of a copy's rate).
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
        if (p.limit && t1 - t0 > p.limit) continue;
        const size_t at = (size_t)s * p.C + c;
        float2 h = p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                : make_float2(0.f, 0.f);
#pragma unroll 4
        for (long long t = t0; t < t1; ++t) {
            const float2 xv = load_pair(x + t * p.ld), av = load_pair(a + t * p.ld),
                         bv = load_pair(b + t * p.ld);
            const Gate g = decay_gate(av, ch);
            h = __ffma2_rn(decay(g.y), h, gated_input<Tin>(xv, bv));
            store_pair(p.out + t * p.C + c, h);
        }
        if (p.final_state) *reinterpret_cast<float2*>(p.final_state + at) = h;
    }
}

// part [gridDim.y][2 C]: this row of CTAs' sums for A_log, then for dt_bias.  Twelve blocks per SM: left
// alone the compiler takes 118 registers for loads ahead, and 64 sequences of 32 tokens x 6144
// channels take 113 us instead of 73.
template <typename Tin>
__global__ void __launch_bounds__(kSeqThreads, 12)
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
        const bool another = p.limit && t1 - t0 > p.limit;
        if (another) t0 = t1;
        const size_t at = (size_t)s * p.C + c;
        float2 D = r.grad_final ? *reinterpret_cast<const float2*>(r.grad_final + at)
                                : make_float2(0.f, 0.f);
        const float2 init = p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                         : make_float2(0.f, 0.f);
#pragma unroll 2
        for (long long t = t1 - 1; t >= t0; --t) {
            const float2 prev = t > t0 ? load_pair(p.out + (t - 1) * p.C + c) : init;
            D = __fadd2_rn(load_pair(r.grad_out + t * p.C + c), D);
            float2 lam, fa, fA, fx, fb;
            decay_factors(load_pair(a + t * p.ld), prev, ch, lam, fa, fA);
            input_factors<Tin>(load_pair(x + t * p.ld), load_pair(b + t * p.ld), fx, fb);
            store_grads(fx, fb, fa, fA, D, dx + t * r.ld_grad, da + t * r.ld_grad, db + t * r.ld_grad,
                        acc_A, acc_bias);
            D = __fmul2_rn(lam, D);
        }
        if (r.grad_init && !another) *reinterpret_cast<float2*>(r.grad_init + at) = D;
    }
    float* row = part + (size_t)blockIdx.y * 2 * p.C;
    *reinterpret_cast<float2*>(row + c) = __fmul2_rn(acc_A, bcast2(kLn2));
    *reinterpret_cast<float2*>(row + p.C + c) = acc_bias;
}

// ------------------------------------------------------------------- tiled form
// One pass over the data with the time axis split three ways.  A CTA owns a strip of 64
// channels of one sequence and takes tiles of WARPS * TOK tokens; warp w holds tokens
// [w TOK, (w + 1) TOK) of the tile in registers, two channels per lane.  K CTAs of a cluster
// take K consecutive tiles at a time.  The recurrence is affine, h_end = P h_start + H, so
// each warp forms (P, H) of its tokens from zero, the CTA composes its warps' pairs through
// shared memory, the cluster its CTAs' through distributed shared memory, and every warp
// then runs its tokens once more from its true start state and stores them.  Nothing is
// read twice.
//
// What bounds it (B200, bf16): with as many units as SMs the backward pass runs at 0.97 of a
// copy's rate ([1, 8192, 9472] 245 us) and the forward pass at 0.86 (137 us), where the
// special-function unit does eight operations per token and channel pair; other calls lose to
// their last wave, to CTA starts and to the exchanges.  The kernels alone, forward: [8, 1024, 6144]
// 87 us (0.88 of a copy's rate), [1, 8192, 6144] 108 us (0.71), [1, 65536, 1024] 157 us (0.65);
// backward 167 us (0.92), 190 us (0.81), 273 us (0.75).
//
// Decays are composed as sums of log-decays.  From tile to tile a factor P near 1 acts
// through W = P - 1, formed as expm1 of its tile's sum: a slow channel's state lasts over
// thousands of tokens, and factors rounded near 1 would lose in every tile what the small
// W does not.  A factor below 2^-0.5 acts as P itself: there S + W S would cancel, and a
// large forgotten state would leave its rounding error in a small new one.
constexpr int kStrip = 64;
constexpr int kMaxCluster = 12;  // above 8 where the device allows it
constexpr size_t kSmemPerSm = 228 * 1024;  // 1 KB of it per CTA is the system's

// Shared memory of a CTA: per slot the x, a, b tiles, and for the backward pass dout's.
// PEERS: CTAs per cluster at most (1: none).
template <typename Tin_, int WARPS_, int TOK_, int STAGES_, int PEERS_, bool Grad>
struct alignas(128) TileSmem {
    using Tin = Tin_;
    static constexpr int WARPS = WARPS_, TOK = TOK_, STAGES = STAGES_, kRows = WARPS * TOK;
    static constexpr int PEERS = PEERS_;
    static constexpr bool Cluster = PEERS > 1;
    struct alignas(128) Slot {
        Tin in[3][kRows][kStrip];
        float dout[Grad ? kRows : 1][Grad ? kStrip : 4];
    };
    Slot slot[STAGES];
    float4 part[2][WARPS][32];       // per warp and lane: P pair, H pair; by step parity
    float2 log_part[2][WARPS][32];   // log2 of P
    // The cluster's tiles: coded factor pair, H pair; by step parity.  A CTA publishes step
    // s + 2 only once it has every peer's step s + 1, which a peer publishes after all its
    // warps are done with step s: nothing still unread is overwritten.
    float4 peer[2][PEERS][32];
    uint64_t full[STAGES], peers_in[2];
    int ticket;
};

// The factor 2^y, y <= 0, coded for carry(): for y > -0.5, W = expm1(y ln 2) with its sign
// bit set (y times the degree-4 polynomial nearest to (2^y - 1) / y on [-0.5, 0], relative error
// 1.6e-8; fitted as above), else 2^y itself, its sign bit clear.
__device__ __forceinline__ float code_factor(float y) {
    float q = 1.159412786e-03f;
    q = fmaf(q, y, 9.546945803e-03f);
    q = fmaf(q, y, 5.549255386e-02f);
    q = fmaf(q, y, 2.402259409e-01f);
    q = fmaf(q, y, 6.931471825e-01f);
    return y > -0.5f ? __int_as_float(__float_as_int(q * y) | 0x80000000) : decay(y);
}
// S <- 2^y S + H, the factor coded.  An infinite S enters the product W S as the largest float: W is
// negative, and W S + S would be -inf + inf.
__device__ __forceinline__ float carry(float S, float code, float H) {
    const float most = 3.402823466e38f, F = fminf(fmaxf(S, -most), most);
    return __float_as_int(code) < 0 ? fmaf(code, F, H) + S : fmaf(code, S, H);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Asynchronous store to the same shared-memory variable of CTA `rank` of this cluster; its 16
// bytes are counted on that CTA's `bar`.  (A cluster barrier per step, whose release also
// waits for the step's global stores, cost a third of the forward pass.)
__device__ __forceinline__ void store_peer(float4* p, uint64_t* bar, uint32_t rank, float4 v) {
    uint32_t a, b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
                 : "memory");
}
// Waits for the phase of `bar` that other CTAs' asynchronous stores complete; false if they did not
// come within the limit.  The stores' completion releases at cluster scope, so the wait acquires
// there too: at the default scope, the CTA's, nothing would order the peers' data before the
// reads behind the wait.  (The TMA barriers' completion is this CTA's own: their waits keep the default.)
__device__ __forceinline__ bool peers_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool peers_wait_slow(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = tc::globaltimer();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            __nanosleep(tc::kPollSleepNs);
            if (peers_test(bar, parity)) return true;
        }
        if (tc::globaltimer() - t0 > tc::kWaitLimitNs) return false;
    }
}
__device__ __forceinline__ bool peers_wait(uint64_t* bar, uint32_t parity) {
    return peers_test(bar, parity) || peers_wait_slow(bar, parity);
}
__device__ __forceinline__ float2 smem_pair(const float* p) {
    return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ float2 smem_pair(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// Tensor maps of a tiled call: boxes of kStrip channels x a tile's tokens.
struct Maps {
    CUtensorMap x, a, b, dout;
};

// Starts the copies of the tile whose first row is token `row` (rows before or past the tensor
// read as zeros) into slot st.
template <bool Grad, typename Smem>
__device__ __forceinline__ void load_tile(Smem& sm, int st, const Maps& m, int c0, int row) {
    auto& s = sm.slot[st];
    tc::mbar_arrive_expect_tx(&sm.full[st],
                              (uint32_t)(sizeof(s.in) + (Grad ? sizeof(s.dout) : 0)));
    tc::tma_load_2d(&s.in[0][0][0], &m.x, c0, row, &sm.full[st]);
    tc::tma_load_2d(&s.in[1][0][0], &m.a, c0, row, &sm.full[st]);
    tc::tma_load_2d(&s.in[2][0][0], &m.b, c0, row, &sm.full[st]);
    if constexpr (Grad) tc::tma_load_2d(&s.dout[0][0], &m.dout, c0, row, &sm.full[st]);
}

// After a wait that gave up, copies may still be in flight: the CTA stays for them (each
// wait is bounded too).
__device__ __noinline__ void wait_in_flight(uint64_t* full, int stages, int issued) {
    for (int s = max(0, issued - stages); s < issued; ++s)
        tc::mbar_wait(&full[s % stages], (uint32_t)(s / stages) & 1u);
}

// What a warp keeps of a step between its two runs over the step's tokens: the pair of the
// tokens before its own in the tile, and (no cluster) the whole tile's, coded.
struct Joined {
    float2 P, H;
    float4 all;
    int step;
};

// Composes the warps' pairs in sm.part (after the barrier behind their stores) and, in a
// cluster, starts the exchange of the CTAs' tiles.
template <bool Cluster, typename Smem>
__device__ __forceinline__ Joined publish(Smem& sm, int step, int warp, int lane) {
    const int buf = step & 1;
    float2 G = make_float2(0.f, 0.f), H = G, Gp = G, Hp = G;
#pragma unroll
    for (int w = 0; w < Smem::WARPS; ++w) {
        if (w == warp) {  // uniform: a branch, not eight times four selects
            Gp = G;
            Hp = H;
            asm volatile("");
        }
        const float4 v = sm.part[buf][w][lane];
        H = __ffma2_rn(make_float2(v.x, v.y), H, make_float2(v.z, v.w));
        G = __fadd2_rn(G, sm.log_part[buf][w][lane]);
    }
    Joined j;
    j.step = step;
    j.P = decay(Gp);
    j.H = Hp;
    j.all = make_float4(code_factor(G.x), code_factor(G.y), H.x, H.y);
    if constexpr (Cluster) {
        uint64_t* bar = &sm.peers_in[step & 1];
        const uint32_t K = cluster_size();
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(bar, K * (uint32_t)sizeof(sm.peer[0][0]));
        for (uint32_t k = warp; k < K; k += Smem::WARPS)
            store_peer(&sm.peer[step & 1][cluster_rank()][lane], bar, k, j.all);
    }
    return j;
}

// The state before this warp's tokens of the step; S moves from before the step to behind it.
template <bool Cluster, typename Smem>
__device__ __forceinline__ float2 start_state(Smem& sm, const Joined& j, int lane, float2& S,
                                              bool& dead) {
    const int step = j.step;
    float2 in = S;
    if constexpr (Cluster) {
        if (!dead && !peers_wait(&sm.peers_in[step & 1], (uint32_t)(step >> 1) & 1u)) {
            dead = true;
            if (lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        const uint32_t K = cluster_size(), rank = cluster_rank();
#pragma unroll 4
        for (uint32_t k = 0; k < K; ++k) {
            if (k == rank) in = S;
            const float4 v = sm.peer[step & 1][k][lane];
            S = make_float2(carry(S.x, v.x, v.z), carry(S.y, v.y, v.w));
        }
    } else {
        S = make_float2(carry(S.x, j.all.x, j.all.z), carry(S.y, j.all.y, j.all.w));
    }
    return __ffma2_rn(j.P, in, j.H);
}

// How a grid's clusters share the units' steps.  Plain (span == 0): cluster i takes unit i from end
// to end.  Split: the units' steps, all of one number, are laid end to end and cluster i takes
// `span` of them, at least a unit's; a unit cut by the border between i and i + 1 has its
// first steps in i and the rest in i + 1.  Every cluster takes its units from the last to
// the first, so it starts with the first steps of a cut unit, which wait for nothing, and
// ends with the last steps of another, whose state the cluster before it handed over long
// ago.  No SM idles for want of whole units: 96 units on 74 clusters of two.  Clusters are
// numbered in the order in which they start, so the one waited for always runs.
struct Schedule {
    int span, steps, total;
    int* ticket;       // clusters started; zero at launch
    uint32_t* ready;   // [clusters], zero at launch: states[i] is there
    float* states;     // [clusters][kStrip]
};

// A unit's part: steps [s0, s1) of `steps`.
struct Part {
    int unit, s0, s1;
};
struct Parts {
    int first, last, lo, hi, index;
};
template <bool Cluster, typename Smem>
__device__ __forceinline__ Parts parts_of(Smem& sm, const Schedule& s) {
    Parts p;
    p.lo = p.hi = 0;
    p.index = blockIdx.x / (Cluster ? (int)cluster_size() : 1);
    p.first = p.last = p.index;
    if (Cluster && s.span) {
        uint32_t a;  // rank 0 drew it
        int t;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(tc::smem_u32(&sm.ticket)));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(t) : "r"(a) : "memory");
        p.index = t;
        p.lo = t * s.span;
        p.hi = min(s.total, p.lo + s.span);
        p.first = p.lo / s.steps;
        p.last = p.lo < p.hi ? (p.hi - 1) / s.steps : p.first - 1;
    }
    return p;
}
template <bool Cluster>
__device__ __forceinline__ Part part_of(const Parts& p, const Schedule& s, int unit, int steps) {
    if (!Cluster || !s.span) return {unit, 0, steps};
    return {unit, max(0, p.lo - unit * s.steps), min(s.steps, p.hi - unit * s.steps)};
}

// Hands the state behind a cut unit's first steps to the next cluster (one warp) ...
__device__ __forceinline__ void hand_over(const Schedule& s, int index, int lane, float2 S) {
    __stcg(reinterpret_cast<float2*>(s.states + (size_t)index * kStrip + 2 * lane), S);
    __threadfence();
    __syncwarp();
    if (lane == 0) asm volatile("st.release.gpu.u32 [%0], %1;" ::"l"(s.ready + index), "r"(1u) : "memory");
}
// ... and takes it there (every warp); false if it did not come within the wait's limit.
__device__ __noinline__ bool wait_ready(const uint32_t* flag) {
    const uint64_t t0 = tc::globaltimer();
    for (;;) {
        uint32_t v;
        asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if (tc::globaltimer() - t0 > tc::kWaitLimitNs) return false;
        __nanosleep(100);
    }
}
__device__ __forceinline__ float2 take_over(const Schedule& s, int index, int lane, bool& dead) {
    int ok = 1;
    if (lane == 0 && !dead) ok = wait_ready(s.ready + index);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) {
        dead = true;
        if (lane == 0) atomicExch(&g_recurrence_status, 1);
    }
    __syncwarp();
    return __ldcg(reinterpret_cast<const float2*>(s.states + (size_t)index * kStrip + 2 * lane));
}

// What the CTAs of both tiled kernels share: their place in a unit, and its tokens.
struct Place {
    int warp, lane, K, rank, seq, c0, c, tiles, steps;
    long long t0, t1;
    bool in_c;
};
template <bool Cluster>
__device__ __forceinline__ Place place_of(const RecurrenceParams& p, int seq, int strip, int rows) {
    Place w;
    w.warp = threadIdx.x / 32;
    w.lane = threadIdx.x % 32;
    w.K = Cluster ? (int)cluster_size() : 1;
    w.rank = Cluster ? (int)cluster_rank() : 0;
    w.seq = seq;
    w.c0 = strip * kStrip;
    w.c = w.c0 + 2 * w.lane;
    w.in_c = w.c < p.C;  // C is even
    seq_bounds(p.cu_seqlens, w.seq, p.T, w.t0, w.t1);
    w.tiles = (int)((w.t1 - w.t0 + rows - 1) / rows);
    w.steps = (w.tiles + w.K - 1) / w.K;
    return w;
}
// The k-th of the packed sequences with more than p.limit tokens (a block of Warps warps; -1: none).
template <int Warps>
__device__ __forceinline__ int kth_long(const RecurrenceParams& p, int k) {
    __shared__ int counts[Warps], found;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int base = 0; base < p.nseq; base += 32 * Warps) {  // nseq is kMostPicked at most
        const int s = base + (int)threadIdx.x;
        bool is = false;
        if (s < p.nseq) {
            long long t0, t1;
            seq_bounds(p.cu_seqlens, s, p.T, t0, t1);
            is = t1 - t0 > p.limit;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, is);
        if (lane == 0) counts[warp] = __popc(mask);
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < Warps; ++w) {
            before += w < warp ? counts[w] : 0;
            all += counts[w];
        }
        if (is && before + __popc(mask & ((1u << lane) - 1)) == k) found = s;
        __syncthreads();
        if (k < all) return found;
        k -= all;
    }
    return -1;
}
// One thread: barriers, and the cluster's number where it is drawn.
template <typename Smem>
__device__ __forceinline__ void init_cta(Smem& sm, const Schedule& s, int rank) {
    for (int i = 0; i < Smem::STAGES; ++i) tc::mbar_init(&sm.full[i], 1);
    for (int i = 0; i < 2; ++i) tc::mbar_init(&sm.peers_in[i], 1);
    tc::mbar_init_fence();
    if (Smem::Cluster && s.span && rank == 0) sm.ticket = atomicAdd(s.ticket, 1);
}

// Pick (no cluster): CTAs k strips .. (k + 1) strips - 1 take the k-th sequence longer than p.limit.
template <typename Smem, int Blocks, bool Pick = false>
__global__ void __launch_bounds__(32 * Smem::WARPS, Blocks)
recurrence_tile_kernel(const __grid_constant__ Maps maps, RecurrenceParams p, int strips,
                       Schedule sched) {
    static_assert(sizeof(Smem) <= kSmemPerSm / Blocks - 1024, "the SM's CTAs have to fit");
    constexpr int TOK = Smem::TOK, STAGES = Smem::STAGES, kRows = Smem::kRows;
    constexpr bool Cluster = Smem::Cluster;
    using Tin = typename Smem::Tin;
    int seq = 0;
    if constexpr (Pick) {
        static_assert(!Cluster, "a picked sequence is one CTA's per strip");
        seq = kth_long<Smem::WARPS>(p, blockIdx.x / strips);
        if (seq < 0) return;
    }
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    if (threadIdx.x == 0) init_cta(sm, sched, Cluster ? (int)cluster_rank() : 0);
    // the barriers are set up; in a cluster, every CTA has started
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    const Parts parts = parts_of<Cluster>(sm, sched);
    struct Held {
        float2 lam[TOK], u[TOK];
        Joined j;
    };
    bool dead = false;
    int issued = 0, taken = 0, turn = 0;  // tiles copied, tiles waited for, steps begun
    for (int unit = parts.last; unit >= parts.first; --unit) {  // without a cluster: once
        const int place = Cluster ? unit : (int)blockIdx.x;
        const Place w = place_of<Cluster>(p, Pick ? seq : place / strips, place % strips, kRows);
        const Part part = part_of<Cluster>(parts, sched, unit, w.steps);
        Channels ch = {};
        if (w.in_c) ch = load_channels(p.A_log, p.dt_bias, w.c);
        const size_t at = (size_t)w.seq * p.C + w.c;
        float2 S = w.in_c && p.init_state && part.s0 == 0
                       ? *reinterpret_cast<const float2*>(p.init_state + at)
                       : make_float2(0.f, 0.f);
        // tokens of this warp in a step: the first one, and how many are within the sequence
        auto first_of = [&](int step) {
            return w.t0 + (long long)(step * w.K + w.rank) * kRows + w.warp * TOK;
        };
        auto live_of = [&](long long first) {
            return (int)min((long long)TOK, max(0LL, w.t1 - first));
        };
        int to_load = part.s0;  // one thread: the step whose tile is copied next
        auto load_next = [&]() {
            const int tile = to_load * w.K + w.rank;
            if (to_load >= part.s1 || tile >= w.tiles) return;
            load_tile<false>(sm, issued % STAGES, maps, w.c0, (int)(w.t0 + (long long)tile * kRows));
            ++to_load;
            ++issued;
        };
        if (Cluster) __syncthreads();  // the part before is done with its tiles
        if (threadIdx.x == 0 && !dead)
            for (int i = 0; i < STAGES; ++i) load_next();
        // The state has arrived in every lane before any barrier or exchange that lets another warp
        // write the final one, which may be the same memory.
        S.x = __shfl_sync(0xffffffffu, S.x, w.lane);
        S.y = __shfl_sync(0xffffffffu, S.y, w.lane);
        // the run from zero, up to the exchange
        auto read_tile = [&](int step, Held& k) {
            const int st = taken % STAGES, buf = turn & 1, live = live_of(first_of(step));
            if (step * w.K + w.rank < w.tiles) {
                if (!dead && !tc::mbar_wait(&sm.full[st], (uint32_t)(taken / STAGES) & 1u)) {
                    dead = true;
                    if (w.lane == 0) atomicExch(&g_recurrence_status, 1);
                }
                ++taken;
            }
            __syncwarp();
            float2 G = make_float2(0.f, 0.f), H = G;
            const auto* row = &sm.slot[st].in[0][w.warp * TOK][2 * w.lane];
            auto gates = [&](int i) {
                const float2 xv = smem_pair(row + i * kStrip);
                const float2 av = smem_pair(row + (kRows + i) * kStrip);
                const float2 bv = smem_pair(row + (2 * kRows + i) * kStrip);
                const float2 y = decay_gate(av, ch).y;
                k.lam[i] = decay(y);
                k.u[i] = gated_input<Tin>(xv, bv);
                G = __fadd2_rn(G, y);
                H = __ffma2_rn(k.lam[i], H, k.u[i]);
            };
            if (live == TOK) {
#pragma unroll
                for (int i = 0; i < TOK; ++i) gates(i);
            } else {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    if (i < live) {
                        gates(i);
                    } else {
                        k.lam[i] = make_float2(1.f, 1.f);
                        k.u[i] = make_float2(0.f, 0.f);
                    }
                }
            }
            sm.part[buf][w.warp][w.lane] = make_float4(decay(G.x), decay(G.y), H.x, H.y);
            sm.log_part[buf][w.warp][w.lane] = G;
            __syncthreads();
            // every warp has read the tile: its slot takes another
            if (threadIdx.x == 0 && !dead) load_next();
            k.j = publish<Cluster>(sm, turn++, w.warp, w.lane);
        };
        // the run from the true start state
        auto write_tile = [&](int step, const Held& k) {
            float2 h = start_state<Cluster>(sm, k.j, w.lane, S, dead);
            const long long first = first_of(step);
            const int live = live_of(first);
            float* out = p.out + first * p.C + w.c;
            if (w.in_c) {
                if (live == TOK) {
#pragma unroll
                    for (int i = 0; i < TOK; ++i) {
                        h = __ffma2_rn(k.lam[i], h, k.u[i]);
                        store_pair(out + (size_t)i * p.C, h);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < TOK; ++i) {
                        h = __ffma2_rn(k.lam[i], h, k.u[i]);
                        if (i < live) store_pair(out + (size_t)i * p.C, h);
                    }
                }
                // the warp with the sequence's last token: its h, so that the two agree
                if (live > 0 && first + live == w.t1 && p.final_state)
                    *reinterpret_cast<float2*>(p.final_state + at) = h;
            }
            __syncwarp();
        };
        Held k;
        for (int step = part.s0; step < part.s1; ++step) {
            read_tile(step, k);
            if (Cluster && step == part.s0 && step > 0) S = take_over(sched, parts.index - 1, w.lane, dead);
            write_tile(step, k);
        }
        if (Cluster && part.s1 < w.steps && w.rank == 0 && w.warp == 0)
            hand_over(sched, parts.index, w.lane, S);
        if (w.tiles == 0 && w.rank == 0 && w.warp == 0 && w.in_c && p.final_state)
            *reinterpret_cast<float2*>(p.final_state + at) = S;
        if (!Cluster) break;
    }
    if (dead && threadIdx.x == 0) wait_in_flight(sm.full, STAGES, issued);
    // no CTA leaves while a peer may still store to it
    if constexpr (Cluster) cluster_barrier();
}

// The same pass against time: with E the gradient that reaches h_t from later tokens,
// D_t = dout_t + E and E <- exp(g_t) D_t, so tokens are taken from the last one back and a
// warp's pair is (P, H) of E.  Tiles are counted from the sequence's end.  What D is multiplied
// with for da and dA_log is formed while the tile is read, for dx and db (sigmoid(b)) in the
// second run, from the slot: three values per token and channel to hold, not five.  h comes by
// plain loads, one step ahead.
// partial [rows][2 C]: each CTA's sums for A_log and dt_bias, one row per (sequence, rank), and
// under a split schedule as many rows again for the units' later parts; Pick: one per k.
template <typename Smem, int Blocks, bool Pick = false>
__global__ void __launch_bounds__(32 * Smem::WARPS, Blocks)
recurrence_tile_backward_kernel(const __grid_constant__ Maps maps, RecurrenceParams p,
                                RecurrenceGrads r, float* partial, int strips, Schedule sched) {
    constexpr int TOK = Smem::TOK, STAGES = Smem::STAGES, kRows = Smem::kRows;
    constexpr bool Cluster = Smem::Cluster;
    using Tin = typename Smem::Tin;
    static_assert(STAGES > 1, "a slot has to be free for the next tile");
    static_assert(sizeof(Smem) <= kSmemPerSm / Blocks - 1024, "the SM's CTAs have to fit");
    int seq = 0;
    if constexpr (Pick) {
        static_assert(!Cluster, "a picked sequence is one CTA's per strip");
        seq = kth_long<Smem::WARPS>(p, blockIdx.x / strips);
        if (seq < 0) {  // its row of sums is added all the same
            const int c = blockIdx.x % strips * kStrip + (int)threadIdx.x;
            float* o = partial + (size_t)(blockIdx.x / strips) * 2 * p.C;
            if (threadIdx.x < kStrip && c < p.C) o[c] = o[p.C + c] = 0.f;
            return;
        }
    }
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    if (threadIdx.x == 0) init_cta(sm, sched, Cluster ? (int)cluster_rank() : 0);
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    const Parts parts = parts_of<Cluster>(sm, sched);
    const float2 zero = make_float2(0.f, 0.f);
    struct Held {
        float2 lam[TOK], a[TOK], A[TOK];
        Joined j;
        int slot;
    };
    bool dead = false;
    int issued = 0, taken = 0, turn = 0;  // tiles copied, tiles waited for, steps begun
    for (int unit = parts.last; unit >= parts.first; --unit) {  // without a cluster: once
        const int place = Cluster ? unit : (int)blockIdx.x;
        const Place w = place_of<Cluster>(p, Pick ? seq : place / strips, place % strips, kRows);
        const Part part = part_of<Cluster>(parts, sched, unit, w.steps);
        Channels ch = {};
        if (w.in_c) ch = load_channels(p.A_log, p.dt_bias, w.c);
        const size_t at = (size_t)w.seq * p.C + w.c;
        float2 S = w.in_c && r.grad_final && part.s0 == 0
                       ? *reinterpret_cast<const float2*>(r.grad_final + at) : zero;
        auto last_of = [&](int step) {
            return w.t1 - (long long)(step * w.K + w.rank) * kRows - w.warp * TOK - 1;
        };
        auto live_of = [&](long long last) {
            return (int)min((long long)TOK, max(0LL, last + 1 - w.t0));
        };
        int to_load = part.s0;  // one thread: the step whose tile is copied next
        auto load_next = [&]() {
            const int tile = to_load * w.K + w.rank;
            if (to_load >= part.s1 || tile >= w.tiles) return;
            // a sequence's first tile may start before it, at a negative row even
            load_tile<true>(sm, issued % STAGES, maps, w.c0,
                            (int)(w.t1 - (long long)(tile + 1) * kRows));
            ++to_load;
            ++issued;
        };
        if (Cluster) __syncthreads();  // the part before is done with its tiles
        if (threadIdx.x == 0 && !dead)
            for (int i = 0; i < STAGES; ++i) load_next();
        // The state has arrived in every lane before any barrier or exchange that lets another warp
        // write the final one, which may be the same memory.
        S.x = __shfl_sync(0xffffffffu, S.x, w.lane);
        S.y = __shfl_sync(0xffffffffu, S.y, w.lane);
        // the states before a step's tokens of this warp: last, last - 1, ...
        float2 prev[TOK];
        auto load_prev = [&](int step) {
            const long long last = last_of(step);
            const float* h = p.out + (last - 1) * p.C + w.c;
            if (last - TOK >= w.t0 && w.in_c) {
#pragma unroll
                for (int i = 0; i < TOK; ++i) prev[i] = load_pair(h - (size_t)i * p.C);
            } else {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    prev[i] = zero;
                    if (w.in_c && last - i > w.t0) prev[i] = load_pair(h - (size_t)i * p.C);
                    if (w.in_c && last - i == w.t0 && p.init_state)
                        prev[i] = *reinterpret_cast<const float2*>(p.init_state + at);
                }
            }
        };
        if (part.s0 < part.s1) load_prev(part.s0);
        float2 acc_A = zero, acc_bias = zero;
        auto read_tile = [&](int step, Held& k) {
            const int st = taken % STAGES, buf = turn & 1, live = live_of(last_of(step));
            k.slot = st;
            if (step * w.K + w.rank < w.tiles) {
                if (!dead && !tc::mbar_wait(&sm.full[st], (uint32_t)(taken / STAGES) & 1u)) {
                    dead = true;
                    if (w.lane == 0) atomicExch(&g_recurrence_status, 1);
                }
                ++taken;
            }
            __syncwarp();
            float2 G = zero, H = zero;
            const auto* a = &sm.slot[st].in[1][kRows - 1 - w.warp * TOK][2 * w.lane];
            const float* dout = &sm.slot[st].dout[kRows - 1 - w.warp * TOK][2 * w.lane];
            auto gates = [&](int i) {
                const float2 y = decay_factors(smem_pair(a - i * kStrip), prev[i], ch, k.lam[i], k.a[i], k.A[i]);
                G = __fadd2_rn(G, y);
                H = __fmul2_rn(k.lam[i], __fadd2_rn(smem_pair(dout - i * kStrip), H));
            };
            if (live == TOK) {
#pragma unroll
                for (int i = 0; i < TOK; ++i) gates(i);
            } else {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    if (i < live) gates(i);
                }
            }
            if (step + 1 < part.s1) load_prev(step + 1);
            sm.part[buf][w.warp][w.lane] = make_float4(decay(G.x), decay(G.y), H.x, H.y);
            sm.log_part[buf][w.warp][w.lane] = G;
            __syncthreads();
            // every warp is done with the step before: its slot takes another tile
            if (threadIdx.x == 0 && !dead && step > part.s0) load_next();
            k.j = publish<Cluster>(sm, turn++, w.warp, w.lane);
        };
        auto write_tile = [&](int step, const Held& k) {
            float2 E = start_state<Cluster>(sm, k.j, w.lane, S, dead);
            const long long last = last_of(step);
            const int live = live_of(last);
            const auto* x = &sm.slot[k.slot].in[0][kRows - 1 - w.warp * TOK][2 * w.lane];
            const float* dout = &sm.slot[k.slot].dout[kRows - 1 - w.warp * TOK][2 * w.lane];
            if (w.in_c) {
                Tin* dx = static_cast<Tin*>(r.grad_x) + last * r.ld_grad + w.c;
                Tin* da = static_cast<Tin*>(r.grad_a) + last * r.ld_grad + w.c;
                Tin* db = static_cast<Tin*>(r.grad_b) + last * r.ld_grad + w.c;
                auto token = [&](int i) {
                    const float2 D = __fadd2_rn(smem_pair(dout - i * kStrip), E);
                    const long long o = i * r.ld_grad;
                    float2 fx, fb;
                    input_factors<Tin>(smem_pair(x - i * kStrip), smem_pair(x + (2 * kRows - i) * kStrip), fx, fb);
                    store_grads(fx, fb, k.a[i], k.A[i], D, dx - o, da - o, db - o, acc_A, acc_bias);
                    E = __fmul2_rn(k.lam[i], D);
                };
                if (live == TOK) {
#pragma unroll
                    for (int i = 0; i < TOK; ++i) token(i);
                } else {
#pragma unroll
                    for (int i = 0; i < TOK; ++i) {
                        if (i < live) token(i);
                    }
                }
                // the warp with the sequence's first token
                if (live > 0 && last + 1 - live == w.t0 && r.grad_init)
                    *reinterpret_cast<float2*>(r.grad_init + at) = E;
            }
            __syncwarp();
        };
        Held k;
        for (int step = part.s0; step < part.s1; ++step) {
            read_tile(step, k);
            if (Cluster && step == part.s0 && step > 0) S = take_over(sched, parts.index - 1, w.lane, dead);
            write_tile(step, k);
        }
        if (Cluster && part.s1 < w.steps && w.rank == 0 && w.warp == 0)
            hand_over(sched, parts.index, w.lane, S);
        if (w.tiles == 0 && w.rank == 0 && w.warp == 0 && w.in_c && r.grad_init)
            *reinterpret_cast<float2*>(r.grad_init + at) = S;
        __syncthreads();
        sm.part[0][w.warp][w.lane] = make_float4(acc_A.x, acc_A.y, acc_bias.x, acc_bias.y);
        __syncthreads();
        if (w.warp == 0 && w.in_c) {
            float4 s = sm.part[0][0][w.lane];
#pragma unroll
            for (int k = 1; k < Smem::WARPS; ++k) {
                const float4 v = sm.part[0][k][w.lane];
                s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
            const float2 sum_A = __fmul2_rn(make_float2(s.x, s.y), bcast2(kLn2));
            const float2 sum_bias = make_float2(s.z, s.w);
            const size_t row = Pick ? (size_t)(blockIdx.x / strips) : (size_t)w.seq * w.K + w.rank;
            const size_t later = (size_t)p.nseq * w.K;
            auto put = [&](size_t row, float2 a, float2 b) {
                float* o = partial + row * 2 * p.C + w.c;
                *reinterpret_cast<float2*>(o) = a;
                *reinterpret_cast<float2*>(o + p.C) = b;
            };
            put(part.s0 > 0 ? row + later : row, sum_A, sum_bias);
            if (Cluster && sched.span && part.s0 == 0 && part.s1 == w.steps) put(row + later, zero, zero);
        }
        if (!Cluster) break;
    }
    if (dead && threadIdx.x == 0) wait_in_flight(sm.full, STAGES, issued);
    if constexpr (Cluster) cluster_barrier();
}

// Rows of CTAs of the sequential form backward, one row of partial sums each: enough threads to
// fill the SMs.
int seq_rows(const RecurrenceParams& p) {
    return std::min(p.nseq, std::max(64, (300000 + p.C - 1) / p.C));
}

// The tokens of a call's mean sequence; the host does not know packed sequences' lengths.
int mean_length(const RecurrenceParams& p) {
    return p.cu_seqlens ? (int)(((long long)p.T + p.nseq - 1) / p.nseq) : p.T;
}

// (sequence, strip of channels) pairs, each one chain of tiles.
long long units_of(const RecurrenceParams& p) {
    return (long long)p.nseq * ((p.C + kStrip - 1) / kStrip);
}

// Clusters of K CTAs of a kernel that the current device holds at once; the runtime is asked once
// per kernel, K and device.
struct Capacity {
    std::atomic<int> fit[64][kMaxCluster + 1];
};
template <typename Kernel>
cudaError_t clusters_held(Capacity& held, Kernel kernel, int threads, size_t smem, int K, int* fit) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    *fit = held.fit[dev][K].load();  // 0: not asked yet, -1: none
    if (*fit != 0) return cudaSuccess;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)K;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)K);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    CaptureRelaxed relaxed;
    e = allow_smem((const void*)kernel, smem);
    if (e == cudaSuccess && K > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(fit, kernel, &cfg);
    if (e != cudaSuccess && K > 8) {  // a device without clusters of this size
        cudaGetLastError();
        e = cudaSuccess;
        *fit = 0;
    }
    if (e == cudaSuccess) held.fit[dev][K].store(*fit = *fit > 0 ? *fit : -1);
    return e;
}

// What a launch of the tiled kernels looks like: which form, K CTAs per cluster, and steps per
// cluster under a split schedule (0: plain).
struct Plan {
    int form, K, span, clusters;
    double time;
};

// Offers `slots` clusters of K CTAs that take `rows` tokens of a unit per step of `ns`, plain and
// (cuttable: equal lengths) split.  The time is that of the busiest slot's steps, and of what
// a CTA does before its first (`start_ns`, less where another CTA of its SM works on).  A split
// schedule spends a start per unit and some 8 us more: another node of the stream sets its
// counters to zero, and a part's first tile is not copied ahead.
void offer(Plan* plan, const RecurrenceParams& p, int form, int K, long long slots, long long rows,
           double ns, double start_ns, bool cuttable) {
    const long long units = units_of(p), steps = (mean_length(p) + rows - 1) / rows;
    double t = (double)((units + slots - 1) / slots) * (steps * ns + start_ns);
    if (!plan->K || t < 0.97 * plan->time) *plan = {form, K, 0, 0, t};
    const long long total = units * steps, span = std::max(steps, (total + slots - 1) / slots);
    if (!cuttable || p.cu_seqlens || total + span > (1 << 30)) return;
    t = (double)(span + 1) * ns + (double)span / steps * start_ns + 8000.0;
    if (t < 0.97 * plan->time)
        *plan = {form, K, (int)span, (int)((total + span - 1) / span), t};
}
template <typename Smem, typename Kernel>
cudaError_t offer_clusters(Plan* plan, const RecurrenceParams& p, int form, Kernel kernel,
                           Capacity& held, double ns, double ns_per_rank, double start_ns) {
    for (int K = 2; K <= Smem::PEERS; ++K) {
        // clusters are for units that leave SMs idle, and for at least a tile each
        if (units_of(p) > 2LL * device_sms() || (long long)(K - 1) * Smem::kRows >= mean_length(p)) break;
        int fit = 0;
        const cudaError_t e = clusters_held(held, kernel, 32 * Smem::WARPS, sizeof(Smem), K, &fit);
        if (e != cudaSuccess) return e;
        if (fit < 1) break;
        offer(plan, p, form, K, fit, (long long)K * Smem::kRows, ns + K * ns_per_rank, start_ns, true);
    }
    return cudaSuccess;
}

template <typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, long long grid, int threads, int K, size_t smem,
                         cudaStream_t stream, Args... args) {
    cudaError_t e = allow_smem((const void*)kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)K;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = K > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool make_maps(Maps& m, const RecurrenceParams& p, const float* dout, int box) {
    const uint64_t rows = p.cu_seqlens ? (uint64_t)p.T : (uint64_t)p.nseq * p.T;
    const bool f32 = p.in == InType::F32;
    return make_map_pitched(&m.x, p.x, f32, p.C, rows, p.ld, kStrip, box) &&
           make_map_pitched(&m.a, p.a, f32, p.C, rows, p.ld, kStrip, box) &&
           make_map_pitched(&m.b, p.b, f32, p.C, rows, p.ld, kStrip, box) &&
           (!dout || make_map_pitched(&m.dout, dout, true, p.C, rows, p.C, kStrip, box));
}

// The forms of each kernel: warps, tokens per warp, slots, CTAs per cluster at most.  One: no
// cluster, a CTA per SM.  Many: no cluster, two CTAs per SM, whose phases and starts overlap.
// Crowd: no cluster, three small ones per SM, for dense calls of more units than Many takes at
// once: their starts and their last wave cost less ([8, 1024, 6144] forward 88 against 98 us,
// [64, 200, 6144] 140 against the sequential form's 182).
// Wide: clusters with one CTA per SM, for few units; its tiles are the largest that the slots
// hold, since a step's exchange costs the same 0.6 us for any.  Pair: clusters with two CTAs
// per SM, for units in between (a cluster's CTAs share SMs, so it needs enough clusters).
// Registers set the tokens of two CTAs per SM (two values per token and channel forward, three
// backward, where a slot is held through its step, too).  Times in ns, a step and a CTA's start, are
// fitted to calls that fill the slots in part: a plan's time ranks the forms and foretells no call
// (where units fill every slot, steps of kCrowd and of fp32's kMany would move 7.3 to 8.3 TB/s).
template <typename Tin> struct Forms;
template <> struct Forms<__nv_bfloat16> {
    using T = __nv_bfloat16;
    struct Fwd {
        using One = TileSmem<T, 8, 20, 2, 1, false>;
        using Many = TileSmem<T, 8, 12, 2, 1, false>;
        using Crowd = TileSmem<T, 4, 16, 2, 1, false>;
        using Wide = TileSmem<T, 8, 32, 2, 12, false>;
        using Pair = TileSmem<T, 8, 12, 2, 4, false>;
        static constexpr double kOne = 2600, kMany = 3140, kCrowd = 2500, kWide = 4450, kPair = 3350;
        static constexpr double kStart = 1500, kManyStart = 300, kCrowdStart = 1800,
                                kWideStart = 4500, kPairStart = 300;
    };
    struct Bwd {
        using One = TileSmem<T, 8, 10, 3, 1, true>;
        using Many = TileSmem<T, 8, 8, 2, 1, true>;
        using Crowd = TileSmem<T, 4, 11, 2, 1, true>;
        using Wide = TileSmem<T, 8, 14, 2, 12, true>;
        using Pair = TileSmem<T, 8, 7, 2, 4, true>;
        static constexpr double kOne = 2200, kMany = 3370, kCrowd = 3300, kWide = 3550, kPair = 3600;
        static constexpr double kStart = 3400, kManyStart = 6000, kCrowdStart = 4000,
                                kWideStart = 6000, kPairStart = 1500;
    };
};
template <> struct Forms<float> {
    using T = float;
    struct Fwd {
        using One = TileSmem<T, 8, 12, 2, 1, false>;
        using Many = TileSmem<T, 8, 8, 2, 1, false>;
        using Crowd = TileSmem<T, 4, 10, 2, 1, false>;
        using Wide = TileSmem<T, 8, 16, 2, 12, false>;
        using Pair = TileSmem<T, 8, 6, 2, 4, false>;
        static constexpr double kOne = 2110, kMany = 2350, kCrowd = 2450, kWide = 2850, kPair = 2250;
        static constexpr double kStart = 1500, kManyStart = 300, kCrowdStart = 1800,
                                kWideStart = 4500, kPairStart = 300;
    };
    struct Bwd {
        using One = TileSmem<T, 8, 6, 3, 1, true>;
        using Many = TileSmem<T, 8, 6, 2, 1, true>;
        using Crowd = TileSmem<T, 4, 7, 2, 1, true>;
        using Wide = TileSmem<T, 8, 12, 2, 12, true>;
        using Pair = TileSmem<T, 8, 5, 2, 4, true>;
        static constexpr double kOne = 2230, kMany = 3490, kCrowd = 3450, kWide = 4100, kPair = 3000;
        static constexpr double kStart = 3400, kManyStart = 6000, kCrowdStart = 2500,
                                kWideStart = 6000, kPairStart = 1500;
    };
};
constexpr double kWideRank = 10, kPairRank = 50;  // a step's further ns for each CTA of the cluster

enum Form { kOneForm, kManyForm, kCrowdForm, kWideForm, kPairForm };

template <typename F>
void offer_single(Plan* plan, const RecurrenceParams& p) {
    const int sms = device_sms();
    if (units_of(p) <= sms)
        offer(plan, p, kOneForm, 1, sms, F::One::kRows, F::kOne, F::kStart, false);
    else
        offer(plan, p, kManyForm, 1, 2LL * sms, F::Many::kRows, F::kMany, F::kManyStart, false);
    // packed sequences may be uneven, and the longest then waits for a slower CTA
    if (units_of(p) > 2LL * sms && !p.cu_seqlens)
        offer(plan, p, kCrowdForm, 1, 3LL * sms, F::Crowd::kRows, F::kCrowd, F::kCrowdStart, false);
}

// Whether the sequential form is the faster one: a chain of tokens, each at least a memory latency
// and at least its bytes' time (backward in fp32, eight streams of wide rows, at half of a
// copy's rate), against a plan.  It is for short sequences (64 sequences of 6144 channels,
// forward: 31 against 82 us at 32 tokens, 59 against 58 at 64, 116 against 90 at 128; one
// sequence: 16 against 8 at 16).  Of packed sequences only the mean length is known here: the long
// ones among them are left to tiles (long_limit); where there are too many to look through, one that
// holds most of the tokens may cost the sequential form at most 20 times a plan.
constexpr int kMostPicked = 16384;
bool sequential(const RecurrenceParams& p, const Plan& plan, double latency_ns, double channel_ns) {
    if (p.cu_seqlens && p.nseq > kMostPicked && p.T * latency_ns > 20 * plan.time) return false;
    return mean_length(p) * std::max(latency_ns, channel_ns * p.nseq * p.C) < plan.time;
}

// Packed sequences that are short in the mean: those of more than `limit` tokens, `groups` at most,
// go to a tiled kernel behind the sequential one, which finds them on the device.  A long prompt
// among single tokens ([8192, 255 x 1], C = 6144) takes 157 us forward and 237 backward so, 5.0 and
// 5.8 ms a token at a time.  The limit is the least whose groups fit four waves of CTAs, which
// without any such sequence cost 5 us (64 x 32: 45 -> 50 us forward, 68 -> 73 backward), and never so
// short that the tiles gain nothing; no limit (0) where one sequence of all the tokens would take
// 0.2 ms at most.
struct Long {
    int limit, groups;
};
Long long_limit(const RecurrenceParams& p, double latency_ns) {
    if (!p.cu_seqlens || p.nseq > kMostPicked || p.T * latency_ns <= 2e5) return {0, 0};
    const int strips = (p.C + kStrip - 1) / kStrip, most = std::max(1, 4 * device_sms() / strips);
    const int limit = std::max(64, (int)(((long long)p.T + most - 1) / most) - 1);
    return p.T > limit ? Long{limit, std::min(p.nseq, p.T / (limit + 1))} : Long{0, 0};
}

// A split schedule's counters and states in `ws`, the counters set to zero.
size_t schedule_bytes(const Plan& plan) {
    return plan.span ? sizeof(float) * plan.clusters * (size_t)kStrip + sizeof(int) * (plan.clusters + 1) : 0;
}
cudaError_t set_schedule(Schedule* s, const Plan& plan, long long units, int steps, void* ws,
                         cudaStream_t stream) {
    *s = {};
    if (!plan.span) return cudaSuccess;
    s->span = plan.span;
    s->steps = steps;
    s->total = (int)(units * steps);
    s->states = static_cast<float*>(ws);
    s->ready = reinterpret_cast<uint32_t*>(s->states + (size_t)plan.clusters * kStrip);
    s->ticket = reinterpret_cast<int*>(s->ready + plan.clusters);
    return cudaMemsetAsync(s->ready, 0, sizeof(int) * (plan.clusters + 1), stream);
}

template <typename Smem, int Blocks>
cudaError_t forward_tiles(const RecurrenceParams& p, const Plan& plan, cudaStream_t stream) {
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long units = units_of(p);
    const long long grid = (plan.span ? plan.clusters : units) * plan.K;
    const long long rows = (long long)Smem::kRows * plan.K;
    Maps m;
    // a cluster's exchange needs a launch in clusters
    if (Smem::Cluster != (plan.K > 1)) return cudaErrorInvalidValue;
    if (grid > 0x7fffffffLL || !make_maps(m, p, nullptr, Smem::kRows)) return cudaErrorNotSupported;
    void* ws = nullptr;
    cudaError_t e = plan.span ? workspace_alloc(&ws, schedule_bytes(plan), stream) : cudaSuccess;
    if (e != cudaSuccess) return e;
    Schedule s;
    e = set_schedule(&s, plan, units, (int)((p.T + rows - 1) / rows), ws, stream);
    if (e == cudaSuccess)
        e = launch_tiles(recurrence_tile_kernel<Smem, Blocks>, grid, 32 * Smem::WARPS, plan.K,
                         sizeof(Smem), stream, m, p, strips, s);
    const cudaError_t f = ws ? cudaFreeAsync(ws, stream) : cudaSuccess;
    return e != cudaSuccess ? e : f;
}

template <typename Smem, int Blocks>
cudaError_t backward_tiles(const RecurrenceParams& p, const RecurrenceGrads& r, const Plan& plan,
                           cudaStream_t stream) {
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long units = units_of(p);
    const long long grid = (plan.span ? plan.clusters : units) * plan.K;
    const long long rows = (long long)Smem::kRows * plan.K;
    // rows of partial sums: one per (sequence, rank), and one for a cut unit's later part
    const long long sums = (long long)p.nseq * plan.K * (plan.span ? 2 : 1);
    Maps m;
    // a cluster's exchange needs a launch in clusters
    if (Smem::Cluster != (plan.K > 1)) return cudaErrorInvalidValue;
    if (grid > 0x7fffffffLL || !make_maps(m, p, r.grad_out, Smem::kRows)) return cudaErrorNotSupported;
    const size_t sum_bytes = sizeof(float) * sums * 2 * p.C;
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sum_bytes + schedule_bytes(plan), stream);
    if (e != cudaSuccess) return e;
    Schedule s;
    e = set_schedule(&s, plan, units, (int)((p.T + rows - 1) / rows),
                     reinterpret_cast<char*>(part) + sum_bytes, stream);
    if (e == cudaSuccess)
        e = launch_tiles(recurrence_tile_backward_kernel<Smem, Blocks>, grid, 32 * Smem::WARPS,
                         plan.K, sizeof(Smem), stream, m, p, r, part, strips, s);
    if (e == cudaSuccess)
        e = launch_column_sum(part, sums, 2 * p.C, r.grad_A_log, p.C, r.grad_dt_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

// The tiled kernels on the sequences longer than p.limit, with a CTA per SM.
template <typename Smem>
cudaError_t forward_long(const RecurrenceParams& p, int groups, cudaStream_t stream) {
    const int strips = (p.C + kStrip - 1) / kStrip;
    Maps m;
    if (!make_maps(m, p, nullptr, Smem::kRows)) return cudaErrorNotSupported;
    return launch_tiles(recurrence_tile_kernel<Smem, 1, true>, (long long)groups * strips,
                        32 * Smem::WARPS, 1, sizeof(Smem), stream, m, p, strips, Schedule{});
}
template <typename Smem>
cudaError_t backward_long(const RecurrenceParams& p, const RecurrenceGrads& r, int groups, float* part,
                          cudaStream_t stream) {
    const int strips = (p.C + kStrip - 1) / kStrip;
    Maps m;
    if (!make_maps(m, p, r.grad_out, Smem::kRows)) return cudaErrorNotSupported;
    return launch_tiles(recurrence_tile_backward_kernel<Smem, 1, true>, (long long)groups * strips,
                        32 * Smem::WARPS, 1, sizeof(Smem), stream, m, p, r, part, strips, Schedule{});
}

template <typename Tin>
cudaError_t forward(const RecurrenceParams& call, cudaStream_t stream) {
    using F = typename Forms<Tin>::Fwd;
    RecurrenceParams p = call;
    static Capacity wide, pair;
    Plan plan = {};
    offer_single<F>(&plan, p);
    if (sequential(p, plan, 620, sizeof(Tin) == 2 ? 0.0023 : 0.0026)) {
        const dim3 grid((unsigned)((p.C / 2 + kSeqThreads - 1) / kSeqThreads),
                        (unsigned)std::min(p.nseq, 65535));
        const Long rest = long_limit(p, 620);
        p.limit = rest.limit;
        recurrence_seq_kernel<Tin><<<grid, kSeqThreads, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        return e != cudaSuccess || !rest.groups ? e
                                                : forward_long<typename F::One>(p, rest.groups, stream);
    }
    cudaError_t e = offer_clusters<typename F::Wide>(
        &plan, p, kWideForm, recurrence_tile_kernel<typename F::Wide, 1>, wide, F::kWide, kWideRank,
        F::kWideStart);
    if (e == cudaSuccess)
        e = offer_clusters<typename F::Pair>(
            &plan, p, kPairForm, recurrence_tile_kernel<typename F::Pair, 2>, pair, F::kPair,
            kPairRank, F::kPairStart);
    if (e != cudaSuccess) return e;
    switch (plan.form) {
        case kOneForm: return forward_tiles<typename F::One, 1>(p, plan, stream);
        case kManyForm: return forward_tiles<typename F::Many, 2>(p, plan, stream);
        case kCrowdForm: return forward_tiles<typename F::Crowd, 3>(p, plan, stream);
        case kWideForm: return forward_tiles<typename F::Wide, 1>(p, plan, stream);
        default: return forward_tiles<typename F::Pair, 2>(p, plan, stream);
    }
}

template <typename Tin>
cudaError_t backward(const RecurrenceParams& call, const RecurrenceGrads& r, cudaStream_t stream) {
    using F = typename Forms<Tin>::Bwd;
    RecurrenceParams p = call;
    static Capacity wide, pair;
    Plan plan = {};
    offer_single<F>(&plan, p);
    if (sequential(p, plan, 750, sizeof(Tin) == 2 ? 0.0038 : 0.0088)) {
        const Long rest = long_limit(p, 750);
        p.limit = rest.limit;
        const int rows = seq_rows(p), all = rows + rest.groups;
        float* part = nullptr;
        cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * all * 2 * p.C, stream);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)((p.C / 2 + kSeqThreads - 1) / kSeqThreads), (unsigned)rows);
        recurrence_seq_backward_kernel<Tin><<<grid, kSeqThreads, 0, stream>>>(p, r, part);
        e = cudaGetLastError();
        if (e == cudaSuccess && rest.groups)
            e = backward_long<typename F::One>(p, r, rest.groups, part + (size_t)rows * 2 * p.C, stream);
        if (e == cudaSuccess)
            e = launch_column_sum(part, all, 2 * p.C, r.grad_A_log, p.C, r.grad_dt_bias, stream);
        const cudaError_t f = cudaFreeAsync(part, stream);
        return e != cudaSuccess ? e : f;
    }
    cudaError_t e = offer_clusters<typename F::Wide>(
        &plan, p, kWideForm, recurrence_tile_backward_kernel<typename F::Wide, 1>, wide, F::kWide,
        kWideRank, F::kWideStart);
    if (e == cudaSuccess)
        e = offer_clusters<typename F::Pair>(
            &plan, p, kPairForm, recurrence_tile_backward_kernel<typename F::Pair, 2>, pair,
            F::kPair, kPairRank, F::kPairStart);
    if (e != cudaSuccess) return e;
    switch (plan.form) {
        case kOneForm: return backward_tiles<typename F::One, 1>(p, r, plan, stream);
        case kManyForm: return backward_tiles<typename F::Many, 2>(p, r, plan, stream);
        case kCrowdForm: return backward_tiles<typename F::Crowd, 3>(p, r, plan, stream);
        case kWideForm: return backward_tiles<typename F::Wide, 1>(p, r, plan, stream);
        default: return backward_tiles<typename F::Pair, 2>(p, r, plan, stream);
    }
}

}  // namespace

cudaError_t launch_recurrence(const RecurrenceParams& p, cudaStream_t stream) {
    return p.in == InType::BF16 ? forward<__nv_bfloat16>(p, stream) : forward<float>(p, stream);
}

cudaError_t launch_recurrence_backward(const RecurrenceParams& p, const RecurrenceGrads& r,
                                       cudaStream_t stream) {
    return p.in == InType::BF16 ? backward<__nv_bfloat16>(p, r, stream)
                                : backward<float>(p, r, stream);
}

int read_and_clear_recurrence_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_recurrence_status, sizeof(int)) != cudaSuccess) return -1;
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_recurrence_status, &zero, sizeof(int));
    }
    return v;
}

}  // namespace gdr

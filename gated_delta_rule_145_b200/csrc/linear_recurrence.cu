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

// The gates of two channels in base 2, as the special-function unit's exponential takes them:
// A = -exp(A_log), bias = dt_bias log2(e).
struct Channels {
    float2 A, bias;
};

// zl = log2(e) z for z = a + dt_bias; t = e^{-|z|} in (0, 1]; y = A log2(e) softplus(z), the
// base-2 log-decay.  softplus(z) = max(z, 0) + log1p(t) and log2(e) log1p(t) = t Q(t), Q the
// degree-8 polynomial whose largest relative error on [0, 1] is smallest (3e-8; a weighted
// least-squares fit).  Small values of softplus are slow channels, whose state sums over
// many tokens: there the relative error of the log-decay, not the absolute one, is what the
// result sees, so log(1 + t) from the special-function unit (absolute error) will not do.
struct Gate {
    float2 zl, t, y;
};
__device__ __forceinline__ Gate decay_gate(float2 a, const Channels& ch) {
    Gate g;
    g.zl = __ffma2_rn(a, bcast2(kLog2e), ch.bias);
    g.t = ex2f2(make_float2(-fabsf(g.zl.x), -fabsf(g.zl.y)));
    float2 q = bcast2(7.549088448e-03f);
    q = __ffma2_rn(q, g.t, bcast2(-4.256669804e-02f));
    q = __ffma2_rn(q, g.t, bcast2(1.128556207e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-1.971185058e-01f));
    q = __ffma2_rn(q, g.t, bcast2(2.756412029e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-3.584084213e-01f));
    q = __ffma2_rn(q, g.t, bcast2(4.806929529e-01f));
    q = __ffma2_rn(q, g.t, bcast2(-7.213401794e-01f));
    q = __ffma2_rn(q, g.t, bcast2(1.442695022e+00f));
    q = __ffma2_rn(q, g.t, make_float2(fmaxf(g.zl.x, 0.f), fmaxf(g.zl.y, 0.f)));
    g.y = __fmul2_rn(ch.A, q);
    return g;
}

// x sigmoid(b)
__device__ __forceinline__ float2 gated_input(float2 x, float2 b) {
    const float2 e = ex2f2(__fmul2_rn(b, bcast2(-kLog2e)));
    return __fmul2_rn(x, rcpf2(__fadd2_rn(e, bcast2(1.f))));
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

// One token's backward step on two channels: its decay (and its base-2 logarithm y), and the
// factors of D, the gradient of its h, in dx, db, da and (times log2 e) dA_log, from the
// inputs and the state before the token.  sigmoid(v) is r = 1 / (1 + t) for v >= 0 and t r
// below, t = e^{-|v|}, so that small values keep their relative accuracy; sigmoid(v) (1 -
// sigmoid(v)) is t r^2 for both signs.  Both forms of the backward pass use it, so they agree
// bit for bit where they add in the same order.
struct GradFactors {
    float2 lam, x, b, a, A;
};
__device__ __forceinline__ GradFactors grad_factors(float2 x, float2 a, float2 b, float2 prev,
                                                    const Channels& ch, float2& y) {
    const Gate g = decay_gate(a, ch);
    y = g.y;
    GradFactors f;
    f.lam = ex2f2(g.y);
    const float2 rz = rcpf2(__fadd2_rn(g.t, bcast2(1.f))), tz = __fmul2_rn(g.t, rz);
    const float2 slope = make_float2(g.zl.x >= 0.f ? rz.x : tz.x, g.zl.y >= 0.f ? rz.y : tz.y);
    const float2 bl = __fmul2_rn(b, bcast2(kLog2e));
    const float2 tb = ex2f2(make_float2(-fabsf(bl.x), -fabsf(bl.y)));
    const float2 rb = rcpf2(__fadd2_rn(tb, bcast2(1.f))), tr = __fmul2_rn(tb, rb);
    f.x = make_float2(bl.x >= 0.f ? rb.x : tr.x, bl.y >= 0.f ? rb.y : tr.y);
    f.b = __fmul2_rn(x, __fmul2_rn(rb, tr));
    const float2 lp = __fmul2_rn(f.lam, prev);
    f.a = __fmul2_rn(__fmul2_rn(lp, ch.A), slope);
    f.A = __fmul2_rn(lp, g.y);
    return f;
}
template <typename Tin>
__device__ __forceinline__ void store_grads(const GradFactors& f, float2 D, Tin* dx, Tin* da,
                                            Tin* db, float2& acc_A, float2& acc_bias) {
    const float2 va = __fmul2_rn(f.a, D);
    store_pair(dx, __fmul2_rn(f.x, D));
    store_pair(da, va);
    store_pair(db, __fmul2_rn(f.b, D));
    acc_A = __ffma2_rn(f.A, D, acc_A);
    acc_bias = __fadd2_rn(acc_bias, va);
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
            h = __ffma2_rn(ex2f2(g.y), h, gated_input(xv, bv));
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
            D = __fadd2_rn(load_pair(r.grad_out + t * p.C + c), D);
            float2 y;
            const GradFactors f = grad_factors(load_pair(x + t * p.ld), load_pair(a + t * p.ld),
                                               load_pair(b + t * p.ld), prev, ch, y);
            store_grads(f, D, dx + t * r.ld_grad, da + t * r.ld_grad, db + t * r.ld_grad, acc_A,
                        acc_bias);
            D = __fmul2_rn(f.lam, D);
        }
        if (r.grad_init) *reinterpret_cast<float2*>(r.grad_init + at) = D;
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
// read twice and no CTA waits for one outside its cluster.
//
// Decays are composed as sums of log-decays.  From tile to tile a factor P near 1 acts
// through W = P - 1, formed as expm1 of its tile's sum: a slow channel's state lasts over
// thousands of tokens, and factors rounded near 1 would lose in every tile what the small
// W does not.  A factor below 2^-0.5 acts as P itself: there S + W S would cancel, and a
// large forgotten state would leave its rounding error in a small new one.
constexpr int kStrip = 64;
constexpr int kMaxCluster = 8;

// Shared memory of a CTA: per slot the x, a, b tiles, and for the backward pass dout's.
template <typename Tin_, int WARPS_, int TOK_, int STAGES_, bool Grad>
struct alignas(128) TileSmem {
    using Tin = Tin_;
    static constexpr int WARPS = WARPS_, TOK = TOK_, STAGES = STAGES_, kRows = WARPS * TOK;
    static_assert(WARPS >= kMaxCluster, "warp w sends to peer w");
    struct alignas(128) Slot {
        Tin in[3][kRows][kStrip];
        float dout[Grad ? kRows : 1][Grad ? kStrip : 4];
    };
    Slot slot[STAGES];
    float4 part[2][WARPS][32];       // per warp and lane: P pair, H pair; by step parity
    float2 log_part[2][WARPS][32];   // log2 of P
    // The cluster's tiles: coded factor pair, H pair; by step modulo 4.  A CTA publishes step
    // s + 4 only once it has every peer's step s + 2, which a peer publishes after all its
    // warps are done with step s: nothing still unread is overwritten.
    float4 peer[4][kMaxCluster][32];
    uint64_t full[STAGES], peers_in[4];
};

// The factor 2^y, y <= 0, coded for carry(): for y > -0.5, W = expm1(y ln 2) with its sign
// bit set (y times the degree-4 polynomial nearest to (2^y - 1) / y on [-0.5, 0], relative error
// 1.3e-8; a weighted least-squares fit), else 2^y itself, its sign bit clear.
__device__ __forceinline__ float code_factor(float y) {
    float q = 1.154452213e-03f;
    q = fmaf(q, y, 9.541281499e-03f);
    q = fmaf(q, y, 5.549040809e-02f);
    q = fmaf(q, y, 2.402256429e-01f);
    q = fmaf(q, y, 6.931471825e-01f);
    return y > -0.5f ? __int_as_float(__float_as_int(q * y) | 0x80000000) : ex2f(y);
}
// S <- 2^y S + H, the factor coded
__device__ __forceinline__ float carry(float S, float code, float H) {
    return fmaf(code, S, H) + (__float_as_int(code) < 0 ? S : 0.f);
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
    j.P = ex2f2(Gp);
    j.H = Hp;
    j.all = make_float4(code_factor(G.x), code_factor(G.y), H.x, H.y);
    if constexpr (Cluster) {
        uint64_t* bar = &sm.peers_in[step & 3];
        const uint32_t K = cluster_size();
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(bar, K * (uint32_t)sizeof(sm.peer[0][0]));
        if (warp < K) store_peer(&sm.peer[step & 3][cluster_rank()][lane], bar, warp, j.all);
    }
    return j;
}

// The state before this warp's tokens of the step; S moves from before the step to behind it.
template <bool Cluster, typename Smem>
__device__ __forceinline__ float2 start_state(Smem& sm, const Joined& j, int step, int lane,
                                              float2& S, bool& dead) {
    float2 in = S;
    if constexpr (Cluster) {
        if (!dead && !tc::mbar_wait(&sm.peers_in[step & 3], (uint32_t)(step >> 2) & 1u)) {
            dead = true;
            if (lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        const uint32_t K = cluster_size(), rank = cluster_rank();
        for (uint32_t k = 0; k < K; ++k) {
            if (k == rank) in = S;
            const float4 v = sm.peer[step & 3][k][lane];
            S = make_float2(carry(S.x, v.x, v.z), carry(S.y, v.y, v.w));
        }
    } else {
        S = make_float2(carry(S.x, j.all.x, j.all.z), carry(S.y, j.all.y, j.all.w));
    }
    return __ffma2_rn(j.P, in, j.H);
}

// What the CTAs of both tiled kernels share: their place, their tokens, their barriers.
struct Place {
    int warp, lane, K, rank, seq, c0, c, tiles, steps;
    long long t0, t1;
    bool in_c;
};
template <bool Cluster>
__device__ __forceinline__ Place place_of(const RecurrenceParams& p, int strips, int rows) {
    Place w;
    w.warp = threadIdx.x / 32;
    w.lane = threadIdx.x % 32;
    w.K = Cluster ? (int)cluster_size() : 1;
    w.rank = Cluster ? (int)cluster_rank() : 0;
    const int unit = blockIdx.x / w.K;
    w.seq = unit / strips;
    w.c0 = unit % strips * kStrip;
    w.c = w.c0 + 2 * w.lane;
    w.in_c = w.c < p.C;  // C is even
    seq_bounds(p.cu_seqlens, w.seq, p.T, w.t0, w.t1);
    w.tiles = (int)((w.t1 - w.t0 + rows - 1) / rows);
    w.steps = (w.tiles + w.K - 1) / w.K;
    return w;
}
template <typename Smem>
__device__ __forceinline__ void init_barriers(Smem& sm) {
    for (int i = 0; i < Smem::STAGES; ++i) tc::mbar_init(&sm.full[i], 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(&sm.peers_in[i], 1);
    tc::mbar_init_fence();
}

template <typename Smem, int Blocks, bool Cluster>
__global__ void __launch_bounds__(32 * Smem::WARPS, Blocks)
recurrence_tile_kernel(const __grid_constant__ Maps maps, RecurrenceParams p, int strips) {
    constexpr int TOK = Smem::TOK, STAGES = Smem::STAGES, kRows = Smem::kRows;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const Place w = place_of<Cluster>(p, strips, kRows);
    Channels ch = {};
    if (w.in_c) ch = load_channels(p.A_log, p.dt_bias, w.c);
    const size_t at = (size_t)w.seq * p.C + w.c;
    float2 S = w.in_c && p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                      : make_float2(0.f, 0.f);
    int issued = 0;
    if (threadIdx.x == 0) {
        init_barriers(sm);
        for (; issued < STAGES && issued * w.K + w.rank < w.tiles; ++issued)
            load_tile<false>(sm, issued, maps, w.c0,
                             (int)(w.t0 + (long long)(issued * w.K + w.rank) * kRows));
    }
    // the barriers are set up; in a cluster, every CTA has started and has read its state
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    bool dead = false;
    struct Held {
        float2 lam[TOK], u[TOK];
        Joined j;
    };
    // tokens of this warp in a step: the first one, and how many are within the sequence
    auto first_of = [&](int step) {
        return w.t0 + (long long)(step * w.K + w.rank) * kRows + w.warp * TOK;
    };
    auto live_of = [&](long long first) { return (int)min((long long)TOK, max(0LL, w.t1 - first)); };
    // the run from zero, up to the exchange
    auto read_tile = [&](int step, Held& k) {
        const int st = step % STAGES, buf = step & 1, live = live_of(first_of(step));
        if (step * w.K + w.rank < w.tiles && !dead &&
            !tc::mbar_wait(&sm.full[st], (uint32_t)(step / STAGES) & 1u)) {
            dead = true;
            if (w.lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        float2 G = make_float2(0.f, 0.f), H = G;
        const auto* row = &sm.slot[st].in[0][w.warp * TOK][2 * w.lane];
        auto gates = [&](int i) {
            const float2 xv = smem_pair(row + i * kStrip);
            const float2 av = smem_pair(row + (kRows + i) * kStrip);
            const float2 bv = smem_pair(row + (2 * kRows + i) * kStrip);
            const float2 y = decay_gate(av, ch).y;
            k.lam[i] = ex2f2(y);
            k.u[i] = gated_input(xv, bv);
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
        sm.part[buf][w.warp][w.lane] = make_float4(ex2f(G.x), ex2f(G.y), H.x, H.y);
        sm.log_part[buf][w.warp][w.lane] = G;
        __syncthreads();
        // every warp has read the tile: its slot takes the tile STAGES steps ahead
        if (threadIdx.x == 0 && !dead && issued * w.K + w.rank < w.tiles) {
            load_tile<false>(sm, st, maps, w.c0,
                             (int)(w.t0 + (long long)(issued * w.K + w.rank) * kRows));
            ++issued;
        }
        k.j = publish<Cluster>(sm, step, w.warp, w.lane);
    };
    // the run from the true start state
    auto write_tile = [&](int step, const Held& k) {
        float2 h = start_state<Cluster>(sm, k.j, step, w.lane, S, dead);
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
    if constexpr (Cluster) {
        // a step's exchange runs while the next step's tile is read
        Held even, odd;
        if (w.steps > 0) read_tile(0, even);
        for (int step = 0; step < w.steps; step += 2) {
            if (step + 1 < w.steps) read_tile(step + 1, odd);
            write_tile(step, even);
            if (step + 1 < w.steps) {
                if (step + 2 < w.steps) read_tile(step + 2, even);
                write_tile(step + 1, odd);
            }
        }
    } else {
        Held k;
        for (int step = 0; step < w.steps; ++step) {
            read_tile(step, k);
            write_tile(step, k);
        }
    }
    if (w.tiles == 0 && w.rank == 0 && w.warp == 0 && w.in_c && p.final_state)
        *reinterpret_cast<float2*>(p.final_state + at) = S;
    if (dead && threadIdx.x == 0) wait_in_flight(sm.full, STAGES, issued);
    // no CTA leaves while a peer may still store to it
    if constexpr (Cluster) cluster_barrier();
}

// The same pass against time: with E the gradient that reaches h_t from later tokens,
// D_t = dout_t + E and E <- exp(g_t) D_t, so tokens are taken from the last one back and a
// warp's pair is (P, H) of E.  Tiles are counted from the sequence's end.  Everything that
// multiplies D is formed while the tile is read, so that the second run over a warp's tokens,
// after the join, is short.  h comes by plain loads, one step ahead.
// part [units * K][2 C]: each CTA's sums for A_log and dt_bias.
template <typename Smem, int Blocks, bool Cluster>
__global__ void __launch_bounds__(32 * Smem::WARPS, Blocks)
recurrence_tile_backward_kernel(const __grid_constant__ Maps maps, RecurrenceParams p,
                                RecurrenceGrads r, float* part, int strips) {
    constexpr int TOK = Smem::TOK, STAGES = Smem::STAGES, kRows = Smem::kRows;
    using Tin = typename Smem::Tin;
    // steps after which a tile's dout is no longer needed: the exchange takes one of two
    constexpr int kHeld = Cluster ? 2 : 1;
    static_assert(STAGES > kHeld, "a slot has to be free for the next tile");
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const Place w = place_of<Cluster>(p, strips, kRows);
    Channels ch = {};
    if (w.in_c) ch = load_channels(p.A_log, p.dt_bias, w.c);
    const size_t at = (size_t)w.seq * p.C + w.c;
    const float2 zero = make_float2(0.f, 0.f);
    float2 S = w.in_c && r.grad_final ? *reinterpret_cast<const float2*>(r.grad_final + at) : zero;
    int issued = 0;
    // a sequence's first tile may start before it, at a negative row even
    auto first_row = [&](int step) {
        return (int)(w.t1 - (long long)(step * w.K + w.rank + 1) * kRows);
    };
    if (threadIdx.x == 0) {
        init_barriers(sm);
        for (; issued < STAGES && issued * w.K + w.rank < w.tiles; ++issued)
            load_tile<true>(sm, issued, maps, w.c0, first_row(issued));
    }
    // the states before a step's tokens of this warp: last, last - 1, ...
    float2 prev[TOK];
    auto load_prev = [&](int step) {
        const long long last = w.t1 - (long long)(step * w.K + w.rank) * kRows - w.warp * TOK - 1;
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
    load_prev(0);
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    float2 acc_A = zero, acc_bias = zero;
    bool dead = false;
    struct Held {
        GradFactors f[TOK];
        Joined j;
    };
    auto last_of = [&](int step) {
        return w.t1 - (long long)(step * w.K + w.rank) * kRows - w.warp * TOK - 1;
    };
    auto live_of = [&](long long last) {
        return (int)min((long long)TOK, max(0LL, last + 1 - w.t0));
    };
    auto read_tile = [&](int step, Held& k) {
        const int st = step % STAGES, buf = step & 1, live = live_of(last_of(step));
        if (step * w.K + w.rank < w.tiles && !dead &&
            !tc::mbar_wait(&sm.full[st], (uint32_t)(step / STAGES) & 1u)) {
            dead = true;
            if (w.lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        float2 G = zero, H = zero;
        const auto* row = &sm.slot[st].in[0][kRows - 1 - w.warp * TOK][2 * w.lane];
        const float* dout = &sm.slot[st].dout[kRows - 1 - w.warp * TOK][2 * w.lane];
        auto gates = [&](int i) {
            float2 y;
            k.f[i] = grad_factors(smem_pair(row - i * kStrip), smem_pair(row + (kRows - i) * kStrip),
                                  smem_pair(row + (2 * kRows - i) * kStrip), prev[i], ch, y);
            G = __fadd2_rn(G, y);
            H = __fmul2_rn(k.f[i].lam, __fadd2_rn(smem_pair(dout - i * kStrip), H));
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
        if (step + 1 < w.steps) load_prev(step + 1);
        sm.part[buf][w.warp][w.lane] = make_float4(ex2f(G.x), ex2f(G.y), H.x, H.y);
        sm.log_part[buf][w.warp][w.lane] = G;
        __syncthreads();
        // every warp is done with step - kHeld: its slot takes the tile STAGES steps later
        if (threadIdx.x == 0 && !dead && step >= kHeld && issued * w.K + w.rank < w.tiles) {
            load_tile<true>(sm, issued % STAGES, maps, w.c0, first_row(issued));
            ++issued;
        }
        k.j = publish<Cluster>(sm, step, w.warp, w.lane);
    };
    auto write_tile = [&](int step, const Held& k) {
        float2 E = start_state<Cluster>(sm, k.j, step, w.lane, S, dead);
        const long long last = last_of(step);
        const int live = live_of(last);
        const float* dout =
            &sm.slot[step % STAGES].dout[kRows - 1 - w.warp * TOK][2 * w.lane];
        if (w.in_c) {
            Tin* dx = static_cast<Tin*>(r.grad_x) + last * r.ld_grad + w.c;
            Tin* da = static_cast<Tin*>(r.grad_a) + last * r.ld_grad + w.c;
            Tin* db = static_cast<Tin*>(r.grad_b) + last * r.ld_grad + w.c;
            auto token = [&](int i) {
                const float2 D = __fadd2_rn(smem_pair(dout - i * kStrip), E);
                const long long o = i * r.ld_grad;
                store_grads(k.f[i], D, dx - o, da - o, db - o, acc_A, acc_bias);
                E = __fmul2_rn(k.f[i].lam, D);
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
    if constexpr (Cluster) {
        // a step's exchange runs while the next step's tile is read
        Held even, odd;
        if (w.steps > 0) read_tile(0, even);
        for (int step = 0; step < w.steps; step += 2) {
            if (step + 1 < w.steps) read_tile(step + 1, odd);
            write_tile(step, even);
            if (step + 1 < w.steps) {
                if (step + 2 < w.steps) read_tile(step + 2, even);
                write_tile(step + 1, odd);
            }
        }
    } else {
        Held k;
        for (int step = 0; step < w.steps; ++step) {
            read_tile(step, k);
            write_tile(step, k);
        }
    }
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
        float* o = part + ((size_t)w.seq * w.K + w.rank) * 2 * p.C + w.c;
        *reinterpret_cast<float2*>(o) = __fmul2_rn(make_float2(s.x, s.y), bcast2(kLn2));
        *reinterpret_cast<float2*>(o + p.C) = make_float2(s.z, s.w);
    }
    if (dead && threadIdx.x == 0) wait_in_flight(sm.full, STAGES, issued);
    if constexpr (Cluster) cluster_barrier();
}

// Rows of CTAs of the sequential form: the partial sums have one row each.
int seq_rows(int nseq) { return std::min(nseq, 64); }

// The tokens of a call's mean sequence; the host does not know packed sequences' lengths.
int mean_length(const RecurrenceParams& p) {
    return p.cu_seqlens ? (p.T + p.nseq - 1) / p.nseq : p.T;
}

// (sequence, strip of channels) pairs, each one chain of tiles.
long long units_of(const RecurrenceParams& p) {
    return (long long)p.nseq * ((p.C + kStrip - 1) / kStrip);
}

// Sequences of up to a warp's tokens leave the tiled form's other warps idle.
bool use_tiles(const RecurrenceParams& p) { return mean_length(p) > 16; }

// CTAs per cluster for `units` (sequence, strip) pairs of `tiles` tiles.  A cluster's CTAs
// take one SM each, so K of them for every unit pay only while the units leave SMs idle: the
// largest K whose clusters the device still holds at once, at one CTA per SM.  (96 units of
// 8192 tokens: 141 us forward with K = 1, 168 with K = 2, 178 with K = 3.)
template <typename Kernel>
cudaError_t cluster_of(Kernel kernel, int threads, size_t smem, long long units, int tiles, int* K) {
    *K = 1;
    const int most = (int)std::min<long long>({(long long)kMaxCluster, (long long)tiles,
                                               device_sms() / units});
    if (most < 2) return cudaSuccess;
    // clusters of k CTAs that the current device holds at once; asked once per kernel and device
    struct Held {
        std::atomic<int> fit[kMaxCluster + 1];
    };
    static Held held[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= 64)) e = cudaErrorInvalidDevice;
    if (e != cudaSuccess) return e;
    for (int k = most; k > 1; --k) {
        int fit = held[dev].fit[k].load();
        if (fit == 0) {
            cudaLaunchAttribute attr = {};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)k;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)k);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = allow_smem((const void*)kernel, smem);
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
            if (e != cudaSuccess) return e;
            held[dev].fit[k].store(std::max(fit, 1));
        }
        if (fit >= units) {
            *K = k;
            break;
        }
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

// Warps, tokens per warp, slots, CTAs per SM of each kernel.  Registers set the tokens (two
// values per token and channel forward, five backward, twice that in a cluster, where a
// warp holds two steps), shared memory the slots.
template <typename Tin, bool Cluster> struct Forms;
template <> struct Forms<__nv_bfloat16, false> {
    using Fwd = TileSmem<__nv_bfloat16, 8, 12, 2, false>;
    using Bwd = TileSmem<__nv_bfloat16, 8, 8, 3, true>;
    static constexpr int kFwdBlocks = 2;
};
template <> struct Forms<__nv_bfloat16, true> {
    using Fwd = TileSmem<__nv_bfloat16, 8, 16, 2, false>;
    using Bwd = TileSmem<__nv_bfloat16, 8, 8, 3, true>;
    static constexpr int kFwdBlocks = 1;
};
template <> struct Forms<float, false> {
    using Fwd = TileSmem<float, 8, 8, 2, false>;
    using Bwd = TileSmem<float, 8, 8, 3, true>;
    static constexpr int kFwdBlocks = 2;
};
template <> struct Forms<float, true> {
    using Fwd = TileSmem<float, 8, 8, 3, false>;
    using Bwd = TileSmem<float, 8, 8, 3, true>;
    static constexpr int kFwdBlocks = 1;
};

template <typename Tin, bool Cluster>
cudaError_t forward_tiles(const RecurrenceParams& p, int K, cudaStream_t stream) {
    using F = Forms<Tin, Cluster>;
    using Smem = typename F::Fwd;
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long grid = (long long)p.nseq * strips * K;
    Maps m;
    if (grid > 0x7fffffffLL || !make_maps(m, p, nullptr, Smem::kRows)) return cudaErrorNotSupported;
    return launch_tiles(recurrence_tile_kernel<Smem, F::kFwdBlocks, Cluster>, grid,
                        32 * Smem::WARPS, K, sizeof(Smem), stream, m, p, strips);
}

template <typename Tin, bool Cluster>
cudaError_t backward_tiles(const RecurrenceParams& p, const RecurrenceGrads& r, int K,
                           cudaStream_t stream) {
    using Smem = typename Forms<Tin, Cluster>::Bwd;
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long grid = (long long)p.nseq * strips * K, rows = (long long)p.nseq * K;
    Maps m;
    if (grid > 0x7fffffffLL || !make_maps(m, p, r.grad_out, Smem::kRows))
        return cudaErrorNotSupported;
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * rows * 2 * p.C, stream);
    if (e != cudaSuccess) return e;
    e = launch_tiles(recurrence_tile_backward_kernel<Smem, 1, Cluster>, grid,
                     32 * Smem::WARPS, K, sizeof(Smem), stream, m, p, r, part, strips);
    if (e == cudaSuccess)
        e = launch_column_sum(part, rows, 2 * p.C, r.grad_A_log, p.C, r.grad_dt_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
}

template <typename Tin>
cudaError_t forward_tiles(const RecurrenceParams& p, cudaStream_t stream) {
    using F = Forms<Tin, true>;
    using Smem = typename F::Fwd;
    int K = 1;
    const cudaError_t e =
        cluster_of(recurrence_tile_kernel<Smem, F::kFwdBlocks, true>, 32 * Smem::WARPS, sizeof(Smem),
                   units_of(p), (mean_length(p) + Smem::kRows - 1) / Smem::kRows, &K);
    if (e != cudaSuccess) return e;
    return K > 1 ? forward_tiles<Tin, true>(p, K, stream) : forward_tiles<Tin, false>(p, 1, stream);
}

template <typename Tin>
cudaError_t backward_tiles(const RecurrenceParams& p, const RecurrenceGrads& r,
                           cudaStream_t stream) {
    using Smem = typename Forms<Tin, true>::Bwd;
    int K = 1;
    const cudaError_t e =
        cluster_of(recurrence_tile_backward_kernel<Smem, 1, true>, 32 * Smem::WARPS, sizeof(Smem),
                   units_of(p), (mean_length(p) + Smem::kRows - 1) / Smem::kRows, &K);
    if (e != cudaSuccess) return e;
    return K > 1 ? backward_tiles<Tin, true>(p, r, K, stream)
                 : backward_tiles<Tin, false>(p, r, 1, stream);
}

}  // namespace

cudaError_t launch_recurrence(const RecurrenceParams& p, cudaStream_t stream) {
    if (use_tiles(p))
        return p.in == InType::BF16 ? forward_tiles<__nv_bfloat16>(p, stream)
                                    : forward_tiles<float>(p, stream);
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
    if (use_tiles(p))
        return p.in == InType::BF16 ? backward_tiles<__nv_bfloat16>(p, r, stream)
                                    : backward_tiles<float>(p, r, stream);
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

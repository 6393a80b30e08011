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
#include "tcgen05.cuh"
#include "tma_map.h"

namespace gdr {

namespace {

// Set by a tiled kernel that gave up a bounded wait; gdr_device_status reads it.
__device__ int g_recurrence_status;

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

// One token's backward step on two channels: its decay (and its base-2 logarithm y), and the
// factors of D, the gradient of its h, in dx, db, da and dA_log, from the inputs and the state
// before the token.  Both forms of the backward pass use it, so they agree bit for bit
// where they add in the same order.
struct GradFactors {
    float2 lam, x, b, a, A;
};
__device__ __forceinline__ GradFactors grad_factors(float2 x, float2 a, float2 b, float2 prev,
                                                    const Channels& ch, float2& y) {
    const Gate g = decay_gate(a, ch);
    float2 sz, si, ci;
    float unused;
    sigmoid_both(g.z.x, g.t.x, sz.x, unused);
    sigmoid_both(g.z.y, g.t.y, sz.y, unused);
    sigmoid_both(b.x, ex2f(-fabsf(b.x) * kLog2e), si.x, ci.x);
    sigmoid_both(b.y, ex2f(-fabsf(b.y) * kLog2e), si.y, ci.y);
    y = __fmul2_rn(ch.A2, g.p);
    GradFactors f;
    f.lam = ex2f2(y);
    const float2 lpA = __fmul2_rn(__fmul2_rn(f.lam, prev), ch.A);
    f.x = si;
    f.b = __fmul2_rn(x, __fmul2_rn(si, ci));
    f.a = __fmul2_rn(lpA, sz);
    f.A = __fmul2_rn(lpA, g.p);
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
    *reinterpret_cast<float2*>(row + c) = acc_A;
    *reinterpret_cast<float2*>(row + p.C + c) = acc_bias;
}

// ------------------------------------------------------------------- tiled form
// One pass over the data with the time axis split three ways.  A CTA owns a strip of 64
// channels of one sequence and takes tiles of kWarps * TOK tokens; warp w holds tokens
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
constexpr int kWarps = 8;
constexpr int kStrip = 64;
constexpr int kMaxCluster = 8;
constexpr int kTileThreads = 32 * kWarps;

template <typename Tin, int TOK, int STAGES>
struct alignas(128) TileSmem {
    static constexpr int kRows = kWarps * TOK;
    Tin in[STAGES][3][kRows][kStrip];
    float4 part[2][kWarps][32];       // per warp and lane: P pair, H pair; by step parity
    float2 log_part[2][kWarps][32];   // log2 of P
    float4 peer[2][kMaxCluster][32];  // the cluster's tiles: coded factor pair, H pair
    uint64_t full[STAGES];
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
// Store to the same shared-memory variable of CTA `rank` of this cluster.
__device__ __forceinline__ void store_peer(float4* p, uint32_t rank, float4 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ float2 smem_pair(const float* p) {
    return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ float2 smem_pair(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// The three input tiles whose first row is token `row` (before or past the tensor: zeros).
template <typename Smem>
__device__ __forceinline__ void load_tile(Smem& sm, int st, const CUtensorMap* mx,
                                          const CUtensorMap* ma, const CUtensorMap* mb, int c0,
                                          int row) {
    tc::mbar_arrive_expect_tx(&sm.full[st], (uint32_t)sizeof(sm.in[0]));
    tc::tma_load_2d(&sm.in[st][0][0][0], mx, c0, row, &sm.full[st]);
    tc::tma_load_2d(&sm.in[st][1][0][0], ma, c0, row, &sm.full[st]);
    tc::tma_load_2d(&sm.in[st][2][0][0], mb, c0, row, &sm.full[st]);
}

// After a wait that gave up, copies may still be in flight: the CTA stays for them (each
// wait is bounded too).
template <typename Smem>
__device__ __noinline__ void wait_in_flight(Smem& sm, int stages, int tiles, int K, int rank) {
    const int last = (tiles - 1 - rank) / K;  // this CTA's last step with a tile
    for (int i = 0; i < stages; ++i) {
        const int s = last - (last - i + stages) % stages;
        if (s >= 0) tc::mbar_wait(&sm.full[i], (uint32_t)(s / stages) & 1u);
    }
}

// From the warps' pairs in sm.part[buf] and the state S before the cluster's step: the state
// before this warp's tokens; S moves past the step.
template <bool Cluster, typename Smem>
__device__ __forceinline__ float2 join(Smem& sm, int buf, int warp, int lane, float2& S) {
    float2 G = make_float2(0.f, 0.f), H = G, Gp = G, Hp = G;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) Gp = G, Hp = H;
        const float4 v = sm.part[buf][w][lane];
        H = __ffma2_rn(make_float2(v.x, v.y), H, make_float2(v.z, v.w));
        G = __fadd2_rn(G, sm.log_part[buf][w][lane]);
    }
    const float4 all = make_float4(code_factor(G.x), code_factor(G.y), H.x, H.y);
    float2 in = S;
    if constexpr (Cluster) {
        const uint32_t K = cluster_size(), rank = cluster_rank();
        if (warp < K) store_peer(&sm.peer[buf][rank][lane], warp, all);
        cluster_barrier();
        for (uint32_t k = 0; k < K; ++k) {
            if (k == rank) in = S;
            const float4 v = sm.peer[buf][k][lane];
            S = make_float2(carry(S.x, v.x, v.z), carry(S.y, v.y, v.w));
        }
    } else {
        S = make_float2(carry(S.x, all.x, all.z), carry(S.y, all.y, all.w));
    }
    return __ffma2_rn(ex2f2(Gp), in, Hp);
}

template <typename Tin, int TOK, int STAGES, bool Cluster>
__global__ void __launch_bounds__(kTileThreads, 2)
recurrence_tile_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb, RecurrenceParams p, int strips) {
    using Smem = TileSmem<Tin, TOK, STAGES>;
    constexpr int kRows = Smem::kRows;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int K = Cluster ? (int)cluster_size() : 1, rank = Cluster ? (int)cluster_rank() : 0;
    const int unit = blockIdx.x / K, strip = unit % strips, seq = unit / strips;
    long long t0, t1;
    seq_bounds(p.cu_seqlens, seq, p.T, t0, t1);
    const int tiles = (int)((t1 - t0 + kRows - 1) / kRows), steps = (tiles + K - 1) / K;
    const int c0 = strip * kStrip, c = c0 + 2 * lane;
    const bool in_c = c < p.C;  // C is even
    Channels ch = {};
    if (in_c) ch = load_channels(p.A_log, p.dt_bias, c);
    const size_t at = (size_t)seq * p.C + c;
    float2 S = in_c && p.init_state ? *reinterpret_cast<const float2*>(p.init_state + at)
                                    : make_float2(0.f, 0.f);
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&sm.full[i], 1);
        tc::mbar_init_fence();
        for (int i = 0; i < STAGES && i * K + rank < tiles; ++i)
            load_tile(sm, i, &mx, &ma, &mb, c0, (int)(t0 + (long long)(i * K + rank) * kRows));
    }
    // the barriers are set up; in a cluster, every CTA has started and has read its state
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    bool dead = false;
    for (int step = 0; step < steps; ++step) {
        const int tile = step * K + rank, st = step % STAGES, buf = step & 1;
        const bool have = tile < tiles;
        // tokens of this warp within the sequence
        const long long w0 = t0 + (long long)tile * kRows + warp * TOK;
        const int live = (int)min((long long)TOK, max(0LL, t1 - w0));
        if (have && !dead && !tc::mbar_wait(&sm.full[st], (uint32_t)(step / STAGES) & 1u)) {
            dead = true;
            if (lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        float2 lam[TOK], u[TOK], G = make_float2(0.f, 0.f), H = G;
        const Tin* row = &sm.in[st][0][warp * TOK][2 * lane];
        auto gates = [&](int i) {
            const float2 xv = smem_pair(row + i * kStrip);
            const float2 av = smem_pair(row + (kRows + i) * kStrip);
            const float2 bv = smem_pair(row + (2 * kRows + i) * kStrip);
            const float2 y = __fmul2_rn(ch.A2, decay_gate(av, ch).p);
            lam[i] = ex2f2(y);
            u[i] = __fmul2_rn(sigmoid2(bv), xv);
            G = __fadd2_rn(G, y);
            H = __ffma2_rn(lam[i], H, u[i]);
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
                    lam[i] = make_float2(1.f, 1.f);
                    u[i] = make_float2(0.f, 0.f);
                }
            }
        }
        sm.part[buf][warp][lane] = make_float4(ex2f(G.x), ex2f(G.y), H.x, H.y);
        sm.log_part[buf][warp][lane] = G;
        __syncthreads();
        // every warp has read the tile: its slot takes the tile STAGES steps ahead
        if (threadIdx.x == 0 && !dead && tile + STAGES * K < tiles)
            load_tile(sm, st, &mx, &ma, &mb, c0,
                      (int)(t0 + (long long)(tile + STAGES * K) * kRows));
        float2 h = join<Cluster>(sm, buf, warp, lane, S);
        float* out = p.out + w0 * p.C + c;
        if (in_c) {
            if (live == TOK) {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    h = __ffma2_rn(lam[i], h, u[i]);
                    store_pair(out + (size_t)i * p.C, h);
                }
            } else {
#pragma unroll
                for (int i = 0; i < TOK; ++i) {
                    h = __ffma2_rn(lam[i], h, u[i]);
                    if (i < live) store_pair(out + (size_t)i * p.C, h);
                }
            }
            // the warp with the sequence's last token: its h, so that the two agree
            if (live > 0 && w0 + live == t1 && p.final_state)
                *reinterpret_cast<float2*>(p.final_state + at) = h;
        }
        __syncwarp();
    }
    if (tiles == 0 && rank == 0 && warp == 0 && in_c && p.final_state)
        *reinterpret_cast<float2*>(p.final_state + at) = S;
    if (dead && threadIdx.x == 0) wait_in_flight(sm, STAGES, tiles, K, rank);
}

// The same pass against time: with E the gradient that reaches h_t from later tokens,
// D_t = dout_t + E and E <- exp(g_t) D_t, so tokens are taken from the last one back and a
// warp's pair is (P, H) of E.  Tiles are counted from the sequence's end.  Everything that
// multiplies D is formed while the tile is read, so that the second run over a warp's tokens,
// after the join, is short.  dout and h come by plain loads issued before the tile is
// waited for.  part [units * K][2 C]: each CTA's sums for A_log and dt_bias.
template <typename Tin, int TOK, int STAGES, bool Cluster>
__global__ void __launch_bounds__(kTileThreads, 2)
recurrence_tile_backward_kernel(const __grid_constant__ CUtensorMap mx,
                                const __grid_constant__ CUtensorMap ma,
                                const __grid_constant__ CUtensorMap mb, RecurrenceParams p,
                                RecurrenceGrads r, float* part, int strips) {
    using Smem = TileSmem<Tin, TOK, STAGES>;
    constexpr int kRows = Smem::kRows;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int K = Cluster ? (int)cluster_size() : 1, rank = Cluster ? (int)cluster_rank() : 0;
    const int unit = blockIdx.x / K, strip = unit % strips, seq = unit / strips;
    long long t0, t1;
    seq_bounds(p.cu_seqlens, seq, p.T, t0, t1);
    const int tiles = (int)((t1 - t0 + kRows - 1) / kRows), steps = (tiles + K - 1) / K;
    const int c0 = strip * kStrip, c = c0 + 2 * lane;
    const bool in_c = c < p.C;  // C is even
    Channels ch = {};
    if (in_c) ch = load_channels(p.A_log, p.dt_bias, c);
    const size_t at = (size_t)seq * p.C + c;
    const float2 zero = make_float2(0.f, 0.f);
    float2 S = in_c && r.grad_final ? *reinterpret_cast<const float2*>(r.grad_final + at) : zero;
    const float2 init = in_c && p.init_state
                            ? *reinterpret_cast<const float2*>(p.init_state + at) : zero;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) tc::mbar_init(&sm.full[i], 1);
        tc::mbar_init_fence();
        // a sequence's first tile may start before it, at a negative row even
        for (int i = 0; i < STAGES && i * K + rank < tiles; ++i)
            load_tile(sm, i, &mx, &ma, &mb, c0, (int)(t1 - (long long)(i * K + rank + 1) * kRows));
    }
    if constexpr (Cluster) cluster_barrier(); else __syncthreads();
    float2 acc_A = zero, acc_bias = zero;
    bool dead = false;
    for (int step = 0; step < steps; ++step) {
        const int tile = step * K + rank, st = step % STAGES, buf = step & 1;
        const bool have = tile < tiles;
        // this warp's tokens: last, last - 1, ...
        const long long last = t1 - (long long)tile * kRows - warp * TOK - 1;
        const int live = have ? (int)min((long long)TOK, max(0LL, last + 1 - t0)) : 0;
        float2 d[TOK], prev[TOK];
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            const bool in = i < live && in_c;
            d[i] = in ? load_pair(r.grad_out + (last - i) * p.C + c) : zero;
            prev[i] = !in ? zero : last - i > t0 ? load_pair(p.out + (last - i - 1) * p.C + c) : init;
        }
        if (have && !dead && !tc::mbar_wait(&sm.full[st], (uint32_t)(step / STAGES) & 1u)) {
            dead = true;
            if (lane == 0) atomicExch(&g_recurrence_status, 1);
        }
        __syncwarp();
        GradFactors f[TOK];
        float2 G = zero, H = zero;
        const Tin* row = &sm.in[st][0][kRows - 1 - warp * TOK][2 * lane];
        auto gates = [&](int i) {
            float2 y;
            f[i] = grad_factors(smem_pair(row - i * kStrip), smem_pair(row + (kRows - i) * kStrip),
                                smem_pair(row + (2 * kRows - i) * kStrip), prev[i], ch, y);
            G = __fadd2_rn(G, y);
            H = __fmul2_rn(f[i].lam, __fadd2_rn(d[i], H));
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
        sm.part[buf][warp][lane] = make_float4(ex2f(G.x), ex2f(G.y), H.x, H.y);
        sm.log_part[buf][warp][lane] = G;
        __syncthreads();
        if (threadIdx.x == 0 && !dead && tile + STAGES * K < tiles)
            load_tile(sm, st, &mx, &ma, &mb, c0,
                      (int)(t1 - (long long)(tile + STAGES * K + 1) * kRows));
        float2 E = join<Cluster>(sm, buf, warp, lane, S);
        if (in_c) {
            Tin* dx = static_cast<Tin*>(r.grad_x) + last * r.ld_grad + c;
            Tin* da = static_cast<Tin*>(r.grad_a) + last * r.ld_grad + c;
            Tin* db = static_cast<Tin*>(r.grad_b) + last * r.ld_grad + c;
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                if (i < live) {
                    const float2 D = __fadd2_rn(d[i], E);
                    store_grads(f[i], D, dx - i * r.ld_grad, da - i * r.ld_grad,
                                db - i * r.ld_grad, acc_A, acc_bias);
                    E = __fmul2_rn(f[i].lam, D);
                }
            }
            // the warp with the sequence's first token
            if (live > 0 && last + 1 - live == t0 && r.grad_init)
                *reinterpret_cast<float2*>(r.grad_init + at) = E;
        }
        __syncwarp();
    }
    if (tiles == 0 && rank == 0 && warp == 0 && in_c && r.grad_init)
        *reinterpret_cast<float2*>(r.grad_init + at) = S;
    __syncthreads();
    sm.part[0][warp][lane] = make_float4(acc_A.x, acc_A.y, acc_bias.x, acc_bias.y);
    __syncthreads();
    if (warp == 0 && in_c) {
        float4 s = sm.part[0][0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 v = sm.part[0][w][lane];
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        float* o = part + ((size_t)seq * K + rank) * 2 * p.C + c;
        *reinterpret_cast<float2*>(o) = make_float2(s.x, s.y);
        *reinterpret_cast<float2*>(o + p.C) = make_float2(s.z, s.w);
    }
    if (dead && threadIdx.x == 0) wait_in_flight(sm, STAGES, tiles, K, rank);
}

// Rows of CTAs of the sequential form: the partial sums have one row each.
int seq_rows(int nseq) { return std::min(nseq, 64); }

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        n = 148;
    return n;
}

// The tokens of a call's mean sequence; the host does not know packed sequences' lengths.
int mean_length(const RecurrenceParams& p) {
    return p.cu_seqlens ? (p.T + p.nseq - 1) / p.nseq : p.T;
}

// Sequences of up to a warp's tokens leave the tiled form's other warps idle.
bool use_tiles(const RecurrenceParams& p) { return mean_length(p) > 16; }

// CTAs per cluster for `units` (sequence, strip) pairs of `tiles` tiles: the K that keeps the
// largest share of the SMs' slots (two CTAs each) at work until the last wave is done.
int cluster_of(long long units, int tiles) {
    const int sms = sm_count(), most = std::min(tiles, kMaxCluster);
    int best = 1;
    double best_share = 0.0;
    for (int K = 1; K <= most; ++K) {
        const long long n = units * K;
        const long long width = n <= sms ? sms : 2LL * sms;
        const double share = (double)n / (double)((n + width - 1) / width * width);
        if (share > best_share + 0.02) best = K, best_share = share;
    }
    return best;
}

template <typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, long long grid, int K, size_t smem, cudaStream_t stream,
                         Args... args) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kTileThreads);
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

struct Maps {
    CUtensorMap x, a, b;
};
bool make_maps(Maps& m, const RecurrenceParams& p, int rows_of_box) {
    const uint64_t rows = p.cu_seqlens ? (uint64_t)p.T : (uint64_t)p.nseq * p.T;
    const bool f32 = p.in == InType::F32;
    return make_map_pitched(&m.x, p.x, f32, p.C, rows, p.ld, kStrip, rows_of_box) &&
           make_map_pitched(&m.a, p.a, f32, p.C, rows, p.ld, kStrip, rows_of_box) &&
           make_map_pitched(&m.b, p.b, f32, p.C, rows, p.ld, kStrip, rows_of_box);
}

// Tokens per warp.  Forward holds two values per token and channel in registers, 16 bf16
// tokens; fp32 tiles are twice as large in shared memory, and backward holds six values.
template <typename Tin> constexpr int kFwdTok = sizeof(Tin) == 2 ? 16 : 8;
constexpr int kBwdTok = 8;
constexpr int kStages = 2;

template <typename Tin>
cudaError_t forward_tiles(const RecurrenceParams& p, cudaStream_t stream) {
    using Smem = TileSmem<Tin, kFwdTok<Tin>, kStages>;
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long units = (long long)p.nseq * strips;
    const int K = cluster_of(units, (mean_length(p) + Smem::kRows - 1) / Smem::kRows);
    Maps m;
    if (units * K > 0x7fffffffLL || !make_maps(m, p, Smem::kRows)) return cudaErrorNotSupported;
    auto kernel = K > 1 ? recurrence_tile_kernel<Tin, kFwdTok<Tin>, kStages, true>
                        : recurrence_tile_kernel<Tin, kFwdTok<Tin>, kStages, false>;
    return launch_tiles(kernel, units * K, K, sizeof(Smem), stream, m.x, m.a, m.b, p, strips);
}

template <typename Tin>
cudaError_t backward_tiles(const RecurrenceParams& p, const RecurrenceGrads& r, cudaStream_t stream) {
    using Smem = TileSmem<Tin, kBwdTok, kStages>;
    const int strips = (p.C + kStrip - 1) / kStrip;
    const long long units = (long long)p.nseq * strips;
    const int K = cluster_of(units, (mean_length(p) + Smem::kRows - 1) / Smem::kRows);
    Maps m;
    if (units * K > 0x7fffffffLL || !make_maps(m, p, Smem::kRows)) return cudaErrorNotSupported;
    const long long rows = (long long)p.nseq * K;
    float* part = nullptr;
    cudaError_t e = workspace_alloc((void**)&part, sizeof(float) * rows * 2 * p.C, stream);
    if (e != cudaSuccess) return e;
    auto kernel = K > 1 ? recurrence_tile_backward_kernel<Tin, kBwdTok, kStages, true>
                        : recurrence_tile_backward_kernel<Tin, kBwdTok, kStages, false>;
    e = launch_tiles(kernel, units * K, K, sizeof(Smem), stream, m.x, m.a, m.b, p, r, part, strips);
    if (e == cudaSuccess)
        e = launch_column_sum(part, rows, 2 * p.C, r.grad_A_log, p.C, r.grad_dt_bias, stream);
    const cudaError_t f = cudaFreeAsync(part, stream);
    return e != cudaSuccess ? e : f;
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

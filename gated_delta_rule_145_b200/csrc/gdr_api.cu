// gdr_api.cu -- the C ABI of libgdr.so (declared in include/gdr.h): argument checks,
// then kernel launches.  Nothing is enqueued unless every check passes; no call
// synchronises the stream.  The tensor-core prefill takes its workspace from a private
// stream-ordered pool (workspace.cu).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdr.h"
#include "gdr_internal.h"

namespace {

using gdr::FwdParams;
using gdr::InType;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

bool head_size_built(int dk, int dv) { return dk == dv && (dk == 32 || dk == 64 || dk == 128); }

int check_common(const FwdParams& p, int elem_bytes) {
    // with no tokens the per-token tensors may be empty (NULL); the per-head ones are read
    if (!p.A_log || !p.dt_bias) return GDR_ERR_NULL;
    if (p.T > 0 && (!p.q || !p.k || !p.v || !p.a || !p.b || !p.out)) return GDR_ERR_NULL;
    if (p.nseq < 1 || p.T < 0 || p.Hk < 1 || p.Hv < 1 || p.Hv % p.Hk != 0) return GDR_ERR_SHAPE;
    if (!head_size_built(p.dk, p.dv)) return GDR_ERR_UNSUPPORTED;
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.out, 16) ||
        !aligned(p.a, elem_bytes) || !aligned(p.b, elem_bytes) || !aligned(p.A_log, 4) ||
        !aligned(p.dt_bias, 4) || !aligned(p.init_state, 16) || !aligned(p.final_state, 16) ||
        !aligned(p.cu_seqlens, 4))
        return GDR_ERR_ALIGN;
    // grids are 1-D over (sequence, head[, slice]); keep them within 2^31 - 1
    if ((long long)p.nseq * p.Hv * 4 > 0x7fffffffLL) return GDR_ERR_SHAPE;
    return GDR_OK;
}

int to_status(cudaError_t e) {
    if (e == cudaSuccess) return GDR_OK;
    cudaGetLastError();  // it is reported here: left behind, the next call's launch would report it again
    if (e == cudaErrorNotSupported) return GDR_ERR_UNSUPPORTED;
    if (e == cudaErrorMemoryAllocation) return GDR_ERR_OOM;
    return GDR_ERR_CUDA;
}

FwdParams make_params(const void* q, const void* k, const void* v, const void* a, const void* b,
                      const float* A_log, const float* dt_bias, const float* init_state,
                      float* out, float* final_state, const int32_t* cu_seqlens, int B, int T,
                      int Hk, int Hv, int dk, int dv, int chunk, InType in) {
    FwdParams p;
    p.q = q; p.k = k; p.v = v; p.a = a; p.b = b;
    p.A_log = A_log; p.dt_bias = dt_bias;
    p.init_state = init_state; p.out = out; p.final_state = final_state;
    p.cu_seqlens = cu_seqlens;
    p.nseq = B; p.T = T; p.Hk = Hk; p.Hv = Hv; p.dk = dk; p.dv = dv; p.chunk = chunk;
    p.in = in;
    return p;
}

int prefill_chunked(const FwdParams& p, cudaStream_t stream) {
    const int rc = check_common(p, p.in == InType::BF16 ? 2 : 4);
    if (rc != GDR_OK) return rc;
    if (p.chunk != 32) return GDR_ERR_UNSUPPORTED;
    if (p.in == InType::BF16 && p.dk == 128 && p.dv == 128) {
        const cudaError_t e = gdr::launch_prefill_tc(p, stream);
        if (e != cudaErrorNotSupported) return to_status(e);
    }
    return to_status(gdr::launch_chunked_simt(p, stream));
}

int prefill_recurrent(const FwdParams& p, cudaStream_t stream) {
    const int rc = check_common(p, p.in == InType::BF16 ? 2 : 4);
    if (rc != GDR_OK) return rc;
    return to_status(gdr::launch_recurrent(p, stream));
}

int decode_step(const void* q, const void* k, const void* v, const void* a, const void* b,
                const float* A_log, const float* dt_bias, float* state, float* out, int B, int Hk,
                int Hv, int dk, int dv, InType in, cudaStream_t stream, int erase = 1) {
    if (!state) return GDR_ERR_NULL;
    // one token per sequence: the dense layout with T = 1, state updated in place
    FwdParams p = make_params(q, k, v, a, b, A_log, dt_bias, state, out, state, nullptr, B, 1, Hk,
                              Hv, dk, dv, 0, in);
    p.erase = erase;
    return prefill_recurrent(p, stream);
}

FwdParams gla(FwdParams p) {
    p.erase = 0;
    return p;
}

// Checks of the segment-map calls: the tensor-core prefill's restrictions (bf16,
// dk = dv = 128, chunk 32, T >= 1) and the common ones, with no output tensor.
int check_segment_maps(FwdParams p, const float* phi, const float* nmap) {
    if (!phi || !nmap) return GDR_ERR_NULL;
    p.out = const_cast<float*>(nmap);  // stands in for the output in the common checks
    const int rc = check_common(p, 2);
    if (rc != GDR_OK) return rc;
    if (!aligned(phi, 16) || !aligned(nmap, 16)) return GDR_ERR_ALIGN;
    if (p.chunk != 32 || p.dk != 128 || p.dv != 128 || p.T < 1) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// N (the run from S = 0) into nmap and Phi (from S = I with v = 0) into phi, over one set
// of records; no outputs.
cudaError_t segment_maps(FwdParams p, float* phi, float* nmap, cudaStream_t stream) {
    p.init_state = nullptr;
    p.out = nullptr;
    void* ws = nullptr;
    cudaError_t e = gdr::workspace_alloc(&ws, gdr::prefill_tc64_workspace_bytes(p), stream);
    if (e != cudaSuccess) return e;
    e = gdr::launch_prefill_tc64_maps_ws(p, ws, phi, nmap, stream);
    const cudaError_t f = cudaFreeAsync(ws, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace

extern "C" {

int gdr_prefill_chunked(const void* q, const void* k, const void* v, const void* a,
                        const void* b, const float* A_log, const float* dt_bias,
                        const float* init_state, float* out, float* final_state,
                        const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk, int dv,
                        int chunk, gdr_stream_t stream) {
    return prefill_chunked(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                       final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                                       InType::BF16),
                           (cudaStream_t)stream);
}

int gdr_prefill_chunked_noalloc(const void* q, const void* k, const void* v, const void* a,
                                const void* b, const float* A_log, const float* dt_bias,
                                const float* init_state, float* out, float* final_state,
                                const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                                int dv, int chunk, gdr_stream_t stream) {
    const FwdParams p = make_params(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                                    cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, InType::BF16);
    const int rc = check_common(p, 2);
    if (rc != GDR_OK) return rc;
    if (p.chunk != 32 || p.dk != 128 || p.dv != 128 || p.T < 1) return GDR_ERR_UNSUPPORTED;
    if (gdr::prefill_tc_workspace_bytes(p) > gdr::noalloc_scratch_bytes()) return GDR_ERR_TOO_LARGE;
    void* ws = nullptr;
    const cudaError_t e = gdr::noalloc_scratch(&ws);
    if (e != cudaSuccess) return to_status(e);  // the first lookup may fail for lack of memory
    return to_status(gdr::launch_prefill_tc_ws(p, ws, (cudaStream_t)stream));
}

int gdr_prefill_segment_maps(const void* q, const void* k, const void* v, const void* a,
                             const void* b, const float* A_log, const float* dt_bias, float* phi,
                             float* nmap, const int32_t* cu_seqlens, int B, int T, int Hk, int Hv,
                             int dk, int dv, int chunk, gdr_stream_t stream) {
    const FwdParams p = make_params(q, k, v, a, b, A_log, dt_bias, nullptr, nullptr, nullptr,
                                    cu_seqlens, B, T, Hk, Hv, dk, dv, chunk, InType::BF16);
    const int rc = check_segment_maps(p, phi, nmap);
    if (rc != GDR_OK) return rc;
    return to_status(segment_maps(p, phi, nmap, (cudaStream_t)stream));
}

int gdr_segment_combine(const float* phi, const float* nmap, const float* init_state,
                        float* seg_init, float* final_state, int G, int Hv, int dk, int dv,
                        gdr_stream_t stream) {
    if (!phi || !nmap) return GDR_ERR_NULL;
    if (G < 1 || Hv < 1 || (long long)Hv * 4 > 0x7fffffffLL) return GDR_ERR_SHAPE;
    if (dk != 128 || dv != 128) return GDR_ERR_UNSUPPORTED;
    if (!aligned(phi, 16) || !aligned(nmap, 16) || !aligned(init_state, 16) ||
        !aligned(seg_init, 16) || !aligned(final_state, 16))
        return GDR_ERR_ALIGN;
    return to_status(gdr::launch_segment_combine(phi, nmap, init_state, seg_init, final_state, G,
                                                 Hv, dk, (cudaStream_t)stream));
}

int gdr_prefill_chunked_cp(const void* q, const void* k, const void* v, const void* a,
                           const void* b, const float* A_log, const float* dt_bias,
                           const float* init_state, float* out, float* final_state, int T,
                           int Hk, int Hv, int dk, int dv, int chunk, int nseg,
                           gdr_stream_t stream) {
    FwdParams p = make_params(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                              nullptr, 1, T, Hk, Hv, dk, dv, chunk, InType::BF16);
    int rc = check_common(p, 2);
    if (rc != GDR_OK) return rc;
    if (nseg < 1) return GDR_ERR_SHAPE;
    if (p.chunk != 32 || p.dk != 128 || p.dv != 128 || p.T < 1) return GDR_ERR_UNSUPPORTED;
    // chunk-aligned segments of L tokens; G <= nseg of them cover T
    const long long per = ((long long)T + nseg - 1) / nseg;
    const int L = (int)((per + 31) / 32 * 32);
    const int G = (int)(((long long)T + L - 1) / L);
    const cudaStream_t st = (cudaStream_t)stream;
    const size_t mat = (size_t)Hv * 128 * 128 * sizeof(float);  // one map per segment
    const size_t cu_bytes = ((size_t)(G + 1) * sizeof(int32_t) + 255) / 256 * 256;
    void* ws = nullptr;
    cudaError_t e = gdr::workspace_alloc(&ws, cu_bytes + 3 * (size_t)G * mat, st);
    if (e != cudaSuccess) return to_status(e);
    int32_t* cu = static_cast<int32_t*>(ws);
    float* phi = reinterpret_cast<float*>(static_cast<char*>(ws) + cu_bytes);
    float* nmap = reinterpret_cast<float*>(reinterpret_cast<char*>(phi) + (size_t)G * mat);
    float* seg_init = reinterpret_cast<float*>(reinterpret_cast<char*>(nmap) + (size_t)G * mat);
    // the segments side by side as the sequences of a packed batch
    FwdParams sp = p;
    sp.cu_seqlens = cu;
    sp.nseq = G;
    void* rec = nullptr;
    e = gdr::workspace_alloc(&rec, gdr::prefill_tc64_workspace_bytes(sp), st);
    if (e != cudaSuccess) {
        cudaFreeAsync(ws, st);
        return to_status(e);
    }
    // one set of intra-block records serves the maps and the prefill of the segments
    e = gdr::launch_segment_bounds(cu, G, L, T, st);
    if (e == cudaSuccess) {
        FwdParams mp = sp;
        mp.init_state = nullptr;
        mp.out = nullptr;
        e = gdr::launch_prefill_tc64_maps_ws(mp, rec, phi, nmap, st);
    }
    if (e == cudaSuccess)
        e = gdr::launch_segment_combine(phi, nmap, init_state, seg_init, final_state, G, Hv, 128,
                                        st);
    if (e == cudaSuccess) {
        sp.init_state = seg_init;
        sp.out = out;
        sp.final_state = nullptr;
        e = gdr::launch_prefill_tc64_state_ws(sp, rec, st);
    }
    const cudaError_t f = cudaFreeAsync(rec, st);
    const cudaError_t f2 = cudaFreeAsync(ws, st);
    return to_status(e != cudaSuccess ? e : f != cudaSuccess ? f : f2);
}

int gdr_prefill_chunked_host(const void* q, const void* k, const void* v, const void* a,
                             const void* b, const float* A_log, const float* dt_bias,
                             const float* init_state, float* out, float* final_state, int B,
                             int T, int Hk, int Hv, int dk, int dv, int chunk, int seg_tokens,
                             gdr_stream_t stream) {
    if (!A_log || !dt_bias) return GDR_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !a || !b || !out)) return GDR_ERR_NULL;
    if (B < 1 || T < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0 || seg_tokens < 0 ||
        seg_tokens % 32 != 0 || (long long)B * Hv * 4 > 0x7fffffffLL)
        return GDR_ERR_SHAPE;
    if (!head_size_built(dk, dv) || chunk != 32) return GDR_ERR_UNSUPPORTED;
    // default segment: an eighth of the tokens, at least 256, chunk-aligned
    int seg = seg_tokens;
    if (seg == 0) {
        const long long s8 = ((long long)T + 7) / 8;
        seg = (int)((s8 < 256 ? 256 : s8) + 31) / 32 * 32;
    }
    FwdParams p = make_params(q, k, v, a, b, A_log, dt_bias, init_state, out, final_state,
                              nullptr, B, T, Hk, Hv, dk, dv, chunk, InType::BF16);
    int status = GDR_OK;
    const cudaError_t e = gdr::launch_prefill_host(p, seg, (cudaStream_t)stream,
                                                   prefill_chunked, &status);
    if (status != GDR_OK) return status;
    return to_status(e);
}

int gdr_prefill_chunked_f32(const float* q, const float* k, const float* v, const float* a,
                            const float* b, const float* A_log, const float* dt_bias,
                            const float* init_state, float* out, float* final_state,
                            const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                            int dv, int chunk, gdr_stream_t stream) {
    return prefill_chunked(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                       final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                                       InType::F32),
                           (cudaStream_t)stream);
}

int gdr_prefill_recurrent(const void* q, const void* k, const void* v, const void* a,
                          const void* b, const float* A_log, const float* dt_bias,
                          const float* init_state, float* out, float* final_state,
                          const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                          int dv, gdr_stream_t stream) {
    return prefill_recurrent(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                         final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, 0,
                                         InType::BF16),
                             (cudaStream_t)stream);
}

int gdr_prefill_recurrent_f32(const float* q, const float* k, const float* v, const float* a,
                              const float* b, const float* A_log, const float* dt_bias,
                              const float* init_state, float* out, float* final_state,
                              const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                              int dv, gdr_stream_t stream) {
    return prefill_recurrent(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                         final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, 0,
                                         InType::F32),
                             (cudaStream_t)stream);
}

int gdr_decode_step(const void* q, const void* k, const void* v, const void* a, const void* b,
                    const float* A_log, const float* dt_bias, float* state, float* out, int B,
                    int Hk, int Hv, int dk, int dv, gdr_stream_t stream) {
    return decode_step(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv,
                       InType::BF16, (cudaStream_t)stream);
}

int gdr_decode_step_f32(const float* q, const float* k, const float* v, const float* a,
                        const float* b, const float* A_log, const float* dt_bias, float* state,
                        float* out, int B, int Hk, int Hv, int dk, int dv, gdr_stream_t stream) {
    return decode_step(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv,
                       InType::F32, (cudaStream_t)stream);
}

// ---- erase=False: gated linear attention through the same kernels

int gdr_gla_prefill_chunked(const void* q, const void* k, const void* v, const void* a,
                            const void* b, const float* A_log, const float* dt_bias,
                            const float* init_state, float* out, float* final_state,
                            const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                            int dv, int chunk, gdr_stream_t stream) {
    return prefill_chunked(gla(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                           final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                                           InType::BF16)),
                           (cudaStream_t)stream);
}

int gdr_gla_prefill_chunked_f32(const float* q, const float* k, const float* v, const float* a,
                                const float* b, const float* A_log, const float* dt_bias,
                                const float* init_state, float* out, float* final_state,
                                const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                                int dv, int chunk, gdr_stream_t stream) {
    return prefill_chunked(gla(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                           final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, chunk,
                                           InType::F32)),
                           (cudaStream_t)stream);
}

int gdr_gla_prefill_recurrent(const void* q, const void* k, const void* v, const void* a,
                              const void* b, const float* A_log, const float* dt_bias,
                              const float* init_state, float* out, float* final_state,
                              const int32_t* cu_seqlens, int B, int T, int Hk, int Hv, int dk,
                              int dv, gdr_stream_t stream) {
    return prefill_recurrent(gla(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                             final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, 0,
                                             InType::BF16)),
                             (cudaStream_t)stream);
}

int gdr_gla_prefill_recurrent_f32(const float* q, const float* k, const float* v, const float* a,
                                  const float* b, const float* A_log, const float* dt_bias,
                                  const float* init_state, float* out, float* final_state,
                                  const int32_t* cu_seqlens, int B, int T, int Hk, int Hv,
                                  int dk, int dv, gdr_stream_t stream) {
    return prefill_recurrent(gla(make_params(q, k, v, a, b, A_log, dt_bias, init_state, out,
                                             final_state, cu_seqlens, B, T, Hk, Hv, dk, dv, 0,
                                             InType::F32)),
                             (cudaStream_t)stream);
}

int gdr_gla_decode_step(const void* q, const void* k, const void* v, const void* a,
                        const void* b, const float* A_log, const float* dt_bias, float* state,
                        float* out, int B, int Hk, int Hv, int dk, int dv, gdr_stream_t stream) {
    return decode_step(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv,
                       InType::BF16, (cudaStream_t)stream, 0);
}

int gdr_gla_decode_step_f32(const float* q, const float* k, const float* v, const float* a,
                            const float* b, const float* A_log, const float* dt_bias,
                            float* state, float* out, int B, int Hk, int Hv, int dk, int dv,
                            gdr_stream_t stream) {
    return decode_step(q, k, v, a, b, A_log, dt_bias, state, out, B, Hk, Hv, dk, dv,
                       InType::F32, (cudaStream_t)stream, 0);
}

// ---- the steps around the rule

int gdr_short_conv_silu(const void* x, const float* weight, const float* bias,
                        const float* conv_state_in, float* conv_state_out, void* y, int B, int T,
                        int C, int width, gdr_stream_t stream) {
    if (!weight || (T > 0 && (!x || !y))) return GDR_ERR_NULL;
    if (B < 1 || T < 0 || C < 8 || C % 8 != 0) return GDR_ERR_SHAPE;
    if (width != 4) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * C * ((long long)T + 64) > 0x3fffffffffffLL) return GDR_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(bias, 4) ||
        !aligned(conv_state_in, 4) || !aligned(conv_state_out, 4))
        return GDR_ERR_ALIGN;
    return to_status(gdr::launch_short_conv_silu(x, weight, bias, conv_state_in, conv_state_out,
                                                 y, B, T, C, (cudaStream_t)stream));
}

static int gated_rmsnorm(const float* o, const void* z, bool z_f32, const float* weight,
                         float* y, long long rows, int d, float eps, cudaStream_t stream) {
    if (!weight || (rows > 0 && (!o || !z || !y))) return GDR_ERR_NULL;
    if (rows < 0 || !(eps >= 0.f)) return GDR_ERR_SHAPE;
    if (d != 32 && d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    if (!aligned(o, 16) || !aligned(y, 16) || !aligned(z, z_f32 ? 16 : 8) || !aligned(weight, 4))
        return GDR_ERR_ALIGN;
    return to_status(gdr::launch_gated_rmsnorm(o, z, z_f32, weight, y, rows, d, eps, stream));
}

int gdr_gated_rmsnorm(const float* o, const void* z, const float* weight, float* y,
                      long long rows, int d, float eps, gdr_stream_t stream) {
    return gated_rmsnorm(o, z, false, weight, y, rows, d, eps, (cudaStream_t)stream);
}

int gdr_gated_rmsnorm_f32(const float* o, const float* z, const float* weight, float* y,
                          long long rows, int d, float eps, gdr_stream_t stream) {
    return gated_rmsnorm(o, z, true, weight, y, rows, d, eps, (cudaStream_t)stream);
}

// ---- gradients of the steps around the rule

int gdr_short_conv_silu_backward(const void* x, const float* weight, const float* bias,
                                 const float* conv_state_in, const void* grad_y,
                                 const float* grad_conv_state_out, void* grad_x,
                                 float* grad_weight, float* grad_bias,
                                 float* grad_conv_state_in, int B, int T, int C, int width,
                                 gdr_stream_t stream) {
    if (!weight || (T > 0 && (!x || !grad_y || !grad_x))) return GDR_ERR_NULL;
    if (B < 1 || T < 0 || T > 0x7fffff00 || C < 8 || C % 8 != 0) return GDR_ERR_SHAPE;
    if (width != 4) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * C * ((long long)T + 64) > 0x3fffffffffffLL || 5LL * C > 0x7fffffffLL ||
        (long long)B * (((long long)T + 63) / 64) > 0x7fffffLL)
        return GDR_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(grad_y, 16) || !aligned(grad_x, 16) || !aligned(weight, 16) ||
        !aligned(bias, 4) || !aligned(conv_state_in, 4) || !aligned(grad_conv_state_out, 4) ||
        !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || !aligned(grad_conv_state_in, 4))
        return GDR_ERR_ALIGN;
    gdr::ConvGrads p;
    p.x = x; p.weight = weight; p.bias = bias; p.state_in = conv_state_in;
    p.grad_y = grad_y; p.grad_state_out = grad_conv_state_out;
    p.grad_x = grad_x; p.grad_weight = grad_weight; p.grad_bias = grad_bias;
    p.grad_state_in = grad_conv_state_in;
    p.B = B; p.T = T; p.C = C;
    return to_status(gdr::launch_short_conv_silu_backward(p, (cudaStream_t)stream));
}

static int gated_rmsnorm_backward(const float* o, const void* z, bool z_f32, const float* weight,
                                  const float* grad_y, float* grad_o, void* grad_z,
                                  float* grad_weight, long long rows, int d, float eps,
                                  cudaStream_t stream) {
    if (!weight || !grad_weight || (rows > 0 && (!o || !z || !grad_y || !grad_o || !grad_z)))
        return GDR_ERR_NULL;
    if (rows < 0 || !(eps >= 0.f)) return GDR_ERR_SHAPE;
    if (d != 32 && d != 64 && d != 128) return GDR_ERR_UNSUPPORTED;
    const uintptr_t za = z_f32 ? 16 : 8;
    if (!aligned(o, 16) || !aligned(grad_y, 16) || !aligned(grad_o, 16) || !aligned(z, za) ||
        !aligned(grad_z, za) || !aligned(weight, 16) || !aligned(grad_weight, 4))
        return GDR_ERR_ALIGN;
    gdr::NormGrads p;
    p.o = o; p.z = z; p.weight = weight; p.grad_y = grad_y;
    p.grad_o = grad_o; p.grad_z = grad_z; p.grad_weight = grad_weight;
    p.rows = rows; p.d = d; p.eps = eps; p.z_f32 = z_f32;
    return to_status(gdr::launch_gated_rmsnorm_backward(p, stream));
}

int gdr_gated_rmsnorm_backward(const float* o, const void* z, const float* weight,
                               const float* grad_y, float* grad_o, void* grad_z,
                               float* grad_weight, long long rows, int d, float eps,
                               gdr_stream_t stream) {
    return gated_rmsnorm_backward(o, z, false, weight, grad_y, grad_o, grad_z, grad_weight, rows,
                                  d, eps, (cudaStream_t)stream);
}

int gdr_gated_rmsnorm_backward_f32(const float* o, const float* z, const float* weight,
                                   const float* grad_y, float* grad_o, float* grad_z,
                                   float* grad_weight, long long rows, int d, float eps,
                                   gdr_stream_t stream) {
    return gated_rmsnorm_backward(o, z, true, weight, grad_y, grad_o, grad_z, grad_weight, rows,
                                  d, eps, (cudaStream_t)stream);
}

// ---- layer normalisation

static int layer_norm(const void* x, const float* weight, const float* bias, void* y, float* mean,
                      float* rstd, long long rows, int d, float eps, InType in,
                      cudaStream_t stream) {
    if (!weight || (rows > 0 && (!x || !y))) return GDR_ERR_NULL;
    if (rows < 0 || d < 8 || d % 8 != 0 || !(eps >= 0.f)) return GDR_ERR_SHAPE;
    if (d > 32768) return GDR_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return GDR_ERR_ALIGN;
    gdr::LayerNormParams p;
    p.x = x; p.weight = weight; p.bias = bias; p.y = y; p.mean = mean; p.rstd = rstd;
    p.rows = rows; p.d = d; p.eps = eps; p.in = in;
    return to_status(gdr::launch_layer_norm(p, stream));
}

int gdr_layer_norm(const void* x, const float* weight, const float* bias, void* y, float* mean,
                   float* rstd, long long rows, int d, float eps, gdr_stream_t stream) {
    return layer_norm(x, weight, bias, y, mean, rstd, rows, d, eps, InType::BF16,
                      (cudaStream_t)stream);
}

int gdr_layer_norm_f32(const float* x, const float* weight, const float* bias, float* y,
                       float* mean, float* rstd, long long rows, int d, float eps,
                       gdr_stream_t stream) {
    return layer_norm(x, weight, bias, y, mean, rstd, rows, d, eps, InType::F32,
                      (cudaStream_t)stream);
}

static int layer_norm_backward(const void* x, const float* weight, const float* mean,
                               const float* rstd, const void* grad_y, void* grad_x,
                               float* grad_weight, float* grad_bias, long long rows, int d,
                               InType in, cudaStream_t stream) {
    if (!weight || (rows > 0 && (!x || !mean || !rstd || !grad_y || !grad_x))) return GDR_ERR_NULL;
    if (rows < 0 || d < 8 || d % 8 != 0) return GDR_ERR_SHAPE;
    if (d > 32768) return GDR_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(grad_y, 16) || !aligned(grad_x, 16) || !aligned(weight, 16) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_weight, 4) ||
        !aligned(grad_bias, 4))
        return GDR_ERR_ALIGN;
    gdr::LayerNormGrads p;
    p.x = x; p.weight = weight; p.mean = mean; p.rstd = rstd; p.grad_y = grad_y;
    p.grad_x = grad_x; p.grad_weight = grad_weight; p.grad_bias = grad_bias;
    p.rows = rows; p.d = d; p.in = in;
    return to_status(gdr::launch_layer_norm_backward(p, stream));
}

int gdr_layer_norm_backward(const void* x, const float* weight, const float* mean,
                            const float* rstd, const void* grad_y, void* grad_x,
                            float* grad_weight, float* grad_bias, long long rows, int d,
                            gdr_stream_t stream) {
    return layer_norm_backward(x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias,
                               rows, d, InType::BF16, (cudaStream_t)stream);
}

int gdr_layer_norm_backward_f32(const float* x, const float* weight, const float* mean,
                                const float* rstd, const float* grad_y, float* grad_x,
                                float* grad_weight, float* grad_bias, long long rows, int d,
                                gdr_stream_t stream) {
    return layer_norm_backward(x, weight, mean, rstd, grad_y, grad_x, grad_weight, grad_bias,
                               rows, d, InType::F32, (cudaStream_t)stream);
}

// ---- the gated linear recurrence (vector state)

static int check_recurrence(const gdr::RecurrenceParams& p) {
    if (!p.A_log || !p.dt_bias) return GDR_ERR_NULL;
    if (p.T > 0 && (!p.x || !p.a || !p.b || !p.out)) return GDR_ERR_NULL;
    if (p.nseq < 1 || p.T < 0 || p.C < 8 || p.C % 8 != 0 || p.ld < p.C || p.ld % 8 != 0 ||
        p.ld > 0x7fffffffLL)
        return GDR_ERR_SHAPE;
    // token rows and parameter columns are indexed in 32 bits, their offsets in 64
    const long long tokens = p.cu_seqlens ? p.T : (long long)p.nseq * p.T;
    if (tokens > 0x7fffff00LL || p.C > 0x3fffff00) return GDR_ERR_SHAPE;
    if (!aligned(p.x, 16) || !aligned(p.a, 16) || !aligned(p.b, 16) || !aligned(p.out, 16) ||
        !aligned(p.A_log, 4) || !aligned(p.dt_bias, 4) || !aligned(p.init_state, 16) ||
        !aligned(p.final_state, 16) || !aligned(p.cu_seqlens, 4))
        return GDR_ERR_ALIGN;
    return GDR_OK;
}

static int recurrence(const void* x, const void* a, const void* b, const float* A_log,
                      const float* dt_bias, const float* init_state, float* out,
                      float* final_state, const int32_t* cu_seqlens, int B, int T, int C,
                      long long ld, InType in, cudaStream_t stream) {
    gdr::RecurrenceParams p;
    p.x = x; p.a = a; p.b = b; p.A_log = A_log; p.dt_bias = dt_bias; p.init_state = init_state;
    p.out = out; p.final_state = final_state; p.cu_seqlens = cu_seqlens;
    p.nseq = B; p.T = T; p.C = C; p.ld = ld; p.in = in;
    const int rc = check_recurrence(p);
    if (rc != GDR_OK) return rc;
    return to_status(gdr::launch_recurrence(p, stream));
}

int gdr_linear_recurrence(const void* x, const void* a, const void* b, const float* A_log,
                          const float* dt_bias, const float* init_state, float* out,
                          float* final_state, const int32_t* cu_seqlens, int B, int T, int C,
                          long long ld, gdr_stream_t stream) {
    return recurrence(x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens, B, T, C,
                      ld, InType::BF16, (cudaStream_t)stream);
}

int gdr_linear_recurrence_f32(const float* x, const float* a, const float* b, const float* A_log,
                              const float* dt_bias, const float* init_state, float* out,
                              float* final_state, const int32_t* cu_seqlens, int B, int T, int C,
                              long long ld, gdr_stream_t stream) {
    return recurrence(x, a, b, A_log, dt_bias, init_state, out, final_state, cu_seqlens, B, T, C,
                      ld, InType::F32, (cudaStream_t)stream);
}

static int recurrence_backward(const void* x, const void* a, const void* b, const float* A_log,
                               const float* dt_bias, const float* init_state, const float* out,
                               const float* grad_out, const float* grad_final_state, void* grad_x,
                               void* grad_a, void* grad_b, float* grad_A_log,
                               float* grad_dt_bias, float* grad_init_state,
                               const int32_t* cu_seqlens, int B, int T, int C, long long ld,
                               long long ld_grad, InType in, cudaStream_t stream) {
    gdr::RecurrenceParams p;
    p.x = x; p.a = a; p.b = b; p.A_log = A_log; p.dt_bias = dt_bias; p.init_state = init_state;
    p.out = const_cast<float*>(out); p.final_state = nullptr; p.cu_seqlens = cu_seqlens;
    p.nseq = B; p.T = T; p.C = C; p.ld = ld; p.in = in;
    gdr::RecurrenceGrads r;
    r.grad_out = grad_out; r.grad_final = grad_final_state;
    r.grad_x = grad_x; r.grad_a = grad_a; r.grad_b = grad_b;
    r.grad_A_log = grad_A_log; r.grad_dt_bias = grad_dt_bias; r.grad_init = grad_init_state;
    r.ld_grad = ld_grad;
    if (!grad_A_log || !grad_dt_bias) return GDR_ERR_NULL;
    if (T > 0 && (!grad_out || !grad_x || !grad_a || !grad_b)) return GDR_ERR_NULL;
    const int rc = check_recurrence(p);
    if (rc != GDR_OK) return rc;
    if (ld_grad < C || ld_grad % 8 != 0 || ld_grad > 0x7fffffffLL) return GDR_ERR_SHAPE;
    if (!aligned(grad_out, 16) || !aligned(grad_final_state, 16) || !aligned(grad_x, 16) ||
        !aligned(grad_a, 16) || !aligned(grad_b, 16) || !aligned(grad_A_log, 4) ||
        !aligned(grad_dt_bias, 4) || !aligned(grad_init_state, 16))
        return GDR_ERR_ALIGN;
    return to_status(gdr::launch_recurrence_backward(p, r, stream));
}

int gdr_linear_recurrence_backward(const void* x, const void* a, const void* b,
                                   const float* A_log, const float* dt_bias,
                                   const float* init_state, const float* out,
                                   const float* grad_out, const float* grad_final_state,
                                   void* grad_x, void* grad_a, void* grad_b, float* grad_A_log,
                                   float* grad_dt_bias, float* grad_init_state,
                                   const int32_t* cu_seqlens, int B, int T, int C, long long ld,
                                   long long ld_grad, gdr_stream_t stream) {
    return recurrence_backward(x, a, b, A_log, dt_bias, init_state, out, grad_out,
                               grad_final_state, grad_x, grad_a, grad_b, grad_A_log, grad_dt_bias,
                               grad_init_state, cu_seqlens, B, T, C, ld, ld_grad, InType::BF16,
                               (cudaStream_t)stream);
}

int gdr_linear_recurrence_backward_f32(const float* x, const float* a, const float* b,
                                       const float* A_log, const float* dt_bias,
                                       const float* init_state, const float* out,
                                       const float* grad_out, const float* grad_final_state,
                                       float* grad_x, float* grad_a, float* grad_b,
                                       float* grad_A_log, float* grad_dt_bias,
                                       float* grad_init_state, const int32_t* cu_seqlens, int B,
                                       int T, int C, long long ld, long long ld_grad,
                                       gdr_stream_t stream) {
    return recurrence_backward(x, a, b, A_log, dt_bias, init_state, out, grad_out,
                               grad_final_state, grad_x, grad_a, grad_b, grad_A_log, grad_dt_bias,
                               grad_init_state, cu_seqlens, B, T, C, ld, ld_grad, InType::F32,
                               (cudaStream_t)stream);
}

int gdr_zero_outer_rows(void* x, void* y, void* z, const int32_t* cu_seqlens, int B, int T,
                        long long row_bytes, long long pitch_bytes, gdr_stream_t stream) {
    if (!cu_seqlens || (T > 0 && !x && !y && !z)) return GDR_ERR_NULL;
    if (B < 1 || T < 0 || row_bytes < 16 || row_bytes % 16 != 0 || pitch_bytes < row_bytes ||
        pitch_bytes % 16 != 0 || pitch_bytes > 0x1ffffffffLL)
        return GDR_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(z, 16) || !aligned(cu_seqlens, 4))
        return GDR_ERR_ALIGN;
    return to_status(gdr::launch_zero_outer_rows(x, y, z, cu_seqlens, B, T, row_bytes, pitch_bytes,
                                                 (cudaStream_t)stream));
}

int gdr_device_status(gdr_stream_t stream) {
    const cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    const int v = e == cudaSuccess ? gdr::read_and_clear_tc_status() : -1;
    if (v < 0) {
        cudaGetLastError();
        return GDR_ERR_CUDA;
    }
    return v ? GDR_ERR_TIMEOUT : GDR_OK;
}

int gdr_selftest_bounded_wait(gdr_stream_t stream) {
    return to_status(gdr::launch_bounded_wait_selftest((cudaStream_t)stream)) == GDR_OK
               ? GDR_OK
               : GDR_ERR_CUDA;
}

void gdr_release_workspace(void) { gdr::workspace_release(); }

const char* gdr_status_string(int status) {
    switch (status) {
        case GDR_OK: return "GDR_OK";
        case GDR_ERR_NULL: return "GDR_ERR_NULL: a required pointer is NULL";
        case GDR_ERR_SHAPE: return "GDR_ERR_SHAPE: inconsistent sizes";
        case GDR_ERR_UNSUPPORTED: return "GDR_ERR_UNSUPPORTED: head or chunk size not built";
        case GDR_ERR_ALIGN: return "GDR_ERR_ALIGN: misaligned pointer";
        case GDR_ERR_OOM: return "GDR_ERR_OOM: the call's workspace could not be allocated";
        case GDR_ERR_CUDA: return "GDR_ERR_CUDA: kernel launch failed";
        case GDR_ERR_TIMEOUT: return "GDR_ERR_TIMEOUT: a kernel abandoned a bounded wait";
        case GDR_ERR_TOO_LARGE:
            return "GDR_ERR_TOO_LARGE: the call needs more workspace than the fixed 64 MiB scratch "
                   "of gdr_prefill_chunked_noalloc";
        default: return "unknown status";
    }
}

}  // extern "C"

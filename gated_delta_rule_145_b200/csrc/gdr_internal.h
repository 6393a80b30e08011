// gdr_internal.h -- launch interface between the C ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

enum class InType { BF16, F32 };

// One forward call, already validated by the ABI layer.
struct FwdParams {
    const void *q, *k, *v, *a, *b;  // inputs (bf16 or fp32, see `in`)
    const float *A_log, *dt_bias;   // [Hv]
    const float* init_state;        // [nseq, Hv, dk, dv] or nullptr
    float* out;                     // [tokens, Hv, dv]
    float* final_state;             // [nseq, Hv, dk, dv] or nullptr
    const int32_t* cu_seqlens;      // [nseq + 1] or nullptr (dense: nseq sequences of T)
    int nseq, T, Hk, Hv, dk, dv, chunk;
    InType in;
    // 1: the gated delta rule; 0: its erase=False special case, gated linear attention
    // (delta = beta v, no k^T S term)
    int erase = 1;
    // Segment maps (tensor-core prefill only): v_zero runs the rule with v = 0 (v is not
    // read), init_identity starts every sequence from S = I (dk = dv; init_state is not
    // read); with out == nullptr no output is written.
    int v_zero = 0, init_identity = 0;
};

// Sequential recurrence (decode step and recurrent prefill); recurrent.cu.
cudaError_t launch_recurrent(const FwdParams& p, cudaStream_t stream);

// Chunked prefill on CUDA cores (any supported head size, fp32 or bf16); chunked_simt.cu.
cudaError_t launch_chunked_simt(const FwdParams& p, cudaStream_t stream);

// Chunked prefill on the tcgen05 tensor cores (bf16, dk = dv = 128, chunk 32): the
// intra-block kernel, then the state-passing kernel, with a workspace of one record per
// (64-token block, value head) taken from the library's stream-ordered pool; workspace.cu.
// Returns cudaErrorNotSupported for shapes it does not handle.
cudaError_t launch_prefill_tc(const FwdParams& p, cudaStream_t stream);

// Bytes of workspace the tensor-core prefill needs for `p`, and the launch on a caller's
// workspace of at least that size (16-byte aligned); workspace.cu.
size_t prefill_tc_workspace_bytes(const FwdParams& p);
cudaError_t launch_prefill_tc_ws(const FwdParams& p, void* ws, cudaStream_t stream);

// The chunked prefill with the state advanced 64 tokens (two 32-token solve blocks) per
// serial step: its workspace and launch (also without outputs, or as the segment map
// Phi: v = 0 from S = I), and both segment maps over one set of records; prefill_tc64.cu.
size_t prefill_tc64_workspace_bytes(const FwdParams& p);
cudaError_t launch_prefill_tc64_ws(const FwdParams& p, void* ws, cudaStream_t stream);
cudaError_t launch_prefill_tc64_maps_ws(const FwdParams& p, void* ws, float* phi, float* nmap,
                                        cudaStream_t stream);
// The state pass with outputs over records already in ws (from either launch above on the
// same q, k, gates and sequence bounds), launched as a programmatic dependent of the grid
// before it in the stream.
cudaError_t launch_prefill_tc64_state_ws(const FwdParams& p, const void* ws,
                                         cudaStream_t stream);
int read_and_clear_tc64_status();
cudaError_t launch_bounded_wait_selftest(cudaStream_t stream);
int read_and_clear_selftest_status();

// Returns the cached workspace memory of every device to the system; workspace.cu.
void workspace_release();

// The steps around the rule (mixer_io.cu): the four-tap causal convolution + SiLU on bf16
// channels (C a multiple of 8; state [B, C, 3] fp32, either pointer may be null, in place allowed),
// and the gated RMS normalisation of fp32 rows of d values (z bf16 or fp32).
cudaError_t launch_short_conv_silu(const void* x, const float* w, const float* bias,
                                   const float* state_in, float* state_out, void* y, int B, int T,
                                   int C, cudaStream_t stream);
cudaError_t launch_gated_rmsnorm(const float* o, const void* z, bool z_f32, const float* weight,
                                 float* y, long long rows, int d, float eps, cudaStream_t stream);
// Reads and clears the tiled convolution's timeout record (nonzero if set, -1 on error).
int read_and_clear_conv_status();

// The gated linear recurrence (vector state), forward and backward; linear_recurrence.cu.
struct RecurrenceParams {
    const void *x, *a, *b;          // [tokens, C], rows ld elements apart (bf16 or fp32)
    const float *A_log, *dt_bias;   // [C]
    const float* init_state;        // [nseq, C] or nullptr (zeros)
    float* out;                     // [tokens, C]: written by forward, read by backward
    float* final_state;             // [nseq, C] or nullptr
    const int32_t* cu_seqlens;      // [nseq + 1] or nullptr (dense: nseq sequences of T)
    int nseq, T, C;
    long long ld;
    InType in;
    int limit = 0;  // packed, 0: none: longer sequences are not the sequential kernel's
};
struct RecurrenceGrads {
    const float *grad_out, *grad_final;  // [tokens, C]; [nseq, C] or nullptr (zeros)
    void *grad_x, *grad_a, *grad_b;      // as x, a, b, rows ld_grad elements apart
    float *grad_A_log, *grad_dt_bias;    // [C]
    float* grad_init;                    // [nseq, C] or nullptr
    long long ld_grad;
};
cudaError_t launch_recurrence(const RecurrenceParams& p, cudaStream_t stream);
cudaError_t launch_recurrence_backward(const RecurrenceParams& p, const RecurrenceGrads& r,
                                       cudaStream_t stream);
// Zeros in the rows of up to three tensors (nullptr: none) outside [cu_seqlens[0], cu_seqlens[B]) of T
// rows, 16-byte aligned, row_bytes and pitch_bytes multiples of 16; outer_rows.cu.
cudaError_t launch_zero_outer_rows(void* x, void* y, void* z, const int32_t* cu_seqlens, int B, int T,
                                   long long row_bytes, long long pitch_bytes, cudaStream_t stream);
// Reads and clears the tiled recurrence's timeout record (nonzero if set, -1 on error).
int read_and_clear_recurrence_status();

// Layer normalisation of rows of d values (d a multiple of 8, at most 32768); layer_norm.cu.
struct LayerNormParams {
    const void* x;
    const float *weight, *bias;  // [d]; bias or nullptr
    void* y;
    float *mean, *rstd;  // [rows], either may be nullptr
    long long rows;
    int d;
    float eps;
    InType in;
};
struct LayerNormGrads {
    const void* x;
    const float *weight, *mean, *rstd;
    const void* grad_y;
    void* grad_x;
    float *grad_weight, *grad_bias;  // [d], either may be nullptr
    long long rows;
    int d;
    InType in;
};
cudaError_t launch_layer_norm(const LayerNormParams& p, cudaStream_t stream);
cudaError_t launch_layer_norm_backward(const LayerNormGrads& p, cudaStream_t stream);
// Reads and clears its timeout record (nonzero if set, -1 on error).
int read_and_clear_layer_norm_status();

// Backward passes of the steps around the rule; mixer_grad.cu.
struct ConvGrads {
    const void* x;                   // [B, T, C] bf16
    const float *weight, *bias;      // [C, 4]; [C] or nullptr
    const float* state_in;           // [B, C, 3] or nullptr (zeros)
    const void* grad_y;              // [B, T, C] bf16
    const float* grad_state_out;     // [B, C, 3] or nullptr (zeros)
    void* grad_x;                    // [B, T, C] bf16
    float *grad_weight, *grad_bias;  // [C, 4], [C]; either may be nullptr
    float* grad_state_in;            // [B, C, 3] or nullptr
    int B, T, C;
};
struct NormGrads {
    const float* o;
    const void* z;
    const float *weight, *grad_y;
    float* grad_o;
    void* grad_z;
    float* grad_weight;
    long long rows;
    int d;
    float eps;
    bool z_f32;
};
cudaError_t launch_short_conv_silu_backward(const ConvGrads& p, cudaStream_t stream);
cudaError_t launch_gated_rmsnorm_backward(const NormGrads& p, cudaStream_t stream);
// Reads and clears the convolution backward's timeout record (nonzero if set, -1 on error).
int read_and_clear_mixer_grad_status();

// out0 [n0] and out1 [N - n0] = the column sums of part [P, N], rows added in a fixed order
// (either output may be nullptr; P = 0 gives zeros); N a multiple of 4, part 16-byte aligned;
// column_sum.cu.
cudaError_t launch_column_sum(const float* part, long long P, int N, float* out0, int n0,
                              float* out1, cudaStream_t stream);

// Composition of per-segment state maps, and segment boundaries of one sequence cut into
// G segments of L tokens; segments.cu.
cudaError_t launch_segment_combine(const float* phi, const float* nmap, const float* init,
                                   float* seg_init, float* final_state, int G, int Hv, int d,
                                   cudaStream_t stream);
cudaError_t launch_segment_bounds(int32_t* cu, int G, int L, int T, cudaStream_t stream);

// The chunked prefill from and to host memory in segments of `seg` tokens (a multiple of
// the chunk), copies overlapped with the kernels; `prefill` runs one device-resident
// segment and its status lands in *status (0 = OK); host_pipeline.cu.
cudaError_t launch_prefill_host(const FwdParams& host_params, int seg, cudaStream_t stream,
                                int (*prefill)(const FwdParams&, cudaStream_t), int* status);

// Multiprocessors of the current device, asked once per device; workspace.cu.
int device_sms();

// Allows `kernel` this much dynamic shared memory on the current device; the runtime is asked
// once per kernel, device and size above the last one.
cudaError_t allow_smem(const void* kernel, size_t bytes);

// While it lives, this thread may make calls that a stream capture elsewhere would otherwise
// forbid (creating the pool, asking for occupancy): they enqueue nothing, so a first call may
// be captured.
class CaptureRelaxed {
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;

  public:
    CaptureRelaxed() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    ~CaptureRelaxed() { cudaThreadExchangeStreamCaptureMode(&mode_); }
    CaptureRelaxed(const CaptureRelaxed&) = delete;
    CaptureRelaxed& operator=(const CaptureRelaxed&) = delete;
};

// The library's stream-ordered workspace pool (workspace.cu).
cudaError_t workspace_alloc(void** ptr, size_t bytes, cudaStream_t stream);

// The fixed scratch area of the no-allocation prefill entry point: its size, and its
// device address on the current device (looked up once per device); noalloc.cu.
size_t noalloc_scratch_bytes();
cudaError_t noalloc_scratch(void** ptr);

// Reads and clears the tensor-core kernels', the tiled convolution's and recurrence's, the
// layer norm's, the convolution backward's and the self-test's
// timeout records (nonzero if set, 0 if not, -1 on a CUDA error); workspace.cu.
int read_and_clear_tc_status();

}  // namespace gdr

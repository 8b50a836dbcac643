// gated.h -- internal interface of the gated delta rule (gated_*.cu) and of layer norm (norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace efla {

// Validated geometry of a gated call.  Strides are in elements: {batch, head, token}.
// packed: the B sequences lie one after another on a single axis of L tokens, sequence b at
// tokens offsets[b] .. offsets[b+1]-1 (device memory); else every sequence has L tokens.
struct GDims {
    int B, H, Hk, L, dk, dv;
    int in_bf16, out_bf16, euler, packed, tensor;
    const int* offsets;
    long long qs[3], ks[3], vs[3], gs[3], bs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];
    long long BH() const { return (long long)B * H; }
    // Chunk slots of a value head, in chunks of C tokens: sequence b's chunks start at slot
    // slot0(b) = b ceil(L / C), or offsets[b] / C + b when packed (never fewer than its
    // ceil(length / C) slots before slot0(b + 1)).
    int slots(int C) const { return packed ? L / C + B : B * ((L + C - 1) / C); }
};

// -------------------------------------------------------------- fp32 CUDA-core kernels
size_t gated_simt_bwd_ws_bytes(const GDims& d);
// Whether the recurrence is the faster forward pass where the tensor-core kernels would do too.
bool gated_fwd_short(const GDims& d);
cudaError_t launch_gated_fwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, void* o, float* S_final, cudaStream_t st);
cudaError_t launch_gated_bwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, const void* dO, const float* dS_final,
                                  void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* ws,
                                  cudaStream_t st);

// -------------------------------------------------------------- tensor-core kernels (gated_tc.cu)
// bf16 tokens whose rows start on 16-byte boundaries (the caller checks the strides).
bool gated_tc_supported(const GDims& d);
size_t gated_tc_fwd_ws_bytes(const GDims& d);
cudaError_t launch_gated_fwd_tc(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, void* o, float* S_final, void* ws,
                                cudaStream_t st);
size_t gated_tc_bwd_ws_bytes(const GDims& d);
cudaError_t launch_gated_bwd_tc(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, const void* dO, const float* dS_final,
                                void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* ws,
                                cudaStream_t st);
// Read and clear the kernels' device status words (synchronous).
cudaError_t gated_bwd_tc_status_read_clear(unsigned int* status);
cudaError_t gated_tc_status_read_clear(unsigned int* status);

// ------------------------------------------------------------------- decode (gated_step.cu)
// slots: null (sequence b's states at S + b H dk dv), or B state indices in [0, nslots); a
// sequence whose index is outside is skipped (its o is zero).
cudaError_t launch_gated_step(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                              const float* beta, float* S, const int* slots, int nslots, void* o, cudaStream_t st);

cudaError_t gated_step_status_read_clear(unsigned int* status);

// ------------------------------------------------------------------- layer norm (norm.cu)
struct NormDims {
    long long rows, x_stride, y_stride;   // y_stride: of y, and of dy in the backward
    int D, bf16, w_bf16;
    float eps;
};
size_t norm_bwd_ws_bytes(const NormDims& d);
cudaError_t launch_norm_fwd(const NormDims& d, const void* x, const void* w, const void* b, void* y, float* stats,
                            cudaStream_t st);
cudaError_t launch_norm_bwd(const NormDims& d, const void* x, const void* w, const void* dy, const float* stats,
                            void* dx, void* dw, void* db, void* ws, cudaStream_t st);

// Reads and clears the kernels' device status word (synchronous).
cudaError_t norm_status_read_clear(unsigned int* status);

}  // namespace efla

// mix.h -- internal interface of the short convolution (conv.cu), the selective scan (scan_*.cu) and the
// residual's RMS norm (rms.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace efla {

// Where the sequences of a call lie: `rows` axes of L tokens.  packed: one axis that B sequences share,
// sequence b at tokens offsets[b] .. offsets[b+1]-1 (device memory, clamped to [0, L] where it is read);
// else axis b is sequence b.
struct Axes {
    int B, L, packed;
    const int* offsets;
    __host__ __device__ int rows() const { return packed ? 1 : B; }
};

// ------------------------------------------------------------------- short causal convolution
// Strides are in elements: {axis, token}; channels are contiguous.
struct ConvDims {
    Axes at;
    int D, W, bf16, w_bf16, silu;
    long long xs[2], ys[2], dys[2], dxs[2];
};
cudaError_t launch_conv_fwd(const ConvDims& d, const void* x, const void* w, const void* bias, const void* S0, void* y,
                            void* S_final, cudaStream_t st);
size_t conv_bwd_ws_bytes(const ConvDims& d);
cudaError_t launch_conv_bwd(const ConvDims& d, const void* x, const void* w, const void* bias, const void* S0, const void* dy,
                            const void* dS, void* dx, void* dw, void* db, void* dS0, void* ws, cudaStream_t st);
// slots: null (sequence b's state at S + b (W - 1) D), or B places in [0, nslots); a sequence whose place is
// outside is skipped (its y is zero).
cudaError_t launch_conv_step(const ConvDims& d, const void* x, const void* w, const void* bias, void* S, const int* slots,
                             int nslots, void* y, cudaStream_t st);

// ------------------------------------------------------------------- selective scan
struct ScanDims {
    Axes at;
    int D, G, N, bf16, softplus;
    long long us[2], ds[2], zs[2], ys[2], dys[2], dus[2], dds[2], dzs[2];   // {axis, token}
    long long bs[3], cs[3];                                                 // {axis, token, group}
};
struct ScanIn {
    const void *u, *delta;
    const float* A;
    const void *Bm, *C;
    const float* skip;      // null: none
    const void* z;          // null: none
    const float* dbias;     // null: none
    const float* S0;        // null: zeros
};
struct ScanGrads {
    const void* dy;
    const float* dS;        // null: zeros
    void *du, *ddelta;
    float* dA;
    void *dB, *dC;
    float* dskip;           // null: not wanted
    void* dz;
    float *ddbias, *dS0;    // null: not wanted
};
size_t scan_fwd_ws_bytes(const ScanDims& d);
cudaError_t launch_scan_fwd(const ScanDims& d, const ScanIn& in, void* y, float* S_final, void* ws, cudaStream_t st);
size_t scan_bwd_ws_bytes(const ScanDims& d);
cudaError_t launch_scan_bwd(const ScanDims& d, const ScanIn& in, const ScanGrads& g, void* ws, cudaStream_t st);
cudaError_t launch_scan_step(const ScanDims& d, const ScanIn& in, float* S, const int* slots, int nslots, void* y,
                             cudaStream_t st);

// ------------------------------------------------------------------- RMS norm on a residual stream
struct RmsDims {
    long long rows, x_stride, r_stride, y_stride, h_stride;   // backward: h, dh, dy, dx
    int D, bf16, w_bf16, group;                               // group: columns a scale (0: y in the type of x)
    float eps;
};
cudaError_t launch_rms_fwd(const RmsDims& d, const void* x, const void* res, const void* w, void* y, float* scale, void* h,
                           float* rstd, cudaStream_t st);
size_t rms_bwd_ws_bytes(const RmsDims& d);
cudaError_t launch_rms_bwd(const RmsDims& d, const void* h, const void* w, const void* dy, const float* rstd, const void* dh,
                           void* dx, void* dw, void* ws, cudaStream_t st);
// Reads and clears the norm kernels' device status word (synchronous).
cudaError_t rms_status_read_clear(unsigned int* status);

}  // namespace efla

// norm.cu -- layer norm over the last dimension, forward and backward.
//
//   y = (x - mean) rstd w + b,   mean and rstd = 1 / sqrt(var + eps) of each row
//   xh = (x - mean) rstd,  p = dy w,  dx = rstd (p - mean(p) - xh mean(p xh))
//   dw = sum over rows of dy xh,   db = sum over rows of dy
// Bound by HBM: one read of x (and dy) and one write.  A row is held in the registers of its
// threads, so the variance is the mean square of the centred values (a second pass over
// registers, not over memory, and no difference of large sums).  Statistics, sums and the
// weight's gradient are fp32.
//
// The weight's gradient: each CTA walks rows CTA, CTA + grid, ... and keeps its threads'
// columns of dw and db in registers; a second kernel adds the CTAs' partial rows in a fixed
// order, so that results do not depend on the order in which CTAs finish.
#include "common.cuh"
#include "gated.h"
#include "launch.h"

namespace efla {

namespace {

constexpr int kSpan = 16;   // most elements of a row that one thread holds

// VEC elements at p (aligned to their size) <-> fp32
template <int VEC>
__device__ __forceinline__ void ld_vec(const float* p, float* x) {
    if (VEC == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1 % VEC] = v.y; x[2 % VEC] = v.z; x[3 % VEC] = v.w;
    } else {
        x[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void ld_vec(const __nv_bfloat16* p, float* x) {
    if (VEC == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __bfloat1622float2(h[i]);
            x[2 * i % VEC] = f.x;
            x[(2 * i + 1) % VEC] = f.y;
        }
    } else {
        x[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void st_vec(float* p, const float* x) {
    if (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1 % VEC], x[2 % VEC], x[3 % VEC]);
    else *p = x[0];
}
template <int VEC>
__device__ __forceinline__ void st_vec(__nv_bfloat16* p, const float* x) {
    if (VEC == 8) {
        uint4 v;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i % VEC], x[(2 * i + 1) % VEC]);
        *reinterpret_cast<uint4*>(p) = v;
    } else {
        *p = __float2bfloat16_rn(x[0]);
    }
}

__device__ __forceinline__ float ld_w(const void* w, int i, int bf16) {
    return bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[i]) : ((const float*)w)[i];
}

// Sum of x over the NT threads of a row (a warp, or several whole warps of the CTA).
template <int NT>
__device__ __forceinline__ float2 row_sum(float2 x, float2* red, int row, int t) {
    x.x = warp_sum(x.x);
    x.y = warp_sum(x.y);
    if (NT <= 32) return x;
    constexpr int W = NT > 32 ? NT / 32 : 1;
    __syncthreads();   // the last use of `red` is over
    if ((t & 31) == 0) red[row * W + t / 32] = x;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s.x += red[row * W + i].x;
        s.y += red[row * W + i].y;
    }
    return s;
}

// NT threads a row, a CTA of max(NT, 256) threads; a thread holds vectors t, t + NT, ...
template <typename T, int VEC, int NT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_norm_fwd(NormDims d, const T* x, const void* w, const void* b,
                                                                  T* y, float* stats) {
    constexpr int NV = kSpan / VEC, CT = NT < 256 ? 256 : NT, RPC = CT / NT;
    __shared__ float2 red[CT / 32];
    const int row = threadIdx.x / NT, t = threadIdx.x % NT;
    const float inv = 1.f / (float)d.D;
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < d.rows; r0 += (long long)gridDim.x * RPC) {
        const long long r = r0 + row;
        const bool live = r < d.rows;
        float v[kSpan];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * NT + t) * VEC;
            if (live && c < d.D) ld_vec<VEC>(x + r * d.x_stride + c, v + m * VEC);
            else
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[m * VEC + i] = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i) s.x += v[m * VEC + i];
        }
        const float mean = row_sum<NT>(s, red, row, t).x * inv;
        s = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * NT + t) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float z = v[m * VEC + i] - mean;
                v[m * VEC + i] = z;
                if (c < d.D) s.x = fmaf(z, z, s.x);
            }
        }
        const float rstd = 1.f / sqrtf(row_sum<NT>(s, red, row, t).x * inv + d.eps);
        if (!live) continue;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * NT + t) * VEC;
            if (c < d.D) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float z = v[m * VEC + i] * rstd;
                    v[m * VEC + i] = b ? fmaf(z, ld_w(w, c + i, d.w_bf16), ld_w(b, c + i, d.w_bf16))
                                       : z * ld_w(w, c + i, d.w_bf16);
                }
                st_vec<VEC>(y + r * d.y_stride + c, v + m * VEC);
            }
        }
        if (t == 0) {
            stats[2 * r] = mean;
            stats[2 * r + 1] = rstd;
        }
    }
}

template <typename T, int VEC, int NT>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT) k_norm_bwd(NormDims d, const T* x, const void* w, const T* dy,
                                                                  const float* stats, T* dx, float* part, int want_db) {
    constexpr int NV = kSpan / VEC, CT = NT < 256 ? 256 : NT, RPC = CT / NT;
    __shared__ float2 red[CT / 32];
    const int row = threadIdx.x / NT, t = threadIdx.x % NT;
    const float inv = 1.f / (float)d.D;
    float aw[kSpan], ab[kSpan];
#pragma unroll
    for (int i = 0; i < kSpan; ++i) aw[i] = ab[i] = 0.f;
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < d.rows; r0 += (long long)gridDim.x * RPC) {
        const long long r = r0 + row;
        const bool live = r < d.rows;
        float z[kSpan], p[kSpan];
        const float mean = live ? stats[2 * r] : 0.f, rstd = live ? stats[2 * r + 1] : 0.f;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * NT + t) * VEC;
            if (live && c < d.D) {
                ld_vec<VEC>(x + r * d.x_stride + c, z + m * VEC);
                ld_vec<VEC>(dy + r * d.y_stride + c, p + m * VEC);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    z[e] = (z[e] - mean) * rstd;
                    aw[e] = fmaf(p[e], z[e], aw[e]);
                    ab[e] += p[e];
                    p[e] *= ld_w(w, c + i, d.w_bf16);
                    s.x += p[e];
                    s.y = fmaf(p[e], z[e], s.y);
                }
            }
        }
        s = row_sum<NT>(s, red, row, t);
        s.x *= inv;
        s.y *= inv;
        if (!live) continue;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * NT + t) * VEC;
            if (c < d.D) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    p[e] = rstd * (p[e] - s.x - z[e] * s.y);
                }
                st_vec<VEC>(dx + r * d.D + c, p + m * VEC);
            }
        }
    }
    float* pw = part + ((size_t)blockIdx.x * RPC + row) * (want_db ? 2 : 1) * d.D;
#pragma unroll
    for (int m = 0; m < NV; ++m)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = (m * NT + t) * VEC + i;
            if (c < d.D) {
                pw[c] = aw[m * VEC + i];
                if (want_db) pw[d.D + c] = ab[m * VEC + i];
            }
        }
}

// dw (and db) = the sum of n partial rows: 32 columns a CTA, 8 groups of rows, then the groups in order
__global__ void __launch_bounds__(256) k_norm_dw(int D, int w_bf16, int n, int two, const float* part, void* dw, void* db) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const size_t ld = (size_t)(two ? 2 : 1) * D;
    const float* p = part + (size_t)blockIdx.y * D + c;
    float s = 0.f;
    if (c < D)
        for (int r = g; r < n; r += 8) s += p[r * ld];
    red[g][lane] = s;
    __syncthreads();
    if (g == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += red[i][lane];
        void* out = blockIdx.y ? db : dw;
        if (w_bf16) ((__nv_bfloat16*)out)[c] = __float2bfloat16_rn(s);
        else ((float*)out)[c] = s;
    }
}

constexpr int kGrid = 304;   // CTAs of the backward: two an SM

int threads_per_row(int D, int vec) {
    const int need = (D + kSpan - 1) / kSpan;
    (void)vec;
    return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : need <= 512 ? 512 : 1024;
}

bool al(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename T, int VEC>
cudaError_t fwd(const NormDims& d, const void* x, const void* w, const void* b, void* y, float* stats, cudaStream_t st) {
#define EFLA_NORM_FWD(NT)                                                                                         \
    case NT: {                                                                                                    \
        constexpr int CT = NT < 256 ? 256 : NT;                                                                   \
        const long long ctas = (d.rows * NT + CT - 1) / CT;                                                       \
        k_norm_fwd<T, VEC, NT><<<(unsigned)(ctas < 65536 ? ctas : 65536), CT, 0, st>>>(d, (const T*)x, w, b, (T*)y, \
                                                                                      stats);                     \
        break;                                                                                                    \
    }
    switch (threads_per_row(d.D, VEC)) {
        EFLA_NORM_FWD(32)
        EFLA_NORM_FWD(64)
        EFLA_NORM_FWD(128)
        EFLA_NORM_FWD(256)
        EFLA_NORM_FWD(512)
        EFLA_NORM_FWD(1024)
    }
#undef EFLA_NORM_FWD
    prof_mark("norm_fwd", st);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd(const NormDims& d, const void* x, const void* w, const void* dy, const float* stats, void* dx,
                void* dw, void* db, void* ws, cudaStream_t st) {
    int n = 0;   // partial rows
#define EFLA_NORM_BWD(NT)                                                                                      \
    case NT: {                                                                                                 \
        constexpr int CT = NT < 256 ? 256 : NT;                                                                \
        const long long ctas = (d.rows * NT + CT - 1) / CT;                                                    \
        const unsigned grid = (unsigned)(ctas < kGrid ? (ctas ? ctas : 1) : kGrid);                            \
        n = (int)grid * (CT / NT);                                                                             \
        k_norm_bwd<T, VEC, NT><<<grid, CT, 0, st>>>(d, (const T*)x, w, (const T*)dy, stats, (T*)dx, (float*)ws, \
                                                    db != nullptr);                                            \
        break;                                                                                                 \
    }
    switch (threads_per_row(d.D, VEC)) {
        EFLA_NORM_BWD(32)
        EFLA_NORM_BWD(64)
        EFLA_NORM_BWD(128)
        EFLA_NORM_BWD(256)
        EFLA_NORM_BWD(512)
        EFLA_NORM_BWD(1024)
    }
#undef EFLA_NORM_BWD
    prof_mark("norm_bwd", st);
    k_norm_dw<<<dim3((d.D + 31) / 32, db ? 2 : 1), 256, 0, st>>>(d.D, d.w_bf16, n, db != nullptr, (const float*)ws, dw, db);
    prof_mark("norm_dw", st);
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_ws_bytes(const NormDims& d) {
    const int nt = threads_per_row(d.D, 1);
    return align256((size_t)kGrid * (nt < 256 ? 256 / nt : 1) * 2 * d.D * 4);
}

cudaError_t launch_norm_fwd(const NormDims& d, const void* x, const void* w, const void* b, void* y, float* stats,
                            cudaStream_t st) {
    const int vec = d.bf16 ? 8 : 4;
    const bool wide = d.D % vec == 0 && d.x_stride % vec == 0 && d.y_stride % vec == 0 && al(x, 16) && al(y, 16);
    if (d.bf16)
        return wide ? fwd<__nv_bfloat16, 8>(d, x, w, b, y, stats, st) : fwd<__nv_bfloat16, 1>(d, x, w, b, y, stats, st);
    return wide ? fwd<float, 4>(d, x, w, b, y, stats, st) : fwd<float, 1>(d, x, w, b, y, stats, st);
}

cudaError_t launch_norm_bwd(const NormDims& d, const void* x, const void* w, const void* dy, const float* stats,
                            void* dx, void* dw, void* db, void* ws, cudaStream_t st) {
    const int vec = d.bf16 ? 8 : 4;
    const bool wide = d.D % vec == 0 && d.x_stride % vec == 0 && d.y_stride % vec == 0 && al(x, 16) && al(dy, 16) && al(dx, 16);
    if (d.bf16)
        return wide ? bwd<__nv_bfloat16, 8>(d, x, w, dy, stats, dx, dw, db, ws, st)
                    : bwd<__nv_bfloat16, 1>(d, x, w, dy, stats, dx, dw, db, ws, st);
    return wide ? bwd<float, 4>(d, x, w, dy, stats, dx, dw, db, ws, st)
                : bwd<float, 1>(d, x, w, dy, stats, dx, dw, db, ws, st);
}

}  // namespace efla

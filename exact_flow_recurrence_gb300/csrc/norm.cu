// norm.cu -- layer norm over the last dimension, forward and backward.
//
//   y = (x - mean) rstd w + b,   mean and rstd = 1 / sqrt(var + eps) of each row
//   xh = (x - mean) rstd,  p = dy w,  dx = rstd (p - mean(p) - xh mean(p xh))
//   dw = sum over rows of dy xh,   db = sum over rows of dy
// Bound by HBM: one read of x (and dy) and one write.  A row is held in the registers of its
// threads as it was stored, so the variance is the mean square of the centred values (another
// pass over registers, not over memory, and no difference of large sums).  Statistics, sums and
// the weight's gradient are fp32.
//
// Forward: up to 2048 elements a row belong to one warp, so that a row needs shuffles only and
// an SM has some thirty rows in flight; longer rows to 4 to 32 warps.  Backward: 16 elements a
// thread (dw and db stay in registers over all rows of a CTA), 32 beyond 8192; the next row is
// loaded while the present one is reduced.  A second kernel adds the CTAs' partial sums in a
// fixed order, so that results do not depend on the order in which CTAs finish.
#include "common.cuh"
#include "gated.h"
#include "launch.h"

namespace efla {

namespace {

// VEC neighbouring elements as stored, and as fp32
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void get(float* x) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float* x) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v = *reinterpret_cast<const uint4*>(h);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
};
template <typename T>
struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void get(float* x) const { x[0] = (float)v; }
    __device__ __forceinline__ void set(const float* x) { v = (T)x[0]; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = (T)0.f; }
};

// VEC weights from column c (fp32 or bf16)
template <int VEC>
__device__ __forceinline__ void weights(const void* w, int c, int bf16, float* x) {
    if (VEC == 1) {
        x[0] = bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[c]) : __ldg((const float*)w + c);
    } else if (bf16) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>((const __nv_bfloat16*)w + c + i));
            x[i] = __uint_as_float(v.x << 16);
            x[(i + 1) % VEC] = __uint_as_float(v.x & 0xffff0000u);
            x[(i + 2) % VEC] = __uint_as_float(v.y << 16);
            x[(i + 3) % VEC] = __uint_as_float(v.y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>((const float*)w + c + i));
            x[i] = v.x;
            x[(i + 1) % VEC] = v.y;
            x[(i + 2) % VEC] = v.z;
            x[(i + 3) % VEC] = v.w;
        }
    }
}

__device__ __forceinline__ void bar_sync(int id, int count) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory"); }

// Sums over the W warps of a row; `red` has room for W pairs and is not in use by an earlier sum
// that a warp of this row may still be reading.
template <int W>
__device__ __forceinline__ float2 row_sum(float2 s, float2* red, int bar, int warp_in_row) {
    s.x = warp_sum(s.x);
    s.y = warp_sum(s.y);
    if (W == 1) return s;
    if ((threadIdx.x & 31) == 0) red[warp_in_row] = s;
    bar_sync(bar, 32 * W);
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        r.x += red[i].x;
        r.y += red[i].y;
    }
    return r;
}

// W warps a row, NV vectors a lane.
template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(W < 8 ? 256 : 32 * W) k_norm_fwd(NormDims d, const T* x, const void* w, const void* b,
                                                                   T* y, float* stats) {
    constexpr int RPC = W < 8 ? 8 / W : 1;   // rows a CTA
    __shared__ float2 red[RPC][2][W];
    const int row = threadIdx.x / (32 * W), t = threadIdx.x % (32 * W), wr = t >> 5;
    const long long r = (long long)blockIdx.x * RPC + row;
    if (r >= d.rows) return;   // (whole rows, so whole barriers)
    Pack<T, VEC> v[NV];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = (m * 32 * W + t) * VEC;
        if (c < d.D) v[m].load(x + r * d.x_stride + c);
        else v[m].zero();
    }
    float f[VEC];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        v[m].get(f);
#pragma unroll
        for (int i = 0; i < VEC; ++i) s.x += f[i];
    }
    const float inv = 1.f / (float)d.D;
    const float mean = row_sum<W>(s, red[row][0], row + 1, wr).x * inv;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        if ((m * 32 * W + t) * VEC < d.D) {
            v[m].get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s.x = fmaf(f[i] - mean, f[i] - mean, s.x);
        }
    }
    const float rstd = 1.f / sqrtf(row_sum<W>(s, red[row][1], row + 1, wr).x * inv + d.eps);
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = (m * 32 * W + t) * VEC;
        if (c < d.D) {
            float wf[VEC], bf[VEC];
            weights<VEC>(w, c, d.w_bf16, wf);
            v[m].get(f);
            if (b) {
                weights<VEC>(b, c, d.w_bf16, bf);
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = fmaf((f[i] - mean) * rstd, wf[i], bf[i]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) f[i] = (f[i] - mean) * rstd * wf[i];
            }
            v[m].set(f);
            v[m].store(y + r * d.y_stride + c);
        }
    }
    if (t == 0) *reinterpret_cast<float2*>(stats + 2 * r) = make_float2(mean, rstd);
}

// W warps a row, 16 / W rows at a time in a CTA of 512 threads; NV vectors a lane.
template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(512, 1) k_norm_bwd(NormDims d, const T* x, const void* w, const T* dy,
                                                     const float* stats, T* dx, float* part, int want_db) {
    constexpr int RPC = 16 / W, SP = NV * VEC;
    __shared__ float2 red[RPC][2][W];
    extern __shared__ float comb[];   // [D] when rows share a CTA
    const int row = threadIdx.x / (32 * W), t = threadIdx.x % (32 * W), wr = t >> 5;
    const float inv = 1.f / (float)d.D;
    const long long step = (long long)gridDim.x * RPC;
    float aw[SP], ab[SP];
#pragma unroll
    for (int i = 0; i < SP; ++i) aw[i] = ab[i] = 0.f;
    Pack<T, VEC> xv[NV], gv[NV];
    float2 st = make_float2(0.f, 0.f);
    const auto fetch = [&](long long r) {
        if (r < d.rows) st = __ldg(reinterpret_cast<const float2*>(stats + 2 * r));
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * 32 * W + t) * VEC;
            if (r < d.rows && c < d.D) {
                xv[m].load(x + r * d.x_stride + c);
                gv[m].load(dy + r * d.y_stride + c);
            }
        }
    };
    long long r = (long long)blockIdx.x * RPC + row;
    fetch(r);
    for (int it = 0; r < d.rows; r += step, it ^= 1) {
        float z[SP], p[SP];
        const float mean = st.x, rstd = st.y;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * 32 * W + t) * VEC;
            if (c < d.D) {
                float wf[VEC];
                weights<VEC>(w, c, d.w_bf16, wf);
                xv[m].get(z + m * VEC);
                gv[m].get(p + m * VEC);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    z[e] = (z[e] - mean) * rstd;
                    aw[e] = fmaf(p[e], z[e], aw[e]);
                    ab[e] += p[e];
                    p[e] *= wf[i];
                    s.x += p[e];
                    s.y = fmaf(p[e], z[e], s.y);
                }
            }
        }
        fetch(r + step);   // in flight over the reduction and the stores
        s = row_sum<W>(s, red[row][it], row + 1, wr);
        s.x *= inv;
        s.y *= inv;
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * 32 * W + t) * VEC;
            if (c < d.D) {
                Pack<T, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    p[e] = rstd * (p[e] - s.x - z[e] * s.y);
                }
                o.set(p + m * VEC);
                o.store(dx + r * d.D + c);
            }
        }
    }
    // the CTA's rows together, one group after another in order, then out as one partial row
    float* pw = part + (size_t)blockIdx.x * (want_db ? 2 : 1) * d.D;
#pragma unroll 1
    for (int what = 0; what < (want_db ? 2 : 1); ++what) {
#pragma unroll 1
        for (int k = 0; k < RPC; ++k) {
            if (RPC > 1) __syncthreads();
            if (row == k) {
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    const int c = (m * 32 * W + t) * VEC;
                    if (c < d.D)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float v = (what ? ab : aw)[m * VEC + i] + (k ? comb[c + i] : 0.f);
                            if (k + 1 < RPC) comb[c + i] = v;
                            else pw[(size_t)what * d.D + c + i] = v;
                        }
                }
            }
        }
    }
}

// dw (and db) = the sum of n partial rows: 32 columns a CTA, 32 groups of rows, then the groups in order
__global__ void __launch_bounds__(1024) k_norm_dw(int D, int w_bf16, int n, int two, const float* part, void* dw, void* db) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const size_t ld = (size_t)(two ? 2 : 1) * D;
    const float* p = part + (size_t)blockIdx.y * D + c;
    float s = 0.f;
    if (c < D) {
#pragma unroll 5
        for (int r = g; r < n; r += 32) s += p[r * ld];
    }
    red[g][lane] = s;
    __syncthreads();
    s = warp_sum(red[lane][g]);   // warp g: column g of the CTA
    const int col = blockIdx.x * 32 + g;
    if (lane == 0 && col < D) {
        void* out = blockIdx.y ? db : dw;
        if (w_bf16) ((__nv_bfloat16*)out)[col] = __float2bfloat16_rn(s);
        else ((float*)out)[col] = s;
    }
}

constexpr int kGrid = 152;   // CTAs of the backward: one an SM

bool al(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

struct FwdArgs {
    const NormDims& d;
    const void *x, *w, *b;
    void* y;
    float* stats;
    cudaStream_t st;
};

template <typename T, int VEC, int NV, int W>
void fwd_launch(const FwdArgs& a) {
    constexpr int RPC = W < 8 ? 8 / W : 1;
    k_norm_fwd<T, VEC, NV, W><<<(unsigned)((a.d.rows + RPC - 1) / RPC), W < 8 ? 256 : 32 * W, 0, a.st>>>(
        a.d, (const T*)a.x, a.w, a.b, (T*)a.y, a.stats);
}

// Lanes hold up to 64 elements (32 one by one): a warp a row up to 2048 (1024), else more warps.
template <typename T, int VEC>
void fwd(const FwdArgs& a) {
    const int D = a.d.D;
    if constexpr (VEC == 8) {
        if (D <= 512) fwd_launch<T, 8, 2, 1>(a);
        else if (D <= 1024) fwd_launch<T, 8, 4, 1>(a);
        else if (D <= 2048) fwd_launch<T, 8, 8, 1>(a);
        else if (D <= 4096) fwd_launch<T, 8, 4, 4>(a);
        else if (D <= 8192) fwd_launch<T, 8, 8, 4>(a);
        else fwd_launch<T, 8, 8, 8>(a);
    } else if constexpr (VEC == 4) {
        if (D <= 512) fwd_launch<T, 4, 4, 1>(a);
        else if (D <= 1024) fwd_launch<T, 4, 8, 1>(a);
        else if (D <= 2048) fwd_launch<T, 4, 16, 1>(a);
        else if (D <= 4096) fwd_launch<T, 4, 8, 4>(a);
        else if (D <= 8192) fwd_launch<T, 4, 16, 4>(a);
        else fwd_launch<T, 4, 16, 8>(a);
    } else {
        if (D <= 256) fwd_launch<T, 1, 8, 1>(a);
        else if (D <= 1024) fwd_launch<T, 1, 32, 1>(a);
        else if (D <= 4096) fwd_launch<T, 1, 32, 4>(a);
        else fwd_launch<T, 1, 32, 16>(a);
    }
}

struct BwdArgs {
    const NormDims& d;
    const void *x, *w, *dy;
    const float* stats;
    void *dx, *dw, *db;
    float* ws;
    cudaStream_t st;
};

template <typename T, int VEC, int NV, int W>
int bwd_launch(const BwdArgs& a) {   // returns the number of partial rows
    constexpr int RPC = 16 / W;
    const long long need = (a.d.rows + RPC - 1) / RPC;
    const int grid = (int)(need < 1 ? 1 : need < kGrid ? need : kGrid);
    const size_t sm = RPC > 1 ? (size_t)a.d.D * 4 : 0;   // (at most 4096 columns where rows share a CTA)
    k_norm_bwd<T, VEC, NV, W><<<grid, 512, sm, a.st>>>(a.d, (const T*)a.x, a.w, (const T*)a.dy, a.stats, (T*)a.dx, a.ws,
                                                       a.db != nullptr);
    return grid;
}

// 16 elements a lane (32 beyond 8192).
template <typename T, int VEC>
int bwd(const BwdArgs& a) {
    const int D = a.d.D;
    if (D <= 512) return bwd_launch<T, VEC, 16 / VEC, 1>(a);
    if (D <= 1024) return bwd_launch<T, VEC, 16 / VEC, 2>(a);
    if (D <= 2048) return bwd_launch<T, VEC, 16 / VEC, 4>(a);
    if (D <= 4096) return bwd_launch<T, VEC, 16 / VEC, 8>(a);
    if (D <= 8192) return bwd_launch<T, VEC, 16 / VEC, 16>(a);
    return bwd_launch<T, VEC, 32 / VEC, 16>(a);
}

}  // namespace

size_t norm_bwd_ws_bytes(const NormDims& d) { return align256((size_t)kGrid * 2 * d.D * 4); }

cudaError_t launch_norm_fwd(const NormDims& d, const void* x, const void* w, const void* b, void* y, float* stats,
                            cudaStream_t st) {
    const int vec = d.bf16 ? 8 : 4;
    const bool wide = d.D % vec == 0 && d.x_stride % vec == 0 && d.y_stride % vec == 0 && al(x, 16) && al(y, 16) &&
                      al(w, 16) && al(b, 16);
    const FwdArgs a{d, x, w, b, y, stats, st};
    if (d.bf16) wide ? fwd<__nv_bfloat16, 8>(a) : fwd<__nv_bfloat16, 1>(a);
    else wide ? fwd<float, 4>(a) : fwd<float, 1>(a);
    prof_mark("norm_fwd", st);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormDims& d, const void* x, const void* w, const void* dy, const float* stats,
                            void* dx, void* dw, void* db, void* ws, cudaStream_t st) {
    const int vec = d.bf16 ? 8 : 4;
    const bool wide = d.D % vec == 0 && d.x_stride % vec == 0 && d.y_stride % vec == 0 && al(x, 16) && al(dy, 16) &&
                      al(dx, 16) && al(w, 16);
    const BwdArgs a{d, x, w, dy, stats, dx, dw, db, (float*)ws, st};
    int n;
    if (d.bf16) n = wide ? bwd<__nv_bfloat16, 8>(a) : bwd<__nv_bfloat16, 1>(a);
    else n = wide ? bwd<float, 4>(a) : bwd<float, 1>(a);
    prof_mark("norm_bwd", st);
    k_norm_dw<<<dim3((d.D + 31) / 32, db ? 2 : 1), 1024, 0, st>>>(d.D, d.w_bf16, n, db != nullptr, (const float*)ws, dw, db);
    prof_mark("norm_dw", st);
    return cudaGetLastError();
}

}  // namespace efla

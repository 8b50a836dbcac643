// rms.cu -- RMS norm over the last dimension of a residual stream, forward and backward.
//
//   h = x + res, rounded to the stream's type (or x itself);   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w
//   8-bit output: q = e4m3(y (1 / scale)),   scale = max |y| of 128 columns (or of the row) / 448
//   xh = h rstd,  p = dy w,  dx = rstd (p - xh mean(p xh)) + dh,   dw = sum over rows of dy xh
// The norm is of the rounded h: what the backward, and the next layer, read.  A scale is at least 2^-126, so
// that a row of zeros gives zeros and 1 / scale is finite.
// Bound by HBM: x and res read once, h and y written once (backward: h, dy, dh and dx).  Rows in registers as
// in the layer norm, which this shares its rings and sums with: a CTA an SM walks rows, 16 elements a thread,
// weights (and the sums of dw) in registers; rows come by bulk copies, several ahead.
// 16384 x 2048 bf16: forward 36 us (268 MB, 7.4 TB/s with what stays in L2; 48 a call among others), backward 41 us and 4 for
// the sums over CTAs (268 MB).  6001 rows in 8 bits, scales of 128 columns: 19 us (86 MB; 13 us at a plain copy's rate): ten
// rounds of a row's chain of steps a group.
#include <cuda_fp8.h>

#include "norm_rows.cuh"
#include "launch.h"
#include "mix.h"

namespace efla {

namespace {

__device__ unsigned int g_rms_status = 0;   // bit 0: a bounded wait expired

constexpr size_t kRmsRing = 200 * 1024;             // most dynamic shared memory of a CTA (the sums of dw, D fp32, fit in it too)
constexpr float kTop = 448.f;                       // largest e4m3
constexpr float kTiny = 1.17549435082228751e-38f;   // 2^-126

__device__ __forceinline__ float warp_max(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 1 / x for normal x, within 2^-23 of it (its error moves a quotient by less than 2^-19 of an e4m3 step)
__device__ __forceinline__ float rcp_of(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int W>
__device__ __forceinline__ void row_sync(int bar) {
    if (W == 1) __syncwarp();
    else group_sync(bar, 32 * W);
}

template <int VEC>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float* f) {
    if constexpr (VEC == 1) {
        *p = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t r[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            r[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
        if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = r[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
    }
}

struct RmsArgs {
    const void *x, *res, *w;     // backward: h, dh, w
    void* y;                     // y or q; backward: dx
    float* scale;
    void* h;
    float* rstd;
    const void* dy;
    float* part;
    int stages;
};

// W warps a row, NV vectors a lane; as many rows at a time as the CTA has groups of W warps.
template <typename T, int VEC, int NV, int W, bool BWD, bool Q>
__global__ void __launch_bounds__((Cta<W, NV * VEC, BWD>::threads), 1) k_rms(RmsDims d, RmsArgs a) {
    constexpr int SP = NV * VEC, RPC = Cta<W, SP, BWD>::threads / 32 / W, H = SP / 2;
    constexpr bool RING = VEC > 1;
    __shared__ float2 red[RPC][2][W];
    __shared__ uint64_t full[RPC][kStages];
    __shared__ unsigned tops[Q ? RPC : 1][2][Q ? 128 : 1];   // largest |y| (its bits) of each scale's columns
    extern __shared__ __align__(128) unsigned char dyn[];   // the rings; at the end [D] fp32 sums of the CTA's rows
    const int grp = threadIdx.x / (32 * W), t = threadIdx.x % (32 * W), wr = t >> 5;
    const float inv = 1.f / (float)d.D;
    const long long step = (long long)gridDim.x * RPC, r0 = (long long)blockIdx.x * RPC + grp;
    const T *x = (const T*)a.x, *res = (const T*)a.res, *dy = (const T*)a.dy;
    // what a stage holds: x (h), then dy, then res (dh)
    const int arrays = 1 + (BWD ? 1 : 0) + (res ? 1 : 0);
    const T* second = BWD ? dy : res;
    const long long second_stride = BWD ? d.y_stride : d.r_stride;
    Ring ring{dyn, full[grp], (uint32_t)(d.D * sizeof(T)), a.stages, arrays, 0, 0};
    long long ahead = r0;   // the next row to copy
    const auto issue = [&](int to) {
        ring.issue(to, x + ahead * d.x_stride, second + ahead * second_stride, BWD ? res + ahead * d.r_stride : nullptr);
    };
    if (RING) {
        ring.buf += (size_t)grp * a.stages * arrays * ring.bytes;
        if (threadIdx.x < RPC * a.stages) mbar_init(&full[threadIdx.x / a.stages][threadIdx.x % a.stages], 1);
        if (threadIdx.x == 0) fence_mbar_init();
    }
    if (Q)
        for (int i = threadIdx.x; i < RPC * 2 * 128; i += blockDim.x) (&tops[0][0][0])[i] = 0u;
    if (RING || Q) __syncthreads();
    if (RING)
        for (int i = 0; i < a.stages && ahead < d.rows; ++i, ahead += step)
            if (t == 0) issue(i);
    float2 wv[H], u[BWD ? H : 1];   // weight; backward: this thread's columns of dw
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = (m * 32 * W + t) * VEC;
        float wf[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) wf[i] = 0.f;
        if (c < d.D) weights<VEC>(a.w, c, d.w_bf16, wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int e = m * VEC + i;
            (e & 1 ? wv[e / 2].y : wv[e / 2].x) = wf[i];
        }
    }
    if (BWD)
#pragma unroll
        for (int e = 0; e < H; ++e) u[BWD ? e : 0] = make_float2(0.f, 0.f);
    int it = 0;
    bool ok = true;
    float rs_next = 0.f;
    if (BWD && r0 < d.rows) rs_next = __ldg(a.rstd + r0);
    for (long long r = r0; r < d.rows; r += step, it ^= 1) {
        float2 z[H], p[H];
        float rstd = rs_next;
        if (BWD && r + step < d.rows) rs_next = __ldg(a.rstd + r + step);
        if (RING && ok) ok = ring.wait();   // (after a wait that gave up the rows run on, without copies: barriers stay whole)
        const auto get = [&](int which, const T* from, float2* to) {   // (zeros past D)
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int c = (m * 32 * W + t) * VEC;
                Pack<T, VEC> q;
                float f[VEC];
                q.zero();
                if (c < d.D) {
                    if (RING) q = *reinterpret_cast<const Pack<T, VEC>*>(ring.row(which) + c * sizeof(T));
                    else q.load(from + c);
                }
                q.get(f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    (e & 1 ? to[e / 2].y : to[e / 2].x) = f[i];
                }
            }
        };
        const auto put = [&](T* out, const float2* from) {
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const int c = (m * 32 * W + t) * VEC;
                float f[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int e = m * VEC + i;
                    f[i] = e & 1 ? from[e / 2].y : from[e / 2].x;
                }
                Pack<T, VEC> o;
                o.set(f);
                if (c < d.D) o.store(out + c);
            }
        };
        get(0, x + r * d.x_stride, z);
        if (BWD) get(1, dy + r * d.y_stride, p);
        else if (res) get(1, res + r * d.r_stride, p);
        float2 s = make_float2(0.f, 0.f);
        if (BWD) {
            const float2 rs = both(rstd);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                z[e] = mul2(z[e], rs);
                u[BWD ? e : 0] = fma2(p[e], z[e], u[BWD ? e : 0]);
                p[e] = mul2(p[e], wv[e]);
                s = fma2(p[e], z[e], s);
            }
        } else {
            if (res) {
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    z[e] = add2(z[e], p[e]);
                    if (sizeof(T) == 2) {   // as it is stored
                        const __nv_bfloat162 b = __floats2bfloat162_rn(z[e].x, z[e].y);
                        z[e] = bf16x2(*reinterpret_cast<const uint32_t*>(&b));
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < H; ++e) s = fma2(z[e], z[e], s);
        }
        s.x = row_sum<W, false>(make_float2(s.x + s.y, 0.f), red[grp][it], grp + 1, wr).x;
        float2 extra[BWD ? H : 1];
        if constexpr (BWD)
            if (res) get(2, res + r * d.r_stride, extra);
        if (RING) {   // every thread of the row has read the stage
            if (W == 1 || (BWD && res)) row_sync<W>(grp + 1);   // (else the sum's barrier came after the last read)
            if (t == 0 && ok && ahead < d.rows) issue(ring.stage);
            ahead += step;
            ring.next();
        }
        if constexpr (BWD) {
            const float2 rs = both(rstd), c = both(-rstd * s.x * inv);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                z[e] = fma2(z[e], c, mul2(p[e], rs));
                if (res) z[e] = add2(z[e], extra[e]);
            }
            put((T*)a.y + r * d.h_stride, z);
        } else {
            if (res) put((T*)a.h + r * d.h_stride, z);
            rstd = 1.f / sqrtf(s.x * inv + d.eps);
            if (t == 0) a.rstd[r] = rstd;
            const float2 rs = both(rstd);
#pragma unroll
            for (int e = 0; e < H; ++e) z[e] = mul2(mul2(z[e], rs), wv[e]);
            if constexpr (!Q) {
                put((T*)a.y + r * d.y_stride, z);
            } else {
                const int groups = (d.D + d.group - 1) / d.group;
                float top[NV];
#pragma unroll
                for (int m = 0; m < NV; ++m) {   // (columns past D are zero)
                    top[m] = 0.f;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int e = m * VEC + i;
                        top[m] = fmaxf(top[m], fabsf(e & 1 ? z[e / 2].y : z[e / 2].x));
                    }
                }
                const bool local = VEC > 1 && d.group == 128;   // 128 columns are 16 (bf16) or 32 neighbouring lanes
                if (local) {
#pragma unroll
                    for (int m = 0; m < NV; ++m) top[m] = warp_max(top[m], VEC > 1 ? 128 / VEC : 32);
                } else {
                    // a warp's 32 VEC columns at m lie in one scale's where VEC = 1 (and in the row's always)
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        const int c = (m * 32 * W + t) * VEC;
                        const float v = warp_max(top[m], 32);
                        if ((threadIdx.x & 31) == 0 && c < d.D) atomicMax(&tops[Q ? grp : 0][it][c / d.group], __float_as_uint(v));
                    }
                    row_sync<W>(grp + 1);
#pragma unroll
                    for (int m = 0; m < NV; ++m) {
                        const int c = (m * 32 * W + t) * VEC;
                        top[m] = c < d.D ? __uint_as_float(tops[Q ? grp : 0][it][c / d.group]) : 0.f;
                    }
                    // the other buffer's readers are past this row's first barrier: cleared for the next row
                    for (int i = t; i < groups; i += 32 * W) tops[Q ? grp : 0][it ^ 1][i] = 0u;
                    if (W == 1) __syncwarp();
                }
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    const int c = (m * 32 * W + t) * VEC;
                    const float scale = fmaxf(top[m] * (1.f / kTop), kTiny), by = rcp_of(scale);
                    float f[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int e = m * VEC + i;
                        f[i] = (e & 1 ? z[e / 2].y : z[e / 2].x) * by;
                    }
                    if (c < d.D) {
                        store_e4m3<VEC>((uint8_t*)a.y + r * d.y_stride + c, f);
                        if (c % d.group == 0) a.scale[r * groups + c / d.group] = scale;
                    }
                }
            }
        }
    }
    if (!ok) {   // the copies under way land before the CTA ends (a stage's copy completes either phase)
        atomicOr(&g_rms_status, 1u);
        if (t == 0)
            for (int i = 0; i < a.stages; ++i) mbar_wait(&full[grp][i], i < ring.stage ? ring.phase ^ 1 : ring.phase, kWaitLimit);
    }
    if constexpr (BWD) {
        griddep_launch_dependents();
        // the CTA's rows together, one group after another in order, then out as one partial row
        float* comb = (float*)dyn;
        float* pw = a.part + (size_t)blockIdx.x * d.D;
#pragma unroll 1
        for (int k = 0; k < RPC; ++k) {
            __syncthreads();
            if (grp == k) {
#pragma unroll
                for (int m = 0; m < NV; ++m) {
                    const int c = (m * 32 * W + t) * VEC;
                    if (c < d.D)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const int e = m * VEC + i;
                            const float2 h = u[e / 2];
                            const float q = (e & 1 ? h.y : h.x) + (k ? comb[c + i] : 0.f);
                            if (k + 1 < RPC) comb[c + i] = q;
                            else pw[c + i] = q;
                        }
                }
            }
        }
    }
}

// dw = the sum of n partial rows: 32 columns a CTA, 32 groups of rows, then the groups in order
__global__ void __launch_bounds__(1024) k_rms_dw(int D, int w_bf16, int n, const float* part, void* dw) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.f;
    griddep_wait();   // (launched while the rows' kernel still runs)
    if (c < D) {
#pragma unroll 5
        for (int r = g; r < n; r += 32) s += part[(size_t)r * D + c];
    }
    red[g][lane] = s;
    __syncthreads();
    s = warp_sum(red[lane][g]);   // warp g: column g of the CTA
    const int col = blockIdx.x * 32 + g;
    if (lane == 0 && col < D) {
        if (w_bf16) ((__nv_bfloat16*)dw)[col] = __float2bfloat16_rn(s);
        else ((float*)dw)[col] = s;
    }
}

constexpr int kRmsGrid = 152;   // CTAs: one an SM

bool on(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <typename T, int VEC, int NV, int W, bool BWD, bool Q>
cudaError_t launch_rows(const RmsDims& d, RmsArgs a, int* ctas, cudaStream_t st) {
    constexpr int CT = Cta<W, NV * VEC, BWD>::threads, RPC = CT / 32 / W;
    const long long need = (d.rows + RPC - 1) / RPC;
    *ctas = (int)(need < 1 ? 1 : need < kRmsGrid ? need : kRmsGrid);
    // stages: as many as fit, at most kStages (one always fits: three rows of 16384 fp32 are 192 KB)
    const int arrays = 1 + (BWD ? 1 : 0) + (a.res ? 1 : 0);
    const size_t stage = VEC > 1 ? (size_t)RPC * arrays * d.D * sizeof(T) : 0;
    a.stages = stage ? (int)(kRmsRing / stage < kStages ? kRmsRing / stage : kStages) : 0;
    size_t bytes = stage * a.stages;
    if (BWD && bytes < (size_t)d.D * 4) bytes = (size_t)d.D * 4;
    const auto k = k_rms<T, VEC, NV, W, BWD, Q>;
    // (the most that any width takes, not this call's: another host thread may be between this line and its own launch)
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRmsRing);
    if (e != cudaSuccess) return e;
    k<<<*ctas, CT, bytes, st>>>(d, a);
    return cudaGetLastError();
}

// 16 elements a thread; 32 beyond 8192.
template <typename T, int VEC, bool BWD, bool Q>
cudaError_t rows_by_width(const RmsDims& d, const RmsArgs& a, int* ctas, cudaStream_t st) {
    const int D = d.D;
    if (D <= 512) return launch_rows<T, VEC, 16 / VEC, 1, BWD, Q>(d, a, ctas, st);
    if (D <= 1024) return launch_rows<T, VEC, 16 / VEC, 2, BWD, Q>(d, a, ctas, st);
    if (D <= 2048) return launch_rows<T, VEC, 16 / VEC, 4, BWD, Q>(d, a, ctas, st);
    if (D <= 4096) return launch_rows<T, VEC, 16 / VEC, 8, BWD, Q>(d, a, ctas, st);
    if (D <= 8192) return launch_rows<T, VEC, 16 / VEC, 16, BWD, Q>(d, a, ctas, st);
    return launch_rows<T, VEC, 32 / VEC, 16, BWD, Q>(d, a, ctas, st);
}

template <bool BWD, bool Q>
cudaError_t rows_by_type(const RmsDims& d, const RmsArgs& a, int* ctas, cudaStream_t st) {
    const int vec = d.bf16 ? 8 : 4;
    const bool wide = d.D % vec == 0 && d.x_stride % vec == 0 && d.r_stride % vec == 0 && d.y_stride % vec == 0 && d.h_stride % vec == 0 &&
                      on(a.x, 16) && on(a.res, 16) && on(a.w, 16) && on(a.y, Q ? vec : 16) && on(a.h, 16) && on(a.dy, 16);
    using B = __nv_bfloat16;
    if (d.bf16) return wide ? rows_by_width<B, 8, BWD, Q>(d, a, ctas, st) : rows_by_width<B, 1, BWD, Q>(d, a, ctas, st);
    return wide ? rows_by_width<float, 4, BWD, Q>(d, a, ctas, st) : rows_by_width<float, 1, BWD, Q>(d, a, ctas, st);
}

}  // namespace

size_t rms_bwd_ws_bytes(const RmsDims& d) { return align256((size_t)kRmsGrid * d.D * 4); }

cudaError_t launch_rms_fwd(const RmsDims& d, const void* x, const void* res, const void* w, void* y, float* scale, void* h,
                           float* rstd, cudaStream_t st) {
    int n;
    const RmsArgs a{x, res, w, y, scale, h, rstd, nullptr, nullptr, 0};
    const cudaError_t e = d.group ? rows_by_type<false, true>(d, a, &n, st) : rows_by_type<false, false>(d, a, &n, st);
    prof_mark("rms_fwd", st);
    return e;
}

cudaError_t launch_rms_bwd(const RmsDims& d, const void* h, const void* w, const void* dy, const float* rstd, const void* dh,
                           void* dx, void* dw, void* ws, cudaStream_t st) {
    int n;
    const RmsArgs a{h, dh, w, dx, nullptr, nullptr, const_cast<float*>(rstd), dy, (float*)ws, 0};
    cudaError_t e = rows_by_type<true, false>(d, a, &n, st);
    if (e != cudaSuccess) return e;
    prof_mark("rms_bwd", st);
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((d.D + 31) / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_rms_dw, d.D, (int)d.w_bf16, n, (const float*)ws, dw);
    prof_mark("rms_dw", st);
    return e;
}

cudaError_t rms_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_rms_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_rms_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

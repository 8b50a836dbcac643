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
// A CTA (one an SM) walks rows CTA, CTA + grid, ...; 16 elements a thread, so that weight and bias
// (forward) or weight and the sums of dw and db (backward) stay in its registers over all its rows.
// Rows arrive by bulk copies into a ring of shared memory, several ahead: what an SM has in flight
// then costs no registers.  Rows that are not 16-byte aligned are loaded element by element.
// A second kernel adds the CTAs' partial sums in a fixed order, so that results do not depend on
// the order in which CTAs finish; it is launched while the first one ends.
// 16384 x 2048 bf16: forward 22.7 to 24.6 us (134 MB: 5.5 to 5.9 TB/s; a plain copy's rate would take
// 19.8 us), backward 42 to 45 us (201 MB, 4.5 to 4.8 TB/s; 29.7 us), of which 38 us the rows and the
// rest the sums over CTAs.  2047 columns, element by element: 36 and 56 us.  4 x 1024: 2.7 us, a launch.
#include "common.cuh"
#include "gated.h"
#include "launch.h"
#include "norm_rows.cuh"

namespace efla {

namespace {

__device__ unsigned int g_nm_status = 0;   // bit 0: a bounded wait expired

// W warps a row, NV vectors a lane; as many rows at a time as the CTA has groups of W warps.
template <typename T, int VEC, int NV, int W, bool BWD>
__global__ void __launch_bounds__((Cta<W, NV * VEC, BWD>::threads), 1) k_norm(NormDims d, const T* x, const void* w, const void* b, const T* dy,
                                                  T* y, float* stats, float* part, int want_db, int stages) {
    constexpr int SP = NV * VEC, RPC = Cta<W, SP, BWD>::threads / 32 / W;
    constexpr bool RING = VEC > 1;
    __shared__ float2 red[RPC][2][W];
    __shared__ uint64_t full[RPC][kStages];
    extern __shared__ __align__(128) unsigned char dyn[];   // the rings; at the end [D] fp32 sums of the CTA's rows
    const int grp = threadIdx.x / (32 * W), t = threadIdx.x % (32 * W), wr = t >> 5;
    const float inv = 1.f / (float)d.D;
    const long long step = (long long)gridDim.x * RPC, r0 = (long long)blockIdx.x * RPC + grp;
    Ring ring{dyn, full[grp], (uint32_t)(d.D * sizeof(T)), stages, BWD ? 2 : 1, 0, 0};
    long long ahead = r0;   // the next row to copy
    if (RING) {
        ring.buf += (size_t)grp * stages * ring.arrays * ring.bytes;
        if (threadIdx.x < RPC * stages) mbar_init(&full[threadIdx.x / stages][threadIdx.x % stages], 1);
        if (threadIdx.x == 0) fence_mbar_init();
        __syncthreads();
        for (int i = 0; i < stages && ahead < d.rows; ++i, ahead += step)
            if (t == 0) ring.issue(i, x + ahead * d.x_stride, BWD ? dy + ahead * d.y_stride : nullptr);
    }
    // forward: weight and bias; backward: weight, and this thread's columns of dw and db
    constexpr int H = SP / 2;
    float2 wv[H], u[H], v[BWD ? H : 1];
#pragma unroll
    for (int m = 0; m < NV; ++m) {
        const int c = (m * 32 * W + t) * VEC;
        float wf[VEC], bf[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) wf[i] = bf[i] = 0.f;
        if (c < d.D) {
            weights<VEC>(w, c, d.w_bf16, wf);
            if (!BWD && b) weights<VEC>(b, c, d.w_bf16, bf);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int e = m * VEC + i;
            (e & 1 ? wv[e / 2].y : wv[e / 2].x) = wf[i];
            (e & 1 ? u[e / 2].y : u[e / 2].x) = bf[i];
        }
    }
    if (BWD)
#pragma unroll
        for (int e = 0; e < H; ++e) v[BWD ? e : 0] = make_float2(0.f, 0.f);
    int it = 0;
    bool ok = true;
    float2 st_next = make_float2(0.f, 0.f);
    if (BWD && r0 < d.rows) st_next = __ldg(reinterpret_cast<const float2*>(stats + 2 * r0));
    for (long long r = r0; r < d.rows; r += step, it ^= 1) {
        float2 z[H], p[BWD ? H : 1];
        float2 st = st_next;
        if (BWD && r + step < d.rows) st_next = __ldg(reinterpret_cast<const float2*>(stats + 2 * (r + step)));
        if (RING && ok) ok = ring.wait();   // (after a wait that gave up the rows run on, without copies: barriers stay whole)
        // columns past D count as the mean (forward) or as a zero gradient (backward)
        const auto get = [&](int which, const T* from, float2* to) {
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
        get(0, x + r * d.x_stride, z);
        if (BWD) get(1, dy + r * d.y_stride, p);
        float2 s = make_float2(0.f, 0.f), s2 = s;
        if (BWD) {
            const float2 rs = both(st.y), off = both(-st.x * st.y);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float2 g = p[BWD ? e : 0];
                z[e] = fma2(z[e], rs, off);
                u[e] = fma2(g, z[e], u[e]);
                v[BWD ? e : 0] = add2(v[BWD ? e : 0], g);
                const float2 q = mul2(g, wv[e]);
                p[BWD ? e : 0] = q;
                s = add2(s, q);
                s2 = fma2(q, z[e], s2);
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) s = add2(s, z[e]);
        }
        s = row_sum<W, BWD>(make_float2(s.x + s.y, s2.x + s2.y), red[grp][BWD ? it : 0], grp + 1, wr);
        if (RING) {   // every thread of the row has read the stage
            if (W == 1) __syncwarp();
            if (t == 0 && ok && ahead < d.rows) ring.issue(ring.stage, x + ahead * d.x_stride, BWD ? dy + ahead * d.y_stride : nullptr);
            ahead += step;
            ring.next();
        }
        T* out = y + r * (BWD ? (long long)d.D : d.y_stride);
        if (BWD) {   // rstd p - rstd mean(p) - xh rstd mean(p xh)
            const float2 rs = both(st.y), a = both(-st.y * s.x * inv), c = both(-st.y * s.y * inv);
#pragma unroll
            for (int e = 0; e < H; ++e) z[e] = fma2(z[e], c, fma2(p[BWD ? e : 0], rs, a));
        } else {
            st.x = s.x * inv;
            const float2 mean = both(-st.x);
            s = make_float2(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < NV; ++m) {
                const bool in = (m * 32 * W + t) * VEC < d.D;
                if constexpr (VEC > 1) {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        float2& q = z[m * VEC / 2 + i];
                        q = add2(q, mean);
                        if (in) s = fma2(q, q, s);
                    }
                } else {
                    float& q = m & 1 ? z[m / 2].y : z[m / 2].x;
                    q -= st.x;
                    if (in) s.x = fmaf(q, q, s.x);
                }
            }
            st.y = 1.f / sqrtf(row_sum<W, false>(make_float2(s.x + s.y, 0.f), red[grp][1], grp + 1, wr).x * inv + d.eps);
            if (t == 0) *reinterpret_cast<float2*>(stats + 2 * r) = st;
            const float2 rs = both(st.y);
#pragma unroll
            for (int e = 0; e < H; ++e) z[e] = fma2(mul2(z[e], rs), wv[e], u[e]);
        }
#pragma unroll
        for (int m = 0; m < NV; ++m) {
            const int c = (m * 32 * W + t) * VEC;
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int e = m * VEC + i;
                f[i] = e & 1 ? z[e / 2].y : z[e / 2].x;
            }
            Pack<T, VEC> o;
            o.set(f);
            if (c < d.D) o.store(out + c);
        }
    }
    if (!ok) {   // the copies under way land before the CTA ends (a stage's copy completes either phase)
        atomicOr(&g_nm_status, 1u);
        if (t == 0)
            for (int i = 0; i < stages; ++i) mbar_wait(&full[grp][i], i < ring.stage ? ring.phase ^ 1 : ring.phase, kWaitLimit);
    }
    if (!BWD) return;
    griddep_launch_dependents();
    // the CTA's rows together, one group after another in order, then out as one partial row
    float* comb = (float*)dyn;
    float* pw = part + (size_t)blockIdx.x * (want_db ? 2 : 1) * d.D;
#pragma unroll 1
    for (int what = 0; what < (want_db ? 2 : 1); ++what) {
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
                            const float2 h = what ? v[BWD ? e / 2 : 0] : u[e / 2];
                            const float q = (e & 1 ? h.y : h.x) + (k ? comb[c + i] : 0.f);
                            if (k + 1 < RPC) comb[c + i] = q;
                            else pw[(size_t)what * d.D + c + i] = q;
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
    griddep_wait();   // (launched while the rows' kernel still runs)
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

constexpr int kGrid = 152;   // CTAs: one an SM

bool al(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

struct NormArgs {
    const NormDims& d;
    const void *x, *w, *b, *dy;
    void* y;
    float* stats;
    float* part;
    int want_db;
    cudaStream_t st;
};

template <typename T, int VEC, int NV, int W, bool BWD>
cudaError_t launch(const NormArgs& a, int* ctas) {
    constexpr int CT = Cta<W, NV * VEC, BWD>::threads, RPC = CT / 32 / W;
    const long long need = (a.d.rows + RPC - 1) / RPC;
    *ctas = (int)(need < 1 ? 1 : need < kGrid ? need : kGrid);
    // stages: as many as fit, at most kStages; the sums at the end need D fp32
    const size_t stage = VEC > 1 ? (size_t)RPC * (BWD ? 2 : 1) * a.d.D * sizeof(T) : 0;
    const int stages = stage ? (int)(kRing / stage < kStages ? kRing / stage : kStages) : 0;
    size_t bytes = stage * stages;
    if (BWD && bytes < (size_t)a.d.D * 4) bytes = (size_t)a.d.D * 4;
    const auto k = k_norm<T, VEC, NV, W, BWD>;
    // (the most that any width takes, not this call's: another host thread may be between this line and its own launch)
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRing);
    if (e != cudaSuccess) return e;
    k<<<*ctas, CT, bytes, a.st>>>(a.d, (const T*)a.x, a.w, a.b, (const T*)a.dy, (T*)a.y, a.stats, a.part, a.want_db, stages);
    return cudaGetLastError();
}

// 16 elements a thread; 32 beyond 8192.
template <typename T, int VEC, bool BWD>
cudaError_t by_width(const NormArgs& a, int* ctas) {
    const int D = a.d.D;
    if (D <= 512) return launch<T, VEC, 16 / VEC, 1, BWD>(a, ctas);
    if (D <= 1024) return launch<T, VEC, 16 / VEC, 2, BWD>(a, ctas);
    if (D <= 2048) return launch<T, VEC, 16 / VEC, 4, BWD>(a, ctas);
    if (D <= 4096) return launch<T, VEC, 16 / VEC, 8, BWD>(a, ctas);
    if (D <= 8192) return launch<T, VEC, 16 / VEC, 16, BWD>(a, ctas);
    return launch<T, VEC, 32 / VEC, 16, BWD>(a, ctas);
}

template <bool BWD>
cudaError_t by_type(const NormArgs& a, int* ctas) {
    const int vec = a.d.bf16 ? 8 : 4;
    const bool wide = a.d.D % vec == 0 && a.d.x_stride % vec == 0 && a.d.y_stride % vec == 0 && al(a.x, 16) && al(a.y, 16) &&
                      al(a.w, 16) && al(a.b, 16) && al(a.dy, 16);
    if (a.d.bf16) return wide ? by_width<__nv_bfloat16, 8, BWD>(a, ctas) : by_width<__nv_bfloat16, 1, BWD>(a, ctas);
    return wide ? by_width<float, 4, BWD>(a, ctas) : by_width<float, 1, BWD>(a, ctas);
}

}  // namespace

size_t norm_bwd_ws_bytes(const NormDims& d) { return align256((size_t)kGrid * 2 * d.D * 4); }

cudaError_t launch_norm_fwd(const NormDims& d, const void* x, const void* w, const void* b, void* y, float* stats,
                            cudaStream_t st) {
    int n;
    const cudaError_t e = by_type<false>(NormArgs{d, x, w, b, nullptr, y, stats, nullptr, 0, st}, &n);
    prof_mark("norm_fwd", st);
    return e;
}

cudaError_t launch_norm_bwd(const NormDims& d, const void* x, const void* w, const void* dy, const float* stats,
                            void* dx, void* dw, void* db, void* ws, cudaStream_t st) {
    int n;
    cudaError_t e =
        by_type<true>(NormArgs{d, x, w, nullptr, dy, dx, const_cast<float*>(stats), (float*)ws, db != nullptr, st}, &n);
    if (e != cudaSuccess) return e;
    prof_mark("norm_bwd", st);
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((d.D + 31) / 32, db ? 2 : 1);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_norm_dw, d.D, (int)d.w_bf16, n, (int)(db != nullptr), (const float*)ws, dw, db);
    prof_mark("norm_dw", st);
    return e;
}

cudaError_t norm_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_nm_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_nm_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

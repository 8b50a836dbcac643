// conv.cu -- short causal convolution of every channel by itself, forward, backward, and one token.
//
//   pre_t = bias + sum_j w_j x_{t - (W - 1) + j},   y_t = pre_t, or pre_t sigmoid(pre_t)
//   dp_t = dy_t y'(pre_t),   dx_t = sum_j w_j dp_{t + W - 1 - j},   dw_j = sum_t dp_t x_{t - (W - 1) + j},   db = sum_t dp_t
// Places before a sequence's first token are the W - 1 rows of its state, oldest first, or zeros.
// Bound by HBM: every token's row is read once and its result written once.  A thread owns VEC
// neighbouring channels and walks a run of tokens with the W - 1 rows (and W gradients) behind it in
// registers; the rows that two runs share come from the caches.  Sums are fp32.
#include "mix.cuh"
#include "launch.h"

namespace efla {

namespace {

// weights [VEC channels][W] and bias of a thread's channels
template <int VEC, int W>
__device__ __forceinline__ void conv_weights(const ConvDims& d, const void* w, const void* bias, int c, float (&wv)[W][VEC], float (&bv)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j)
            wv[j][i] = d.w_bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[(size_t)(c + i) * W + j])
                                : __ldg((const float*)w + (size_t)(c + i) * W + j);
        bv[i] = !bias ? 0.f : d.w_bf16 ? __bfloat162float(((const __nv_bfloat16*)bias)[c + i]) : __ldg((const float*)bias + c + i);
    }
}

// The row at place t of sequence s (t may lie up to W - 1 before its start).  xa: the axis's rows.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_row(const ConvDims& d, const T* xa, const T* S0, const Seq& s, int t, int c, float (&out)[VEC]) {
    Vec<T, VEC> v;
    if (t >= s.start) v.load(xa + t * d.xs[1] + c);
    else if (S0) v.load(S0 + ((size_t)s.b * (W - 1) + (W - 1 + t - s.start)) * d.D + c);
    else v.zero();
    v.get(out);
}

// Threads past `items` copy the final states: one row and VEC channels each.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256) k_conv_fwd(ConvDims d, const T* x, const void* w, const void* bias, const T* S0, T* y,
                                                   T* S_final, int nv, int run, int runs, long long items) {
    constexpr int NB = 4;   // rows in flight
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(idx % nv) * VEC;
    if (idx >= items) {
        const long long r = (idx - items) / nv;   // (items is a multiple of nv)
        if (!S_final || r >= (long long)d.at.B * (W - 1)) return;
        const int b = (int)(r / (W - 1)), row = (int)(r % (W - 1));
        const Seq s = seq_at(d.at, b);
        const T* xa = x + (d.at.packed ? 0 : b * d.xs[0]);
        float f[VEC];
        conv_row<T, VEC, W>(d, xa, S0, s, s.end - (W - 1) + row, c, f);
        Vec<T, VEC> v;
        v.set(f);
        v.store(S_final + ((size_t)b * (W - 1) + row) * d.D + c);
        return;
    }
    const long long r = idx / nv;
    const int axis = (int)(r / runs), t0 = (int)(r % runs) * run, t1 = min(t0 + run, d.at.L);
    const T* xa = x + axis * d.xs[0];
    T* ya = y + axis * d.ys[0] + c;
    float wv[W][VEC], bv[VEC];
    conv_weights<VEC, W>(d, w, bias, c, wv, bv);
    Seq s = seq_of(d.at, axis, t0);
    for (int t = next_inside(d.at, s, t0, t1); t < t1; t = next_inside(d.at, s, t, t1)) {
        const int hi = min(t1, s.end);
        float win[W - 1][VEC];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv_row<T, VEC, W>(d, xa, S0, s, t - (W - 1) + j, c, win[j]);
#pragma unroll 1
        for (; t < hi; t += NB) {
            Vec<T, VEC> q[NB];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                q[i].zero();
                if (t + i < hi) q[i].load(xa + (t + i) * d.xs[1] + c);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float cur[VEC], o[VEC];
                q[i].get(cur);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float a = bv[e];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) a = fmaf(wv[j][e], win[j][e], a);
                    a = fmaf(wv[W - 1][e], cur[e], a);
                    o[e] = d.silu ? silu_of(a) : a;
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                    win[W - 2][e] = cur[e];
                }
                if (t + i < hi) {
                    Vec<T, VEC> v;
                    v.set(o);
                    v.store(ya + (t + i) * d.ys[1]);
                }
            }
        }
        t = hi;
    }
}

constexpr int kBwdWarps = 8;   // runs a CTA

// A warp walks one run of tokens of 32 VEC channels.  part [CTA rows][W + 1][D]: the CTA's sums of dw and db.
// CTAs with blockIdx.z = 1 compute dS0, a thread a channel vector of a sequence.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kBwdWarps) k_conv_bwd(ConvDims d, const T* x, const void* w, const void* bias, const T* S0,
                                                            const T* dy, const T* dS, T* dx, T* dS0, float* part, int run, int runs,
                                                            long long nruns) {
    constexpr int NB = 4;
    __shared__ float red[kBwdWarps][W + 1][32 * VEC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const bool in = c < d.D;
    float wv[W][VEC], bv[VEC], dw[W][VEC], db[VEC];
    if (in) conv_weights<VEC, W>(d, w, bias, c, wv, bv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    // dp of one token from its window
    const auto grad = [&](const float (&win)[W][VEC], const float (&g)[VEC], float (&dp)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float a = bv[e];
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(wv[j][e], win[j][e], a);
            dp[e] = d.silu ? g[e] * dsilu_of(a) : g[e];
        }
    };
    const long long r = (long long)blockIdx.x * kBwdWarps + warp;
    if (in && r < nruns) {
        const int axis = (int)(r / runs), t0 = (int)(r % runs) * run, t1 = min(t0 + run, d.at.L);
        const T* xa = x + axis * d.xs[0];
        const T* ga = dy + axis * d.dys[0] + c;
        T* da = dx + axis * d.dxs[0] + c;
        Seq s = seq_of(d.at, axis, t0);
        for (int t = next_inside(d.at, s, t0, t1); t < t1; t = next_inside(d.at, s, t, t1)) {
            const int lo = t, hi = min(t1, s.end), stop = hi + W - 1;   // dx_{u - (W - 1)} leaves at step u
            float win[W][VEC], old[W][VEC];                             // x_{u - (W - 1)} .. x_u, dp_{u - (W - 1)} .. dp_u
#pragma unroll
            for (int j = 1; j < W; ++j) conv_row<T, VEC, W>(d, xa, S0, s, lo - W + j, c, win[j]);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) old[j][e] = 0.f;
#pragma unroll 1
            for (int u = lo; u < stop; u += NB) {
                Vec<T, VEC> qx[NB], qg[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    qx[i].zero();
                    qg[i].zero();
                    if (u + i < min(stop, s.end)) {
                        qx[i].load(xa + (u + i) * d.xs[1] + c);
                        qg[i].load(ga + (u + i) * d.dys[1]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int v = u + i;
                    float g[VEC], dp[VEC];
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            win[j][e] = win[j + 1][e];
                            old[j][e] = old[j + 1][e];
                        }
                    qx[i].get(win[W - 1]);
                    qg[i].get(g);
                    grad(win, g, dp);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) old[W - 1][e] = v < s.end ? dp[e] : 0.f;
                    if (v < hi)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            db[e] += dp[e];
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][e] = fmaf(dp[e], win[j][e], dw[j][e]);
                        }
                    const int q = v - (W - 1);
                    if (q >= lo && v < stop) {
                        float o[VEC];
                        if (dS && q >= s.end - (W - 1)) {
                            Vec<T, VEC> f;
                            f.load(dS + ((size_t)s.b * (W - 1) + (q - (s.end - (W - 1)))) * d.D + c);
                            f.get(o);
                        } else {
#pragma unroll
                            for (int e = 0; e < VEC; ++e) o[e] = 0.f;
                        }
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
#pragma unroll
                            for (int j = 0; j < W; ++j) o[e] = fmaf(wv[W - 1 - j][e], old[j][e], o[e]);
                        Vec<T, VEC> f;
                        f.set(o);
                        f.store(da + q * d.dxs[1]);
                    }
                }
            }
            t = hi;
        }
    }
    // dS0: row k of a state is read by the sequence's tokens 0 .. k, with tap k - i at token i; a sequence
    // shorter than W - 1 also hands its later rows on to the final state.  Sequence b belongs to warp b of the CTAs.
    if (dS0 && in) {
        for (long long b = r; b < d.at.B; b += (long long)gridDim.x * kBwdWarps) {
            const Seq s = seq_at(d.at, (int)b);
            const int len = s.end - s.start;
            const T* xa = x + (d.at.packed ? 0 : b * d.xs[0]);
            const T* ga = dy + (d.at.packed ? 0 : b * d.dys[0]) + c;
            float dp[W - 1][VEC];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) dp[i][e] = 0.f;
                if (i < len) {
                    float win[W][VEC], g[VEC];
#pragma unroll
                    for (int j = 0; j < W; ++j) conv_row<T, VEC, W>(d, xa, S0, s, s.start + i - (W - 1) + j, c, win[j]);
                    Vec<T, VEC> v;
                    v.load(ga + (s.start + i) * d.dys[1]);
                    v.get(g);
                    grad(win, g, dp[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                float o[VEC];
                Vec<T, VEC> v;
                v.zero();
                if (dS && k >= len) v.load(dS + ((size_t)b * (W - 1) + (k - len)) * d.D + c);
                v.get(o);
#pragma unroll
                for (int i = 0; i <= k; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = fmaf(wv[k - i][e], dp[i][e], o[e]);
                v.set(o);
                v.store(dS0 + ((size_t)b * (W - 1) + k) * d.D + c);
            }
        }
    }
    // the CTA's runs together, in order
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[warp][j][lane * VEC + e] = dw[j][e];
        red[warp][W][lane * VEC + e] = db[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * VEC; i += 32 * kBwdWarps) {
        const int j = i / (32 * VEC), e = i % (32 * VEC), ch = blockIdx.y * 32 * VEC + e;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kBwdWarps; ++k) sum += red[k][j][e];
        if (ch < d.D) part[((size_t)blockIdx.x * (W + 1) + j) * d.D + ch] = sum;
    }
}

// dw [D][W] and db [D]: the CTAs' sums in order, 32 channels of one tap a CTA, 8 groups of rows
template <int W>
__global__ void __launch_bounds__(256) k_conv_dw(ConvDims d, const float* part, int n, void* dw, void* db) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, j = blockIdx.y;
    float s = 0.f;
    if (c < d.D)
        for (int r = g; r < n; r += 8) s += part[((size_t)r * (W + 1) + j) * d.D + c];
    red[g][lane] = s;
    __syncthreads();
    if (g || c >= d.D) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][lane];
    if (j == W) {
        if (d.w_bf16) ((__nv_bfloat16*)db)[c] = __float2bfloat16_rn(s);
        else ((float*)db)[c] = s;
    } else if (d.w_bf16) {
        ((__nv_bfloat16*)dw)[(size_t)c * W + j] = __float2bfloat16_rn(s);
    } else {
        ((float*)dw)[(size_t)c * W + j] = s;
    }
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256) k_conv_step(ConvDims d, const T* x, const void* w, const void* bias, T* S, const int* slots,
                                                    int nslots, T* y, int nv) {
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long b = idx / nv;
    const int c = (int)(idx % nv) * VEC;
    if (b >= d.at.B) return;
    const long long sl = slots ? __ldg(slots + b) : b;
    Vec<T, VEC> o;
    o.zero();
    if (sl >= 0 && sl < nslots) {
        T* Sb = S + sl * (W - 1) * d.D + c;
        Vec<T, VEC> q[W];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) q[j] = *reinterpret_cast<const Vec<T, VEC>*>(Sb + (size_t)j * d.D);
        q[W - 1].load(x + b * d.xs[0] + c);
        float wv[W][VEC], bv[VEC], a[VEC];
        conv_weights<VEC, W>(d, w, bias, c, wv, bv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[e] = bv[e];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float f[VEC];
            q[j].get(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) a[e] = fmaf(wv[j][e], f[e], a[e]);
            if (j) q[j].store(Sb + (size_t)(j - 1) * d.D);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[e] = d.silu ? silu_of(a[e]) : a[e];
        o.set(a);
    }
    o.store(y + b * d.ys[0] + c);
}

constexpr int kSms = 152;

struct ConvArgs {
    const void *x, *w, *bias, *S0, *dy, *dS;
    void *y, *S_final, *dx, *dw, *db, *dS0;
    float* part;
    const int* slots;
    int nslots;
};

template <typename T, int VEC, int W>
cudaError_t fwd(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    const int nv = d.D / VEC;
    // runs of 32 tokens, shorter while they do not fill the SMs with 512 threads each
    int run = 32;
    while (run > 4 && (long long)nv * d.at.rows() * ((d.at.L + run - 1) / run) < 512LL * kSms) run /= 2;
    const int runs = (d.at.L + run - 1) / run;
    const long long items = (long long)nv * d.at.rows() * runs;
    const long long all = items + (a.S_final ? (long long)nv * d.at.B * (W - 1) : 0);
    if (all == 0) return cudaSuccess;
    k_conv_fwd<T, VEC, W><<<(unsigned)((all + 255) / 256), 256, 0, st>>>(d, (const T*)a.x, a.w, a.bias, (const T*)a.S0, (T*)a.y,
                                                                      (T*)a.S_final, nv, run, runs, items);
    return cudaGetLastError();
}

// tokens a warp of the backward walks, and CTAs along them
struct BwdGrid {
    int run, runs, ctas;
    long long nruns;
};
BwdGrid bwd_grid(const ConvDims& d) {
    const int vec = 4;
    const long long cols = (d.D + 32 * vec - 1) / (32 * vec);
    BwdGrid g;
    g.run = 64;   // shorter while the SMs are not full with 2 CTAs each
    while (g.run > 8 && cols * d.at.rows() * ((d.at.L + g.run - 1) / g.run) < 2LL * kSms * kBwdWarps) g.run /= 2;
    g.runs = (d.at.L + g.run - 1) / g.run;
    g.nruns = (long long)d.at.rows() * g.runs;
    const long long n = (g.nruns + kBwdWarps - 1) / kBwdWarps;
    g.ctas = (int)(n < 1 ? 1 : n);
    return g;
}

template <typename T, int VEC, int W>
cudaError_t bwd(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    const BwdGrid g = bwd_grid(d);
    k_conv_bwd<T, VEC, W><<<dim3(g.ctas, (d.D + 32 * VEC - 1) / (32 * VEC)), 32 * kBwdWarps, 0, st>>>(
        d, (const T*)a.x, a.w, a.bias, (const T*)a.S0, (const T*)a.dy, (const T*)a.dS, (T*)a.dx, (T*)a.dS0, a.part, g.run, g.runs, g.nruns);
    prof_mark("conv_bwd", st);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    k_conv_dw<W><<<dim3((d.D + 31) / 32, a.db ? W + 1 : W), 256, 0, st>>>(d, a.part, g.ctas, a.dw, a.db);
    prof_mark("conv_dw", st);
    return cudaGetLastError();
}

template <typename T, int VEC, int W>
cudaError_t step(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    const int nv = d.D / VEC;
    const long long n = (long long)nv * d.at.B;
    k_conv_step<T, VEC, W><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(d, (const T*)a.x, a.w, a.bias, (T*)a.S_final, a.slots,
                                                                     a.nslots, (T*)a.y, nv);
    return cudaGetLastError();
}

enum Which { kFwd, kBwd, kStep };
template <Which K, typename T, int VEC>
cudaError_t by_taps(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    const auto go = [&](auto taps) {
        constexpr int W = decltype(taps)::value;
        if constexpr (K == kFwd) return fwd<T, VEC, W>(d, a, st);
        else if constexpr (K == kBwd) return bwd<T, VEC, W>(d, a, st);
        else return step<T, VEC, W>(d, a, st);
    };
    if (d.W == 2) return go(std::integral_constant<int, 2>{});
    if (d.W == 3) return go(std::integral_constant<int, 3>{});
    return go(std::integral_constant<int, 4>{});
}

// Whether `bytes` can be moved at once: every row of the call starts on such a boundary.
bool wide(const ConvDims& d, const ConvArgs& a, int vec, bool step) {
    const int es = d.bf16 ? 2 : 4, bytes = vec * es, n = d.at.rows(), L = step ? 1 : d.at.L;
    if (d.D % vec) return false;
    const auto ok = [&](const void* p, const long long (&s)[2]) { return !p || aligned_rows(p, s, n, L, bytes, es); };
    for (const void* p : {a.S0, (const void*)a.S_final, a.dS, (const void*)a.dS0})
        if ((uintptr_t)p % bytes) return false;
    return ok(a.x, d.xs) && ok(a.y, d.ys) && ok(a.dy, d.dys) && ok(a.dx, d.dxs);
}

// 8 channels a thread forward and 4 backward (bf16), where rows allow it
template <Which K>
cudaError_t by_type(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    constexpr int V = K == kBwd ? 4 : 8;
    if (d.bf16)
        return wide(d, a, V, K == kStep) ? by_taps<K, __nv_bfloat16, V>(d, a, st) : by_taps<K, __nv_bfloat16, 1>(d, a, st);
    return wide(d, a, 4, K == kStep) ? by_taps<K, float, 4>(d, a, st) : by_taps<K, float, 1>(d, a, st);
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvDims& d, const void* x, const void* w, const void* bias, const void* S0, void* y,
                            void* S_final, cudaStream_t st) {
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.S0 = S0; a.y = y; a.S_final = S_final;
    const cudaError_t e = by_type<kFwd>(d, a, st);
    prof_mark("conv_fwd", st);
    return e;
}

size_t conv_bwd_ws_bytes(const ConvDims& d) { return align256((size_t)bwd_grid(d).ctas * (d.W + 1) * d.D * 4); }

cudaError_t launch_conv_bwd(const ConvDims& d, const void* x, const void* w, const void* bias, const void* S0, const void* dy,
                            const void* dS, void* dx, void* dw, void* db, void* dS0, void* ws, cudaStream_t st) {
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.S0 = S0; a.dy = dy; a.dS = dS;
    a.dx = dx; a.dw = dw; a.db = db; a.dS0 = dS0; a.part = (float*)ws;
    return by_type<kBwd>(d, a, st);
}

cudaError_t launch_conv_step(const ConvDims& d, const void* x, const void* w, const void* bias, void* S, const int* slots,
                             int nslots, void* y, cudaStream_t st) {
    ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.S_final = S; a.slots = slots; a.nslots = nslots; a.y = y;
    const cudaError_t e = by_type<kStep>(d, a, st);
    prof_mark("conv_step", st);
    return e;
}

}  // namespace efla

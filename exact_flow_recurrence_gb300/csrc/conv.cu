// conv.cu -- short causal convolution of every channel by itself, forward, backward, and one token.
//
//   pre_t = bias + sum_j w_j x_{t - (W - 1) + j},   y_t = pre_t, or pre_t sigmoid(pre_t)
//   dp_t = dy_t y'(pre_t),   dx_t = sum_j w_j dp_{t + W - 1 - j},   dw_j = sum_t dp_t x_{t - (W - 1) + j},   db = sum_t dp_t
// Places before a sequence's first token are the W - 1 rows of its state, oldest first, or zeros.
// A thread owns four neighbouring channels, two of them an instruction, and walks a run of tokens with the W - 1 rows (and W
// gradients) behind it in registers; rows come a batch ahead of the stores, which would hold back the loads behind them;
// the rows that two runs share come from the caches.  A run is as long as fills the SMs evenly (run_of).  Sums are fp32:
// dw and db in registers over a run, then over a CTA's eight, then over CTAs, in order.
// Its floor is HBM: every token's row is read once and its result written once.  B8 L2048 D2048 W4 bf16 with silu: 28 us (134 MB,
// 4.8 TB/s; 20 us at a plain copy's rate), bound by issue (a third: exponent, reciprocal and conversions) and latency at 24
// warps an SM.  Backward, B4 L4096: 54 us and 4 for the sums (201 MB, 3.7 TB/s; 30 us), at 16 warps of 128 registers; two
// channels a thread, 24 warps: 105 us (spills, twice the addresses).  Eight channels a thread forward: 60 us.
#include "mix.cuh"
#include "launch.h"

namespace efla {

namespace {

// VEC values as pairs (a single one with a zero)
template <int VEC>
constexpr int kPairs = (VEC + 1) / 2;
template <typename T, int VEC>
__device__ __forceinline__ void pairs_of(const Vec<T, VEC>& v, float2 (&to)[kPairs<VEC>]) {
    float f[VEC + 1];
    f[VEC] = 0.f;
    v.get(f);
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) to[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pairs(T* p, const float2 (&x)[kPairs<VEC>]) {
    float f[VEC + 1];
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) {
        f[2 * i] = x[i].x;
        f[2 * i + 1 < VEC ? 2 * i + 1 : VEC] = x[i].y;
    }
    Vec<T, VEC> v;
    v.set(f);
    v.store(p);
}

// weights [VEC channels][W] and bias of a thread's channels, as pairs of channels
template <int VEC, int W>
__device__ __forceinline__ void conv_weights(const ConvDims& d, const void* w, const void* bias, int c, float2 (&wv)[W][kPairs<VEC>],
                                             float2 (&bv)[kPairs<VEC>]) {
    float f[VEC * W], b[VEC + 1];
    if (VEC % 4 == 0 && !d.w_bf16 && ((uintptr_t)w & 15) == 0) {   // (16 bytes at a time: VEC W elements from element c W on)
#pragma unroll
        for (int i = 0; i < VEC * W; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>((const float*)w + (size_t)c * W + i));
            f[i] = v.x;
            f[(i + 1) % (VEC * W)] = v.y;
            f[(i + 2) % (VEC * W)] = v.z;
            f[(i + 3) % (VEC * W)] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC * W; ++i)
            f[i] = d.w_bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[(size_t)c * W + i]) : __ldg((const float*)w + (size_t)c * W + i);
    }
    b[VEC] = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        b[i] = !bias ? 0.f : d.w_bf16 ? __bfloat162float(((const __nv_bfloat16*)bias)[c + i]) : __ldg((const float*)bias + c + i);
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) {
        bv[i] = make_float2(b[2 * i], b[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < W; ++j) wv[j][i] = make_float2(f[2 * i * W + j], 2 * i + 1 < VEC ? f[(2 * i + 1) % VEC * W + j] : 0.f);
    }
}

// The row at place t of sequence s (t may lie up to W - 1 before its start).  xa: the axis's rows.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_row(const ConvDims& d, const T* xa, const T* S0, const Seq& s, int t, int c, float2 (&out)[kPairs<VEC>]) {
    Vec<T, VEC> v;
    if (t >= s.start) v.load(xa + t * d.xs[1] + c);
    else if (S0) v.load(S0 + ((size_t)s.b * (W - 1) + (W - 1 + t - s.start)) * d.D + c);
    else v.zero();
    pairs_of(v, out);
}

// Threads past `items` copy the final states: one row and VEC channels each.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(256, 3) k_conv_fwd(ConvDims d, const T* x, const void* w, const void* bias, const T* S0, T* y,
                                                   T* S_final, int nv, int run, int runs, long long items) {
    constexpr int NB = 4, P = kPairs<VEC>;   // rows a batch
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const int c = (int)(idx % nv) * VEC;
    if (idx >= items) {
        const long long r = (idx - items) / nv;   // (items is a multiple of nv)
        if (!S_final || r >= (long long)d.at.B * (W - 1)) return;
        const int b = (int)(r / (W - 1)), row = (int)(r % (W - 1));
        const Seq s = seq_at(d.at, b);
        const T* xa = x + (d.at.packed ? 0 : b * d.xs[0]);
        float2 f[P];
        conv_row<T, VEC, W>(d, xa, S0, s, s.end - (W - 1) + row, c, f);
        store_pairs<T, VEC>(S_final + ((size_t)b * (W - 1) + row) * d.D + c, f);
        return;
    }
    const long long r = idx / nv;
    const int axis = (int)(r / runs), t0 = (int)(r % runs) * run, t1 = min(t0 + run, d.at.L);
    const T* xa = x + axis * d.xs[0];
    T* ya = y + axis * d.ys[0] + c;
    float2 wv[W][P], bv[P];
    conv_weights<VEC, W>(d, w, bias, c, wv, bv);
    Seq s = seq_of(d.at, axis, t0);
    for (int t = next_inside(d.at, s, t0, t1); t < t1; t = next_inside(d.at, s, t, t1)) {
        const int hi = min(t1, s.end);
        float2 win[W - 1][P];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) conv_row<T, VEC, W>(d, xa, S0, s, t - (W - 1) + j, c, win[j]);
        Vec<T, VEC> q[2][NB];   // a batch ahead: a store holds back the loads behind it
        const T* px = xa + t * d.xs[1] + c;   // (running pointers: a row's address is an addition)
        T* py = ya + t * d.ys[1];
        const auto bring = [&](int u, int k) {   // (past the last row: the last again)
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                q[k][i].load(px);
                if (u + i + 1 < hi) px += d.xs[1];
            }
        };
        const auto walk = [&](int u, int k) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                float2 cur[P], o[P];
                pairs_of(q[k][i], cur);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    float2 a = bv[e];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) a = fma2(wv[j][e], win[j][e], a);
                    a = fma2(wv[W - 1][e], cur[e], a);
                    o[e] = d.silu ? mul2(a, sigmoid2(a)) : a;
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                    win[W - 2][e] = cur[e];
                }
                if (u + i < hi) store_pairs<T, VEC>(py, o);
                py += d.ys[1];
            }
        };
        bring(t, 0);
#pragma unroll 1
        for (; t < hi; t += 2 * NB) {
            bring(t + NB, 1);
            walk(t, 0);
            bring(t + 2 * NB, 0);
            walk(t + NB, 1);
        }
        t = hi;
    }
}

constexpr int kBwdWarps = 8;   // runs a CTA
constexpr int kBwdVec = 4, kBwdCtas = 2;

// A warp walks one run of tokens of 32 VEC channels.  part [CTA rows][W + 1][D]: the CTA's sums of dw and db.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(32 * kBwdWarps, kBwdCtas) k_conv_bwd(ConvDims d, const T* x, const void* w, const void* bias, const T* S0,
                                                            const T* dy, const T* dS, T* dx, T* dS0, float* part, int run, int runs,
                                                            long long nruns) {
    constexpr int NB = 4, P = kPairs<VEC>;
    __shared__ float2 red[kBwdWarps][W + 1][32 * P];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * VEC;
    const bool in = c < d.D;
    float2 wv[W][P], bv[P], dw[W][P], db[P];
    if (in) conv_weights<VEC, W>(d, w, bias, c, wv, bv);
#pragma unroll
    for (int e = 0; e < P; ++e) {
        db[e] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = make_float2(0.f, 0.f);
    }
    // dp of one token from its window
    const auto grad = [&](const float2 (&win)[W][P], const float2 (&g)[P], float2 (&dp)[P]) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
            if (d.silu) {
                float2 a = bv[e];
#pragma unroll
                for (int j = 0; j < W; ++j) a = fma2(wv[j][e], win[j][e], a);
                const float2 s = sigmoid2(a);   // s (1 + a (1 - s))
                dp[e] = mul2(mul2(g[e], s), fma2(a, fma2(s, both(-1.f), both(1.f)), both(1.f)));
            } else {
                dp[e] = g[e];
            }
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
            float2 win[W][P], old[W][P];                                // x_{u - (W - 1)} .. x_u, dp_{u - (W - 1)} .. dp_u
#pragma unroll
            for (int j = 1; j < W; ++j) conv_row<T, VEC, W>(d, xa, S0, s, lo - W + j, c, win[j]);
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int e = 0; e < P; ++e) old[j][e] = make_float2(0.f, 0.f);
            const int last = min(stop, s.end) - 1;   // the last token read
            Vec<T, VEC> qx[2][NB], qg[2][NB];        // a batch ahead: a store holds back the loads behind it
            const T *px = xa + lo * d.xs[1] + c, *pg = ga + lo * d.dys[1];
            T* pd = da + lo * d.dxs[1];
            const auto bring = [&](int u, int k) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    qx[k][i].load(px);
                    qg[k][i].load(pg);
                    if (u + i < last) {
                        px += d.xs[1];
                        pg += d.dys[1];
                    }
                }
            };
            const auto walk = [&](int u, int k) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int v = u + i;
                    float2 g[P], dp[P];
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            win[j][e] = win[j + 1][e];
                            old[j][e] = old[j + 1][e];
                        }
                    pairs_of(qx[k][i], win[W - 1]);
                    pairs_of(qg[k][i], g);
                    grad(win, g, dp);
#pragma unroll
                    for (int e = 0; e < P; ++e) old[W - 1][e] = v < s.end ? dp[e] : make_float2(0.f, 0.f);
                    if (v < hi)
#pragma unroll
                        for (int e = 0; e < P; ++e) {
                            db[e] = add2(db[e], dp[e]);
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][e] = fma2(dp[e], win[j][e], dw[j][e]);
                        }
                    const int q = v - (W - 1);
                    if (q >= lo && v < stop) {
                        float2 o[P];
                        if (dS && q >= s.end - (W - 1)) {
                            Vec<T, VEC> f;
                            f.load(dS + ((size_t)s.b * (W - 1) + (q - (s.end - (W - 1)))) * d.D + c);
                            pairs_of(f, o);
                        } else {
#pragma unroll
                            for (int e = 0; e < P; ++e) o[e] = make_float2(0.f, 0.f);
                        }
#pragma unroll
                        for (int e = 0; e < P; ++e)
#pragma unroll
                            for (int j = 0; j < W; ++j) o[e] = fma2(wv[W - 1 - j][e], old[j][e], o[e]);
                        store_pairs<T, VEC>(pd, o);
                        pd += d.dxs[1];
                    }
                }
            };
            bring(lo, 0);
#pragma unroll 1
            for (int u = lo; u < stop; u += 2 * NB) {
                bring(u + NB, 1);
                walk(u, 0);
                bring(u + 2 * NB, 0);
                walk(u + NB, 1);
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
            float2 dp[W - 1][P];
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
#pragma unroll
                for (int e = 0; e < P; ++e) dp[i][e] = make_float2(0.f, 0.f);
                if (i < len) {
                    float2 win[W][P], g[P];
#pragma unroll
                    for (int j = 0; j < W; ++j) conv_row<T, VEC, W>(d, xa, S0, s, s.start + i - (W - 1) + j, c, win[j]);
                    Vec<T, VEC> v;
                    v.load(ga + (s.start + i) * d.dys[1]);
                    pairs_of(v, g);
                    grad(win, g, dp[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < W - 1; ++k) {
                float2 o[P];
                Vec<T, VEC> v;
                v.zero();
                if (dS && k >= len) v.load(dS + ((size_t)b * (W - 1) + (k - len)) * d.D + c);
                pairs_of(v, o);
#pragma unroll
                for (int i = 0; i <= k; ++i)
#pragma unroll
                    for (int e = 0; e < P; ++e) o[e] = fma2(wv[k - i][e], dp[i][e], o[e]);
                store_pairs<T, VEC>(dS0 + ((size_t)b * (W - 1) + k) * d.D + c, o);
            }
        }
    }
    // the CTA's runs together, in order
#pragma unroll
    for (int e = 0; e < P; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[warp][j][lane * P + e] = dw[j][e];
        red[warp][W][lane * P + e] = db[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32 * P; i += 32 * kBwdWarps) {
        const int j = i / (32 * P), e = i % (32 * P), ch = VEC == 1 ? blockIdx.y * 32 + e : blockIdx.y * 32 * VEC + 2 * e;
        float2 sum = red[0][j][e];
#pragma unroll
        for (int k = 1; k < kBwdWarps; ++k) sum = add2(sum, red[k][j][e]);
        float* p = part + ((size_t)blockIdx.x * (W + 1) + j) * d.D + ch;
        if (ch < d.D) p[0] = sum.x;
        if (VEC > 1 && ch < d.D) p[1] = sum.y;   // (D is a multiple of VEC)
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
        constexpr int P = kPairs<VEC>;
        float2 wv[W][P], a[P];
        conv_weights<VEC, W>(d, w, bias, c, wv, a);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float2 f[P];
            pairs_of(q[j], f);
#pragma unroll
            for (int e = 0; e < P; ++e) a[e] = fma2(wv[j][e], f[e], a[e]);
            if (j) q[j].store(Sb + (size_t)(j - 1) * d.D);
        }
        float f[VEC + 1];
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const float2 v = d.silu ? mul2(a[e], sigmoid2(a[e])) : a[e];
            f[2 * e] = v.x;
            f[2 * e + 1 < VEC ? 2 * e + 1 : VEC] = v.y;
        }
        o.set(f);
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

// Tokens a run: as many CTAs as run at once (`each` an SM), or a multiple of them, so that none comes late; 128 at most, since
// a longer run saves no more of the rows that two of them share, and `least` at least.
int run_of(int L, double ctas_a_run, int each, int least) {
    int run = L;
    if (ctas_a_run <= 0) return least;
    for (int m = 1; m == 1 || run > 128; ++m) {
        const double runs = each * kSms * (double)m / ctas_a_run;
        run = runs <= 1 ? L : (int)((L + (long long)runs - 1) / (long long)runs);
        if (runs > L) break;
    }
    return run < least ? least : run > 128 ? 128 : run;
}

template <typename T, int VEC, int W>
cudaError_t fwd(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    const int nv = d.D / VEC;
    const int run = run_of(d.at.L, (double)nv * d.at.rows() / 256, 3, 4), runs = (d.at.L + run - 1) / run;
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
    const int vec = kBwdVec;
    const long long cols = (d.D + 32 * vec - 1) / (32 * vec);
    BwdGrid g;
    g.run = run_of(d.at.L, (double)cols * d.at.rows() / kBwdWarps, kBwdCtas, 8);
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

// Channels a thread where rows allow it
template <Which K>
cudaError_t by_type(const ConvDims& d, const ConvArgs& a, cudaStream_t st) {
    constexpr int V = K == kBwd ? kBwdVec : 4;
    if (d.bf16)
        return wide(d, a, V, K == kStep) ? by_taps<K, __nv_bfloat16, V>(d, a, st) : by_taps<K, __nv_bfloat16, 1>(d, a, st);
    return wide(d, a, V, K == kStep) ? by_taps<K, float, V>(d, a, st) : by_taps<K, float, 1>(d, a, st);
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

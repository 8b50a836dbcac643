// gated_simt.cu -- the gated delta rule on the fp32 CUDA cores, any supported size, type,
// stride and alignment.
//
// For each sequence and value head, with log decays g_t and alpha_t (beta_t, or the exact
// flow's (1 - e^{-beta lambda}) / lambda):
//   S <- e^{g_t} S,   S <- S + alpha_t k_t (v_t - S^T k_t)^T,   o_t = S^T q_t.
// In chunks of C tokens, with c_i the sum of the chunk's g up to token i, D_ij = e^{c_i - c_j}
// for j <= i (never above 1 for decays: no quotient of two products is formed), S the state
// entering the chunk:
//   A = strict_lower(alpha_i D_ij k_i.k_j),  T = (I + A)^{-1},  P = lower(D_ij q_i.k_j)
//   R = V - diag(e^c) K S,   U = T diag(alpha) R
//   O = diag(e^c) Q S + P U,   S' = e^{c_last} S + K^T diag(e^{c_last - c}) U
// and backwards, G the gradient of S':
//   dU = P^T dO + diag(e^{c_last - c}) K G,   dX = T^T dU,   dV = diag(alpha) dX
//   dA = -strict_lower(dX U^T),   dP = lower(dO U^T)
//   dQ = diag(e^c) dO S^T + (dP D) K
//   dK = (dP D)^T Q + diag(e^{c_last - c}) U G^T - diag(e^c) dV S^T
//        + (dA alpha D) K + (dA alpha D)^T K  (+ 2 dlambda k)
//   dalpha_i = dX_i . R_i + sum_j dA_ij D_ij k_i.k_j
//   dc_i from every e^{c}, then dg_t = sum_{i >= t} dc_i inside the chunk
//   G <- e^{c_last} G + (diag(e^c) Q)^T dO - (diag(e^c) K)^T dV
// These kernels take the calls that the tensor-core kernels do not (fp32 tokens, odd strides).
// They are bound by the fp32 multiply-adds and by shared-memory reads of their operands; the
// sequential scans run one CTA for each 16 value columns so that a few heads still fill SMs.
#include "gated_seq.cuh"
#include "launch.h"

namespace efla {

namespace {

constexpr int kC = 32;        // tokens a chunk: the triangular inverse stays short
constexpr int kNT = 256;
constexpr int kDVS = 16;      // value columns of a scan CTA
constexpr int kLd = 129;      // row stride of a [32][<=128] tile in shared memory (odd: no bank conflicts by rows or columns)
constexpr int kLs = 33;       // of a [32][32] tile
constexpr int kLv = 17;       // of a [..][16] tile

struct SimtWs {
    float *T, *P, *cs, *al;       // [H][slots][32][32] x 2, [H][slots][2][32] (c: hi, lo), [H][slots][32]
    float *S, *R, *U, *G, *dX;    // backward only: [H][slots][dk][dv], [..][32][dv] x 2, [..][dk][dv], [..][32][dv]
};

size_t carve(const GDims& d, bool bwd, void* base, SimtWs* w) {
    const size_t n = (size_t)d.H * d.slots(kC);
    char* p = (char*)base;
    const auto take = [&](size_t floats) {
        float* r = (float*)p;
        p += align256(floats * 4);
        return r;
    };
    w->T = take(n * kC * kC);
    w->P = take(n * kC * kC);
    w->cs = take(n * 2 * kC);
    w->al = take(n * kC);
    w->S = w->R = w->U = w->G = w->dX = nullptr;
    if (bwd) {
        w->S = take(n * d.dk * d.dv);
        w->R = take(n * kC * d.dv);
        w->U = take(n * kC * d.dv);
        w->G = take(n * d.dk * d.dv);
        w->dX = take(n * kC * d.dv);
    }
    return (size_t)(p - (char*)base);
}

template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, long long stride, int n, int width) {
    for (int e = threadIdx.x; e < kC * width; e += kNT) {
        const int r = e / width, x = e - r * width;
        dst[r * ld + x] = r < n ? ld_elem(src + r * stride + x) : 0.f;
    }
}

// -------------------------------------------------- per chunk: T, P, c, alpha
template <typename Tin>
__global__ void __launch_bounds__(kNT) k_gated_prep(GDims d, const Tin* q, const Tin* k, const float* g,
                                                    const float* beta, SimtWs w, int slots) {
    __shared__ float Ks[kC * kLd], Qs[kC * kLd], A[kC * kLs];
    __shared__ float cs[2 * kC], al[kC];
    const int slot = blockIdx.x, h = blockIdx.y, hk = h / (d.H / d.Hk), tid = threadIdx.x;
    const int b = seq_of_slot(d, slot, kC);
    const SeqAt s = seq_at(d, b, kC);
    const int t0 = (slot - s.slot0) * kC, n = min(kC, s.len - t0);
    if (n <= 0) return;
    load_rows(Ks, kLd, k + at3(d.ks, s.batch, hk, s.start + t0), d.ks[2], n, d.dk);
    load_rows(Qs, kLd, q + at3(d.qs, s.batch, hk, s.start + t0), d.qs[2], n, d.dk);
    __syncthreads();
    if (tid < 32) {
        const int t = s.start + t0 + tid;
        double c = tid < n ? (double)log_decay(g[at3(d.gs, s.batch, h, t)]) : 0.0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, c, o);
            if (tid >= o) c += x;
        }
        float lam = 0.f;
        for (int i = 0; i < d.dk; ++i) lam = fmaf(Ks[tid * kLd + i], Ks[tid * kLd + i], lam);
        cs[tid] = (float)c;
        cs[kC + tid] = (float)(c - (double)cs[tid]);
        al[tid] = tid < n ? alpha_of(beta[at3(d.bs, s.batch, h, t)], lam, d.euler) : 0.f;
    }
    __syncthreads();
    const size_t rec = (size_t)h * slots + slot;
    float* P = w.P + rec * kC * kC;
    block_mm<kNT>(kC, kC, d.dk, [&](int i, int x) { return Ks[i * kLd + x]; },
                  [&](int x, int j) { return Ks[j * kLd + x]; },
                  [&](int i, int j, float v) { A[i * kLs + j] = j < i ? al[i] * decay(cs[i], cs[kC + i], cs[j], cs[kC + j]) * v : 0.f; });
    block_mm<kNT>(kC, kC, d.dk, [&](int i, int x) { return Qs[i * kLd + x]; },
                  [&](int x, int j) { return Ks[j * kLd + x]; },
                  [&](int i, int j, float v) { P[i * kC + j] = j <= i ? decay(cs[i], cs[kC + i], cs[j], cs[kC + j]) * v : 0.f; });
    __syncthreads();
    if (tid < 32) {   // column tid of T by forward substitution
        float x[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) x[i] = i == tid ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < kC - 1; ++j)
#pragma unroll
            for (int i = j + 1; i < kC; ++i) x[i] = fmaf(-A[i * kLs + j], x[j], x[i]);
        float* T = w.T + rec * kC * kC;
#pragma unroll
        for (int i = 0; i < kC; ++i) T[i * kC + tid] = x[i];
        w.cs[rec * 2 * kC + tid] = cs[tid];
        w.cs[rec * 2 * kC + kC + tid] = cs[kC + tid];
        w.al[rec * kC + tid] = al[tid];
    }
}

// -------------------------------------------------- forward scan over the chunks
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kNT) k_gated_scan(GDims d, const Tin* q, const Tin* k, const Tin* v, const float* S0,
                                                    Tout* o, float* S_final, SimtWs w, int slots) {
    __shared__ float Ks[kC * kLd], S[128 * kLv], X[kC * kLv], U[kC * kLv], O[kC * kLv];
    __shared__ float Ts[kC * kLs], cs[2 * kC], al[kC];
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), c0 = blockIdx.y * kDVS;
    const int tid = threadIdx.x, dk = d.dk, dv = d.dv;
    const SeqAt s = seq_at(d, b, kC);
    const size_t sb = (size_t)blockIdx.x * dk * dv + c0;
    for (int e = tid; e < dk * kDVS; e += kNT) {
        const int r = e / kDVS, x = e % kDVS;
        S[r * kLv + x] = S0 ? S0[sb + (size_t)r * dv + x] : 0.f;
    }
    for (int t0 = 0; t0 < s.len; t0 += kC) {
        const int n = min(kC, s.len - t0), t = s.start + t0;
        const size_t rec = (size_t)h * slots + s.slot0 + t0 / kC;
        __syncthreads();
        load_rows(Ks, kLd, q + at3(d.qs, s.batch, hk, t), d.qs[2], n, dk);   // the queries first
        load_rows(X, kLv, v + at3(d.vs, s.batch, h, t) + c0, d.vs[2], n, kDVS);
        if (tid < 2 * kC) cs[tid] = w.cs[rec * 2 * kC + tid];
        if (tid < kC) {
            al[tid] = w.al[rec * kC + tid];
        }
        for (int e = tid; e < kC * kC; e += kNT) Ts[(e / kC) * kLs + e % kC] = w.T[rec * kC * kC + e];
        if (w.S)
            for (int e = tid; e < dk * kDVS; e += kNT)
                w.S[rec * dk * dv + (size_t)(e / kDVS) * dv + c0 + e % kDVS] = S[(e / kDVS) * kLv + e % kDVS];
        __syncthreads();
        block_mm<kNT>(kC, kDVS, dk, [&](int i, int x) { return Ks[i * kLd + x]; },
                      [&](int x, int j) { return S[x * kLv + j]; },
                      [&](int i, int j, float y) { O[i * kLv + j] = expf(cs[i]) * y; });
        __syncthreads();
        load_rows(Ks, kLd, k + at3(d.ks, s.batch, hk, t), d.ks[2], n, dk);
        __syncthreads();
        block_mm<kNT>(kC, kDVS, dk, [&](int i, int x) { return Ks[i * kLd + x]; },
                      [&](int x, int j) { return S[x * kLv + j]; },
                      [&](int i, int j, float y) {
                          const float r = i < n ? X[i * kLv + j] - expf(cs[i]) * y : 0.f;
                          if (w.R) w.R[(rec * kC + i) * dv + c0 + j] = r;
                          X[i * kLv + j] = al[i] * r;
                      });
        __syncthreads();
        block_mm_ranged<kNT>(kC, kDVS, [&](int i, int x) { return Ts[i * kLs + x]; },
                             [&](int x, int j) { return X[x * kLv + j]; },
                             [&](int i, int, int& lo, int& hi) { lo = 0; hi = i + 1; },
                             [&](int i, int j, float y) {
                                 U[i * kLv + j] = y;
                                 if (w.U) w.U[(rec * kC + i) * dv + c0 + j] = y;
                             });
        __syncthreads();
        for (int e = tid; e < kC * kC; e += kNT) Ts[(e / kC) * kLs + e % kC] = w.P[rec * kC * kC + e];
        const float cl = cs[n - 1], el = expf(cl);
        block_mm<kNT>(dk, kDVS, kC, [&](int r, int i) { return Ks[i * kLd + r]; },
                      [&](int i, int j) { return i < n ? decay(cl, cs[kC + n - 1], cs[i], cs[kC + i]) * U[i * kLv + j] : 0.f; },
                      [&](int r, int j, float y) { S[r * kLv + j] = fmaf(el, S[r * kLv + j], y); });
        __syncthreads();
        if (o)
            block_mm_ranged<kNT>(kC, kDVS, [&](int i, int x) { return Ts[i * kLs + x]; },
                                 [&](int x, int j) { return U[x * kLv + j]; },
                                 [&](int i, int, int& lo, int& hi) { lo = 0; hi = i < n ? i + 1 : 0; },
                                 [&](int i, int j, float y) {
                                     if (i < n) st_elem(o + at3(d.os, s.batch, h, t + i) + c0 + j, O[i * kLv + j] + y);
                                 });
    }
    __syncthreads();
    if (S_final)
        for (int e = tid; e < dk * kDVS; e += kNT)
            S_final[sb + (size_t)(e / kDVS) * dv + e % kDVS] = S[(e / kDVS) * kLv + e % kDVS];
}

// -------------------------------------------------- reverse scan: G and dX of every chunk
template <typename Tin>
__global__ void __launch_bounds__(kNT) k_gated_rscan(GDims d, const Tin* q, const Tin* k, const Tin* dO,
                                                     const float* dS_final, float* dS0, SimtWs w, int slots) {
    __shared__ float Ks[kC * kLd], G[128 * kLv], X[kC * kLv], D[kC * kLv], U[kC * kLv];
    __shared__ float Ts[kC * kLs], cs[2 * kC], al[kC];
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), c0 = blockIdx.y * kDVS;
    const int tid = threadIdx.x, dk = d.dk, dv = d.dv;
    const SeqAt s = seq_at(d, b, kC);
    const size_t sb = (size_t)blockIdx.x * dk * dv + c0;
    for (int e = tid; e < dk * kDVS; e += kNT)
        G[(e / kDVS) * kLv + e % kDVS] = dS_final ? dS_final[sb + (size_t)(e / kDVS) * dv + e % kDVS] : 0.f;
    for (int t0 = (s.len - 1) / kC * kC; s.len > 0 && t0 >= 0; t0 -= kC) {
        const int n = min(kC, s.len - t0), t = s.start + t0;
        const size_t rec = (size_t)h * slots + s.slot0 + t0 / kC;
        __syncthreads();
        load_rows(Ks, kLd, k + at3(d.ks, s.batch, hk, t), d.ks[2], n, dk);
        load_rows(D, kLv, dO + at3(d.dos, s.batch, h, t) + c0, d.dos[2], n, kDVS);
        if (tid < 2 * kC) cs[tid] = w.cs[rec * 2 * kC + tid];
        if (tid < kC) {
            al[tid] = w.al[rec * kC + tid];
        }
        for (int e = tid; e < kC * kC; e += kNT) Ts[(e / kC) * kLs + e % kC] = w.P[rec * kC * kC + e];
        for (int e = tid; e < dk * kDVS; e += kNT)
            w.G[rec * dk * dv + (size_t)(e / kDVS) * dv + c0 + e % kDVS] = G[(e / kDVS) * kLv + e % kDVS];
        __syncthreads();
        const float cl = cs[n - 1], el = expf(cl);
        block_mm<kNT>(kC, kDVS, dk, [&](int i, int x) { return Ks[i * kLd + x]; },
                      [&](int x, int j) { return G[x * kLv + j]; },
                      [&](int i, int j, float y) { U[i * kLv + j] = i < n ? decay(cl, cs[kC + n - 1], cs[i], cs[kC + i]) * y : 0.f; });
        __syncthreads();
        block_mm_ranged<kNT>(kC, kDVS, [&](int i, int x) { return Ts[x * kLs + i]; },
                             [&](int x, int j) { return D[x * kLv + j]; },
                             [&](int i, int, int& lo, int& hi) { lo = i; hi = n; },
                             [&](int i, int j, float y) { U[i * kLv + j] += y; });
        __syncthreads();
        for (int e = tid; e < kC * kC; e += kNT) Ts[(e / kC) * kLs + e % kC] = w.T[rec * kC * kC + e];
        __syncthreads();
        block_mm_ranged<kNT>(kC, kDVS, [&](int i, int x) { return Ts[x * kLs + i]; },
                             [&](int x, int j) { return U[x * kLv + j]; },
                             [&](int i, int, int& lo, int& hi) { lo = i; hi = n; },
                             [&](int i, int j, float y) {
                                 w.dX[(rec * kC + i) * dv + c0 + j] = y;
                                 X[i * kLv + j] = al[i] * y;
                             });
        __syncthreads();
        block_mm<kNT>(dk, kDVS, kC, [&](int r, int i) { return Ks[i * kLd + r]; },
                      [&](int i, int j) { return expf(cs[i]) * X[i * kLv + j]; },
                      [&](int r, int j, float y) { G[r * kLv + j] = fmaf(el, G[r * kLv + j], -y); });
        __syncthreads();
        load_rows(Ks, kLd, q + at3(d.qs, s.batch, hk, t), d.qs[2], n, dk);
        __syncthreads();
        block_mm<kNT>(dk, kDVS, kC, [&](int r, int i) { return Ks[i * kLd + r]; },
                      [&](int i, int j) { return expf(cs[i]) * D[i * kLv + j]; },
                      [&](int r, int j, float y) { G[r * kLv + j] += y; });
    }
    __syncthreads();
    if (dS0)
        for (int e = tid; e < dk * kDVS; e += kNT)
            dS0[sb + (size_t)(e / kDVS) * dv + e % kDVS] = G[(e / kDVS) * kLv + e % kDVS];
}

// -------------------------------------------------- gradients of a chunk, all value heads of a key head
struct GradSmem {
    float K[kC * kLd], Q[kC * kLd], dQ[kC * kLd], dK[kC * kLd], V[kC * kLd], Y[kC * kLd], Z[kC * kLd];
    float dP[kC * kLs], dA[kC * kLs], KK[kC * kLs], P[kC * kLs], W[kC * kLs];
    float cs[2 * kC], al[kC], be[kC], lam[kC], dc[kC], da[kC], dl[kC], part[8];
};

// acc += diag(f) Z and sum[i] += w sum_x f_i Z[i][x] Y[i][x], one warp a row (a fixed order: no atomics)
template <typename F>
__device__ __forceinline__ void add_rows(float* acc, const float* Z, const float* Y, int width, F f, float w, float* sum) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < kC; i += kNT / 32) {
        const float c = f(i);
        float dot = 0.f;
        for (int x = lane; x < width; x += 32) {
            const float z = c * Z[i * kLd + x];
            acc[i * kLd + x] += z;
            dot = fmaf(z, Y[i * kLd + x], dot);
        }
        dot = warp_sum(dot);
        if (lane == 0) sum[i] = fmaf(w, dot, sum[i]);
    }
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kNT) k_gated_grad(GDims d, const Tin* q, const Tin* k, const Tin* dO,
                                                    const float* beta, Tout* dq, Tout* dk_, Tout* dv_, float* dg,
                                                    float* dbeta, SimtWs w, int slots) {
    extern __shared__ float gsm[];
    GradSmem& m = *reinterpret_cast<GradSmem*>(gsm);
    const int slot = blockIdx.x, hk = blockIdx.y, rep = d.H / d.Hk, tid = threadIdx.x, dk = d.dk, dv = d.dv;
    const int b = seq_of_slot(d, slot, kC);
    const SeqAt s = seq_at(d, b, kC);
    const int t0 = (slot - s.slot0) * kC, n = min(kC, s.len - t0), t = s.start + t0;
    if (n <= 0) return;
    load_rows(m.K, kLd, k + at3(d.ks, s.batch, hk, t), d.ks[2], n, dk);
    load_rows(m.Q, kLd, q + at3(d.qs, s.batch, hk, t), d.qs[2], n, dk);
    for (int e = tid; e < kC * kLd; e += kNT) m.dQ[e] = m.dK[e] = 0.f;
    __syncthreads();
    block_mm<kNT>(kC, kC, dk, [&](int i, int x) { return m.K[i * kLd + x]; },
                  [&](int x, int j) { return m.K[j * kLd + x]; },
                  [&](int i, int j, float y) { m.KK[i * kLs + j] = y; });
    for (int h = hk * rep; h < (hk + 1) * rep; ++h) {
        const size_t rec = (size_t)h * slots + slot;
        const float* S = w.S + rec * dk * dv;
        const float* G = w.G + rec * dk * dv;
        const float* R = w.R + rec * kC * dv;
        const float* U = w.U + rec * kC * dv;
        const float* dX = w.dX + rec * kC * dv;
        __syncthreads();
        if (tid < 2 * kC) m.cs[tid] = w.cs[rec * 2 * kC + tid];
        if (tid < kC) {
            m.al[tid] = w.al[rec * kC + tid];
            m.be[tid] = tid < n ? beta[at3(d.bs, s.batch, h, t + tid)] : 0.f;
            m.lam[tid] = m.KK[tid * kLs + tid];
            m.da[tid] = m.dc[tid] = m.dl[tid] = 0.f;
        }
        for (int e = tid; e < kC * kC; e += kNT) m.P[(e / kC) * kLs + e % kC] = w.P[rec * kC * kC + e];
        load_rows(m.V, kLd, dO + at3(d.dos, s.batch, h, t), d.dos[2], n, dv);
        load_rows(m.Y, kLd, U, dv, n, dv);
        __syncthreads();
        const float cl = m.cs[n - 1];
        // dP = lower(dO U^T); dO S^T; U G^T
        block_mm<kNT>(kC, kC, dv, [&](int i, int x) { return m.V[i * kLd + x]; },
                      [&](int x, int j) { return m.Y[j * kLd + x]; },
                      [&](int i, int j, float y) { m.dP[i * kLs + j] = j <= i ? y : 0.f; });
        block_mm<kNT>(kC, dk, dv, [&](int i, int x) { return m.V[i * kLd + x]; },
                      [&](int x, int j) { return S[(size_t)j * dv + x]; },
                      [&](int i, int j, float y) { m.Z[i * kLd + j] = y; });
        __syncthreads();
        add_rows(m.dQ, m.Z, m.Q, dk, [&](int i) { return expf(m.cs[i]); }, 1.f, m.dc);
        __syncthreads();
        block_mm<kNT>(kC, dk, dv, [&](int i, int x) { return m.Y[i * kLd + x]; },
                      [&](int x, int j) { return G[(size_t)j * dv + x]; },
                      [&](int i, int j, float y) { m.Z[i * kLd + j] = y; });
        load_rows(m.V, kLd, dX, dv, n, dv);
        __syncthreads();
        add_rows(m.dK, m.Z, m.K, dk, [&](int i) { return i < n ? decay(cl, m.cs[kC + n - 1], m.cs[i], m.cs[kC + i]) : 0.f; }, 1.f, m.dl);
        // dA = -strict_lower(dX U^T); dV; (alpha dX) S^T
        block_mm<kNT>(kC, kC, dv, [&](int i, int x) { return m.V[i * kLd + x]; },
                      [&](int x, int j) { return m.Y[j * kLd + x]; },
                      [&](int i, int j, float y) { m.dA[i * kLs + j] = j < i ? -y : 0.f; });
        for (int i = tid >> 5; i < n; i += kNT / 32) {
            float dot = 0.f;
            for (int x = tid & 31; x < dv; x += 32) {
                const float y = m.V[i * kLd + x];
                st_elem(dv_ + at3(d.dvs, s.batch, h, t + i) + x, m.al[i] * y);
                dot = fmaf(y, R[(size_t)i * dv + x], dot);
            }
            dot = warp_sum(dot);
            if ((tid & 31) == 0) m.da[i] = dot;
        }
        __syncthreads();
        block_mm<kNT>(kC, dk, dv, [&](int i, int x) { return m.al[i] * m.V[i * kLd + x]; },
                      [&](int x, int j) { return S[(size_t)j * dv + x]; },
                      [&](int i, int j, float y) { m.Z[i * kLd + j] = -y; });
        __syncthreads();
        add_rows(m.dK, m.Z, m.K, dk, [&](int i) { return expf(m.cs[i]); }, 1.f, m.dc);
        float gs = 0.f;   // <G, S> e^{c_last}, through the decay of the whole chunk
        for (int e = tid; e < dk * dv; e += kNT) gs = fmaf(S[e], G[e], gs);
        gs = warp_sum(gs);
        if (tid % 32 == 0) m.part[tid / 32] = gs;
        __syncthreads();
        // the chunk's own pairs: dP D, dA alpha D, and the sums by rows and columns of
        // dP P + dA A (into dc) and of dA D K K^T (into dalpha)
        for (int e = tid; e < kC * kC; e += kNT) {
            const int i = e / kC, j = e % kC, at = i * kLs + j;
            if (j > i || i >= n) {
                m.dP[at] = m.dA[at] = m.W[at] = m.Z[i * kLd + j] = 0.f;
                continue;
            }
            const float D = decay(m.cs[i], m.cs[kC + i], m.cs[j], m.cs[kC + j]), p = m.dP[at], a = m.dA[at];
            const float ak = a * D * m.KK[at];
            m.W[at] = fmaf(p, m.P[at], m.al[i] * ak);
            m.Z[i * kLd + j] = ak;
            m.dP[at] = p * D;
            m.dA[at] = m.al[i] * a * D;
        }
        __syncthreads();
        if (tid < kC) {
            float c = m.dc[tid] - m.dl[tid], a = m.da[tid];
            for (int j = 0; j < kC; ++j) {
                c += m.W[tid * kLs + j] - m.W[j * kLs + tid];
                a += m.Z[tid * kLd + j];
            }
            m.dc[tid] = c;
            m.da[tid] = a;
        }
        __syncthreads();
        block_mm<kNT>(kC, dk, kC, [&](int i, int x) { return m.dP[i * kLs + x]; },
                      [&](int x, int j) { return m.K[x * kLd + j]; },
                      [&](int i, int j, float y) { m.dQ[i * kLd + j] += y; });
        block_mm<kNT>(kC, dk, kC, [&](int i, int x) { return m.dP[x * kLs + i]; },
                      [&](int x, int j) { return m.Q[x * kLd + j]; },
                      [&](int i, int j, float y) { m.dK[i * kLd + j] += y; });
        block_mm<kNT>(kC, dk, kC, [&](int i, int x) { return m.dA[i * kLs + x] + m.dA[x * kLs + i]; },
                      [&](int x, int j) { return m.K[x * kLd + j]; },
                      [&](int i, int j, float y) {
                          const float dl = m.da[i] * dalpha_dlambda_of(m.be[i], m.lam[i], d.euler);
                          m.dK[i * kLd + j] += fmaf(2.f * dl, m.K[i * kLd + j], y);
                      });
        if (tid < 32) {
            float x = tid < n ? m.dc[tid] : 0.f;
            if (tid == n - 1) {
                float y = 0.f;
                for (int e = 0; e < 8; ++e) y += m.part[e];
                x = fmaf(expf(cl), y, x);
                for (int i = 0; i < n; ++i) x += m.dl[i];   // U G^T's e^{c_last - c_i}
            }
#pragma unroll
            for (int o2 = 1; o2 < 32; o2 <<= 1) {   // sums from token tid to the chunk's end
                const float y = __shfl_down_sync(0xffffffffu, x, o2);
                if (tid + o2 < 32) x += y;
            }
            if (tid < n) {
                const size_t at = ((size_t)(d.packed ? 0 : b) * d.H + h) * d.L + t + tid;
                dg[at] = x;
                dbeta[at] = m.da[tid] * dalpha_dbeta_of(m.be[tid], m.lam[tid], d.euler);
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < kC * dk; e += kNT) {
        const int i = e / dk, x = e - i * dk;
        if (i < n) {
            st_elem(dq + at3(d.dqs, s.batch, hk, t + i) + x, m.dQ[i * kLd + x]);
            st_elem(dk_ + at3(d.dks, s.batch, hk, t + i) + x, m.dK[i * kLd + x]);
        }
    }
}

template <typename Tin, typename Tout>
cudaError_t fwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, void* o, float* S_final, const SimtWs& w, cudaStream_t st) {
    const int slots = d.slots(kC);
    if (slots) {
        k_gated_prep<Tin><<<dim3(slots, d.H), kNT, 0, st>>>(d, (const Tin*)q, (const Tin*)k, g, beta, w, slots);
        prof_mark("gated_prep_simt", st);
    }
    k_gated_scan<Tin, Tout><<<dim3((unsigned)d.BH(), d.dv / kDVS), kNT, 0, st>>>(
        d, (const Tin*)q, (const Tin*)k, (const Tin*)v, S0, (Tout*)o, S_final, w, slots);
    prof_mark("gated_scan_simt", st);
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t bwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                float* dbeta, float* dS0, const SimtWs& w, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_gated_grad<Tin, Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(GradSmem));
    if (e == cudaSuccess) e = fwd<Tin, Tout>(d, q, k, v, g, beta, S0, nullptr, nullptr, w, st);
    if (e != cudaSuccess) return e;
    const int slots = d.slots(kC);
    k_gated_rscan<Tin><<<dim3((unsigned)d.BH(), d.dv / kDVS), kNT, 0, st>>>(
        d, (const Tin*)q, (const Tin*)k, (const Tin*)dO, dS_final, dS0, w, slots);
    prof_mark("gated_rscan_simt", st);
    if (!slots) return cudaGetLastError();
    k_gated_grad<Tin, Tout><<<dim3(slots, d.Hk), kNT, sizeof(GradSmem), st>>>(
        d, (const Tin*)q, (const Tin*)k, (const Tin*)dO, beta, (Tout*)dq, (Tout*)dk, (Tout*)dv, dg, dbeta, w, slots);
    prof_mark("gated_grad_simt", st);
    return cudaGetLastError();
}

}  // namespace

size_t gated_simt_fwd_ws_bytes(const GDims& d) {
    SimtWs w;
    return carve(d, false, nullptr, &w);
}
size_t gated_simt_bwd_ws_bytes(const GDims& d) {
    SimtWs w;
    return carve(d, true, nullptr, &w);
}

cudaError_t launch_gated_fwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, void* o, float* S_final, void* ws,
                                  cudaStream_t st) {
    SimtWs w;
    carve(d, false, ws, &w);
    using B = __nv_bfloat16;
    if (d.in_bf16)
        return d.out_bf16 ? fwd<B, B>(d, q, k, v, g, beta, S0, o, S_final, w, st)
                          : fwd<B, float>(d, q, k, v, g, beta, S0, o, S_final, w, st);
    return d.out_bf16 ? fwd<float, B>(d, q, k, v, g, beta, S0, o, S_final, w, st)
                      : fwd<float, float>(d, q, k, v, g, beta, S0, o, S_final, w, st);
}

cudaError_t launch_gated_bwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, const void* dO, const float* dS_final,
                                  void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* ws,
                                  cudaStream_t st) {
    SimtWs w;
    carve(d, true, ws, &w);
    using B = __nv_bfloat16;
    if (d.in_bf16)
        return d.out_bf16 ? bwd<B, B>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st)
                          : bwd<B, float>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st);
    return d.out_bf16 ? bwd<float, B>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st)
                      : bwd<float, float>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st);
}

}  // namespace efla

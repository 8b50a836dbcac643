// gated_simt.cu -- the gated delta rule on the fp32 CUDA cores, any supported size, type,
// stride and alignment.
//
// For each sequence and value head, with log decays g_t and alpha_t (beta_t, or the exact
// flow's (1 - e^{-beta lambda}) / lambda):
//   S <- e^{g_t} S,   r_t = v_t - S^T k_t,   S <- S + alpha_t k_t r_t^T,   o_t = S^T q_t
// and backwards, G the gradient of the state after token t, from the tokens that follow:
//   w_t = (G + q_t dO_t^T)^T k_t,   dv_t = alpha_t w_t,   G <- e^{g_t} (G + q_t dO_t^T - alpha_t k_t w_t^T)
// Both recurrences are taken a token at a time, on states that stay in registers: the fp32
// multiply-adds are as many as in chunked products of 32 tokens, and none of their operands
// but k and q come from shared memory.  A state column needs no other column, so a CTA has 16 of
// them, and a column's dk rows lie on eight lanes.  Every token is one chain, because
// o_t = e^g S^T q + alpha (k.q) r takes both sums from the state before it: two dots (32 multiply-adds a
// lane), three steps of a butterfly, the update.
//
// The gradients of q, k and the gates then come from the states recorded every C tokens, in
// products over a chunk: with c_i the sum of the chunk's g up to token i, D_ij = e^{c_i - c_j}
// for j <= i (never above 1 for decays: no quotient of two products is formed), S the state
// entering the chunk, G the gradient of the one that leaves it, U = diag(alpha) R:
//   dA = -strict_lower(W U^T),   dP = lower(dO U^T)
//   dQ = diag(e^c) dO S^T + (dP D) K
//   dK = (dP D)^T Q + diag(e^{c_last - c}) U G^T - diag(e^c) dV S^T
//        + (dA alpha D) K + (dA alpha D)^T K  (+ 2 dlambda k)
//   dalpha_i = w_i . r_i
//   dc_i from every e^{c}, then dg_t = sum_{i >= t} dc_i inside the chunk
// These kernels take the calls that the tensor-core kernels do not (fp32 tokens, odd strides), and
// short forward passes (gated_fwd_short).  A token takes 0.17 us at dk 128 where a warp has its scheduler to
// itself, 0.13 us at dk 64; with every SM full, the shared-memory reads of k and q (eight 16-byte reads a
// lane and token for 96 multiply-adds) bound them.  H4 L77 dk 64 dv 48 fp32: 13 us; chunked
// products of 32 tokens in shared memory, this file's first form, took 45 us.  One chain of tokens is
// what a long fp32 prompt costs, whatever the rest of the GPU does: B1 H16 L4096 d 128 0.70 ms (its
// bytes: 0.02), B8 H8 L2048 1.01 ms; backward B8 H8 L256 0.40 ms, B4 H16 L1024 1.48 ms.  Taking the dots
// one token early, from a state that lacks the token between, costs more instructions than the
// overlap gives a warp that issues in order: 0.23 us a token.
#include "gated_seq.cuh"
#include "launch.h"
#include "packed2.cuh"

namespace efla {

namespace {

constexpr int kC = 32;        // tokens a chunk of the gradients
constexpr int kNT = 256;
constexpr int kLd = 132;      // row strides of a [32][<= 128] tile in shared memory and of a [..][32] one: 16-byte
constexpr int kLs = 36;       // reads of the same columns in eight rows find different banks

struct SimtWs {   // backward only
    float *S, *R, *G, *W;    // [H][slots][dk][dv], [..][32][dv], [..][dk][dv], [..][32][dv]
};

size_t carve(const GDims& d, void* base, SimtWs* w) {
    const size_t n = (size_t)d.H * d.slots(kC);
    char* p = (char*)base;
    const auto take = [&](size_t floats) {
        float* r = (float*)p;
        p += align256(floats * 4);
        return r;
    };
    w->S = take(n * d.dk * d.dv);
    w->R = take(n * kC * d.dv);
    w->G = take(n * d.dk * d.dv);
    w->W = take(n * kC * d.dv);
    return (size_t)(p - (char*)base);
}

template <typename T>
__device__ __forceinline__ void load_rows(float* dst, int ld, const T* src, long long stride, int n, int width) {
    for (int e = threadIdx.x; e < kC * width; e += kNT) {
        const int r = e / width, x = e - r * width;
        dst[r * ld + x] = r < n ? ld_elem(src + r * stride + x) : 0.f;
    }
}

// -------------------------------------------------- the recurrences
constexpr int kRT = 128;      // threads: four warps of four columns
constexpr int kCols = 16;
constexpr int kTS = 16;       // tokens a stage of k, q, v in shared memory (two stages)

enum { FWD, RECORD, REVERSE };

struct RecArgs {
    const void *q, *k, *v;    // REVERSE: v is dO
    const float *g, *beta;
    const float* state;       // S0, or the final state's gradient
    void* o;                  // FWD
    float* last;              // the final state, or S0's gradient
    float *rec_S, *rec_R;     // RECORD: S and r;  REVERSE: G and w
    int slots;
};

template <typename Tin, typename Tout, int KW, int MODE>
__global__ void __launch_bounds__(kRT, 3) k_gated_rec(GDims d, RecArgs a) {
    constexpr int RJ = KW / 32, NL = kTS * KW / kRT;   // float4s of a lane's rows; elements a thread stages
    constexpr bool Q = MODE != RECORD;
    __shared__ __align__(16) float Ks[2][kTS][KW], Qs[2][Q ? kTS : 1][KW], Vs[2][kTS][kCols], Eg[2][kTS], Al[2][kTS], Kq[2][kTS];
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), c0 = blockIdx.y * kCols;
    const int tid = threadIdx.x, lane = tid & 31, l = lane & 7, cx = (tid >> 5) * 4 + (lane >> 3), col = c0 + cx;
    const int dk = d.dk, dv = d.dv;
    const SeqAt s = seq_at(d, b, kC);
    // rows 4 (l + 8 j) .. + 3 of column col, two a register pair
    float2 S[2 * RJ];
    const size_t sb = (size_t)blockIdx.x * dk * dv + col;
    const auto row = [&](int j, int e) { return 4 * (l + 8 * j) + e; };
#pragma unroll
    for (int j = 0; j < RJ; ++j) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a.state && row(j, e) < dk ? a.state[sb + (size_t)row(j, e) * dv] : 0.f;
        S[2 * j] = make_float2(x[0], x[1]);
        S[2 * j + 1] = make_float2(x[2], x[3]);
    }
    const auto put_state = [&](float* p) {
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            if (row(j, 0) < dk) {   // (dk is a multiple of 4)
                p[(size_t)row(j, 0) * dv] = S[2 * j].x;
                p[(size_t)row(j, 1) * dv] = S[2 * j].y;
                p[(size_t)row(j, 2) * dv] = S[2 * j + 1].x;
                p[(size_t)row(j, 3) * dv] = S[2 * j + 1].y;
            }
        }
    };
    float kr[NL], qr[Q ? NL : 1], vr[2], gr = 0.f, br = 0.f;   // the next stage, on its way
    const auto fetch = [&](int t0) {
        const int n = min(kTS, s.len - t0), t = s.start + t0;
        const Tin* kp = (const Tin*)a.k + at3(d.ks, s.batch, hk, t);
        const Tin* qp = (const Tin*)a.q + at3(d.qs, s.batch, hk, t);
#pragma unroll
        for (int e = 0; e < NL; ++e) {
            const int r = (tid + e * kRT) / KW, x = (tid + e * kRT) % KW;
            const bool in = r < n && x < dk;
            kr[e] = in ? ld_elem(kp + r * d.ks[2] + x) : 0.f;
            if (Q) qr[e] = in ? ld_elem(qp + r * d.qs[2] + x) : 0.f;
        }
        const long long (&vst)[3] = MODE == REVERSE ? d.dos : d.vs;
        const Tin* vp = (const Tin*)a.v + at3(vst, s.batch, h, t) + c0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = (tid + e * kRT) / kCols, x = tid % kCols;
            vr[e] = r < n ? ld_elem(vp + r * vst[2] + x) : 0.f;
        }
        if ((tid & 7) == 0) {   // eight threads a token below: the first of them
            const bool in = tid / 8 < n;
            gr = in ? a.g[at3(d.gs, s.batch, h, t + tid / 8)] : 0.f;
            br = in ? a.beta[at3(d.bs, s.batch, h, t + tid / 8)] : 0.f;
        }
    };
    const int stages = (s.len + kTS - 1) / kTS;
    const auto begin = [&](int it) { return (MODE == REVERSE ? stages - 1 - it : it) * kTS; };
    if (stages) fetch(begin(0));
    for (int it = 0; it < stages; ++it) {
        const int u = it & 1, t0 = begin(it), n = min(kTS, s.len - t0);
        const size_t rec = (size_t)h * a.slots + s.slot0 + t0 / kC;
#pragma unroll
        for (int e = 0; e < NL; ++e) {
            const int r = (tid + e * kRT) / KW, x = (tid + e * kRT) % KW;
            Ks[u][r][x] = kr[e];
            if (Q) Qs[u][r][x] = qr[e];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) Vs[u][(tid + e * kRT) / kCols][tid % kCols] = vr[e];
        __syncthreads();
        {   // the stage's k.q, lambda, alpha and decays: eight threads a token
            float2 kq = both(0.f), lam = both(0.f);
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&Ks[u][tid >> 3][4 * (l + 8 * j)]);
                lam = fma2(make_float2(x.x, x.y), make_float2(x.x, x.y), lam);
                lam = fma2(make_float2(x.z, x.w), make_float2(x.z, x.w), lam);
                if (Q) {
                    const float4 y = *reinterpret_cast<const float4*>(&Qs[u][tid >> 3][4 * (l + 8 * j)]);
                    kq = fma2(make_float2(x.x, x.y), make_float2(y.x, y.y), kq);
                    kq = fma2(make_float2(x.z, x.w), make_float2(y.z, y.w), kq);
                }
            }
            float x = lam.x + lam.y, y = kq.x + kq.y;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                x += __shfl_xor_sync(0xffffffffu, x, o);
                y += __shfl_xor_sync(0xffffffffu, y, o);
            }
            if (l == 0) {
                Eg[u][tid >> 3] = expf(log_decay(gr));
                Al[u][tid >> 3] = tid >> 3 < n ? alpha_of(br, x, d.euler) : 0.f;
                Kq[u][tid >> 3] = y;
            }
        }
        __syncthreads();
        if (it + 1 < stages) fetch(begin(it + 1));
        if (MODE == RECORD && t0 % kC == 0) put_state(a.rec_S + rec * dk * dv + col);
        if (MODE == REVERSE && (it == 0 || t0 % kC != 0)) put_state(a.rec_S + rec * dk * dv + col);
        float keep = 0.f;   // lane l's of eight tokens' results of this column
#pragma unroll 4
        for (int m = 0; m < n; ++m) {
            const int i = MODE == REVERSE ? n - 1 - m : m;
            float2 k[2 * RJ], q[2 * RJ];
#pragma unroll
            for (int j = 0; j < RJ; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&Ks[u][i][4 * (l + 8 * j)]);
                k[2 * j] = make_float2(x.x, x.y);
                k[2 * j + 1] = make_float2(x.z, x.w);
                if (Q) {
                    const float4 y = *reinterpret_cast<const float4*>(&Qs[u][i][4 * (l + 8 * j)]);
                    q[2 * j] = make_float2(y.x, y.y);
                    q[2 * j + 1] = make_float2(y.z, y.w);
                }
            }
            const float eg = Eg[u][i], al = Al[u][i], kq = Q ? Kq[u][i] : 0.f, v = Vs[u][i][cx];
            float2 x[2] = {mul2(S[0], k[0]), mul2(S[1], k[1])}, y[2] = {both(0.f), both(0.f)};
#pragma unroll
            for (int j = 2; j < 2 * RJ; ++j) x[j & 1] = fma2(S[j], k[j], x[j & 1]);
            x[0] = add2(x[0], x[1]);
            float sk = x[0].x + x[0].y, sq = 0.f;
            if (MODE == FWD) {
                y[0] = mul2(S[0], q[0]);
                y[1] = mul2(S[1], q[1]);
#pragma unroll
                for (int j = 2; j < 2 * RJ; ++j) y[j & 1] = fma2(S[j], q[j], y[j & 1]);
                y[0] = add2(y[0], y[1]);
                sq = y[0].x + y[0].y;
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                sk += __shfl_xor_sync(0xffffffffu, sk, o);
                if (MODE == FWD) sq += __shfl_xor_sync(0xffffffffu, sq, o);
            }
            float res;
            if (MODE == REVERSE) {
                res = fmaf(kq, v, sk);   // w
                const float2 a1 = both(eg * v), a2 = both(-eg * al * res);
#pragma unroll
                for (int j = 0; j < 2 * RJ; ++j) S[j] = fma2(both(eg), S[j], fma2(a1, q[j], mul2(a2, k[j])));
            } else {
                const float r = fmaf(-eg, sk, v), ar = al * r;
                res = MODE == FWD ? fmaf(kq, ar, eg * sq) : r;
#pragma unroll
                for (int j = 0; j < 2 * RJ; ++j) S[j] = fma2(both(ar), k[j], mul2(both(eg), S[j]));
            }
            if ((i & 7) == l) keep = res;
            if (MODE == REVERSE ? (i & 7) == 0 : (i & 7) == 7 || i == n - 1) {
                const int ti = (i & ~7) + l;
                if (ti < n) {
                    if (MODE == FWD) st_elem((Tout*)a.o + at3(d.os, s.batch, h, s.start + t0 + ti) + col, keep);
                    else a.rec_R[(rec * kC + t0 % kC + ti) * dv + col] = keep;
                }
            }
        }
    }
    if (a.last) put_state(a.last + sb);
}

// -------------------------------------------------- gradients of a chunk, all value heads of a key head
// A thread has rows i = warp + 8 r and columns j = lane + 32 c of every product (r, c < 4), dQ's and
// dK's among them, which stay in registers over the value heads.  A row's columns are one warp's, so
// the sums by rows are warp sums, in a fixed order.  Bound by the fp32 multiply-adds and the
// shared-memory reads that feed them (one 16-byte read for 8 multiply-adds).
struct GradSmem {
    float K[kC * kLd], Q[kC * kLd], V[kC * kLd], Y[kC * kLd];
    float St[128 * kLs];                                            // 32 columns of S or G
    float dP[kC * kLs], dA[kC * kLs], KK[kC * kLs], QK[kC * kLs], W[kC * kLs];
    float cs[2 * kC], al[kC], be[kC], lam[kC], dc[kC], da[kC], dl[kC], part[8];
};
using Acc = float[4][4];

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// y[r][c] += sum_x A[i][x] B[j][x], x < width (a multiple of 4), rows j < nj of B
template <int NC>
__device__ __forceinline__ void mm_nt(float (&y)[4][NC], const float* A, int lda, const float* B, int ldb, int width, int nj) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int x = 0; x < width; x += 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = ld4(A + (w + 8 * r) * lda + x);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (32 * c >= nj) break;
            const float4 q = ld4(B + (lane + 32 * c) * ldb + x);
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r][c] = dot4(p[r], q, y[r][c]);
        }
    }
}
// y[r][c] += sum_x A(i, x) B[x][j], x < 32
template <typename F>
__device__ __forceinline__ void mm_nn(Acc& y, F A, const float* B, int nj) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 4
    for (int x = 0; x < kC; ++x) {
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = A(w + 8 * r, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (32 * c >= nj) break;
            const float q = B[x * kLd + lane + 32 * c];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r][c] = fmaf(p[r], q, y[r][c]);
        }
    }
}
// y = A M^T for a recorded M [dk][dv], 32 of its columns at a time
__device__ __forceinline__ void mm_state(GradSmem& m, Acc& y, const float* A, const float* M, int dk, int dv) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) y[r][c] = 0.f;
    for (int x0 = 0; x0 < dv; x0 += 32) {
        const int nx = min(32, dv - x0);
        __syncthreads();
        for (int e = threadIdx.x; e < dk * 8; e += kNT)   // (a row's 32 columns: eight 16-byte pieces)
            if (4 * (e & 7) < nx)
                *reinterpret_cast<float4*>(m.St + (e >> 3) * kLs + 4 * (e & 7)) = ld4(M + (size_t)(e >> 3) * dv + x0 + 4 * (e & 7));
        __syncthreads();
        mm_nt<4>(y, A + x0, kLd, m.St, kLs, nx, dk);
    }
}
// acc += f_i y and sum[i] += f_i sum_j y X[i][j]
template <typename F>
__device__ __forceinline__ void add_rows(Acc& acc, const Acc& y, const float* X, F f, float* sum, int dk) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = w + 8 * r;
        const float fi = f(i);
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (lane + 32 * c >= dk) break;
            const float z = fi * y[r][c];
            acc[r][c] += z;
            dot = fmaf(z, X[i * kLd + lane + 32 * c], dot);
        }
        dot = warp_sum(dot);
        if (lane == 0) sum[i] += dot;
    }
}

template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kNT, 2) k_gated_grad(GDims d, const Tin* q, const Tin* k, const Tin* dO,
                                                       const float* g, const float* beta, Tout* dq, Tout* dk_, Tout* dv_,
                                                       float* dg, float* dbeta, SimtWs w, int slots) {
    extern __shared__ __align__(16) float gsm[];
    GradSmem& m = *reinterpret_cast<GradSmem*>(gsm);
    const int slot = blockIdx.x, hk = blockIdx.y, rep = d.H / d.Hk, tid = threadIdx.x, dk = d.dk, dv = d.dv;
    const int wp = tid >> 5, lane = tid & 31;
    int b, t0;
    SeqAt s;
    const int n = chunk_at(d, slot, kC, b, s, t0), t = s.start + t0;
    if (n <= 0) return;
    load_rows(m.K, kLd, k + at3(d.ks, s.batch, hk, t), d.ks[2], n, dk);
    load_rows(m.Q, kLd, q + at3(d.qs, s.batch, hk, t), d.qs[2], n, dk);
    __syncthreads();
    {
        float y[4][1] = {}, z[4][1] = {};
        mm_nt<1>(y, m.K, kLd, m.K, kLd, dk, kC);
        mm_nt<1>(z, m.Q, kLd, m.K, kLd, dk, kC);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m.KK[(wp + 8 * r) * kLs + lane] = y[r][0];
            m.QK[(wp + 8 * r) * kLs + lane] = z[r][0];
        }
    }
    Acc aq = {}, ak = {};
    for (int h = hk * rep; h < (hk + 1) * rep; ++h) {
        const size_t rec = (size_t)h * slots + slot;
        const float* S = w.S + rec * dk * dv;
        const float* G = w.G + rec * dk * dv;
        const float* R = w.R + rec * kC * dv;
        const float* W = w.W + rec * kC * dv;
        __syncthreads();
        if (tid < kC) {
            double c = tid < n ? (double)log_decay(g[at3(d.gs, s.batch, h, t + tid)]) : 0.0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_up_sync(0xffffffffu, c, o);
                if (tid >= o) c += x;
            }
            const float be = tid < n ? beta[at3(d.bs, s.batch, h, t + tid)] : 0.f, lam = m.KK[tid * kLs + tid];
            m.cs[tid] = (float)c;
            m.cs[kC + tid] = (float)(c - (double)m.cs[tid]);
            m.be[tid] = be;
            m.lam[tid] = lam;
            m.al[tid] = tid < n ? alpha_of(be, lam, d.euler) : 0.f;
            m.dc[tid] = m.dl[tid] = 0.f;
        }
        load_rows(m.V, kLd, dO + at3(d.dos, s.batch, h, t), d.dos[2], n, dv);
        __syncthreads();
        for (int e = tid; e < kC * dv; e += kNT) {   // U = alpha r
            const int i = e / dv, x = e - i * dv;
            m.Y[i * kLd + x] = i < n ? m.al[i] * R[e] : 0.f;
        }
        __syncthreads();
        const float cl = m.cs[n - 1], cl2 = m.cs[kC + n - 1];
        const auto rest = [&](int i) { return i < n ? decay(cl, cl2, m.cs[i], m.cs[kC + i]) : 0.f; };
        Acc y;
        {   // dP = lower(dO U^T)
            float z[4][1] = {};
            mm_nt<1>(z, m.V, kLd, m.Y, kLd, dv, kC);
#pragma unroll
            for (int r = 0; r < 4; ++r) m.dP[(wp + 8 * r) * kLs + lane] = lane <= wp + 8 * r ? z[r][0] : 0.f;
        }
        mm_state(m, y, m.V, S, dk, dv);      // dO S^T
        add_rows(aq, y, m.Q, [&](int i) { return expf(m.cs[i]); }, m.dc, dk);
        mm_state(m, y, m.Y, G, dk, dv);      // U G^T
        add_rows(ak, y, m.K, rest, m.dl, dk);
        load_rows(m.V, kLd, W, dv, n, dv);   // (the products with dO are over: mm_state's barriers)
        __syncthreads();
        {   // dA = -strict_lower(W U^T); dV, dalpha
            float z[4][1] = {};
            mm_nt<1>(z, m.V, kLd, m.Y, kLd, dv, kC);
#pragma unroll
            for (int r = 0; r < 4; ++r) m.dA[(wp + 8 * r) * kLs + lane] = lane < wp + 8 * r ? -z[r][0] : 0.f;
        }
        for (int i = wp; i < n; i += kNT / 32) {
            float dot = 0.f;
            for (int x = lane; x < dv; x += 32) {
                const float z = m.V[i * kLd + x];
                st_elem(dv_ + at3(d.dvs, s.batch, h, t + i) + x, m.al[i] * z);
                dot = fmaf(z, R[(size_t)i * dv + x], dot);
            }
            dot = warp_sum(dot);
            if (lane == 0) m.da[i] = dot;
        }
        mm_state(m, y, m.V, S, dk, dv);      // W S^T
        add_rows(ak, y, m.K, [&](int i) { return -expf(m.cs[i]) * m.al[i]; }, m.dc, dk);
        float gs = 0.f;   // <G, S> e^{c_last}, through the decay of the whole chunk
        for (int e = 4 * tid; e < dk * dv; e += 4 * kNT) gs = dot4(ld4(S + e), ld4(G + e), gs);
        gs = warp_sum(gs);
        if (lane == 0) m.part[wp] = gs;
        __syncthreads();
        // the chunk's own pairs: dP D, dA alpha D, and the sums by rows and columns of
        // dP P + dA A (into dc)
        for (int e = tid; e < kC * kC; e += kNT) {
            const int i = e / kC, j = e % kC, at = i * kLs + j;
            if (j > i || i >= n) {
                m.dP[at] = m.dA[at] = m.W[at] = 0.f;
                continue;
            }
            const float D = decay(m.cs[i], m.cs[kC + i], m.cs[j], m.cs[kC + j]), p = m.dP[at], a = m.dA[at];
            m.W[at] = D * fmaf(p, m.QK[at], m.al[i] * a * m.KK[at]);
            m.dP[at] = p * D;
            m.dA[at] = m.al[i] * a * D;
        }
        __syncthreads();
        mm_nn(aq, [&](int i, int x) { return m.dP[i * kLs + x]; }, m.K, dk);
        mm_nn(ak, [&](int i, int x) { return m.dP[x * kLs + i]; }, m.Q, dk);
        mm_nn(ak, [&](int i, int x) { return m.dA[i * kLs + x] + m.dA[x * kLs + i]; }, m.K, dk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wp + 8 * r;
            const float dl = i < n ? 2.f * dlambda_of(m.da[i], m.be[i], m.lam[i], d.euler) : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (lane + 32 * c < dk) ak[r][c] = fmaf(dl, m.K[i * kLd + lane + 32 * c], ak[r][c]);
        }
        if (tid < 32) {
            // (the last token's U G^T decays by nothing inside the chunk: left out of both sums, not added and taken off)
            float x = m.dc[tid] - (tid == n - 1 ? 0.f : m.dl[tid]);
            for (int j = 0; j < kC; ++j) x += m.W[tid * kLs + j] - m.W[j * kLs + tid];
            if (tid >= n) x = 0.f;
            if (tid == n - 1) {
                float z = 0.f;
                for (int e = 0; e < 8; ++e) z += m.part[e];
                x = fmaf(expf(cl), z, x);
                for (int i = 0; i < n - 1; ++i) x += m.dl[i];   // U G^T's e^{c_last - c_i}
            }
#pragma unroll
            for (int o2 = 1; o2 < 32; o2 <<= 1) {   // sums from token tid to the chunk's end
                const float z = __shfl_down_sync(0xffffffffu, x, o2);
                if (tid + o2 < 32) x += z;
            }
            if (tid < n) {
                const size_t at = ((size_t)(d.packed ? 0 : b) * d.H + h) * d.L + t + tid;
                dg[at] = x;
                dbeta[at] = m.da[tid] * dalpha_dbeta_of(m.be[tid], m.lam[tid], d.euler);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = wp + 8 * r;
        if (i >= n) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = lane + 32 * c;
            if (j >= dk) continue;
            st_elem(dq + at3(d.dqs, s.batch, hk, t + i) + j, aq[r][c]);
            st_elem(dk_ + at3(d.dks, s.batch, hk, t + i) + j, ak[r][c]);
        }
    }
}

template <typename Tin, typename Tout, int MODE>
cudaError_t rec(const GDims& d, const RecArgs& a, cudaStream_t st) {
    const auto k = d.dk <= 64 ? k_gated_rec<Tin, Tout, 64, MODE> : k_gated_rec<Tin, Tout, 128, MODE>;
    k<<<dim3((unsigned)d.BH(), d.dv / kCols), kRT, 0, st>>>(d, a);
    prof_mark(MODE == FWD ? "gated_scan_simt" : MODE == RECORD ? "gated_record_simt" : "gated_rscan_simt", st);
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t bwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                float* dbeta, float* dS0, const SimtWs& w, cudaStream_t st) {
    const int slots = d.slots(kC);
    cudaError_t e = cudaFuncSetAttribute(k_gated_grad<Tin, Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(GradSmem));
    if (e == cudaSuccess && slots)
        e = rec<Tin, float, RECORD>(d, RecArgs{q, k, v, g, beta, S0, nullptr, nullptr, w.S, w.R, slots}, st);
    if (e == cudaSuccess)
        e = rec<Tin, float, REVERSE>(d, RecArgs{q, k, dO, g, beta, dS_final, nullptr, dS0, w.G, w.W, slots}, st);
    if (e != cudaSuccess || !slots) return e;
    k_gated_grad<Tin, Tout><<<dim3(slots, d.Hk), kNT, sizeof(GradSmem), st>>>(
        d, (const Tin*)q, (const Tin*)k, (const Tin*)dO, g, beta, (Tout*)dq, (Tout*)dk, (Tout*)dv, dg, dbeta, w, slots);
    prof_mark("gated_grad_simt", st);
    return cudaGetLastError();
}

}  // namespace

// The tensor-core kernels take two launches and a whole chunk's products for any length: 14 us up to
// 64 tokens (d 128).  The recurrence takes one launch and a time that grows with the tokens and, once
// its CTAs no longer all run at once, with their number.  H 4 / H 32, B 1, in us, tensor cores first:
//   L 1: 13.7, 3.5 / 14.3, 4.3    L 16: 13.7, 5.5 / 14.5, 7.5    L 32: 13.9, 8.6 / 14.5, 12.0
//   L 64: 13.9, 15.0 / 14.7, 20.9;    B 16 H 16 (2048 CTAs) L 32: 41, 63
bool gated_fwd_short(const GDims& d) { return d.L <= 32 && d.BH() * (d.dv / kCols) <= 3 * 152; }

size_t gated_simt_bwd_ws_bytes(const GDims& d) {
    SimtWs w;
    return carve(d, nullptr, &w);
}

cudaError_t launch_gated_fwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, void* o, float* S_final, cudaStream_t st) {
    const RecArgs a{q, k, v, g, beta, S0, o, S_final, nullptr, nullptr, 0};
    using B = __nv_bfloat16;
    if (d.in_bf16) return d.out_bf16 ? rec<B, B, FWD>(d, a, st) : rec<B, float, FWD>(d, a, st);
    return d.out_bf16 ? rec<float, B, FWD>(d, a, st) : rec<float, float, FWD>(d, a, st);
}

cudaError_t launch_gated_bwd_simt(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                  const float* beta, const float* S0, const void* dO, const float* dS_final,
                                  void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* ws,
                                  cudaStream_t st) {
    SimtWs w;
    carve(d, ws, &w);
    using B = __nv_bfloat16;
    if (d.in_bf16)
        return d.out_bf16 ? bwd<B, B>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st)
                          : bwd<B, float>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st);
    return d.out_bf16 ? bwd<float, B>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st)
                      : bwd<float, float>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, w, st);
}

}  // namespace efla

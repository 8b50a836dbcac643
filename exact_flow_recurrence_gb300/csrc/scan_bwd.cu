// scan_bwd.cu -- gradients of the selective scan, from its inputs alone.
//
// With g_t = dy_t z sigmoid(z), a_t = e^{dt_t A} and p_t the gradient of the state behind token t:
//   p_t = C_t g_t + a_{t+1} p_{t+1},   dC_t = sum_d h_t g_t,   dB_t = sum_d p_t dt_t u_t
//   s1 = sum_n p_t B_t,   e_t = a_t p_t h_{t-1},   du = dt s1 + skip g,   d(dt) = sum_n A e_t + u s1,   dA = sum_t dt e_t
// The tokens are cut into chunks (32 tokens from 9 states on).  Both recurrences are linear, so one launch takes every chunk
// from a zero state to its last token and, with the running product of its decays, its gradients back to its first:
// all chunks at once.  A second launch chains the chunks' maps, and the third has every chunk's entering state and
// gradient at hand: it walks the chunk forward to the state in front of every kSub tokens (shared memory),
// then back, kSub tokens' states in registers.  Sums over channels (dB, dC) and tokens (dA, dskip, dbias) are
// partial sums of CTAs, added in a fixed order by the last launch.
// B4 L4096 D2048 N16 bf16 with gate: 0.97 ms (473 MB; 70 us at a plain copy's rate, 175 us for the twelve fp32 operations and the
// exponential that a gradient needs at least): every chunk by itself 206 us (issue slots 61% used), the chain 41 us (268 MB:
// a plain copy's rate), gradients 695 us (422 instructions a warp's token of 32 channels, 230 of them the walk back; slots
// half used, by two warps a scheduler: 255 registers), sums 9 us (two launches, one value a thread: 17).  Chunks of 64 tokens with a tile a barrier: 2.43 ms;
// loads in batches ahead of stores took 1.60 to 0.96.
#include "scan.cuh"
#include "launch.h"

namespace efla {

namespace {

constexpr int kSub = 4;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMost = 3.402823466e38f;   // the largest finite fp32

// Tokens a chunk: dt, u and the gated gradient of a CTA's channels take 48 KB at most
constexpr int chunk_of(int lanes) { return lanes >= 4 ? 32 : lanes == 2 ? 16 : 8; }

// ends, grads [axis][chunk][D][states]: the chunk's last state from a zero one, and its gradient in front of its first
// token; after the chain: the state that it starts from, and the gradient that reaches its last token from behind.
// dts [axis][chunk][D]; alive [axis][chunk][2]: whether state and gradient pass through the whole chunk.
// bc [channel block][axis L + token][G][2 states], ch [grid x][D][states], then skip and bias [D] each (ch_stride): partial sums.
struct ScanWs {
    int chunks, gx;
    float *ends, *grads, *dts;
    int* alive;
    float *bc, *ch;
};

// floats a CTA row of `ch`: whole float4
__host__ __device__ inline size_t ch_stride(const ScanDims& d, int S) { return ((size_t)d.D * (S + 2) + 3) / 4 * 4; }

// The arrays of one axis from a CTA's first channel on
template <typename T>
struct Rows {
    const T *u, *delta, *z, *Bm, *C, *dy;
    __device__ __forceinline__ Rows(const ScanDims& d, const ScanIn& in, const void* gy, int axis, const ChBlock& cb) {
        u = (const T*)in.u + axis * d.us[0] + cb.c0;
        delta = (const T*)in.delta + axis * d.ds[0] + cb.c0;
        z = in.z ? (const T*)in.z + axis * d.zs[0] + cb.c0 : nullptr;
        Bm = (const T*)in.Bm + axis * d.bs[0] + cb.g * d.bs[2];
        C = (const T*)in.C + axis * d.cs[0] + cb.g * d.cs[2];
        dy = (const T*)gy + axis * d.dys[0] + cb.c0;
    }
};

constexpr int kBatch = 8;   // tokens of four channels a thread loads at once

// A chunk in shared memory: dt, u, g [tokens][CH] fp32 (g = dy z sigmoid(z)), B and C [tokens][NL][4 and 4] fp32,
// and what its tokens are.
template <typename T, int NL>
struct Chunk {
    static constexpr int CH = ScanTile<NL>::ch, S = ScanTile<NL>::states, C = chunk_of(NL);
    // (One pair of channels a thread, in twice the threads of half the registers, adds up over channels twice as often:
    // B4 L4096 D2048 N16 takes 1.01 ms so, 0.96 with two.)
    static constexpr int NP = kNP, TH = 256 / NP;
    static constexpr int floats = 3 * C * CH + C * NL * 8;
    float *dt, *u, *g;
    float* bc;
    int *what, *seq;    // [C]
    __device__ __forceinline__ Chunk(float* base, int* flags)
        : dt(base), u(base + C * CH), g(base + 2 * C * CH), bc(base + 3 * C * CH), what(flags), seq(flags + C) {}
    // tokens ta .. tb-1 (every thread of the CTA; ends with a barrier)
    template <bool WIDE>
    __device__ __forceinline__ void load(const ScanDims& d, const Rows<T>& r, const ChBlock& cb, int axis, int ta, int tb, float4 bias) const {
        constexpr int V = CH / 4, rows = TH / V, items = C / rows, batch = items < kBatch ? items : kBatch;
        const int tid = threadIdx.x, c = tid % V * 4, row = tid / V, n = min(4, cb.n - c);
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();   // (the last readers of what was here)
        if (tid < C) {
            const TokenAt a = token_at(d.at, axis, ta + tid, tb);
            what[tid] = a.what;
            seq[tid] = a.seq;
        }
        __syncthreads();
        // (every load of a batch before its first use, and before the first store, which would hold the loads behind it back; tokens
        // past the last read the last one again, and count as zeros)
        constexpr int groups = 2 * C * NL, bcs = (groups + TH - 1) / TH;
        Vec<T, 4> vb[bcs];
#pragma unroll
        for (int j = 0; j < bcs; ++j) {
            const int e = tid + j * TH, q = e % NL, t = e / NL % C;
            vb[j].zero();
            if (e < groups && !(what[t] & kOutside) && 4 * q < d.N)
                take4<T, WIDE>(vb[j], (e >= C * NL ? r.C + (ta + t) * d.cs[1] : r.Bm + (ta + t) * d.bs[1]) + 4 * q, min(4, d.N - 4 * q));
        }
        const auto batch_of = [&](int j0) {
            Vec<T, 4> vd[batch], vu[batch], vg[batch], vz[batch];
#pragma unroll
            for (int j = 0; j < batch; ++j) {
                const long long tt = min(ta + row + (j0 + j) * rows, tb - 1);
                vd[j].zero(); vu[j].zero(); vg[j].zero(); vz[j].zero();
                if (n > 0) {
                    take4<T, WIDE>(vd[j], r.delta + tt * d.ds[1] + c, n);
                    take4<T, WIDE>(vu[j], r.u + tt * d.us[1] + c, n);
                    take4<T, WIDE>(vg[j], r.dy + tt * d.dys[1] + c, n);
                    if (r.z) take4<T, WIDE>(vz[j], r.z + tt * d.zs[1] + c, n);
                }
            }
#pragma unroll
            for (int j = 0; j < batch; ++j) {
                const int t = row + (j0 + j) * rows, o = t * CH + c;
                const bool in_range = n > 0 && !(what[t] & kOutside);
                float4 xg = as4(vg[j]);
                const float4 xd = steps(d, add4(as4(vd[j]), bias), n), xu = as4(vu[j]);
                if (r.z) {
                    const float4 z = as4(vz[j]);
                    xg = mul4(xg, mul4(z, sigmoid4(z)));
                }
                *reinterpret_cast<float4*>(dt + o) = in_range ? xd : none;
                *reinterpret_cast<float4*>(u + o) = in_range ? xu : none;
                *reinterpret_cast<float4*>(g + o) = in_range ? xg : none;
            }
        };
#pragma unroll
        for (int j0 = 0; j0 < items; j0 += batch) batch_of(j0);
#pragma unroll
        for (int j = 0; j < bcs; ++j) {
            const int e = tid + j * TH, q = e % NL, t = e / NL % C;
            if (e < groups) *reinterpret_cast<float4*>(bc + (t * NL + q) * 8 + (e >= C * NL ? 4 : 0)) = as4(vb[j]);
        }
        __syncthreads();
    }
};


// ------------------------------------------------------------------- every chunk by itself
// the values of the thread's four channels, from p on
__device__ __forceinline__ void load_pairs(const float* p, float2 (&to)[kNP]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    to[0] = lo(v);
    to[1] = hi(v);
}
template <typename T, int NL, bool WIDE>
__global__ void __launch_bounds__((Chunk<T, NL>::TH)) k_scan_local(ScanDims d, ScanIn in, ScanGrads gr, ScanWs ws) {
    using Ck = Chunk<T, NL>;
    constexpr int CH = Ck::CH, S = Ck::S, C = Ck::C, NP = Ck::NP;
    extern __shared__ __align__(16) float dyn[];
    __shared__ int flags[2 * C];
    const Ck ck(dyn, flags);
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const int axis = blockIdx.z, k = blockIdx.x, ta = k * C, tb = min(ta + C, d.at.L);
    const ScanLane<NL, NP> l;
    const Rows<T> r(d, in, gr.dy, axis, cb);
    {
        const int c = threadIdx.x % (CH / 4) * 4;
        ck.template load<WIDE>(d, r, cb, axis, ta, tb,
                               in.dbias ? load4<float, false>(in.dbias + cb.c0 + c, min(4, cb.n - c)) : make_float4(0.f, 0.f, 0.f, 0.f));
    }
    float2 a2[NP][4], h[NP][4], cp[NP][4], q[NP][4], dts[NP];
    l.pairs(in.A, 0, d, cb, a2);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        dts[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            a2[i][n] = mul2(a2[i][n], both(kLog2eF));
            h[i][n] = q[i][n] = make_float2(0.f, 0.f);
            cp[i][n] = both(1.f);
        }
    }
    // whether the state before the chunk, and gradients back to it, still pass
    bool alive = true, open = !(ck.what[0] & kOutside);
#pragma unroll 2
    for (int t = 0; t < tb - ta; ++t) {
        const int w = ck.what[t];
        const size_t at = (size_t)ck.seq[t] * d.D * d.N;
        if (w & kFirst) {
            alive = false;
            l.pairs(in.S0, at, d, cb, h);
        }
        float2 dt[NP], u[NP], g[NP];
        load_pairs(ck.dt + t * CH + l.cl, dt);
        load_pairs(ck.u + t * CH + l.cl, u);
        load_pairs(ck.g + t * CH + l.cl, g);
        Bc bc;
        bc.load(ck.bc + (t * NL + l.nl) * 8, true);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float2 du = mul2(dt[i], u[i]);
            dts[i] = add2(dts[i], dt[i]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 a = decay2(dt[i], a2[i][n]);
                h[i][n] = fma2(a, h[i][n], mul2(du, both(bc.bn(n))));
                if (open) {
                    cp[i][n] = mul2(cp[i][n], a);
                    q[i][n] = fma2(cp[i][n], mul2(g[i], both(bc.cn(n))), q[i][n]);
                }
            }
        }
        if (open && (w & kLast)) {
            open = false;
            if (gr.dS) {
                float2 f[NP][4];
                l.pairs(gr.dS, at, d, cb, f);
#pragma unroll
                for (int i = 0; i < NP; ++i)
#pragma unroll
                    for (int n = 0; n < 4; ++n) q[i][n] = fma2(cp[i][n], f[i][n], q[i][n]);
            }
        }
    }
    // A product of decays above one that has left fp32 says nothing (inf times a zero gradient is not a number): then the
    // gradient is taken back a token at a time instead.  (A product that vanishes and grows again loses less than 2^-21 of a
    // gradient, or one that is infinite token by token too.)
    bool whole = true;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) whole = whole && fabsf(cp[i][n].x) <= kMost && fabsf(cp[i][n].y) <= kMost;
    if (!whole) {
        int t = 0;   // the last token that a gradient in front of the chunk's first one passes
        while (t + 1 < tb - ta && !(ck.what[t] & (kLast | kOutside))) ++t;
        l.pairs(ck.what[t] & kLast ? gr.dS : nullptr, (size_t)ck.seq[t] * d.D * d.N, d, cb, q);
#pragma unroll 1
        for (; t >= 0; --t) {
            float2 dt[NP], g[NP];
            load_pairs(ck.dt + t * CH + l.cl, dt);
            load_pairs(ck.g + t * CH + l.cl, g);
            Bc bc;
            bc.load(ck.bc + (t * NL + l.nl) * 8, true);
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n) q[i][n] = mul2(decay2(dt[i], a2[i][n]), fma2(g[i], both(bc.cn(n)), q[i][n]));
        }
    }
    const size_t at = (size_t)axis * ws.chunks + k;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        ws.alive[2 * at] = alive;
        ws.alive[2 * at + 1] = open;
    }
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
        if (l.cl + i >= cb.n) continue;
        const size_t ch = at * d.D + cb.c0 + l.cl + i;
        *reinterpret_cast<float4*>(ws.ends + ch * S + 4 * l.nl) = one_of<NP>(h, i);
        *reinterpret_cast<float4*>(ws.grads + ch * S + 4 * l.nl) = one_of<NP>(q, i);
        if (l.nl == 0) ws.dts[ch] = i & 1 ? dts[i / 2].y : dts[i / 2].x;
    }
}

// ------------------------------------------------------------------- the chunks' maps chained
// A thread takes four states of a channel through its axis's chunks: blockIdx.y 0 forward, 1 backward.
__global__ void __launch_bounds__(128) k_scan_chain(ScanDims d, const float* A, ScanWs ws, int nl) {
    constexpr int AHEAD = 16;   // chunks loaded at once (188 chunks of one axis: 28 us; 38 with eight)
    const long long idx = (long long)blockIdx.x * 128 + threadIdx.x;
    if (idx >= (long long)d.D * nl) return;
    const int c = (int)(idx / nl), q = (int)(idx % nl), axis = blockIdx.z, back = blockIdx.y, n = ws.chunks;
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = 4 * q + i < d.N ? A[(size_t)c * d.N + 4 * q + i] * kLog2eF : 0.f;
    float4* at = reinterpret_cast<float4*>(back ? ws.grads : ws.ends) + (size_t)axis * n * d.D * nl + idx;
    const float* dts = ws.dts + (size_t)axis * n * d.D + c;
    const int* alive = ws.alive + 2 * (size_t)axis * n + back;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += AHEAD) {
        float4 e[AHEAD];
        float x[AHEAD];
        int on[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int k = back ? n - 1 - (k0 + j) : k0 + j;
            if (k0 + j < n) {
                e[j] = at[(size_t)k * d.D * nl];
                x[j] = dts[(size_t)k * d.D];
                on[j] = alive[2 * k];
            }
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int k = back ? n - 1 - (k0 + j) : k0 + j;
            if (k0 + j < n) {
                at[(size_t)k * d.D * nl] = s;
                s = on[j] ? add4(make_float4(times_ex2(s.x, a[0] * x[j]), times_ex2(s.y, a[1] * x[j]), times_ex2(s.z, a[2] * x[j]),
                                             times_ex2(s.w, a[3] * x[j])), e[j])
                          : e[j];
            }
        }
    }
}

// ------------------------------------------------------------------- gradients
// Sums of 8 values over the lanes along the channels (32 / NL of them); `first`: which values this lane holds
// afterwards, and whether it is the one to write them.
template <int NL>
struct ChannelSum {
    static constexpr int lanes = 32 / NL, steps = lanes >= 8 ? 3 : lanes == 4 ? 2 : 1, held = 8 >> steps;
    int first;
    bool writes;
    __device__ __forceinline__ ChannelSum() {
        const int g = (threadIdx.x & 31) / NL;
        first = (g & 1) * 4 + (steps > 1 ? (g >> 1 & 1) * 2 : 0) + (steps > 2 ? g >> 2 & 1 : 0);
        writes = (g >> steps) == 0;
    }
    __device__ __forceinline__ void sum(float (&v)[8]) const {   // the sums: v[0 .. held - 1]
        const int g = (threadIdx.x & 31) / NL;
#pragma unroll
        for (int s = 0; s < steps; ++s) {
            const int half = 4 >> s;
            const bool b = g >> s & 1;
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const float give = b ? v[i] : v[i + half], keep = b ? v[i + half] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, NL << s);
            }
        }
#pragma unroll
        for (int o = NL << steps; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < held; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
};

// Shared memory of the gradients: the chunk, the states in front of its subs but the first ([sub][warp][2 NP][lane] float4 of
// four states each), and room for the first sub's sums.  A sub's sums of dB and dC ([token][2 states] a warp) take the place
// of the warp's states in front of it.
template <typename T, int NL>
struct GradSmem {
    using Ck = Chunk<T, NL>;
    static constexpr int NP = Ck::NP, warps = Ck::TH / 32;
    static constexpr int subs = Ck::C / kSub, warp = 2 * NP * 32 * 4;   // floats of a warp's states
    static constexpr int sums = kSub * 2 * Ck::S;                       // floats of a warp's sums
    static_assert(sums <= warp, "a sub's sums fit in its states' place");
    static constexpr size_t bytes = sizeof(float) * (Ck::floats + (subs - 1) * warps * warp + warps * sums);
};

template <typename T, int NL, bool WIDE>
__global__ void __launch_bounds__((Chunk<T, NL>::TH), 2) k_scan_grad(ScanDims d, ScanIn in, ScanGrads gr, ScanWs ws) {
    using Ck = Chunk<T, NL>;
    using Sm = GradSmem<T, NL>;
    constexpr int CH = Ck::CH, S = Ck::S, C = Ck::C, TH = Ck::TH, V = CH / 4, NP = Sm::NP, W = Sm::warps;
    extern __shared__ __align__(16) float dyn[];
    __shared__ int flags[2 * C];
    const Ck ck(dyn, flags);
    float* const place = dyn + Ck::floats;   // of subs 1 .. , then the first sub's sums
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const ScanLane<NL, NP> l;
    const ChannelSum<NL> cs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const auto sums_of = [&](int sub, int w) { return sub ? place + ((sub - 1) * W + w) * Sm::warp : place + (Sm::subs - 1) * W * Sm::warp + w * Sm::sums; };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 a2[NP][4], dA[NP][4];
    l.pairs(in.A, 0, d, cb, a2);
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            a2[i][n] = mul2(a2[i][n], both(kLog2eF));
            dA[i][n] = make_float2(0.f, 0.f);
        }
    // what the thread adds up over tokens: channels ec .. ec + 3
    const int ec = threadIdx.x % V * 4, en = min(4, cb.n - ec);
    float4 dskip = none, dbias = none;
    if (gr.dS0 && blockIdx.x == 0)   // empty sequences hand their gradients on
        for (int b = 0; b < d.at.B; ++b) {
            const Seq s = seq_at(d.at, b);
            if (s.end > s.start) continue;
            const size_t at = (size_t)b * d.D * d.N;
            float2 f[NP][4];
            l.pairs(gr.dS, at, d, cb, f);
            l.put_pairs(gr.dS0 + at, d, cb, f);
        }
    const int tasks = d.at.rows() * ws.chunks;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int axis = task / ws.chunks, ta = task % ws.chunks * C, tb = min(ta + C, d.at.L);
        const int subs = (tb - ta + kSub - 1) / kSub;
        const Rows<T> r(d, in, gr.dy, axis, cb);
        const float4 skip = in.skip ? load4<float, false>(in.skip + cb.c0 + ec, en) : none;
        const float4 bias = in.dbias ? load4<float, false>(in.dbias + cb.c0 + ec, en) : none;
        float2 q[NP][4], h0[NP][4];   // the gradient from behind, and the chunk's entering state
        {
            const size_t at0 = ((size_t)task * d.D + cb.c0 + l.cl) * S + 4 * l.nl;
            float4 e[2 * NP], f[2 * NP];
#pragma unroll
            for (int i = 0; i < 2 * NP; ++i) {
                const bool in_range = l.cl + i < cb.n;
                e[i] = in_range ? *reinterpret_cast<const float4*>(ws.ends + at0 + (size_t)i * S) : none;
                f[i] = in_range ? *reinterpret_cast<const float4*>(ws.grads + at0 + (size_t)i * S) : none;
            }
            ck.template load<WIDE>(d, r, cb, axis, ta, tb, bias);
#pragma unroll
            for (int i = 0; i < 2 * NP; ++i) {
                set_one<NP>(h0, i, e[i]);
                set_one<NP>(q, i, f[i]);
            }
        }
        // the state behind token t from the one before it
        const auto advance = [&](int t, float2 (&h)[NP][4]) {
            float2 dt[NP], u[NP];
            load_pairs(ck.dt + t * CH + l.cl, dt);
            load_pairs(ck.u + t * CH + l.cl, u);
            Bc bc;
            bc.load(ck.bc + (t * NL + l.nl) * 8, false);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float2 du = mul2(dt[i], u[i]);
#pragma unroll
                for (int n = 0; n < 4; ++n) h[i][n] = fma2(decay2(dt[i], a2[i][n]), h[i][n], mul2(du, both(bc.bn(n))));
            }
        };
        const auto copy = [](float2 (&to)[NP][4], const float2 (&from)[NP][4]) {
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n) to[i][n] = from[i][n];
        };
        const auto enter = [&](int sub, float2 (&h)[NP][4]) {   // the state in front of a sub
            if (sub) {
                const float4* p = reinterpret_cast<const float4*>(place + ((sub - 1) * W + warp) * Sm::warp) + lane;
#pragma unroll
                for (int i = 0; i < 2 * NP; ++i) set_one<NP>(h, i, p[i * 32]);
            } else {
                copy(h, h0);
            }
        };
        const auto mixed = [&](int sub) {   // whether a sequence begins or ends in a sub
            int w = 0;
#pragma unroll
            for (int e = 0; e < kSub; ++e) w |= ck.what[sub * kSub + e];
            return (w & (kFirst | kLast)) != 0;
        };
        {   // the states in front of the subs
            float2 h[NP][4];
            copy(h, h0);
#pragma unroll 1
            for (int sub = 0; sub + 1 < subs; ++sub) {
                if (!mixed(sub)) {
#pragma unroll
                    for (int e = 0; e < kSub; ++e) advance(sub * kSub + e, h);
                } else {
#pragma unroll 1
                    for (int e = 0; e < kSub; ++e) {
                        const int t = sub * kSub + e;
                        if (ck.what[t] & kFirst) l.pairs(in.S0, (size_t)ck.seq[t] * d.D * d.N, d, cb, h);
                        advance(t, h);
                    }
                }
                float4* p = reinterpret_cast<float4*>(place + (sub * W + warp) * Sm::warp) + lane;
#pragma unroll
                for (int i = 0; i < 2 * NP; ++i) p[i * 32] = one_of<NP>(h, i);
            }
        }
        // token t backwards, from the states behind (h) and in front of it (hp): its sums, of which this lane holds some
        using Cs = ChannelSum<NL>;
        constexpr int K = kSums<NL>;
        struct Sums {
            float bc[Cs::held], s1[K], s2[K], y[K];
        };
        const auto back = [&](int t, const float2 (&h)[NP][4], const float2 (&hp)[NP][4]) {
            const int o = t * CH + l.cl;
            float2 dt[NP], u[NP], g[NP];
            load_pairs(ck.dt + o, dt);
            load_pairs(ck.u + o, u);
            load_pairs(ck.g + o, g);
            Bc bc;
            bc.load(ck.bc + (t * NL + l.nl) * 8, true);
            float2 db[4], dc[4], x1[NP], x2[NP], xy[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float2 du = mul2(dt[i], u[i]);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 b = both(bc.bn(n)), c = both(bc.cn(n));
                    const float2 p = fma2(g[i], c, q[i][n]);
                    dc[n] = i ? fma2(g[i], h[i][n], dc[n]) : mul2(g[i], h[i][n]);
                    db[n] = i ? fma2(du, p, db[n]) : mul2(du, p);
                    x1[i] = n ? fma2(p, b, x1[i]) : mul2(p, b);
                    xy[i] = n ? fma2(c, h[i][n], xy[i]) : mul2(c, h[i][n]);
                    q[i][n] = mul2(p, decay2(dt[i], a2[i][n]));
                    const float2 e = mul2(q[i][n], hp[i][n]);
                    dA[i][n] = fma2(dt[i], e, dA[i][n]);
                    x2[i] = n ? fma2(a2[i][n], e, x2[i]) : mul2(a2[i][n], e);
                }
            }
            float v[8] = {db[0].x + db[0].y, db[1].x + db[1].y, db[2].x + db[2].y, db[3].x + db[3].y,
                          dc[0].x + dc[0].y, dc[1].x + dc[1].y, dc[2].x + dc[2].y, dc[3].x + dc[3].y};
            cs.sum(v);
            Sums to;
#pragma unroll
            for (int i = 0; i < Cs::held; ++i) to.bc[i] = v[i];
            sum_states<NL>(x1, l.nl, to.s1);
            sum_states<NL>(x2, l.nl, to.s2);
            if (r.z) sum_states<NL>(xy, l.nl, to.y);
            return to;
        };
        // ... and where they go: the gradients' in the place of the token's inputs, dt s1 of u, that of dt of dt, sum_n C h of g
        const auto keep = [&](int t, float* sums, const Sums& v) {
            if (cs.writes)
#pragma unroll
                for (int i = 0; i < Cs::held; ++i) {
                    const int j = cs.first + i;
                    sums[(j >> 2) * S + 4 * l.nl + (j & 3)] = v.bc[i];
                }
            if (sums_here(l.nl)) {
                const int first = t * CH + l.cl + its_channel<NL>(l.nl);
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    const float dti = ck.dt[first + i], ui = ck.u[first + i];
                    ck.u[first + i] = dti * v.s1[i];
                    ck.dt[first + i] = fmaf(ui, v.s1[i], kLn2 * v.s2[i]);
                    if (r.z) ck.g[first + i] = v.y[i];
                }
            }
        };
#pragma unroll 1
        for (int sub = subs - 1; sub >= 0; --sub) {
            float* const sums = sums_of(sub, warp);
            const int t0 = sub * kSub;
            float2 hp[NP][4];
            enter(sub, hp);
            __syncwarp();   // (the sums take the states' place)
            if (!mixed(sub)) {
                float2 hs[kSub][NP][4];
                Sums got[kSub];   // (their stores would hold back the next token's loads)
#pragma unroll
                for (int e = 0; e < kSub; ++e) {
                    if (e) copy(hs[e], hs[e ? e - 1 : 0]);
                    else copy(hs[0], hp);
                    advance(t0 + e, hs[e]);
                }
#pragma unroll
                for (int e = kSub - 1; e >= 0; --e) got[e] = back(t0 + e, hs[e], e ? hs[e ? e - 1 : 0] : hp);
                __syncwarp();   // (every lane has read what the results replace)
#pragma unroll
                for (int e = 0; e < kSub; ++e) keep(t0 + e, sums + e * 2 * S, got[e]);
            } else {
#pragma unroll 1
                for (int e = kSub - 1; e >= 0; --e) {
                    const int t = t0 + e, w = ck.what[t];
                    const size_t at = (size_t)ck.seq[t] * d.D * d.N;
                    float2 h[NP][4], before[NP][4];
                    copy(h, hp);
#pragma unroll 1
                    for (int f = 0; f <= e; ++f) {
                        if (ck.what[t0 + f] & kFirst) l.pairs(in.S0, (size_t)ck.seq[t0 + f] * d.D * d.N, d, cb, h);
                        copy(before, h);
                        advance(t0 + f, h);
                    }
                    if (w & kLast) l.pairs(gr.dS, at, d, cb, q);
                    const Sums got = back(t, h, before);
                    __syncwarp();
                    keep(t, sums + e * 2 * S, got);
                    if (w & kFirst) {
                        if (gr.dS0) l.put_pairs(gr.dS0 + at, d, cb, q);
#pragma unroll
                        for (int i = 0; i < NP; ++i)
#pragma unroll
                            for (int n = 0; n < 4; ++n) q[i][n] = make_float2(0.f, 0.f);
                    }
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < subs * kSub * 2 * S; i += TH) {
            const int t = i / (2 * S), j = i % (2 * S), at = (t % kSub) * 2 * S + j;
            if (ck.what[t] & kOutside) continue;
            float v = sums_of(t / kSub, 0)[at];
#pragma unroll
            for (int w = 1; w < W; ++w) v += sums_of(t / kSub, w)[at];
            ws.bc[((((size_t)cb.cb * d.at.rows() + axis) * d.at.L + ta + t) * d.G + cb.g) * 2 * S + j] = v;
        }
        if (en > 0) {
            constexpr int rows = TH / V, items = C / rows, batch = items < kBatch ? items : kBatch;
#pragma unroll
            for (int j0 = 0; j0 < items; j0 += batch) {
                Vec<T, 4> vd[batch], vu[batch], vg[batch], vz[batch];
#pragma unroll
                for (int j = 0; j < batch; ++j) {
                    const long long tt = min(ta + (int)threadIdx.x / V + (j0 + j) * rows, tb - 1);
                    vd[j].zero(); vz[j].zero();
                    take4<T, WIDE>(vu[j], r.u + tt * d.us[1] + ec, en);
                    take4<T, WIDE>(vg[j], r.dy + tt * d.dys[1] + ec, en);
                    if (d.softplus) take4<T, WIDE>(vd[j], r.delta + tt * d.ds[1] + ec, en);
                    if (r.z) take4<T, WIDE>(vz[j], r.z + tt * d.zs[1] + ec, en);
                }
#pragma unroll
                for (int j = 0; j < batch; ++j) {
                    const int t = threadIdx.x / V + (j0 + j) * rows, o = t * CH + ec;
                    if (ck.what[t] & kOutside) continue;
                    const long long tt = ta + t;
                    const float4 u = as4(vu[j]), dy = as4(vg[j]);
                    const float4 x1 = *reinterpret_cast<const float4*>(ck.u + o), y = *reinterpret_cast<const float4*>(ck.g + o);
                    float4 dd = *reinterpret_cast<const float4*>(ck.dt + o), g = dy;
                    if (r.z) {
                        const float4 z = as4(vz[j]);
                        const float4 s = sigmoid4(z), f = mul4(z, s);
                        // dz = dy (y + skip u) (s + z s (1 - s))
                        const float4 yy = mul4(dy, add4(y, mul4(skip, u)));
                        store4<T, WIDE>((T*)gr.dz + axis * d.dzs[0] + tt * d.dzs[1] + cb.c0 + ec,
                                        mul4(yy, make_float4(fmaf(f.x, 1.f - s.x, s.x), fmaf(f.y, 1.f - s.y, s.y), fmaf(f.z, 1.f - s.z, s.z),
                                                             fmaf(f.w, 1.f - s.w, s.w))), en);
                        g = mul4(dy, f);
                    }
                    store4<T, WIDE>((T*)gr.du + axis * d.dus[0] + tt * d.dus[1] + cb.c0 + ec, add4(x1, mul4(skip, g)), en);
                    if (d.softplus) {
                        dd = mul4(dd, sigmoid4(add4(as4(vd[j]), bias)));
                    }
                    store4<T, WIDE>((T*)gr.ddelta + axis * d.dds[0] + tt * d.dds[1] + cb.c0 + ec, dd, en);
                    dbias = add4(dbias, dd);
                    dskip = add4(dskip, mul4(g, u));
                }
            }
        }
    }
    // the CTA's sums over its tokens
    float* out = ws.ch + blockIdx.x * ch_stride(d, S);
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i)
        if (l.cl + i < cb.n) *reinterpret_cast<float4*>(out + (size_t)(cb.c0 + l.cl + i) * S + 4 * l.nl) = one_of<NP>(dA, i);
    __syncthreads();
    float4* red = reinterpret_cast<float4*>(dyn);
    red[threadIdx.x] = dskip;
    red[TH + threadIdx.x] = dbias;
    __syncthreads();
    if (threadIdx.x < V) {
        for (int k = 1; k < TH / V; ++k) {
            dskip = add4(dskip, red[k * V + threadIdx.x]);
            dbias = add4(dbias, red[TH + k * V + threadIdx.x]);
        }
        float* p = out + (size_t)d.D * S + cb.c0 + ec;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < en) {
                p[i] = at4(dskip, i);
                p[d.D + i] = at4(dbias, i);
            }
    }
}

// ------------------------------------------------------------------- partial sums together, in order
// CTAs before `first` add up dB and dC, four neighbouring states of a token and group a thread; the others dA, dskip, dbias.
template <typename T, int NL>
__global__ void __launch_bounds__(256) k_scan_sums(ScanDims d, ScanWs ws, int blocks, unsigned first, T* dB, T* dC, float* dA, float* dskip,
                                                   float* dbias) {
    constexpr int S = ScanTile<NL>::states;
    if (blockIdx.x < first) {
        const long long idx = (long long)blockIdx.x * 256 + threadIdx.x, n = (long long)d.at.rows() * d.at.L * d.G * 2 * NL;
        if (idx >= n) return;
        const int q = (int)(idx % NL) * 4;
        const long long tg = idx / (2 * NL);   // token and group
        if (q >= d.N) return;
        if (d.at.packed) {   // (tokens outside every sequence keep what they hold)
            const int t = (int)(tg / d.G);
            const Seq s = seq_of(d.at, 0, t);
            if (t < s.start || t >= s.end) return;
        }
        const float4* p = reinterpret_cast<const float4*>(ws.bc) + idx;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < blocks; ++k) v = add4(v, p[k * n]);
        store4<T, false>((idx / NL & 1 ? dC : dB) + tg * d.N + q, v, min(4, d.N - q));
        return;
    }
    const long long idx = (long long)(blockIdx.x - first) * 256 + threadIdx.x, n = (long long)d.D * (S + 2);
    if (idx >= n) return;
    float* out;
    if (idx < (long long)d.D * S) {
        const int state = (int)(idx % S);
        if (state >= d.N) return;
        out = dA + idx / S * d.N + state;
    } else {
        const int c = (int)(idx - (long long)d.D * S);
        float* p = c < d.D ? dskip : dbias;
        if (!p) return;
        out = p + (c < d.D ? c : c - d.D);
    }
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < ws.gx; ++k) v += ws.ch[k * ch_stride(d, S) + idx];
    *out = v;
}

// Sizes of a backward call's workspace; CTAs along the chunks: about two an SM in all.
size_t carve(const ScanDims& d, char* base, ScanWs* ws) {
    const int S = 4 * state_lanes(d.N), ch = 16 * 32 / (S / 4), blocks = ch_blocks(d, ch) / d.G;
    const int C = chunk_of(state_lanes(d.N));
    ws->chunks = (d.at.L + C - 1) / C;
    const long long tasks = (long long)d.at.rows() * ws->chunks, all = (long long)blocks * d.G;
    const long long most = (2 * kScanSms + all - 1) / all, per = tasks ? (tasks + most - 1) / most : 1;
    ws->gx = (int)(tasks ? (tasks + per - 1) / per : 1);
    size_t off = 0;
    const auto take = [&](size_t n) {
        const size_t at = off;
        off += align256(n);
        return base ? base + at : nullptr;
    };
    ws->ends = (float*)take((size_t)tasks * d.D * S * 4);
    ws->grads = (float*)take((size_t)tasks * d.D * S * 4);
    ws->dts = (float*)take((size_t)tasks * d.D * 4);
    ws->alive = (int*)take((size_t)tasks * 8);
    ws->bc = (float*)take((size_t)blocks * d.at.rows() * d.at.L * d.G * 2 * S * 4);
    ws->ch = (float*)take(ws->gx * ch_stride(d, S) * 4);
    return off;
}

template <typename T, int NL, bool WIDE>
cudaError_t run(const ScanDims& d, const ScanIn& in, const ScanGrads& g, const ScanWs& ws, cudaStream_t st) {
    using Tile = ScanTile<NL>;
    using Sm = GradSmem<T, NL>;
    const int blocks = ch_blocks(d, Tile::ch), rows = d.at.rows();
    cudaError_t e;
    if (ws.chunks && rows) {
        constexpr size_t smem = sizeof(float) * Chunk<T, NL>::floats;
        const auto local = k_scan_local<T, NL, WIDE>;
        if ((e = cudaFuncSetAttribute(local, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        local<<<dim3(ws.chunks, blocks, rows), Chunk<T, NL>::TH, smem, st>>>(d, in, g, ws);
        prof_mark("scan_local", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        k_scan_chain<<<dim3((unsigned)(((long long)d.D * NL + 127) / 128), 2, rows), 128, 0, st>>>(d, in.A, ws, NL);
        prof_mark("scan_chain", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const auto grad = k_scan_grad<T, NL, WIDE>;
    if ((e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sm::bytes)) != cudaSuccess) return e;
    grad<<<dim3(ws.gx, blocks), Chunk<T, NL>::TH, Sm::bytes, st>>>(d, in, g, ws);
    prof_mark("scan_grad", st);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const unsigned first = (unsigned)(((long long)rows * d.at.L * d.G * 2 * NL + 255) / 256),
                   rest = (unsigned)(((long long)d.D * (Tile::states + 2) + 255) / 256);
    k_scan_sums<T, NL><<<first + rest, 256, 0, st>>>(d, ws, blocks / d.G, first, (T*)g.dB, (T*)g.dC, g.dA, g.dskip, g.ddbias);
    prof_mark("scan_sums", st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const ScanDims& d, const ScanIn& in, const ScanGrads& g, const ScanWs& ws, cudaStream_t st) {
    const bool wide = wide4(d, in.u, d.us) && wide4(d, in.delta, d.ds) && wide4(d, in.z, d.zs) && wide4(d, g.dy, d.dys) &&
                      wide4(d, g.du, d.dus) && wide4(d, g.ddelta, d.dds) && wide4(d, g.dz, d.dzs) && wide4(d, in.Bm, d.bs) &&
                      wide4(d, in.C, d.cs);
    return by_lanes(d.N, [&](auto nl) {
        constexpr int NL = decltype(nl)::value;
        return wide ? run<T, NL, true>(d, in, g, ws, st) : run<T, NL, false>(d, in, g, ws, st);
    });
}

}  // namespace

size_t scan_bwd_ws_bytes(const ScanDims& d) {
    ScanWs ws;
    return carve(d, nullptr, &ws);
}

cudaError_t launch_scan_bwd(const ScanDims& d, const ScanIn& in, const ScanGrads& g, void* workspace, cudaStream_t st) {
    ScanWs ws;
    carve(d, (char*)workspace, &ws);
    return d.bf16 ? bwd<__nv_bfloat16>(d, in, g, ws, st) : bwd<float>(d, in, g, ws, st);
}

}  // namespace efla

// scan_bwd.cu -- gradients of the selective scan, from its inputs alone.
//
// With g_t = dy_t z sigmoid(z), a_t = e^{dt_t A} and p_t the gradient of the state behind token t:
//   p_t = C_t g_t + a_{t+1} p_{t+1},   dC_t = sum_d h_t g_t,   dB_t = sum_d p_t dt_t u_t
//   s1 = sum_n p_t B_t,   e_t = a_t p_t h_{t-1},   du = dt s1 + skip g,   d(dt) = sum_n A e_t + u s1,   dA = sum_t dt e_t
// The tokens are cut into chunks of kChunk.  Both recurrences are linear, so one launch takes every chunk from a
// zero state to its last token and, with the running product of its decays, its gradients back to its first:
// all chunks at once.  A second launch chains the chunks' maps, and the third has every chunk's entering state and
// gradient at hand: it walks the chunk forward to the state in front of every kSub tokens (shared memory),
// then back, kSub tokens' states in registers.  Sums over channels (dB, dC) and tokens (dA, dskip, dbias) are
// partial sums of CTAs, added in a fixed order by the last launch.
#include "scan.cuh"
#include "launch.h"

namespace efla {

namespace {

constexpr int kChunk = 64, kSub = 8;
constexpr float kLn2 = 0.6931471805599453f;

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

template <typename T, bool WIDE>
__device__ __forceinline__ float4 gated(const T* dy, const T* z, int n) {   // dy z sigmoid(z)
    const float4 g = load4<T, WIDE>(dy, n);
    if (!z) return g;
    const float4 v = load4<T, WIDE>(z, n);
    return mul4(g, make_float4(silu_of(v.x), silu_of(v.y), silu_of(v.z), silu_of(v.w)));
}

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

// dt, dt u and g of TT tokens from t0 on
template <typename T, bool WIDE, int CH, int TT, bool GRAD>
__device__ __forceinline__ void load_tile(const ScanDims& d, const ScanIn& in, const Rows<T>& r, const ChBlock& cb, int t0, const int* what,
                                          float* s_dt, float* s_du, float* s_g) {
    for (int i = threadIdx.x; i < TT * CH / 4; i += kScanThreads) {
        const int t = i / (CH / 4), c = i % (CH / 4) * 4, n = min(4, cb.n - c);
        float4 dt = make_float4(0.f, 0.f, 0.f, 0.f), du = dt, g = dt;
        if (!(what[t] & kOutside) && n > 0) {
            const long long tt = t0 + t;
            const float4 raw = load4<T, WIDE>(r.delta + tt * d.ds[1] + c, n);
            dt = steps(d, in.dbias ? add4(raw, load4<float, false>(in.dbias + cb.c0 + c, n)) : raw, n);
            du = mul4(dt, load4<T, WIDE>(r.u + tt * d.us[1] + c, n));
            if (GRAD) g = gated<T, WIDE>(r.dy + tt * d.dys[1] + c, r.z ? r.z + tt * d.zs[1] + c : nullptr, n);
        }
        *reinterpret_cast<float4*>(s_dt + t * CH + c) = dt;
        *reinterpret_cast<float4*>(s_du + t * CH + c) = du;
        if (GRAD) *reinterpret_cast<float4*>(s_g + t * CH + c) = g;
    }
}
template <typename T, int S, int TT>
__device__ __forceinline__ void load_rows(float* to, const T* from, long long stride, int N, int t0, const int* what) {
    for (int i = threadIdx.x; i < TT * S; i += kScanThreads) {
        const int t = i / S, n = i % S;
        to[i] = n < N && !(what[t] & kOutside) ? (float)from[(t0 + t) * stride + n] : 0.f;
    }
}

__device__ __forceinline__ float2 lo(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi(const float4& v) { return make_float2(v.z, v.w); }

// ------------------------------------------------------------------- every chunk by itself
template <typename T, int NL, bool WIDE>
__global__ void __launch_bounds__(kScanThreads) k_scan_local(ScanDims d, ScanIn in, ScanGrads gr, ScanWs ws) {
    using Tile = ScanTile<NL>;
    constexpr int CH = Tile::ch, S = Tile::states;
    extern __shared__ __align__(16) float dyn[];
    float *s_dt = dyn, *s_du = s_dt + kTile * CH, *s_g = s_du + kTile * CH, *s_b = s_g + kTile * CH, *s_c = s_b + kTile * S;
    __shared__ int what[kTile], seq[kTile];
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const int axis = blockIdx.z, k = blockIdx.x, ta = k * kChunk, tb = min(ta + kChunk, d.at.L);
    const ScanLane<NL> l;
    const Rows<T> r(d, in, gr.dy, axis, cb);
    float2 a2[4][2], h[4][2], cp[4][2], q[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = l.states(in.A, d, cb, i);
        a2[i][0] = mul2(lo(v), both(kLog2eF));
        a2[i][1] = mul2(hi(v), both(kLog2eF));
        h[i][0] = h[i][1] = q[i][0] = q[i][1] = make_float2(0.f, 0.f);
        cp[i][0] = cp[i][1] = make_float2(1.f, 1.f);
    }
    float4 dts = make_float4(0.f, 0.f, 0.f, 0.f);
    bool alive = true, open = true;   // whether the state before the chunk, and gradients back to it, still pass
    for (int t0 = ta; t0 < tb; t0 += kTile) {
        __syncthreads();
        if (threadIdx.x < kTile) {
            const TokenAt a = token_at(d.at, axis, t0 + threadIdx.x, tb);
            what[threadIdx.x] = a.what;
            seq[threadIdx.x] = a.seq;
        }
        __syncthreads();
        if (t0 == ta && (what[0] & kOutside)) open = false;
        load_rows<T, S, kTile>(s_b, r.Bm, d.bs[1], d.N, t0, what);
        load_rows<T, S, kTile>(s_c, r.C, d.cs[1], d.N, t0, what);
        load_tile<T, WIDE, CH, kTile, true>(d, in, r, cb, t0, what, s_dt, s_du, s_g);
        __syncthreads();
        for (int t = 0; t < kTile; ++t) {
            const int w = what[t];
            const size_t at = (size_t)seq[t] * d.D * d.N;
            if (w & kFirst) {
                alive = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = in.S0 ? l.states(in.S0 + at, d, cb, i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    h[i][0] = lo(v);
                    h[i][1] = hi(v);
                }
            }
            const float4 dt = *reinterpret_cast<const float4*>(s_dt + t * CH + l.cl), du = *reinterpret_cast<const float4*>(s_du + t * CH + l.cl),
                         g = *reinterpret_cast<const float4*>(s_g + t * CH + l.cl), b = *reinterpret_cast<const float4*>(s_b + t * S + 4 * l.nl),
                         c = *reinterpret_cast<const float4*>(s_c + t * S + 4 * l.nl);
            dts = add4(dts, dt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 dt2 = both(at4(dt, i)), du2 = both(at4(du, i)), g2 = both(at4(g, i));
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 a = decay2(dt2, a2[i][p]);
                    h[i][p] = fma2(a, h[i][p], mul2(du2, p ? hi(b) : lo(b)));
                    if (open) {
                        cp[i][p] = mul2(cp[i][p], a);
                        q[i][p] = fma2(cp[i][p], mul2(g2, p ? hi(c) : lo(c)), q[i][p]);
                    }
                }
            }
            if (open && (w & kLast)) {
                open = false;
                if (gr.dS)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = l.states(gr.dS + at, d, cb, i);
                        q[i][0] = fma2(cp[i][0], lo(v), q[i][0]);
                        q[i][1] = fma2(cp[i][1], hi(v), q[i][1]);
                    }
            }
        }
    }
    const size_t at = (size_t)axis * ws.chunks + k;
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        ws.alive[2 * at] = alive;
        ws.alive[2 * at + 1] = open;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (l.cl + i >= cb.n) continue;
        const size_t ch = at * d.D + cb.c0 + l.cl + i;
        *reinterpret_cast<float4*>(ws.ends + ch * S + 4 * l.nl) = make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y);
        *reinterpret_cast<float4*>(ws.grads + ch * S + 4 * l.nl) = make_float4(q[i][0].x, q[i][0].y, q[i][1].x, q[i][1].y);
        if (l.nl == 0) ws.dts[ch] = at4(dts, i);
    }
}

// ------------------------------------------------------------------- the chunks' maps chained
// A thread takes four states of a channel through its axis's chunks: blockIdx.y 0 forward, 1 backward.
__global__ void __launch_bounds__(128) k_scan_chain(ScanDims d, const float* A, ScanWs ws, int nl) {
    constexpr int AHEAD = 8;
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
                s = on[j] ? make_float4(fmaf(ex2(a[0] * x[j]), s.x, e[j].x), fmaf(ex2(a[1] * x[j]), s.y, e[j].y),
                                        fmaf(ex2(a[2] * x[j]), s.z, e[j].z), fmaf(ex2(a[3] * x[j]), s.w, e[j].w))
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

template <int NL>
struct GradSmem {
    using Tile = ScanTile<NL>;
    static constexpr int CH = Tile::ch, S = Tile::states;
    static constexpr int entries = kChunk / kSub * 4 * kScanThreads * 4;   // floats
    static constexpr size_t bytes = sizeof(float) * (entries + 6 * kSub * CH + 2 * kSub * S + 4 * kSub * 2 * S);
};

template <typename T, int NL, bool WIDE>
__global__ void __launch_bounds__(kScanThreads, NL == 1 ? 1 : 2) k_scan_grad(ScanDims d, ScanIn in, ScanGrads gr, ScanWs ws) {
    using Tile = ScanTile<NL>;
    constexpr int CH = Tile::ch, S = Tile::states, V = CH / 4;
    extern __shared__ __align__(16) float dyn[];
    float4* entry = reinterpret_cast<float4*>(dyn);   // [sub][channel i][thread]
    float *s_dt = dyn + GradSmem<NL>::entries, *s_du = s_dt + kSub * CH, *s_g = s_du + kSub * CH, *s_1 = s_g + kSub * CH, *s_2 = s_1 + kSub * CH,
          *s_y = s_2 + kSub * CH, *s_b = s_y + kSub * CH, *s_c = s_b + kSub * S, *s_bc = s_c + kSub * S;   // s_bc [warp][token][2 S]
    __shared__ int what[kSub], seq[kSub];
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const ScanLane<NL> l;
    const ChannelSum<NL> cs;
    const int warp = threadIdx.x >> 5;
    float2 a2[4][2], dA[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = l.states(in.A, d, cb, i);
        a2[i][0] = mul2(lo(v), both(kLog2eF));
        a2[i][1] = mul2(hi(v), both(kLog2eF));
        dA[i][0] = dA[i][1] = make_float2(0.f, 0.f);
    }
    // what the thread adds up over tokens: channels ec .. ec + 3
    const int ec = threadIdx.x % V * 4, en = min(4, cb.n - ec);
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 dskip = none, dbias = none;
    const float4 skip = in.skip ? load4<float, false>(in.skip + cb.c0 + ec, en) : none;
    const float4 bias = in.dbias ? load4<float, false>(in.dbias + cb.c0 + ec, en) : none;
    if (gr.dS0 && blockIdx.x == 0)   // empty sequences hand their gradients on
        for (int b = 0; b < d.at.B; ++b) {
            const Seq s = seq_at(d.at, b);
            if (s.end > s.start) continue;
            const size_t at = (size_t)b * d.D * d.N;
#pragma unroll
            for (int i = 0; i < 4; ++i) l.put_states(gr.dS0 + at, d, cb, i, gr.dS ? l.states(gr.dS + at, d, cb, i) : none);
        }
    const int tasks = d.at.rows() * ws.chunks;
    for (int task = blockIdx.x; task < tasks; task += gridDim.x) {
        const int axis = task / ws.chunks, ta = task % ws.chunks * kChunk, tb = min(ta + kChunk, d.at.L);
        const int subs = (tb - ta + kSub - 1) / kSub;
        const Rows<T> r(d, in, gr.dy, axis, cb);
        float2 q[4][2], hs[kSub][4][2];
        // the chunk's entering state and gradient
        const size_t at0 = ((size_t)task * d.D + cb.c0 + l.cl) * S + 4 * l.nl;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in_range = l.cl + i < cb.n;
            const float4 e = in_range ? *reinterpret_cast<const float4*>(ws.ends + at0 + (size_t)i * S) : none;
            const float4 f = in_range ? *reinterpret_cast<const float4*>(ws.grads + at0 + (size_t)i * S) : none;
            entry[i * kScanThreads + threadIdx.x] = e;
            q[i][0] = lo(f);
            q[i][1] = hi(f);
        }
        const auto fetch = [&](int sub, bool grad) {   // the sub's tokens into shared memory
            const int t0 = ta + sub * kSub;
            __syncthreads();
            if (threadIdx.x < kSub) {
                const TokenAt a = token_at(d.at, axis, t0 + threadIdx.x, tb);
                what[threadIdx.x] = a.what;
                seq[threadIdx.x] = a.seq;
            }
            __syncthreads();
            load_rows<T, S, kSub>(s_b, r.Bm, d.bs[1], d.N, t0, what);
            if (grad) {
                load_rows<T, S, kSub>(s_c, r.C, d.cs[1], d.N, t0, what);
                load_tile<T, WIDE, CH, kSub, true>(d, in, r, cb, t0, what, s_dt, s_du, s_g);
            } else {
                load_tile<T, WIDE, CH, kSub, false>(d, in, r, cb, t0, what, s_dt, s_du, s_g);
            }
            __syncthreads();
        };
        // the sub's states from its entering one
        const auto forward = [&](int sub) {
            float2 h[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 e = entry[(sub * 4 + i) * kScanThreads + threadIdx.x];
                h[i][0] = lo(e);
                h[i][1] = hi(e);
            }
#pragma unroll
            for (int t = 0; t < kSub; ++t) {
                if (what[t] & kFirst)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = in.S0 ? l.states(in.S0 + (size_t)seq[t] * d.D * d.N, d, cb, i) : none;
                        h[i][0] = lo(v);
                        h[i][1] = hi(v);
                    }
                const float4 dt = *reinterpret_cast<const float4*>(s_dt + t * CH + l.cl), du = *reinterpret_cast<const float4*>(s_du + t * CH + l.cl),
                             b = *reinterpret_cast<const float4*>(s_b + t * S + 4 * l.nl);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 a = decay2(both(at4(dt, i)), a2[i][p]);
                        h[i][p] = fma2(a, h[i][p], mul2(both(at4(du, i)), p ? hi(b) : lo(b)));
                        hs[t][i][p] = h[i][p];
                    }
            }
        };
        for (int sub = 0; sub + 1 < subs; ++sub) {
            fetch(sub, false);
            forward(sub);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                entry[((sub + 1) * 4 + i) * kScanThreads + threadIdx.x] =
                    make_float4(hs[kSub - 1][i][0].x, hs[kSub - 1][i][0].y, hs[kSub - 1][i][1].x, hs[kSub - 1][i][1].y);
        }
        for (int sub = subs - 1; sub >= 0; --sub) {
            const int t0 = ta + sub * kSub;
            fetch(sub, true);
            forward(sub);
#pragma unroll
            for (int t = kSub - 1; t >= 0; --t) {
                const int w = what[t];
                const size_t at = (size_t)seq[t] * d.D * d.N;
                if (w & kLast)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = gr.dS ? l.states(gr.dS + at, d, cb, i) : none;
                        q[i][0] = lo(v);
                        q[i][1] = hi(v);
                    }
                const float4 dt = *reinterpret_cast<const float4*>(s_dt + t * CH + l.cl), du = *reinterpret_cast<const float4*>(s_du + t * CH + l.cl),
                             g = *reinterpret_cast<const float4*>(s_g + t * CH + l.cl), b = *reinterpret_cast<const float4*>(s_b + t * S + 4 * l.nl),
                             c = *reinterpret_cast<const float4*>(s_c + t * S + 4 * l.nl);
                float2 db[2], dc[2];
                db[0] = db[1] = dc[0] = dc[1] = make_float2(0.f, 0.f);
                float o1[4], o2[4], oy[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 dt2 = both(at4(dt, i)), du2 = both(at4(du, i)), g2 = both(at4(g, i));
                    float2 hp[2];
                    if (w & kFirst) {
                        const float4 v = in.S0 ? l.states(in.S0 + at, d, cb, i) : none;
                        hp[0] = lo(v);
                        hp[1] = hi(v);
                    } else if (t > 0) {
                        hp[0] = hs[t > 0 ? t - 1 : 0][i][0];
                        hp[1] = hs[t > 0 ? t - 1 : 0][i][1];
                    } else {
                        const float4 e = entry[(sub * 4 + i) * kScanThreads + threadIdx.x];
                        hp[0] = lo(e);
                        hp[1] = hi(e);
                    }
                    float2 x1 = make_float2(0.f, 0.f), x2 = x1, xy = x1;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 bp = p ? hi(b) : lo(b), cp = p ? hi(c) : lo(c), h = hs[t][i][p];
                        const float2 pt = fma2(g2, cp, q[i][p]);
                        dc[p] = fma2(g2, h, dc[p]);
                        db[p] = fma2(du2, pt, db[p]);
                        x1 = fma2(pt, bp, x1);
                        xy = fma2(cp, h, xy);
                        q[i][p] = mul2(pt, decay2(dt2, a2[i][p]));
                        const float2 e = mul2(q[i][p], hp[p]);
                        dA[i][p] = fma2(dt2, e, dA[i][p]);
                        x2 = fma2(a2[i][p], e, x2);
                    }
                    o1[i] = x1.x + x1.y;
                    o2[i] = x2.x + x2.y;
                    oy[i] = xy.x + xy.y;
                }
                if (w & kFirst)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (gr.dS0) l.put_states(gr.dS0 + at, d, cb, i, make_float4(q[i][0].x, q[i][0].y, q[i][1].x, q[i][1].y));
                        q[i][0] = q[i][1] = make_float2(0.f, 0.f);
                    }
                put_sums<NL>(s_1 + t * CH, l, o1);
                put_sums<NL>(s_2 + t * CH, l, o2);
                if (r.z) put_sums<NL>(s_y + t * CH, l, oy);
                float v[8] = {db[0].x, db[0].y, db[1].x, db[1].y, dc[0].x, dc[0].y, dc[1].x, dc[1].y};
                cs.sum(v);
                if (cs.writes)
#pragma unroll
                    for (int i = 0; i < ChannelSum<NL>::held; ++i) {
                        const int j = cs.first + i;
                        s_bc[(warp * kSub + t) * 2 * S + (j >> 2) * S + 4 * l.nl + (j & 3)] = v[i];
                    }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < kSub * 2 * S; i += kScanThreads) {
                const int t = i / (2 * S), j = i % (2 * S);
                if (what[t] & kOutside) continue;
                float v = s_bc[i];
#pragma unroll
                for (int k = 1; k < 4; ++k) v += s_bc[k * kSub * 2 * S + i];
                ws.bc[((((size_t)cb.cb * d.at.rows() + axis) * d.at.L + t0 + t) * d.G + cb.g) * 2 * S + j] = v;
            }
            for (int t = threadIdx.x / V; t < kSub; t += kScanThreads / V) {
                if ((what[t] & kOutside) || en <= 0) continue;
                const long long tt = t0 + t;
                const int o = t * CH + ec;
                const float4 dt = *reinterpret_cast<const float4*>(s_dt + o), g = *reinterpret_cast<const float4*>(s_g + o),
                             x1 = *reinterpret_cast<const float4*>(s_1 + o), x2 = *reinterpret_cast<const float4*>(s_2 + o);
                const float4 u = load4<T, WIDE>(r.u + tt * d.us[1] + ec, en);
                store4<T, WIDE>((T*)gr.du + axis * d.dus[0] + tt * d.dus[1] + cb.c0 + ec, add4(mul4(dt, x1), mul4(skip, g)), en);
                float4 dd = add4(mul4(x2, make_float4(kLn2, kLn2, kLn2, kLn2)), mul4(u, x1));
                if (d.softplus) {
                    const float4 raw = add4(load4<T, WIDE>(r.delta + tt * d.ds[1] + ec, en), bias);
                    dd = mul4(dd, make_float4(sigmoid_of(raw.x), sigmoid_of(raw.y), sigmoid_of(raw.z), sigmoid_of(raw.w)));
                }
                store4<T, WIDE>((T*)gr.ddelta + axis * d.dds[0] + tt * d.dds[1] + cb.c0 + ec, dd, en);
                dbias = add4(dbias, dd);
                dskip = add4(dskip, mul4(g, u));
                if (r.z) {
                    const float4 y = add4(*reinterpret_cast<const float4*>(s_y + o), mul4(skip, u)), z = load4<T, WIDE>(r.z + tt * d.zs[1] + ec, en);
                    const float4 dy = load4<T, WIDE>(r.dy + tt * d.dys[1] + ec, en);
                    const float4 f = make_float4(dsilu_of(z.x), dsilu_of(z.y), dsilu_of(z.z), dsilu_of(z.w));
                    store4<T, WIDE>((T*)gr.dz + axis * d.dzs[0] + tt * d.dzs[1] + cb.c0 + ec, mul4(mul4(dy, y), f), en);
                }
            }
        }
    }
    // the CTA's sums over its tokens
    float* out = ws.ch + blockIdx.x * ch_stride(d, S);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (l.cl + i < cb.n)
            *reinterpret_cast<float4*>(out + (size_t)(cb.c0 + l.cl + i) * S + 4 * l.nl) = make_float4(dA[i][0].x, dA[i][0].y, dA[i][1].x, dA[i][1].y);
    __syncthreads();
    float4* red = reinterpret_cast<float4*>(dyn);
    red[threadIdx.x] = dskip;
    red[kScanThreads + threadIdx.x] = dbias;
    __syncthreads();
    if (threadIdx.x < V) {
        for (int k = 1; k < kScanThreads / V; ++k) {
            dskip = add4(dskip, red[k * V + threadIdx.x]);
            dbias = add4(dbias, red[kScanThreads + k * V + threadIdx.x]);
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
template <typename T>
__global__ void __launch_bounds__(256) k_scan_sum_bc(ScanDims d, const float* bc, int blocks, int S, T* dB, T* dC) {
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x, tokens = (long long)d.at.rows() * d.at.L;
    const long long n = tokens * d.G * 2 * S;
    if (idx >= n) return;
    const int j = (int)(idx % (2 * S)), state = j % S;
    if (state >= d.N) return;
    const long long tg = idx / (2 * S);   // token and group
    if (d.at.packed) {   // (tokens outside every sequence keep what they hold)
        const int t = (int)(tg / d.G);
        const Seq s = seq_of(d.at, 0, t);
        if (t < s.start || t >= s.end) return;
    }
    float v = 0.f;
#pragma unroll 4
    for (int k = 0; k < blocks; ++k) v += bc[(size_t)k * n + idx];
    st_elem((j < S ? dB : dC) + tg * d.N + state, v);
}

__global__ void __launch_bounds__(256) k_scan_sum_ch(ScanDims d, const float* ch, int gx, int S, float* dA, float* dskip, float* dbias) {
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x, n = (long long)d.D * (S + 2);
    if (idx >= n) return;
    float* out;
    if (idx < (long long)d.D * S) {
        const int state = (int)(idx % S);
        if (state >= d.N) return;
        out = dA + idx / S * d.N + state;
    } else {
        const long long c = idx - (long long)d.D * S;
        float* p = c < d.D ? dskip : dbias;
        if (!p) return;
        out = p + c % d.D;
    }
    float v = 0.f;
#pragma unroll 4
    for (int k = 0; k < gx; ++k) v += ch[k * ch_stride(d, S) + idx];
    *out = v;
}

// Sizes of a backward call's workspace; CTAs along the chunks: about two an SM in all.
size_t carve(const ScanDims& d, char* base, ScanWs* ws) {
    const int S = 4 * state_lanes(d.N), ch = 16 * 32 / (S / 4), blocks = ch_blocks(d, ch) / d.G;
    ws->chunks = (d.at.L + kChunk - 1) / kChunk;
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
    const int blocks = ch_blocks(d, Tile::ch), rows = d.at.rows();
    cudaError_t e;
    if (ws.chunks && rows) {
        const size_t smem = sizeof(float) * kTile * (3 * Tile::ch + 2 * Tile::states);
        const auto local = k_scan_local<T, NL, WIDE>;
        if ((e = cudaFuncSetAttribute(local, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        local<<<dim3(ws.chunks, blocks, rows), kScanThreads, smem, st>>>(d, in, g, ws);
        prof_mark("scan_local", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        k_scan_chain<<<dim3((unsigned)(((long long)d.D * NL + 127) / 128), 2, rows), 128, 0, st>>>(d, in.A, ws, NL);
        prof_mark("scan_chain", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const auto grad = k_scan_grad<T, NL, WIDE>;
    if ((e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GradSmem<NL>::bytes)) != cudaSuccess) return e;
    grad<<<dim3(ws.gx, blocks), kScanThreads, GradSmem<NL>::bytes, st>>>(d, in, g, ws);
    prof_mark("scan_grad", st);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long n = (long long)rows * d.at.L * d.G * 2 * Tile::states;
    if (n) k_scan_sum_bc<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(d, ws.bc, blocks / d.G, Tile::states, (T*)g.dB, (T*)g.dC);
    k_scan_sum_ch<<<(unsigned)(((long long)d.D * (Tile::states + 2) + 255) / 256), 256, 0, st>>>(d, ws.ch, ws.gx, Tile::states, g.dA, g.dskip, g.ddbias);
    prof_mark("scan_sums", st);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const ScanDims& d, const ScanIn& in, const ScanGrads& g, const ScanWs& ws, cudaStream_t st) {
    const bool wide = wide4(d, in.u, d.us) && wide4(d, in.delta, d.ds) && wide4(d, in.z, d.zs) && wide4(d, g.dy, d.dys) &&
                      wide4(d, g.du, d.dus) && wide4(d, g.ddelta, d.dds) && wide4(d, g.dz, d.dzs);
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

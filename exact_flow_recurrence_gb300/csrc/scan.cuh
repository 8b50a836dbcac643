// scan.cuh -- parts that the selective scan's forward and backward kernels share.
//
// Channel d keeps N states; with the A, B, C of its group:
//   dt = softplus(delta + bias)  (or delta + bias),   h <- e^{dt A} h + dt u B,   y = (sum_n C h + skip u) z sigmoid(z)
//
// A thread owns four neighbouring channels, two and two the halves of its packed instructions, and four neighbouring states
// of each: N/4 lanes (rounded up to a power of two, NL) lie side by side along the states, the warp's other lanes along
// the channels.  A CTA has 512 / NL channels of one group, all on the same tokens, which pass through shared memory in tiles:
// what depends on a channel alone (dt, the gated gradient) is worked out once there.
// Tokens outside every sequence, and channels and states past the last, are zeros: e^0 h + 0 leaves a state alone.
#pragma once

#include "mix.cuh"

namespace efla {

constexpr int kNP = 2;   // pairs of channels a thread

// NL: lanes along the states
template <int NL>
struct ScanTile {
    static constexpr int states = 4 * NL;   // padded
    static constexpr int ch = 512 / NL;     // channels a CTA
};

// A CTA's channels c0 .. c0 + n - 1, of group g; block `cb` of that group's.
struct ChBlock {
    int g, cb, c0, n;
};
template <int NL>
__device__ __forceinline__ ChBlock ch_block(const ScanDims& d, int index) {
    const int per = d.D / d.G, blocks = (per + ScanTile<NL>::ch - 1) / ScanTile<NL>::ch;
    const int g = index / blocks, cb = index % blocks;
    return ChBlock{g, cb, g * per + cb * ScanTile<NL>::ch, min(ScanTile<NL>::ch, per - cb * ScanTile<NL>::ch)};
}
inline int ch_blocks(const ScanDims& d, int ch) { return d.G * ((d.D / d.G + ch - 1) / ch); }

// n (0 .. 4) neighbouring elements as fp32, zeros behind them; WIDE: whole and aligned where n = 4
template <typename T, bool WIDE>
__device__ __forceinline__ float4 load4(const T* p, int n) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (WIDE && n >= 4) {
        Vec<T, 4> v;
        v.load(p);
        v.get(f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) f[i] = (float)p[i];
    }
    return make_float4(f[0], f[1], f[2], f[3]);
}
// ... and as they are stored, into v
template <typename T, bool WIDE>
__device__ __forceinline__ void take4(Vec<T, 4>& v, const T* p, int n) {
    if (WIDE) {
        v.load(p);
    } else {
        const float4 x = load4<T, false>(p, n);
        const float f[4] = {x.x, x.y, x.z, x.w};
        v.set(f);
    }
}
template <typename T>
__device__ __forceinline__ float4 as4(const Vec<T, 4>& v) {
    float f[4];
    v.get(f);
    return make_float4(f[0], f[1], f[2], f[3]);
}
template <typename T, bool WIDE>
__device__ __forceinline__ void store4(T* p, float4 x, int n) {
    const float f[4] = {x.x, x.y, x.z, x.w};
    if (WIDE && n >= 4) {
        Vec<T, 4> v;
        v.set(f);
        v.store(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = (T)f[i];
    }
}

// log(1 + e^x) = max(x, 0) + log1p(w), w = e^{-|x|}: log1p(w) / w on [0, 1] as its Chebyshev fit of degree 9 (1.2e-8 of it),
// two values an instruction.  Within (1.3 |x| + 8) 2^-24 of the result: below zero w's exponent, rounded to |x| 2^-24, is most of it.
__device__ __forceinline__ float2 softplus2(float2 x) {
    const float2 w = make_float2(ex2(-kLog2eF * fabsf(x.x)), ex2(-kLog2eF * fabsf(x.y)));
    float2 p = both(-0.0032438531052321196f);
    p = fma2(p, w, both(0.01985068805515766f));
    p = fma2(p, w, both(-0.05695807933807373f));
    p = fma2(p, w, both(0.10603507608175278f));
    p = fma2(p, w, both(-0.15305505692958832f));
    p = fma2(p, w, both(0.19675908982753754f));
    p = fma2(p, w, both(-0.2495412826538086f));
    p = fma2(p, w, both(0.3332996070384979f));
    p = fma2(p, w, both(-0.4999990165233612f));
    p = fma2(p, w, both(1.f));
    return fma2(p, w, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float step_of(const ScanDims& d, float x) { return d.softplus ? softplus2(both(x)).x : x; }
// dt of four channels from their delta + bias, zeros past the n-th
__device__ __forceinline__ float4 steps(const ScanDims& d, float4 raw, int n) {
    if (d.softplus) {
        const float2 a = softplus2(make_float2(raw.x, raw.y)), b = softplus2(make_float2(raw.z, raw.w));
        raw = make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(raw.x, n > 1 ? raw.y : 0.f, n > 2 ? raw.z : 0.f, n > 3 ? raw.w : 0.f);
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }
__device__ __forceinline__ float4 sigmoid4(float4 x) {
    const float2 a = sigmoid2(make_float2(x.x, x.y)), b = sigmoid2(make_float2(x.z, x.w));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float2 lo(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi(const float4& v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float at4(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// e^{dt A} from a2 = A log2(e).  ex2.approx gives a little too small a result: -5e-9 of it on average for exponents of
// -2^-17 .. -2^-9, -1e-8 to -3e-8 up to -2^-3 (measured over all of each binade).  A state that remembers a thousand tokens
// would collect that, so 1.1e-8 is added to the exponent, in the product's own rounding (it leaves e^0 = 1 as it is).
constexpr float kEx2Mean = 1.1e-8f * kLog2eF;
__device__ __forceinline__ float2 decay2(float2 dt, float2 a2) {
    const float2 x = fma2(dt, a2, both(kEx2Mean));
    return make_float2(ex2(x.x), ex2(x.y));
}

// h 2^x, the map of many tokens together, in two halves: 2^x alone may leave fp32 where h 2^x is inside (a state of zeros behind
// tokens that would grow it: inf 0 is not a number).  From x = 254 on every normal h but 0 is infinite either way.
__device__ __forceinline__ float times_ex2(float h, float x) {
    const float f = ex2(fminf(0.5f * x, 127.f));
    return h * f * f;
}

// What a token is, a bit each: the first or last of its sequence, outside every sequence.
enum { kFirst = 1, kLast = 2, kOutside = 4 };
struct TokenAt {
    int what, seq;
};
__device__ __forceinline__ TokenAt token_at(const Axes& a, int axis, int t, int t1) {
    if (t >= t1) return TokenAt{kOutside, 0};
    const Seq s = seq_of(a, axis, t);
    if (t < s.start || t >= s.end) return TokenAt{kOutside, 0};
    return TokenAt{(t == s.start ? kFirst : 0) | (t == s.end - 1 ? kLast : 0), s.b};
}

// The thread's 2 NP channels of four states: its place in a warp, and where its values lie.
template <int NL, int NP>
struct ScanLane {
    int nl, cl;      // first state / 4; first channel in the CTA
    __device__ __forceinline__ ScanLane() {
        const int lane = threadIdx.x & 31;
        nl = lane % NL;
        cl = (threadIdx.x >> 5) * (2 * NP * 32 / NL) + lane / NL * 2 * NP;
    }
    // of x [D][N] fp32: channel i's states, zeros past the last
    __device__ __forceinline__ float4 states(const float* x, const ScanDims& d, const ChBlock& b, int i) const {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (cl + i < b.n) {
            const float* p = x + (size_t)(b.c0 + cl + i) * d.N + 4 * nl;
            if (4 * nl < d.N) v.x = p[0];
            if (4 * nl + 1 < d.N) v.y = p[1];
            if (4 * nl + 2 < d.N) v.z = p[2];
            if (4 * nl + 3 < d.N) v.w = p[3];
        }
        return v;
    }
    __device__ __forceinline__ void put_states(float* x, const ScanDims& d, const ChBlock& b, int i, float4 v) const {
        if (cl + i < b.n) {
            float* p = x + (size_t)(b.c0 + cl + i) * d.N + 4 * nl;
            if (4 * nl < d.N) p[0] = v.x;
            if (4 * nl + 1 < d.N) p[1] = v.y;
            if (4 * nl + 2 < d.N) p[2] = v.z;
            if (4 * nl + 3 < d.N) p[3] = v.w;
        }
    }
    // pairs of channels (2 i, 2 i + 1), states 4 nl + n, of x + at (null: zeros), and back
    __device__ __forceinline__ void pairs(const float* x, size_t at, const ScanDims& d, const ChBlock& b, float2 (&to)[NP][4]) const {
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float4 p = x ? states(x + at, d, b, 2 * i) : none, q = x ? states(x + at, d, b, 2 * i + 1) : none;
#pragma unroll
            for (int n = 0; n < 4; ++n) to[i][n] = make_float2(at4(p, n), at4(q, n));
        }
    }
    __device__ __forceinline__ void put_pairs(float* x, const ScanDims& d, const ChBlock& b, const float2 (&v)[NP][4]) const {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            put_states(x, d, b, 2 * i, make_float4(v[i][0].x, v[i][1].x, v[i][2].x, v[i][3].x));
            put_states(x, d, b, 2 * i + 1, make_float4(v[i][0].y, v[i][1].y, v[i][2].y, v[i][3].y));
        }
    }
};

// the four states of the thread's channel i
template <int NP>
__device__ __forceinline__ float4 one_of(const float2 (&v)[NP][4], int i) {
    return i & 1 ? make_float4(v[i / 2][0].y, v[i / 2][1].y, v[i / 2][2].y, v[i / 2][3].y)
                 : make_float4(v[i / 2][0].x, v[i / 2][1].x, v[i / 2][2].x, v[i / 2][3].x);
}
template <int NP>
__device__ __forceinline__ void set_one(float2 (&v)[NP][4], int i, const float4& x) {
#pragma unroll
    for (int n = 0; n < 4; ++n) (i & 1 ? v[i / 2][n].y : v[i / 2][n].x) = at4(x, n);
}

// Sums over a channel's NL lanes of a value for each of the thread's four channels.  Afterwards the lanes that sums_here()
// names hold the sums of kSums channels from its_channel() on.
template <int NL>
constexpr int kSums = NL < 4 ? 4 / NL : 1;
template <int NL>
__device__ __forceinline__ int its_channel(int nl) { return NL == 1 ? 0 : NL == 2 ? 2 * (nl & 1) : 2 * (nl & 1) + (nl >> 1 & 1); }
__device__ __forceinline__ bool sums_here(int nl) { return nl < 4; }
template <int NL>
__device__ __forceinline__ void sum_states(const float2 (&v)[2], int nl, float (&out)[kSums<NL>]) {
    if constexpr (NL == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            out[2 * i] = v[i].x;
            out[2 * i + 1] = v[i].y;
        }
    } else {
        const bool b0 = nl & 1;
        const float z0 = (b0 ? v[1].x : v[0].x) + __shfl_xor_sync(0xffffffffu, b0 ? v[0].x : v[1].x, 1);
        const float z1 = (b0 ? v[1].y : v[0].y) + __shfl_xor_sync(0xffffffffu, b0 ? v[0].y : v[1].y, 1);
        if constexpr (NL == 2) {
            out[0] = z0;
            out[1] = z1;
        } else {
            const bool b1 = nl & 2;
            float z = (b1 ? z1 : z0) + __shfl_xor_sync(0xffffffffu, b1 ? z0 : z1, 2);
#pragma unroll
            for (int o = 4; o < NL; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            out[0] = z;
        }
    }
}

// The four B and four C of a token
struct Bc {
    float4 b, c;
    __device__ __forceinline__ void load(const float* p, bool both_) {
        b = *reinterpret_cast<const float4*>(p);
        if (both_) c = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ float bn(int n) const { return at4(b, n); }
    __device__ __forceinline__ float cn(int n) const { return at4(c, n); }
};

// Lanes along the states for N of them
inline int state_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

constexpr int kScanSms = 152;

// Calls f with an integral_constant: the lanes along the states
template <typename F>
cudaError_t by_lanes(int N, F f) {
    switch (state_lanes(N)) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 8: return f(std::integral_constant<int, 8>{});
        default: return f(std::integral_constant<int, 16>{});
    }
}

// Whether rows of channels, or of B and C, can be read four elements at a time
inline bool wide4(const ScanDims& d, const void* p, const long long (&s)[2]) {
    const int es = d.bf16 ? 2 : 4;
    return !p || ((d.D / d.G) % 4 == 0 && aligned_rows(p, s, d.at.rows(), d.at.L, 4 * es, es));
}
inline bool wide4(const ScanDims& d, const void* p, const long long (&s)[3]) {
    const int es = d.bf16 ? 2 : 4;
    const long long rows[2] = {s[0], s[1]};
    return d.N % 4 == 0 && (d.G < 2 || s[2] % 4 == 0) && aligned_rows(p, rows, d.at.rows(), d.at.L, 4 * es, es);
}

}  // namespace efla

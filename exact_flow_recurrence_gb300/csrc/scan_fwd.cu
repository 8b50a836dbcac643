// scan_fwd.cu -- the selective scan over whole sequences, and one token of it.
//
// Four fp32 operations and one exponential for every token, channel and state: their pipes, not HBM, bound it
// from 8 states on.  The recurrence runs along the tokens; channels and states are independent.  Where those are
// too few to fill the SMs the tokens are cut into segments: a first launch takes every segment from a zero state
// to its last one and adds up its dt, the second works out the state that a segment starts from (a fold over the
// segments before it) and takes it from there.
#include "scan.cuh"
#include "launch.h"

namespace efla {

namespace {

// Segments of `seg` tokens; ends [axis][segment][D][states], dts [axis][segment][D], alive [axis][segment] (whether the
// state that a segment starts from reaches its last token).
struct Segments {
    int seg, count;
    float *ends, *dts;
    int* alive;
};

template <typename T, int NL, bool WIDE, bool PART>
__global__ void __launch_bounds__(kScanThreads) k_scan_fwd(ScanDims d, ScanIn in, T* y, float* S_final, Segments sg) {
    using Tile = ScanTile<NL>;
    constexpr int CH = Tile::ch, S = Tile::states;
    extern __shared__ __align__(16) float dyn[];
    float *s_dt = dyn, *s_du = s_dt + kTile * CH, *s_b = s_du + kTile * CH, *s_c = s_b + kTile * S, *s_y = s_c + kTile * S;
    __shared__ int what[kTile], seq[kTile];
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const int axis = blockIdx.z, k = blockIdx.x, ta = k * sg.seg, tb = min(ta + sg.seg, d.at.L);
    const ScanLane<NL> l;
    const T* u = (const T*)in.u + axis * d.us[0] + cb.c0;
    const T* delta = (const T*)in.delta + axis * d.ds[0] + cb.c0;
    const T* z = in.z ? (const T*)in.z + axis * d.zs[0] + cb.c0 : nullptr;
    const T* Bm = (const T*)in.Bm + axis * d.bs[0] + cb.g * d.bs[2];
    const T* C = (const T*)in.C + axis * d.cs[0] + cb.g * d.cs[2];
    if (!PART) y += axis * d.ys[0] + cb.c0;
    float2 a2[4][2], h[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = l.states(in.A, d, cb, i);
        a2[i][0] = make_float2(v.x * kLog2eF, v.y * kLog2eF);
        a2[i][1] = make_float2(v.z * kLog2eF, v.w * kLog2eF);
        h[i][0] = h[i][1] = make_float2(0.f, 0.f);
    }
    if (!PART)   // the state that this segment starts from
        for (int j = 0; j < k; ++j) {
            const size_t at = (size_t)axis * sg.count + j;
            const bool alive = sg.alive[at];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (l.cl + i >= cb.n) continue;
                const float4 e = *reinterpret_cast<const float4*>(sg.ends + (at * d.D + cb.c0 + l.cl + i) * S + 4 * l.nl);
                const float2 sum = both(sg.dts[at * d.D + cb.c0 + l.cl + i]);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 x = mul2(a2[i][p], sum), f = p ? make_float2(e.z, e.w) : make_float2(e.x, e.y);
                    h[i][p] = alive ? fma2(make_float2(ex2(x.x), ex2(x.y)), h[i][p], f) : f;
                }
            }
        }
    // empty sequences hand their states on
    if (!PART && S_final && d.at.packed && k == 0)
        for (int b = 0; b < d.at.B; ++b) {
            const Seq s = seq_at(d.at, b);
            if (s.end > s.start) continue;
            const size_t at = (size_t)b * d.D * d.N;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                l.put_states(S_final + at, d, cb, i, in.S0 ? l.states(in.S0 + at, d, cb, i) : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    float4 dts = make_float4(0.f, 0.f, 0.f, 0.f);
    bool alive = true;
    for (int t0 = ta; t0 < tb; t0 += kTile) {
        __syncthreads();
        if (threadIdx.x < kTile) {
            const TokenAt a = token_at(d.at, axis, t0 + threadIdx.x, tb);
            what[threadIdx.x] = a.what;
            seq[threadIdx.x] = a.seq;
        }
        __syncthreads();
        load_bc<T, NL>(s_b, Bm, d.bs[1], d.N, t0, what);
        if (!PART) load_bc<T, NL>(s_c, C, d.cs[1], d.N, t0, what);
        for (int i = threadIdx.x; i < kTile * CH / 4; i += kScanThreads) {
            const int t = i / (CH / 4), c = i % (CH / 4) * 4, n = min(4, cb.n - c);
            float4 dt = make_float4(0.f, 0.f, 0.f, 0.f), du = dt;
            if (!(what[t] & kOutside) && n > 0) {
                const long long tt = t0 + t;
                const float4 x = load4<T, WIDE>(delta + tt * d.ds[1] + c, n);
                const float4 bias = in.dbias ? load4<float, false>(in.dbias + cb.c0 + c, n) : dt;
                dt.x = step_of(d, x.x + bias.x);
                if (n > 1) dt.y = step_of(d, x.y + bias.y);
                if (n > 2) dt.z = step_of(d, x.z + bias.z);
                if (n > 3) dt.w = step_of(d, x.w + bias.w);
                du = mul4(dt, load4<T, WIDE>(u + tt * d.us[1] + c, n));
            }
            *reinterpret_cast<float4*>(s_dt + t * CH + c) = dt;
            *reinterpret_cast<float4*>(s_du + t * CH + c) = du;
        }
        __syncthreads();
#pragma unroll 2
        for (int t = 0; t < kTile; ++t) {
            const int w = what[t];
            if (w & kFirst) {
                alive = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = in.S0 ? l.states(in.S0 + (size_t)seq[t] * d.D * d.N, d, cb, i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    h[i][0] = make_float2(v.x, v.y);
                    h[i][1] = make_float2(v.z, v.w);
                }
            }
            const float4 dt = *reinterpret_cast<const float4*>(s_dt + t * CH + l.cl), du = *reinterpret_cast<const float4*>(s_du + t * CH + l.cl);
            const float4 b = *reinterpret_cast<const float4*>(s_b + t * S + 4 * l.nl);
            float4 c = b;
            if (!PART) c = *reinterpret_cast<const float4*>(s_c + t * S + 4 * l.nl);
            float out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 dt2 = both(at4(dt, i)), du2 = both(at4(du, i));
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 bp = p ? make_float2(b.z, b.w) : make_float2(b.x, b.y);
                    h[i][p] = fma2(decay2(dt2, a2[i][p]), h[i][p], mul2(du2, bp));
                    if (!PART) acc = fma2(p ? make_float2(c.z, c.w) : make_float2(c.x, c.y), h[i][p], acc);
                }
                out[i] = acc.x + acc.y;
            }
            if (PART) dts = add4(dts, dt);
            else put_sums<NL>(s_y + t * CH, l, out);
            if (!PART && S_final && (w & kLast))
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    l.put_states(S_final + (size_t)seq[t] * d.D * d.N, d, cb, i, make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y));
        }
        if (PART) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * CH / 4; i += kScanThreads) {
            const int t = i / (CH / 4), c = i % (CH / 4) * 4, n = min(4, cb.n - c);
            if ((what[t] & kOutside) || n <= 0) continue;
            const long long tt = t0 + t;
            float4 v = *reinterpret_cast<const float4*>(s_y + t * CH + c);
            if (in.skip) v = add4(v, mul4(load4<float, false>(in.skip + cb.c0 + c, n), load4<T, WIDE>(u + tt * d.us[1] + c, n)));
            if (z) {
                const float4 g = load4<T, WIDE>(z + tt * d.zs[1] + c, n);
                v = mul4(v, make_float4(silu_of(g.x), silu_of(g.y), silu_of(g.z), silu_of(g.w)));
            }
            store4<T, WIDE>(y + tt * d.ys[1] + c, v, n);
        }
    }
    if (PART) {
        const size_t at = (size_t)axis * sg.count + k;
        if (threadIdx.x == 0 && blockIdx.y == 0) sg.alive[at] = alive;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (l.cl + i >= cb.n) continue;
            const size_t ch = at * d.D + cb.c0 + l.cl + i;
            *reinterpret_cast<float4*>(sg.ends + ch * S + 4 * l.nl) = make_float4(h[i][0].x, h[i][0].y, h[i][1].x, h[i][1].y);
            if (l.nl == 0) sg.dts[ch] = at4(dts, i);
        }
    }
}

// Segments of a forward pass: one, unless four-warp CTAs of whole sequences leave most SMs idle.
int segments(const ScanDims& d, int ch, int* seg) {
    const long long ctas = (long long)ch_blocks(d, ch) * d.at.rows();
    int count = 1;
    if (ctas < 96 && d.at.L >= 256) {
        count = (int)((2 * kScanSms + ctas - 1) / ctas);
        count = count < 32 ? count : 32;
        count = count < d.at.L / 64 ? count : d.at.L / 64;
    }
    *seg = ((d.at.L + count - 1) / count + kTile - 1) / kTile * kTile;
    return *seg ? (d.at.L + *seg - 1) / *seg : 1;
}

size_t seg_bytes(const ScanDims& d, int count, int states, size_t* dts, size_t* alive) {
    const size_t n = (size_t)d.at.rows() * count;
    *dts = align256(n * d.D * states * 4);
    *alive = *dts + align256(n * d.D * 4);
    return count > 1 ? *alive + align256(n * 4) : 0;
}

template <typename T, int NL, bool WIDE>
cudaError_t run(const ScanDims& d, const ScanIn& in, void* y, float* S_final, void* ws, cudaStream_t st) {
    using Tile = ScanTile<NL>;
    Segments sg{};
    sg.count = segments(d, Tile::ch, &sg.seg);
    size_t dts, alive;
    seg_bytes(d, sg.count, Tile::states, &dts, &alive);
    sg.ends = (float*)ws;
    sg.dts = (float*)((char*)ws + dts);
    sg.alive = (int*)((char*)ws + alive);
    const size_t smem = sizeof(float) * kTile * (3 * Tile::ch + 2 * Tile::states);
    const auto whole = k_scan_fwd<T, NL, WIDE, false>;
    const auto part = k_scan_fwd<T, NL, WIDE, true>;
    cudaError_t e = cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(sg.count, ch_blocks(d, Tile::ch), d.at.rows());
    if (sg.count > 1) {
        e = cudaFuncSetAttribute(part, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        part<<<dim3(sg.count - 1, grid.y, grid.z), kScanThreads, smem, st>>>(d, in, nullptr, nullptr, sg);
        prof_mark("scan_part", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    whole<<<grid, kScanThreads, smem, st>>>(d, in, (T*)y, S_final, sg);
    prof_mark("scan_fwd", st);
    return cudaGetLastError();
}

// ------------------------------------------------------------------- one token
// A thread takes four states of a channel; S [nslots][D][N].
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) k_scan_step(ScanDims d, ScanIn in, float* S, const int* slots, int nslots, T* y, int nl) {
    // (nl lanes a channel: a power of two, so that they lie in one warp)
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long ch = idx / nl, b = ch / d.D;
    const int q = (int)(idx % nl) * 4, c = (int)(ch % d.D);
    float acc = 0.f;
    const bool in_range = b < d.at.B;
    long long sl = -1;
    if (in_range) {
        sl = slots ? __ldg(slots + b) : b;
        if (sl >= nslots) sl = -1;
    }
    float x = 0.f;
    if (sl >= 0) {
        float* p = S + (sl * d.D + c) * d.N + q;
        const int n = min(4, d.N - q);
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n > 0) h = WIDE ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
        const int g = c / (d.D / d.G);
        x = ld_elem((const T*)in.u + b * d.us[0] + c);
        const float dt = step_of(d, ld_elem((const T*)in.delta + b * d.ds[0] + c) + (in.dbias ? __ldg(in.dbias + c) : 0.f));
        if (n > 0) {
            const float4 A = load4<float, WIDE>(in.A + (size_t)c * d.N + q, n);
            const float4 Bv = load4<T, false>((const T*)in.Bm + b * d.bs[0] + g * d.bs[2] + q, n);
            const float4 Cv = load4<T, false>((const T*)in.C + b * d.cs[0] + g * d.cs[2] + q, n);
            const float du = dt * x;
            const float2 a0 = decay2(both(dt), make_float2(A.x * kLog2eF, A.y * kLog2eF)), a1 = decay2(both(dt), make_float2(A.z * kLog2eF, A.w * kLog2eF));
            h.x = fmaf(a0.x, h.x, du * Bv.x);
            h.y = fmaf(a0.y, h.y, du * Bv.y);
            h.z = fmaf(a1.x, h.z, du * Bv.z);
            h.w = fmaf(a1.y, h.w, du * Bv.w);
            acc = fmaf(Cv.x, h.x, Cv.y * h.y) + fmaf(Cv.z, h.z, Cv.w * h.w);
            if (WIDE) {
                *reinterpret_cast<float4*>(p) = h;
            } else {
                p[0] = h.x;
                if (n > 1) p[1] = h.y;
                if (n > 2) p[2] = h.z;
                if (n > 3) p[3] = h.w;
            }
        }
    }
    for (int o = nl / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (!in_range || q) return;
    if (sl >= 0) {
        if (in.skip) acc = fmaf(__ldg(in.skip + c), x, acc);
        if (in.z) acc *= silu_of(ld_elem((const T*)in.z + b * d.zs[0] + c));
    }
    st_elem(y + b * d.ys[0] + c, sl >= 0 ? acc : 0.f);
}

template <typename T>
cudaError_t fwd(const ScanDims& d, const ScanIn& in, void* y, float* S_final, void* ws, cudaStream_t st) {
    const bool wide = wide4(d, in.u, d.us) && wide4(d, in.delta, d.ds) && wide4(d, in.z, d.zs) && wide4(d, y, d.ys);
    return by_lanes(d.N, [&](auto nl) {
        constexpr int NL = decltype(nl)::value;
        return wide ? run<T, NL, true>(d, in, y, S_final, ws, st) : run<T, NL, false>(d, in, y, S_final, ws, st);
    });
}

template <typename T>
cudaError_t step(const ScanDims& d, const ScanIn& in, float* S, const int* slots, int nslots, void* y, cudaStream_t st) {
    const int nl = state_lanes(d.N);
    const long long n = (long long)d.at.B * d.D * nl;
    const unsigned grid = (unsigned)((n + 255) / 256);
    const bool wide = d.N % 4 == 0 && ((uintptr_t)S & 15) == 0 && ((uintptr_t)in.A & 15) == 0;
    if (wide) k_scan_step<T, true><<<grid, 256, 0, st>>>(d, in, S, slots, nslots, (T*)y, nl);
    else k_scan_step<T, false><<<grid, 256, 0, st>>>(d, in, S, slots, nslots, (T*)y, nl);
    prof_mark("scan_step", st);
    return cudaGetLastError();
}

}  // namespace

size_t scan_fwd_ws_bytes(const ScanDims& d) {
    const int s = 4 * state_lanes(d.N);   // (CTAs of 16 * 32 / (s / 4) channels)
    int seg;
    size_t a, b;
    return seg_bytes(d, segments(d, 16 * 32 / (s / 4), &seg), s, &a, &b);
}

cudaError_t launch_scan_fwd(const ScanDims& d, const ScanIn& in, void* y, float* S_final, void* ws, cudaStream_t st) {
    if (d.at.L == 0) return cudaSuccess;
    return d.bf16 ? fwd<__nv_bfloat16>(d, in, y, S_final, ws, st) : fwd<float>(d, in, y, S_final, ws, st);
}

cudaError_t launch_scan_step(const ScanDims& d, const ScanIn& in, float* S, const int* slots, int nslots, void* y,
                             cudaStream_t st) {
    return d.bf16 ? step<__nv_bfloat16>(d, in, S, slots, nslots, y, st) : step<float>(d, in, S, slots, nslots, y, st);
}

}  // namespace efla

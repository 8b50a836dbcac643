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

// Named barriers of a CTA: a buffer filled, and a buffer's states done.
__device__ __forceinline__ void bar_wait(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}

// Tiles of TT tokens: two buffers of dt, dt u, y [TT][CH] and B, C [TT][S], and a ring of kRing raw tiles.
constexpr int kRing = 4, kWhat = 4;
template <typename T, int NL, bool PART>
struct FwdTile {
    static constexpr int CH = ScanTile<NL>::ch, S = ScanTile<NL>::states;
    static constexpr int TT = NL == 1 ? 4 : NL == 2 ? 8 : 16;
    static constexpr int items = TT * CH / 4 / kScanThreads;                       // a producer's groups of four channels a tile
    static constexpr int bc = TT * NL * (PART ? 1 : 2);                            // groups of four states of B and C a tile
    static constexpr int bc_items = (bc + kScanThreads - 1) / kScanThreads;
    static constexpr int arrays = PART ? 2 : 3;
    static constexpr int buffer = TT * CH * (PART ? 2 : 3) + TT * S * 2;           // floats
    static constexpr int slot = (items * arrays + bc_items) * kScanThreads;        // Vec<T, 4>
    static constexpr size_t bytes = 2 * buffer * sizeof(float) + kRing * slot * sizeof(Vec<T, 4>);
};

// Warps 0 .. 3 carry the states; warps 4 .. 7 bring the tokens (asynchronous copies, kRing tiles ahead), work out dt and dt u
// for them, and finish the y that they left: skip, gate, store.
template <typename T, int NL, bool WIDE, bool PART>
__global__ void __launch_bounds__(2 * kScanThreads, 2) k_scan_fwd(ScanDims d, ScanIn in, T* y, float* S_final, Segments sg) {
    using Tile = FwdTile<T, NL, PART>;
    using V = Vec<T, 4>;
    constexpr int CH = Tile::CH, S = Tile::S, TT = Tile::TT;
    extern __shared__ __align__(16) float dyn[];
    __shared__ int what[kWhat][TT], seq[kWhat][TT], any[kWhat];
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const int axis = blockIdx.z, k = blockIdx.x, ta = k * sg.seg, tb = min(ta + sg.seg, d.at.L);
    const int tiles = (tb - ta + TT - 1) / TT;
    const auto buffer = [&](int i) { return dyn + (i & 1) * Tile::buffer; };   // dt, dt u, B, C, y
    if (threadIdx.x >= kScanThreads) {
        const int tid = threadIdx.x - kScanThreads;
        const T* u = (const T*)in.u + axis * d.us[0] + cb.c0;
        const T* delta = (const T*)in.delta + axis * d.ds[0] + cb.c0;
        const T* z = in.z ? (const T*)in.z + axis * d.zs[0] + cb.c0 : nullptr;
        const T* Bm = (const T*)in.Bm + axis * d.bs[0] + cb.g * d.bs[2];
        const T* C = (const T*)in.C + axis * d.cs[0] + cb.g * d.cs[2];
        if (!PART) y += axis * d.ys[0] + cb.c0;
        V* raw = reinterpret_cast<V*>(dyn + 2 * Tile::buffer) + tid;
        // its channels c .. c + n - 1 (n <= 4), and tokens row, row + rows, .. of a tile
        constexpr int rows = kScanThreads / (CH / 4 < kScanThreads ? CH / 4 : kScanThreads);
        const int c = tid % (CH / 4) * 4, row = tid / (CH / 4), n = min(4, cb.n - c);
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 bias = in.dbias ? load4<float, false>(in.dbias + cb.c0 + c, n) : none;
        const float4 skip = in.skip ? load4<float, false>(in.skip + cb.c0 + c, n) : none;
        const auto bring = [&](V* to, const T* from, int m) {
            if (WIDE) {
                copy_async(to, from, sizeof(V));
            } else {
                const float4 v = load4<T, false>(from, m);
                const float f[4] = {v.x, v.y, v.z, v.w};
                to->set(f);
            }
        };
        const auto issue = [&](int i) {   // tile i into its slot
            if (i < tiles) {
                V* slot = raw + (i % kRing) * Tile::slot;
                const int t0 = ta + i * TT;
                if (n > 0)
#pragma unroll
                    for (int j = 0; j < Tile::items; ++j) {
                        const long long t = t0 + row + j * rows;
                        if (t >= tb) continue;
                        bring(slot + j * Tile::arrays * kScanThreads, u + t * d.us[1] + c, n);
                        bring(slot + (j * Tile::arrays + 1) * kScanThreads, delta + t * d.ds[1] + c, n);
                        if (!PART && z) bring(slot + (j * Tile::arrays + 2) * kScanThreads, z + t * d.zs[1] + c, n);
                    }
#pragma unroll
                for (int j = 0; j < Tile::bc_items; ++j) {
                    const int e = tid + j * kScanThreads, q = e % NL * 4, t = e / NL % TT;
                    if (e >= Tile::bc || t0 + t >= tb || q >= d.N) continue;
                    const T* from = e < TT * NL ? Bm + (t0 + t) * d.bs[1] + q : C + (t0 + t) * d.cs[1] + q;
                    bring(slot + (Tile::items * Tile::arrays + j) * kScanThreads, from, min(4, d.N - q));
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const auto look = [&](int i) {   // what tile i's tokens are
            if (i < tiles && tid < 32) {
                int w = 0;
                if (tid < TT) {
                    const TokenAt a = token_at(d.at, axis, ta + i * TT + tid, tb);
                    what[i % kWhat][tid] = w = a.what;
                    seq[i % kWhat][tid] = a.seq;
                }
                w = __any_sync(0xffffffffu, w & (kFirst | kLast));
                if (tid == 0) any[i % kWhat] = w;
            }
        };
        const auto get = [](const V* p) {
            float f[4];
            p->get(f);
            return make_float4(f[0], f[1], f[2], f[3]);
        };
        const auto fill = [&](int i) {
            const V* slot = raw + (i % kRing) * Tile::slot;
            float *s_dt = buffer(i), *s_du = s_dt + TT * CH, *s_bc = s_du + TT * CH;
            const int* w = what[i % kWhat];
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                const int t = row + j * rows;
                float4 dt = none, du = none;
                if (!(w[t] & kOutside) && n > 0) {
                    dt = steps(d, add4(get(slot + (j * Tile::arrays + 1) * kScanThreads), bias), n);
                    du = mul4(dt, get(slot + j * Tile::arrays * kScanThreads));
                }
                *reinterpret_cast<float4*>(s_dt + t * CH + c) = dt;
                *reinterpret_cast<float4*>(s_du + t * CH + c) = du;
            }
#pragma unroll
            for (int j = 0; j < Tile::bc_items; ++j) {
                const int e = tid + j * kScanThreads, q = e % NL * 4, t = e / NL % TT;
                if (e >= Tile::bc) continue;
                const bool in_range = !(w[t] & kOutside) && q < d.N;
                *reinterpret_cast<float4*>(s_bc + (e / NL) * S + q) = in_range ? get(slot + (Tile::items * Tile::arrays + j) * kScanThreads) : none;
            }
        };
        const auto finish = [&](int i) {
            const V* slot = raw + (i % kRing) * Tile::slot;
            const float* s_y = buffer(i) + 2 * TT * CH + 2 * TT * S;
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                const int t = row + j * rows;
                if ((what[i % kWhat][t] & kOutside) || n <= 0) continue;
                const long long tt = ta + i * TT + t;
                float4 v = *reinterpret_cast<const float4*>(s_y + t * CH + c);
                const float4 uu = get(slot + j * Tile::arrays * kScanThreads);
                v = make_float4(fmaf(skip.x, uu.x, v.x), fmaf(skip.y, uu.y, v.y), fmaf(skip.z, uu.z, v.z), fmaf(skip.w, uu.w, v.w));
                if (z) {
                    const float4 g = get(slot + (j * Tile::arrays + 2) * kScanThreads);
                    v = mul4(v, make_float4(silu_of(g.x), silu_of(g.y), silu_of(g.z), silu_of(g.w)));
                }
                store4<T, WIDE>(y + tt * d.ys[1] + c, v, n);
            }
        };
        for (int i = 0; i < kRing; ++i) issue(i);
        look(0);
        look(1);
        asm volatile("bar.sync 5, 128;" ::: "memory");
        for (int i = 0; i < tiles; ++i) {
            // tile i is group i, and i + 2 is the last one under way (a thread reads only what it copied itself)
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            fill(i);
            bar_arrive(1 + (i & 1));
            if (i > 0) {
                look(i + 1);   // (the others read it behind the next barrier; its slot's last readers are behind the one before)
                bar_wait(3 + ((i - 1) & 1));
                if (!PART) finish(i - 1);
                issue(i - 1 + kRing);
            }
        }
        bar_wait(3 + ((tiles - 1) & 1));
        if (!PART) finish(tiles - 1);
        return;
    }
    const ScanLane<NL> l;
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
    for (int i = 0; i < tiles; ++i) {
        float* const s_dt = buffer(i);
        const float *s_du = s_dt + TT * CH, *s_b = s_du + TT * CH, *s_c = s_b + TT * S;
        float* const s_y = s_dt + 2 * TT * CH + 2 * TT * S;
        bar_wait(1 + (i & 1));
        const auto token = [&](int t) {
            const float4 dt = *reinterpret_cast<const float4*>(s_dt + t * CH + l.cl), du = *reinterpret_cast<const float4*>(s_du + t * CH + l.cl);
            const float4 b = *reinterpret_cast<const float4*>(s_b + t * S + 4 * l.nl);
            float4 c = b;
            if (!PART) c = *reinterpret_cast<const float4*>(s_c + t * S + 4 * l.nl);
            float out[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 dt2 = both(at4(dt, j)), du2 = both(at4(du, j));
                float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float2 bp = p ? make_float2(b.z, b.w) : make_float2(b.x, b.y), cp = p ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
                    h[j][p] = fma2(decay2(dt2, a2[j][p]), h[j][p], mul2(du2, bp));
                    if (!PART) acc = p ? fma2(cp, h[j][p], acc) : mul2(cp, h[j][p]);
                }
                out[j] = acc.x + acc.y;
            }
            if (PART) dts = add4(dts, dt);
            else put_sums<NL>(s_y + t * CH, l, out);
        };
        if (!any[i % kWhat]) {
#pragma unroll 4
            for (int t = 0; t < TT; ++t) token(t);
        } else {
#pragma unroll 1
            for (int t = 0; t < TT; ++t) {
                const int w = what[i % kWhat][t];
                const size_t at = (size_t)seq[i % kWhat][t] * d.D * d.N;
                if (w & kFirst) {
                    alive = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = in.S0 ? l.states(in.S0 + at, d, cb, j) : make_float4(0.f, 0.f, 0.f, 0.f);
                        h[j][0] = make_float2(v.x, v.y);
                        h[j][1] = make_float2(v.z, v.w);
                    }
                }
                token(t);
                if (!PART && S_final && (w & kLast))
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        l.put_states(S_final + at, d, cb, j, make_float4(h[j][0].x, h[j][0].y, h[j][1].x, h[j][1].y));
            }
        }
        bar_arrive(3 + (i & 1));
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
    *seg = ((d.at.L + count - 1) / count + 15) / 16 * 16;
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
    using Whole = FwdTile<T, NL, false>;
    using Part = FwdTile<T, NL, true>;
    const auto whole = k_scan_fwd<T, NL, WIDE, false>;
    const auto part = k_scan_fwd<T, NL, WIDE, true>;
    cudaError_t e = cudaFuncSetAttribute(whole, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Whole::bytes);
    if (e != cudaSuccess) return e;
    const dim3 grid(sg.count, ch_blocks(d, Tile::ch), d.at.rows());
    if (sg.count > 1) {
        e = cudaFuncSetAttribute(part, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Part::bytes);
        if (e != cudaSuccess) return e;
        part<<<dim3(sg.count - 1, grid.y, grid.z), 2 * kScanThreads, Part::bytes, st>>>(d, in, nullptr, nullptr, sg);
        prof_mark("scan_part", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    whole<<<grid, 2 * kScanThreads, Whole::bytes, st>>>(d, in, (T*)y, S_final, sg);
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
    const bool wide = wide4(d, in.u, d.us) && wide4(d, in.delta, d.ds) && wide4(d, in.z, d.zs) && wide4(d, y, d.ys) &&
                      wide4(d, in.Bm, d.bs) && wide4(d, in.C, d.cs);
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

// scan_fwd.cu -- the selective scan over whole sequences, and one token of it.
//
// Four fp32 operations and one exponential for every token, channel and state: their pipes, not HBM, bound it
// from 8 states on (a warp's token of 32 channels and 16 states: 64 cycles of a scheduler's FMA pipe, 64 of its exponentials).
// The recurrence runs along the tokens; channels and states are independent: B D N / 16 threads in all, one carrying warp a
// scheduler at the training size, so that what counts is how little else that warp does and waits for.  Hence a
// thread's 4 x 4 tile (B, C read once for four channels), everything that depends on a channel alone in other warps, and
// loads of the next four tokens before the stores of these.
// Where channels are too few to fill the SMs the tokens are cut into segments: a first launch takes every segment from a zero
// state to its last one and adds up its dt, the second works out the state that a segment starts from (a fold over the
// segments before it) and takes it from there.
// B8 L2048 D2048 N16 bf16 with gate: 195 us on 128 SMs (272 MB, 1.4 TB/s; 40 us at a plain copy's rate, 69 us at its pipes' on these SMs),
// issue slots 60% used.  Steps on the way: warps that do all by themselves 1574, carrying and bringing warps 280, loads ahead of
// stores 229, four buffers 213, B and C as fp32 in shared memory 197; B and C there twice, for packed operands: 254 (shared
// memory's loads then bound it).  13 packed prompts, 16384 tokens: 309 us in two launches (nine segments).
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

// Threads that carry states; and those that bring tokens, in kGroups groups that take turns
constexpr int kCarry = 256 / kNP, kBring = 128, kGroups = 2;

// Named barriers of a CTA: a buffer filled, and a buffer's states done.
__device__ __forceinline__ void bar_wait(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kCarry + kBring) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kCarry + kBring) : "memory"); }
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
}

// Tiles of TT tokens.  kBuffers buffers: (dt, dt, dt u, dt u) of two channels [TT][CH / 2], y [TT][CH], and (B, C) of four states
// [TT][NL], fp32; and for each group a ring of raw tiles.
constexpr int kBuffers = 4, kWhat = 8;
static_assert(kBuffers == 2 * kGroups, "a group fills a buffer while the carriers may still read the one that it filled before");
static_assert(kWhat >= 2 * kBuffers && 2 * kBuffers + kGroups < 16, "slots of flags, named barriers");
template <typename T, int NL, bool PART>
struct FwdTile {
    static constexpr int CH = ScanTile<NL>::ch, S = ScanTile<NL>::states;
    static constexpr int TT = NL == 1 ? 4 : NL == 2 ? 8 : 16;
    static constexpr int items = (TT * CH / 4 + kBring - 1) / kBring;               // a thread's groups of four channels a tile
    static constexpr int bc = TT * NL * (PART ? 1 : 2);                            // groups of four states of B and C a tile
    static constexpr int bc_items = (bc + kBring - 1) / kBring;
    static constexpr int arrays = PART ? 2 : 3;
    static constexpr int y_at = TT * CH * 2, bc_at = y_at + (PART ? 0 : TT * CH);  // floats
    static constexpr int buffer = bc_at + TT * NL * 8;
    static constexpr int slot = (items * arrays + bc_items) * kBring;              // Vec<T, 4>
    static constexpr int ring = sizeof(T) == 2 ? 3 : 2;
    static constexpr size_t bytes = kBuffers * buffer * sizeof(float) + kGroups * ring * slot * sizeof(Vec<T, 4>);
};

// Warps 0 .. 3 carry the states, four neighbouring channels of four states a thread (two and two in one instruction's halves);
// warps 4 .. 11, two groups of four that take a tile each in turn, bring the tokens, work out dt and dt u for them, and finish the
// y that the carriers left: skip, gate, store.  A barrier joins the carriers and one group.  Both sides are chains of short steps;
// four buffers and two groups keep either from waiting for the other.  Rows come by asynchronous copies into a group's ring: three
// tiles for bf16, so that one is under way while the one before it is waited for; two for fp32, where a turn waits for the copies
// that the turn before it issued at its end.  Rows that are not aligned to four elements are loaded and stored at once.
template <typename T, int NL, bool WIDE, bool PART>
__global__ void __launch_bounds__(kCarry + kGroups * kBring, 1) k_scan_fwd(ScanDims d, ScanIn in, T* y, float* S_final, Segments sg) {
    using Tile = FwdTile<T, NL, PART>;
    using V = Vec<T, 4>;
    constexpr int CH = Tile::CH, S = Tile::S, TT = Tile::TT;
    extern __shared__ __align__(16) float dyn[];
    __shared__ int what[kWhat][TT], seq[kWhat][TT], any[kWhat];
    const ChBlock cb = ch_block<NL>(d, blockIdx.y);
    const int axis = blockIdx.z, k = blockIdx.x, ta = k * sg.seg, tb = min(ta + sg.seg, d.at.L);
    const int tiles = (tb - ta + TT - 1) / TT;
    const auto buffer = [&](int i) { return dyn + (i % kBuffers) * Tile::buffer; };
    if (threadIdx.x >= kCarry) {
        const int group = (threadIdx.x - kCarry) / kBring, tid = (threadIdx.x - kCarry) % kBring;
        const T* u = (const T*)in.u + axis * d.us[0] + cb.c0;
        const T* delta = (const T*)in.delta + axis * d.ds[0] + cb.c0;
        const T* z = in.z ? (const T*)in.z + axis * d.zs[0] + cb.c0 : nullptr;
        const T* Bm = (const T*)in.Bm + axis * d.bs[0] + cb.g * d.bs[2];
        const T* C = (const T*)in.C + axis * d.cs[0] + cb.g * d.cs[2];
        if (!PART) y += axis * d.ys[0] + cb.c0;
        V* raw = reinterpret_cast<V*>(dyn + kBuffers * Tile::buffer) + group * Tile::ring * Tile::slot + tid;
        // its channels c .. c + n - 1 (n <= 4), and tokens row, row + rows, .. of a tile
        constexpr int rows = kBring / (CH / 4);
        const int c = tid % (CH / 4) * 4, row = tid / (CH / 4), n = row < TT ? min(4, cb.n - c) : 0;
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
                V* slot = raw + (i / kGroups % Tile::ring) * Tile::slot;
                const int t0 = ta + i * TT;
                if (n > 0)
#pragma unroll
                    for (int j = 0; j < Tile::items; ++j) {
                        const long long t = t0 + row + j * rows;
                        if (t >= tb) continue;
                        bring(slot + j * Tile::arrays * kBring, u + t * d.us[1] + c, n);
                        bring(slot + (j * Tile::arrays + 1) * kBring, delta + t * d.ds[1] + c, n);
                        if (!PART && z) bring(slot + (j * Tile::arrays + 2) * kBring, z + t * d.zs[1] + c, n);
                    }
#pragma unroll
                for (int j = 0; j < Tile::bc_items; ++j) {
                    const int e = tid + j * kBring, q = e % NL * 4, t = e / NL % TT;
                    if (e >= Tile::bc || t0 + t >= tb || q >= d.N) continue;
                    const T* from = e < TT * NL ? Bm + (t0 + t) * d.bs[1] + q : C + (t0 + t) * d.cs[1] + q;
                    bring(slot + (Tile::items * Tile::arrays + j) * kBring, from, min(4, d.N - q));
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
            const V* slot = raw + (i / kGroups % Tile::ring) * Tile::slot;
            float* const s_dd = buffer(i);
            float* const s_bc = s_dd + Tile::bc_at;
            const int* w = what[i % kWhat];
            // (every load before the first store: a store holds back the loads behind it)
            float4 dt[Tile::items], du[Tile::items];
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                dt[j] = get(slot + (j * Tile::arrays + 1) * kBring);
                du[j] = get(slot + j * Tile::arrays * kBring);
            }
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                const bool in_range = n > 0 && !(w[row + j * rows] & kOutside);
                dt[j] = steps(d, add4(dt[j], bias), n);
                du[j] = in_range ? mul4(dt[j], du[j]) : none;
                if (!in_range) dt[j] = none;
            }
            if (row < TT)
#pragma unroll
                for (int j = 0; j < Tile::items; ++j) {
                    float4* p = reinterpret_cast<float4*>(s_dd + ((row + j * rows) * CH + c) * 2);
                    p[0] = make_float4(dt[j].x, dt[j].y, du[j].x, du[j].y);
                    p[1] = make_float4(dt[j].z, dt[j].w, du[j].z, du[j].w);
                }
#pragma unroll
            for (int j = 0; j < Tile::bc_items; ++j) {
                const int e = tid + j * kBring, q = e % NL, t = e / NL % TT;
                if (e >= Tile::bc) continue;
                V v;
                v.zero();
                if (!(w[t] & kOutside) && 4 * q < d.N) v = slot[(Tile::items * Tile::arrays + j) * kBring];
                *reinterpret_cast<float4*>(s_bc + (t * NL + q) * 8 + (e < TT * NL ? 0 : 4)) = as4(v);
            }
        };
        const auto finish = [&](int i) {
            const V* slot = raw + (i / kGroups % Tile::ring) * Tile::slot;
            const float* s_y = buffer(i) + Tile::y_at;
            if (n <= 0) return;
            float4 v[Tile::items], uu[Tile::items], g[Tile::items];
            bool in_range[Tile::items];
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                in_range[j] = !(what[i % kWhat][row + j * rows] & kOutside);
                v[j] = *reinterpret_cast<const float4*>(s_y + (row + j * rows) * CH + c);
                uu[j] = get(slot + j * Tile::arrays * kBring);
                if (z) g[j] = get(slot + (j * Tile::arrays + 2) * kBring);
            }
#pragma unroll
            for (int j = 0; j < Tile::items; ++j) {
                v[j] = make_float4(fmaf(skip.x, uu[j].x, v[j].x), fmaf(skip.y, uu[j].y, v[j].y), fmaf(skip.z, uu[j].z, v[j].z),
                                   fmaf(skip.w, uu[j].w, v[j].w));
                if (z) v[j] = mul4(v[j], mul4(g[j], sigmoid4(g[j])));
            }
#pragma unroll
            for (int j = 0; j < Tile::items; ++j)
                if (in_range[j]) store4<T, WIDE>(y + (long long)(ta + i * TT + row + j * rows) * d.ys[1] + c, v[j], n);
        };
        for (int j = 0; j < Tile::ring; ++j) issue(group + j * kGroups);
        look(group);
        look(group + kGroups);
        asm volatile("bar.sync %0, %1;" ::"r"(9 + group), "n"(kBring) : "memory");
        int last = -1;
        for (int i = group; i < tiles; last = i, i += kGroups) {
            // the group's tile n is its copies' group n, and n + ring - 2 is the last one under way (a thread reads only what it
            // copied itself)
            asm volatile("cp.async.wait_group %0;" ::"n"(Tile::ring - 2) : "memory");
            fill(i);
            bar_arrive(1 + i % kBuffers);
            if (last >= 0) {
                look(i + kGroups);   // (the others read it behind the next barrier; its slot's last readers are behind the one before)
                bar_wait(1 + kBuffers + last % kBuffers);
                if (!PART) finish(last);
                issue(last + Tile::ring * kGroups);
            }
        }
        if (last >= 0) {
            bar_wait(1 + kBuffers + last % kBuffers);
            if (!PART) finish(last);
        }
        return;
    }
    constexpr int NP = kNP;
    const ScanLane<NL, NP> l;
    float2 a2[NP][4], h[NP][4];
    l.pairs(in.A, 0, d, cb, a2);
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            a2[j][n] = mul2(a2[j][n], both(kLog2eF));
            h[j][n] = make_float2(0.f, 0.f);
        }
    if (!PART && S_final && d.at.packed && k == 0)   // empty sequences hand their states on
        for (int b = 0; b < d.at.B; ++b) {
            const Seq s = seq_at(d.at, b);
            if (s.end > s.start) continue;
            const size_t at = (size_t)b * d.D * d.N;
            float2 keep[NP][4];
            l.pairs(in.S0, at, d, cb, keep);
            l.put_pairs(S_final + at, d, cb, keep);
        }
    if (!PART)   // the state that this segment starts from
        for (int j = 0; j < k; ++j) {
            const size_t at = (size_t)axis * sg.count + j;
            const bool alive = sg.alive[at];
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const size_t ch = at * d.D + cb.c0 + l.cl + 2 * i;
                const bool in0 = l.cl + 2 * i < cb.n, in1 = l.cl + 2 * i + 1 < cb.n;
                const float4 e0 = in0 ? *reinterpret_cast<const float4*>(sg.ends + ch * S + 4 * l.nl) : none,
                             e1 = in1 ? *reinterpret_cast<const float4*>(sg.ends + (ch + 1) * S + 4 * l.nl) : none;
                const float2 sum = make_float2(in0 ? sg.dts[ch] : 0.f, in1 ? sg.dts[ch + 1] : 0.f);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 x = mul2(a2[i][n], sum), e = make_float2(at4(e0, n), at4(e1, n));
                    h[i][n] = alive ? add2(make_float2(times_ex2(h[i][n].x, x.x), times_ex2(h[i][n].y, x.y)), e) : e;
                }
            }
        }
    float2 dts[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) dts[j] = make_float2(0.f, 0.f);
    bool alive = true;
    for (int i = 0; i < tiles; ++i) {
        const float* const s_dd = buffer(i) + l.cl * 2;
        const float* const s_bc = buffer(i) + Tile::bc_at + l.nl * 8;
        float* const s_y = buffer(i) + Tile::y_at;
        bar_wait(1 + i % kBuffers);
        // what KT tokens read, and the tokens: a store holds back the loads behind it, so that the next tokens' are loaded before
        const auto load = [&](int t, auto& dd, auto& bc, auto kt) {
#pragma unroll
            for (int e = 0; e < decltype(kt)::value; ++e) {
#pragma unroll
                for (int j = 0; j < NP; ++j) dd[e][j] = *reinterpret_cast<const float4*>(s_dd + (t + e) * CH * 2 + 4 * j);
                bc[e].load(s_bc + (t + e) * NL * 8, !PART);
            }
        };
        const auto tokens = [&](int t, const auto& dd, const auto& bc, auto kt) {
            constexpr int KT = decltype(kt)::value;
            float2 out[KT][NP];
#pragma unroll
            for (int e = 0; e < KT; ++e) {
                float2 dt[NP], du[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    dt[j] = lo(dd[e][j]);
                    du[j] = hi(dd[e][j]);
                    if (PART) dts[j] = add2(dts[j], dt[j]);
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 b = both(bc[e].bn(n)), c = PART ? b : both(bc[e].cn(n));
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        h[j][n] = fma2(decay2(dt[j], a2[j][n]), h[j][n], mul2(du[j], b));
                        if (!PART) out[e][j] = n ? fma2(c, h[j][n], out[e][j]) : mul2(c, h[j][n]);
                    }
                }
            }
            if constexpr (PART) {
            } else if constexpr (KT == 4 && NL >= 4) {   // lane nl < 4 gets the sums of token t + nl
                const bool b0 = l.nl & 1, b1 = l.nl & 2;
                const auto add_other = [](float2 keep, float2 give, int mask) {
                    return make_float2(keep.x + __shfl_xor_sync(0xffffffffu, give.x, mask), keep.y + __shfl_xor_sync(0xffffffffu, give.y, mask));
                };
                float2 s[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    float2 z[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) z[e] = add_other(b1 ? out[e + 2][j] : out[e][j], b1 ? out[e][j] : out[e + 2][j], 2);
                    s[j] = add_other(b0 ? z[1] : z[0], b0 ? z[0] : z[1], 1);
                    if constexpr (NL >= 8) s[j] = add_other(s[j], s[j], 4);
                    if constexpr (NL >= 16) s[j] = add_other(s[j], s[j], 8);
                }
                if (NL == 4 || l.nl < 4)
#pragma unroll
                    for (int j = 0; j < NP; ++j) *reinterpret_cast<float2*>(s_y + (t + (l.nl & 3)) * CH + l.cl + 2 * j) = s[j];
            } else {
#pragma unroll
                for (int e = 0; e < KT; ++e)
#pragma unroll
                    for (int j = 0; j < NP; ++j) {
                        float2 s = out[e][j];
#pragma unroll
                        for (int o = 1; o < NL; o <<= 1)
                            s = make_float2(s.x + __shfl_xor_sync(0xffffffffu, s.x, o), s.y + __shfl_xor_sync(0xffffffffu, s.y, o));
                        if (l.nl == 0) *reinterpret_cast<float2*>(s_y + (t + e) * CH + l.cl + 2 * j) = s;
                    }
            }
        };
        if (!any[i % kWhat]) {
            constexpr std::integral_constant<int, 4> four{};
            float4 dd[2][4][NP];
            Bc bc[2][4];
            load(0, dd[0], bc[0], four);
#pragma unroll
            for (int t = 0; t < TT; t += 4) {
                if (t + 4 < TT) load(t + 4, dd[(t / 4 + 1) & 1], bc[(t / 4 + 1) & 1], four);
                tokens(t, dd[t / 4 & 1], bc[t / 4 & 1], four);
            }
        } else {
#pragma unroll 1
            for (int t = 0; t < TT; ++t) {
                const int w = what[i % kWhat][t];
                const size_t at = (size_t)seq[i % kWhat][t] * d.D * d.N;
                if (w & kFirst) {
                    alive = false;
                    l.pairs(in.S0, at, d, cb, h);
                }
                constexpr std::integral_constant<int, 1> one{};
                float4 dd[1][NP];
                Bc bc[1];
                load(t, dd, bc, one);
                tokens(t, dd, bc, one);
                if (!PART && S_final && (w & kLast)) l.put_pairs(S_final + at, d, cb, h);
            }
        }
        bar_arrive(1 + kBuffers + i % kBuffers);
    }
    if (PART) {
        const size_t at = (size_t)axis * sg.count + k;
        if (threadIdx.x == 0 && blockIdx.y == 0) sg.alive[at] = alive;
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) {
            if (l.cl + i >= cb.n) continue;
            const size_t ch = at * d.D + cb.c0 + l.cl + i;
            *reinterpret_cast<float4*>(sg.ends + ch * S + 4 * l.nl) = one_of<NP>(h, i);
            if (l.nl == 0) sg.dts[ch] = i & 1 ? dts[i / 2].y : dts[i / 2].x;
        }
    }
}

// Segments of a forward pass: one, unless CTAs of whole sequences (one an SM) leave a third of the SMs idle.  Two launches take
// 1.6 times the work of one.
int segments(const ScanDims& d, int ch, int* seg) {
    const long long ctas = (long long)ch_blocks(d, ch) * d.at.rows();
    int count = 1;
    if (ctas < 96 && d.at.L >= 256) {
        count = (int)(kScanSms / ctas);
        if (count < 3) count = (int)(2 * kScanSms / ctas);
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
        part<<<dim3(sg.count - 1, grid.y, grid.z), kCarry + kGroups * kBring, Part::bytes, st>>>(d, in, nullptr, nullptr, sg);
        prof_mark("scan_part", st);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    whole<<<grid, kCarry + kGroups * kBring, Whole::bytes, st>>>(d, in, (T*)y, S_final, sg);
    prof_mark("scan_fwd", st);
    return cudaGetLastError();
}

// ------------------------------------------------------------------- one token
// S [nslots][D][N].  Bound by HBM: the states, read and written once.
//   h <- e^{dt A} h + dt u B of four states, and their part of sum_n C h
__device__ __forceinline__ float step4(float dt, float u, float2 a0, float2 a1, float4& h, const float4& B, const float4& C) {
    const float2 du = both(dt * u), h0 = fma2(decay2(both(dt), a0), make_float2(h.x, h.y), mul2(du, make_float2(B.x, B.y))),
                 h1 = fma2(decay2(both(dt), a1), make_float2(h.z, h.w), mul2(du, make_float2(B.z, B.w)));
    h = make_float4(h0.x, h0.y, h1.x, h1.y);
    const float2 s = fma2(make_float2(C.z, C.w), h1, mul2(make_float2(C.x, C.y), h0));
    return s.x + s.y;
}

// A thread takes four states of a channel of a sequence; nl lanes a channel, a power of two, so that they lie in one warp.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) k_scan_step(ScanDims d, ScanIn in, float* S, const int* slots, int nslots, T* y, int nl) {
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x, ch = idx / nl, b = ch / d.D;
    const int q = (int)(idx % nl) * 4, c = (int)(ch % d.D), n = min(4, d.N - q);
    const bool here = b < d.at.B;
    long long sl = !here ? -1 : slots ? __ldg(slots + b) : b;
    if (sl >= nslots) sl = -1;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 h = none, A = none, Bv = none, Cv = none;
    float u = 0.f, raw = 0.f, acc = 0.f;
    float* p = S + (sl * d.D + c) * d.N + q;
    if (sl >= 0) {
        if (n > 0) {
            const int g = c / (d.D / d.G);
            h = WIDE ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
            A = load4<float, WIDE>(in.A + (size_t)c * d.N + q, n);
            Bv = load4<T, WIDE>((const T*)in.Bm + b * d.bs[0] + g * d.bs[2] + q, n);
            Cv = load4<T, WIDE>((const T*)in.C + b * d.cs[0] + g * d.cs[2] + q, n);
        }
        u = ld_elem((const T*)in.u + b * d.us[0] + c);
        raw = ld_elem((const T*)in.delta + b * d.ds[0] + c) + (in.dbias ? __ldg(in.dbias + c) : 0.f);
        acc = step4(step_of(d, raw), u, mul2(make_float2(A.x, A.y), both(kLog2eF)), mul2(make_float2(A.z, A.w), both(kLog2eF)), h, Bv, Cv);
        if (WIDE) {
            if (n > 0) *reinterpret_cast<float4*>(p) = h;
        } else {
            if (n > 0) p[0] = h.x;
            if (n > 1) p[1] = h.y;
            if (n > 2) p[2] = h.z;
            if (n > 3) p[3] = h.w;
        }
    }
    for (int o = nl / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (!here || q) return;
    if (sl >= 0) {
        if (in.skip) acc = fmaf(__ldg(in.skip + c), u, acc);
        if (in.z) acc *= silu_of(ld_elem((const T*)in.z + b * d.zs[0] + c));
    }
    st_elem(y + b * d.ys[0] + c, sl >= 0 ? acc : 0.f);
}

// A batch: a CTA keeps its channels (16 KB of a state: their A, skip and bias stay in registers) and takes every
// gridDim.x-th sequence.  States and token rows come by asynchronous copies, kStepStages - 1 sequences ahead, so that what is in
// flight costs no registers.  N = 4 nl, nl = 1 << shift.
constexpr int kStepStages = 6, kStepFour = 4;   // groups of four states a thread
template <typename T>
__global__ void __launch_bounds__(256, 2) k_scan_step_ring(ScanDims d, ScanIn in, float* S, const int* slots, int nslots, T* y, int shift) {
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ int s_slot[kStepStages];
    const int tid = threadIdx.x, nl = 1 << shift, CT = (256 * kStepFour) >> shift, c0 = blockIdx.y * CT, n = min(CT, d.D - c0), g = c0 / (d.D / d.G);
    const uint32_t states = 256 * kStepFour * 16, stage = states + (3 * CT + 8 * nl) * (uint32_t)sizeof(T);
    float2 a0[kStepFour], a1[kStepFour];
    float bias[kStepFour], skip[kStepFour];
#pragma unroll
    for (int i = 0; i < kStepFour; ++i) {
        const int f = i * 256 + tid, c = f >> shift;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        bias[i] = skip[i] = 0.f;
        if (c < n) {
            A = __ldg(reinterpret_cast<const float4*>(in.A + (size_t)c0 * d.N) + f);
            if (in.dbias) bias[i] = __ldg(in.dbias + c0 + c);
            if (in.skip) skip[i] = __ldg(in.skip + c0 + c);
        }
        a0[i] = mul2(make_float2(A.x, A.y), both(kLog2eF));
        a1[i] = mul2(make_float2(A.z, A.w), both(kLog2eF));
    }
    const int count = (d.at.B - (int)blockIdx.x + gridDim.x - 1) / gridDim.x;   // this CTA's sequences
    const auto place = [&](int k) {
        const int b = blockIdx.x + k * gridDim.x;
        return k >= count ? -1 : slots ? __ldg(slots + b) : b;
    };
    int next = place(0);
    const auto issue = [&](int k) {
        if (k < count) {
            const long long b = blockIdx.x + (long long)k * gridDim.x;
            unsigned char* to = ring + (k % kStepStages) * stage;
            const int sl = next >= 0 && next < nslots ? next : -1;
            if (tid == 0) s_slot[k % kStepStages] = sl;
            if (sl >= 0) {
                const float4* from = reinterpret_cast<const float4*>(S + ((long long)sl * d.D + c0) * d.N);
#pragma unroll
                for (int i = 0; i < kStepFour; ++i)
                    if (i * 256 + tid < n * nl) copy_async(to + (i * 256 + tid) * 16, from + i * 256 + tid, 16);
                T* rows = reinterpret_cast<T*>(to + states);   // u, delta, z [CT], B, C [4 nl]
                for (int j = tid; j < 3 * (CT / 4) + 2 * nl; j += 256) {
                    const int row = j >> (8 - shift), at = (j & (CT / 4 - 1)) * 4, e = j - 3 * (CT / 4);
                    if (e >= 0)
                        copy_async(rows + j * 4, e < nl ? (const T*)in.Bm + b * d.bs[0] + g * d.bs[2] + 4 * e
                                                        : (const T*)in.C + b * d.cs[0] + g * d.cs[2] + 4 * (e - nl), 4 * sizeof(T));
                    else if (at < n && (row < 2 || in.z))
                        copy_async(rows + j * 4, row == 0 ? (const T*)in.u + b * d.us[0] + c0 + at
                                                 : row == 1 ? (const T*)in.delta + b * d.ds[0] + c0 + at : (const T*)in.z + b * d.zs[0] + c0 + at,
                                   4 * sizeof(T));
                }
            }
            next = place(k + 1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k < kStepStages - 1; ++k) issue(k);
    for (int k = 0; k < count; ++k) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStepStages - 2) : "memory");
        __syncthreads();   // (the stage is whole, and the one before it free)
        issue(k + kStepStages - 1);
        const long long b = blockIdx.x + (long long)k * gridDim.x;
        const unsigned char* from = ring + (k % kStepStages) * stage;
        const T* rows = reinterpret_cast<const T*>(from + states);
        const int sl = s_slot[k % kStepStages];
        if (sl < 0) {
            for (int c = tid; c < n; c += 256) st_elem(y + b * d.ys[0] + c0 + c, 0.f);
            continue;
        }
        const int q = tid & (nl - 1);
        const float4 Bv = as4(*reinterpret_cast<const Vec<T, 4>*>(rows + 3 * CT + 4 * q)),
                     Cv = as4(*reinterpret_cast<const Vec<T, 4>*>(rows + 3 * CT + 4 * (nl + q)));
        float4* to = reinterpret_cast<float4*>(S + ((long long)sl * d.D + c0) * d.N);
        float acc[kStepFour];
#pragma unroll
        for (int i = 0; i < kStepFour; ++i) {
            const int f = i * 256 + tid, c = min(f >> shift, n - 1);
            float4 h = *reinterpret_cast<const float4*>(from + f * 16);
            acc[i] = step4(step_of(d, (float)rows[CT + c] + bias[i]), (float)rows[c], a0[i], a1[i], h, Bv, Cv);
            if (f < n * nl) to[f] = h;
        }
#pragma unroll
        for (int i = 0; i < kStepFour; ++i) {
            const int c = (i * 256 + tid) >> shift;
            for (int o = nl / 2; o > 0; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (q == 0 && c < n) {
                acc[i] = fmaf(skip[i], (float)rows[c], acc[i]);
                if (in.z) acc[i] *= silu_of((float)rows[2 * CT + c]);
                st_elem(y + b * d.ys[0] + c0 + c, acc[i]);
            }
        }
    }
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
    const int nl = state_lanes(d.N), es = sizeof(T), B = d.at.B;
    const long long rows[2] = {d.bs[0], d.bs[2]}, rows_c[2] = {d.cs[0], d.cs[2]};
    const bool wide = d.N % 4 == 0 && ((uintptr_t)S & 15) == 0 && ((uintptr_t)in.A & 15) == 0 &&
                      aligned_rows(in.Bm, rows, B, d.G, 4 * es, es) && aligned_rows(in.C, rows_c, B, d.G, 4 * es, es);
    // the ring: whole groups of four, a tile in one group, and four sequences a CTA at least with two CTAs an SM
    // (256 x 4096 x 16 bf16: 34 us; element by element, one state group a thread, 53).  Six stages are 98 KB plus the token rows:
    // two CTAs share an SM for bf16 from 16 states on and for fp32 from 32, else they follow one another.
    const int CT = 256 * kStepFour / nl, tiles = (d.D + CT - 1) / CT;
    const auto ok = [&](const void* p, const long long (&s)[2]) { return !p || aligned_rows(p, s, B, 1, 4 * es, es); };
    if (wide && d.N == 4 * nl && d.D % 4 == 0 && (d.G == 1 || d.D / d.G % CT == 0) && (long long)tiles * B >= 4 * 2 * kScanSms && tiles <= 2 * kScanSms &&
        ok(in.u, d.us) && ok(in.delta, d.ds) && ok(in.z, d.zs)) {
        const auto bytes = [](int ct, int lanes) { return kStepStages * (256 * kStepFour * 16 + (3 * ct + 8 * lanes) * (int)sizeof(T)); };
        const int smem = bytes(CT, nl);
        // (the most that any N takes, not this call's: another host thread may be between this line and its own launch)
        const cudaError_t e = cudaFuncSetAttribute(k_scan_step_ring<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(256 * kStepFour, 1));
        if (e != cudaSuccess) return e;
        int shift = 0;
        while (1 << shift < nl) ++shift;
        k_scan_step_ring<T><<<dim3(2 * kScanSms / tiles, tiles), 256, smem, st>>>(d, in, S, slots, nslots, (T*)y, shift);
    } else {
        const unsigned grid = (unsigned)(((long long)B * d.D * nl + 255) / 256);
        if (wide) k_scan_step<T, true><<<grid, 256, 0, st>>>(d, in, S, slots, nslots, (T*)y, nl);
        else k_scan_step<T, false><<<grid, 256, 0, st>>>(d, in, S, slots, nslots, (T*)y, nl);
    }
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

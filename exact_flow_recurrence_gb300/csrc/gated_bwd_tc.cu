// gated_bwd_tc.cu -- the gated delta rule's backward on the tcgen05 tensor cores (bf16 tokens).
//
// The formulas of gated_simt.cu's head comment with 64-token chunks, in four kernels:
//   k_gt_prep (gated_tc.cu)  T, P T, decays of every chunk, three bf16 parts
//   k_gt_scan (gated_tc.cu)  recording pass: S entering every chunk and its U, fp32
//   k_gt_rscan               the chunks backwards: G (the gradient of the state that leaves the
//                            chunk) and dX, fp32; dv = alpha dX; dS0
//   k_gt_grad                every chunk at once: dq, dk, dg, dbeta
// dg and dbeta are fp32 results of the whole chain, so every computed operand enters as three
// bf16 parts (about fp32 accuracy); only the last products, which reach dq and dk alone, take two.
//
// dalpha needs the token's residual r_i = v_i - f_i S^T k_i, and U_i = alpha_i r_i: then dalpha_i =
// dX_i . r_i is the diagonal of dX U^T over alpha_i, and neither r nor a second product is kept.
// For this alpha = 0 (beta = 0) is taken as 1e-25, which no fp32 result can tell from 0.
#include "common.cuh"
#include "gated_tc.cuh"
#include "launch.h"

namespace efla {

namespace {

__device__ unsigned int g_gb_status = 0;   // bit 0: a bounded wait expired; kStatusBounds (debug builds): a write was skipped

constexpr int NP = 3;
constexpr float kFloorAlpha = 1e-25f;

// ------------------------------------------------------------------ reverse scan
// As k_gt_scan: one CTA for N columns of a head's G [dk][N], in fp32 registers.  Per chunk:
//   D1 = [K; Q] G  (lanes 0..63: K G);   E = e^c dO as parts (the warps of lanes 64..127)
//   D2 = (P T)^T dO + T^T Y,  Y = e^{c_last - c} K G as parts;   dX = D2
//   D3 = Q^T E + K^T Z,  Z = -alpha e^c dX as parts;   G = e^{c_last} G + D3
constexpr int kRsThreads = 288;

template <int N>
struct RscanSmem {
    static constexpr int BLK = (NP * N + 63) / 64;
    static constexpr uint32_t KQ = 0;                     // 2 stages x 2 blocks x [K rows | Q rows]
    static constexpr uint32_t TP = 65536;                 // [T; P T], NP parts, one stage
    static constexpr uint32_t DO = TP + NP * 16384;       // 2 stages
    static constexpr uint32_t G = DO + 2 * 8192;          // BLK x [128 rows][64]
    static constexpr uint32_t X = G + BLK * 16384;        // BLK x [64 rows][64]: Y, then Z
    static constexpr uint32_t E = X + BLK * 8192;
    static constexpr uint32_t VEC = E + BLK * 8192;       // 2 stages of up, rest, al
    static constexpr uint32_t BAR = VEC + 2 * 768;
    static constexpr size_t bytes = 1024 + BAR + 128;
};
static_assert(RscanSmem<64>::bytes <= 232448, "shared memory per CTA");
static_assert(offsetof(GVec, chi) == 768, "up, rest, al come first");

struct RscanArgs {
    const unsigned char* img;
    const GVec* vec;
    const float* dS_final;
    float* dS0;
    void* dv;
    float* rec_G;    // [H][slots][dk][dv]
    float* rec_dX;   // [H][slots][64][dv]
    int slots;
};

template <int N, typename Tout>
__global__ void __launch_bounds__(kRsThreads, 1) k_gt_rscan(GDims d, RscanArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                            const __grid_constant__ CUtensorMap tm_k,
                                                            const __grid_constant__ CUtensorMap tm_do) {
    using M = RscanSmem<N>;
    constexpr int NC = N / 2, G3 = N == 32 ? NP : 1;   // D3's column groups: tensor memory has room for one at N = 64
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t* full = (uint64_t*)(sm + M::BAR);   // [2]
    uint64_t* full_tp = full + 2;
    uint64_t* g_ready = full + 3;
    uint64_t* e_ready = full + 4;
    uint64_t* y_ready = full + 5;
    uint64_t* z_ready = full + 6;
    uint64_t* d1 = full + 7;
    uint64_t* d2 = full + 8;
    uint64_t* d3 = full + 9;
    uint32_t* tslot = (uint32_t*)(full + 10);
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), c0 = blockIdx.y * N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SeqAt s = seq_at(d, b, kGC);
    const int nch = (s.len + kGC - 1) / kGC;
    const size_t rec0 = (size_t)h * a.slots + s.slot0;
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(full + i, 1);
        mbar_init(g_ready, 8);   // warps
        mbar_init(e_ready, 4);
        mbar_init(y_ready, 4);
        mbar_init(z_ready, 4);
        for (int i = 7; i < 10; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot, t1 = tb, t2 = tb + 192, t3 = tb + 384;

    if (warp == 8) {
        if (lane == 0 && nch > 0) {
            int issued = 0, issued_tp = 0;
            const auto load = [&](int it) {
                const int c = nch - 1 - it, t = s.start + c * kGC;
                unsigned char* kq = sm + M::KQ + (it & 1) * 32768;
                uint64_t* f = &full[it & 1];
                mbar_arrive_expect_tx(f, 5u * 8192u + 768u);
                for (int blk = 0; blk < 2; ++blk) {
                    tma_load_4d(kq + blk * 16384, &tm_k, 64 * blk, t, hk, s.batch, f);
                    tma_load_4d(kq + blk * 16384 + 8192, &tm_q, 64 * blk, t, hk, s.batch, f);
                }
                tma_load_4d(sm + M::DO + (it & 1) * 8192, &tm_do, c0, t, h, s.batch, f);
                bulk_g2s(sm + M::VEC + (it & 1) * 768, a.vec + rec0 + c, 768, f);
                issued = it + 1;
            };
            const auto load_tp = [&](int it) {
                mbar_arrive_expect_tx(full_tp, NP * 16384u);
                bulk_g2s(sm + M::TP, a.img + (rec0 + nch - 1 - it) * NP * 16384, NP * 16384u, full_tp);
                issued_tp = it + 1;
            };
            const int nblk = (d.dk + 63) / 64;
            const uint64_t dG = sdesc_sw128(smem_u32(sm + M::G), 16384), dX = sdesc_sw128(smem_u32(sm + M::X), 8192),
                           dE = sdesc_sw128(smem_u32(sm + M::E), 8192);
            // T^T and (P T)^T: the image's rows are K indices and its 64 columns the product's rows 0..63;
            // rows 64..127 (the next 64 columns, which do not exist) read what follows and are not used
            const uint64_t dT = sdesc_sw128(smem_u32(sm + M::TP), 16384);
            load(0);
            load_tp(0);
            bool ok = true;
            for (int it = 0; it < nch && ok; ++it) {
                const uint32_t ph = it & 1;
                const uint64_t kqK = sdesc_sw128(smem_u32(sm + M::KQ + (it & 1) * 32768));            // K-major
                const uint64_t kqM = sdesc_sw128(smem_u32(sm + M::KQ + (it & 1) * 32768), 16384);     // MN-major
                const uint64_t dDO = sdesc_sw128(smem_u32(sm + M::DO + (it & 1) * 8192));
                ok = mbar_wait(g_ready, ph, kWaitLimit);
                if (!ok) break;
                if (it + 1 < nch) load(it + 1);
                ok = mbar_wait(&full[it & 1], (it >> 1) & 1, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int blk = 0; blk < nblk; ++blk)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t1, kqK + blk * 1024 + ks * 2, dG + blk * 512 + ks * 128,
                                   idesc_f16(128, NP * N, false, true, true), blk + ks > 0);
                mma_commit(d1);
                ok = mbar_wait(full_tp, ph, kWaitLimit) && mbar_wait(e_ready, ph, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                // what does not wait for K G: (P T)^T dO (rows 64..127 of the image, 8 KB in) ...
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ss(t2, dT + (NP - 1) * 1024 + 512 + ks * 128, dDO + ks * 128, idesc_f16(128, N, true, true, true), ks > 0);
#pragma unroll
                for (int p = NP - 2; p >= 0; --p)   // (small parts first: the accumulator cuts off, it does not round)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t2, dT + p * 1024 + 512 + ks * 128, dDO + ks * 128, idesc_f16(128, N, true, true, true), 1u);
                // ... and Q^T E (rows 64..127 of [K; Q])
                if constexpr (G3 == 1) {
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(t3, kqM + 512 + ks * 128, dE + p * 512 + ks * 128, idesc_f16(128, N, true, true, true),
                                       p < NP - 1 || ks > 0);
                } else {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t3, kqM + 512 + ks * 128, dE + ks * 128, idesc_f16(128, NP * N, true, true, true), ks > 0);
                }
                ok = mbar_wait(y_ready, ph, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                // T^T Y into column groups of its own (t2 + N: parts of Y side by side; the first product fills them)
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t2 + N, dT + p * 1024 + ks * 128, dX + ks * 128,
                                   idesc_f16(128, N == 64 && p == 0 ? 2 * N : (NP - p) * N, true, true, true), p + ks > 0);
                if constexpr (N == 64) {   // (two groups fit: T_0 Y_2 joins the first product's columns)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t2, dT + ks * 128, dX + 2 * 512 + ks * 128, idesc_f16(128, N, true, true, true), 1u);
                }
                mma_commit(d2);
                ok = mbar_wait(z_ready, ph, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (it + 1 < nch) load_tp(it + 1);   // (D2 is done: z_ready came from it)
                if constexpr (G3 == 1) {
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(t3, kqM + ks * 128, dX + p * 512 + ks * 128, idesc_f16(128, N, true, true, true), 1u);
                } else {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(t3, kqM + ks * 128, dX + ks * 128, idesc_f16(128, NP * N, true, true, true), 1u);
                }
                mma_commit(d3);
            }
            if (!ok) {   // a wait gave up: the copies under way land before the CTA ends
                atomicOr(&g_gb_status, 1u);
                for (int it = issued > 1 ? issued - 2 : 0; it < issued; ++it)
                    mbar_wait(&full[it & 1], (it >> 1) & 1, kWaitLimit);
                if (issued_tp) mbar_wait(full_tp, (issued_tp - 1) & 1, kWaitLimit);
            }
        }
    } else {
        const int row = 32 * (warp & 3) + lane, half = warp >> 2, cc = half * NC;
        const int i = row & 63;
        const bool top = row < 64;
        const int nv = min(max(d.dv - c0 - cc, 0), NC);
        const size_t sb = ((size_t)blockIdx.x * d.dk + row) * d.dv + c0 + cc;
        const uint32_t lq = 32 * (warp & 3);
        const auto put = [&](uint32_t base, uint32_t blk, int r, int e, const float* x) {
            uint4 w[NP];
            split8<NP>(x, w);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int j = p * N + cc + e;
                *reinterpret_cast<uint4*>(sm + base + (j >> 6) * blk + sw128(r, j & 63)) = w[p];
            }
        };
        // this thread's lane of an accumulator: the sum of GR column groups
        const auto get = [&](uint32_t t, float* y, auto groups) {
            constexpr int GR = decltype(groups)::value;
#pragma unroll
            for (int e = 0; e < NC; e += 16) {
                float x[GR][16];
#pragma unroll
                for (int p = 0; p < GR; ++p) tmem_ld16(taddr(t, lq, p * N + cc + e), x[p]);
                tmem_ld_wait();
#pragma unroll
                for (int p = 0; p < GR; ++p) loaded16(x[p]);
#pragma unroll
                for (int m = 0; m < 16; ++m) {
                    y[e + m] = x[GR - 1][m];
#pragma unroll
                    for (int p = GR - 2; p >= 0; --p) y[e + m] += x[p][m];
                }
            }
        };
        const auto arrive = [&](uint64_t* bar) {
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        const auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, mbar_wait(bar, ph, kWaitLimit)) != 0; };
        float G[NC];
#pragma unroll
        for (int e = 0; e < NC; e += 4) {
            const float4 x = a.dS_final && row < d.dk && e < nv ? *reinterpret_cast<const float4*>(a.dS_final + sb + e)
                                                                : make_float4(0.f, 0.f, 0.f, 0.f);
            G[e] = x.x; G[e + 1] = x.y; G[e + 2] = x.z; G[e + 3] = x.w;
        }
        bool ok = true;
        for (int it = 0; it < nch && ok; ++it) {
            const uint32_t ph = it & 1;
            const int c = nch - 1 - it, n = min(kGC, s.len - c * kGC);
            const float* vec = (const float*)(sm + M::VEC + (it & 1) * 768);
            const unsigned char* dt = sm + M::DO + (it & 1) * 8192;
#pragma unroll
            for (int e = 0; e < NC; e += 8) put(M::G, 16384, row, e, G + e);
            if (d.packed && n < kGC) {   // rows past the sequence are another's: zero them (0 x NaN is not 0)
                ok = wait(&full[it & 1], (it >> 1) & 1);
                unsigned char* kq = sm + M::KQ + (it & 1) * 32768;
                for (int e = tid; e < (kGC - n) * 40; e += 256) {   // five tiles of 64 rows of eight 16-byte chunks
                    const int tile = e % 5, r = n + e / 40, ch = (e / 5) & 7;
                    *reinterpret_cast<uint4*>((tile < 4 ? kq + tile * 8192 : (unsigned char*)dt) + r * 128 + ch * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
            }
            arrive(g_ready);
            if (row < d.dk) {
                float* rg = a.rec_G + ((rec0 + c) * d.dk + row) * d.dv + c0 + cc;
#pragma unroll
                for (int e = 0; e < NC; e += 16)
                    if (e < nv) st16(rg + e, G + e);
            }
            ok = ok && wait(&full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const float up = vec[i], last = vec[63];
            float y[NC];
            if (top) {
                const float rest = vec[64 + i], al = vec[128 + i];
                if (!(ok = wait(d1, ph))) break;
                tc_fence_after();
                get(t1, y, std::integral_constant<int, NP>{});
#pragma unroll
                for (int e = 0; e < NC; e += 8) {
                    float x[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) x[m] = i < n ? rest * y[e + m] : 0.f;
                    put(M::X, 8192, i, e, x);
                }
                arrive(y_ready);
                if (!(ok = wait(d2, ph))) break;
                tc_fence_after();
                get(t2, y, std::integral_constant<int, N == 64 ? 3 : NP + 1>{});
                const float z = -al * up;
#pragma unroll
                for (int e = 0; e < NC; e += 8) {
                    float x[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) x[m] = z * y[e + m];
                    put(M::X, 8192, i, e, x);
                }
                arrive(z_ready);
                float* rx = a.rec_dX + ((rec0 + c) * kGC + i) * d.dv + c0 + cc;
#pragma unroll
                for (int e = 0; e < NC; e += 16)
                    if (e < nv) st16(rx + e, y + e);
                if (i < n) {
                    Tout* vp = (Tout*)a.dv + at3(d.dvs, s.batch, h, s.start + c * kGC + i) + c0 + cc;
#pragma unroll
                    for (int e = 0; e < NC; ++e) y[e] *= al;
#pragma unroll
                    for (int e = 0; e < NC; e += 16)
                        if (e < nv) st16(vp + e, y + e);
                }
            } else {
#pragma unroll
                for (int e = 0; e < NC; e += 8) {
                    const uint4 raw8 = *reinterpret_cast<const uint4*>(dt + sw128(i, cc + e));
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw8);
                    float x[8];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        x[2 * m] = i < n ? up * __uint_as_float(w[m] << 16) : 0.f;
                        x[2 * m + 1] = i < n ? up * __uint_as_float(w[m] & 0xffff0000u) : 0.f;
                    }
                    put(M::E, 8192, i, e, x);
                }
                arrive(e_ready);
            }
            if (!(ok = wait(d3, ph))) break;
            tc_fence_after();
            get(t3, y, std::integral_constant<int, G3>{});
#pragma unroll
            for (int e = 0; e < NC; ++e) G[e] = fmaf(last, G[e], y[e]);
        }
        if (!ok) atomicOr(&g_gb_status, 1u);
        if (a.dS0 && row < d.dk) {
#pragma unroll
            for (int e = 0; e < NC; e += 4)
                if (e < nv) *reinterpret_cast<float4*>(a.dS0 + sb + e) = make_float4(G[e], G[e + 1], G[e + 2], G[e + 3]);
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tb, 512);
}

// ------------------------------------------------------------------ gradients of a chunk
// One chunk of a key head per CTA of 512 threads, its value heads one after another; the value
// columns in slices of 64.  With (dX, U, S, G as three parts)
//   Da = [dO; dX] S^T    D6 = [.; U] G^T    D3 = [dO; dX] U^T    D4 = [Q; K] K^T
//   (lanes 0..63 the first row block, 64..127 the second; every D with M = 128)
//   dPD = lower(D3 D)  and  dAD = -strict_lower(alpha D3 D)  from lanes 0..63 and 64..127
//   D5 = [dPD; dAD] K + [0; dAD^T] K + [0; dPD^T] Q
//   dQ = e^c Da + D5 (lanes 0..63);  dK = -alpha e^c Da + e^{c_last - c} D6 + D5 (lanes 64..127)
// so that a lane is a token: decays scale lanes, and the dot products with q and k that dg needs
// are sums within a thread.
constexpr int kGrThreads = 512;
constexpr uint32_t kGrQK = 0;                    // 2 blocks of 64 dk x [Q rows | K rows]
constexpr uint32_t kGrAX = 32768;                // per 64 columns: dO | dX_0 | 0 | dX_1 | 0 | dX_2, 8 KB each
constexpr uint32_t kGrU = kGrAX + 49152;         // U_0 | U_1 | U_2 (as an A operand, the tile before fills rows 0..63)
constexpr uint32_t kGrS = kGrU + 24576;          // 3 x [128 dk rows][64]; then [dPD; dAD], two parts
constexpr uint32_t kGrG = kGrS + 49152;          // 3 x [128 dk rows][64]
constexpr uint32_t kGrMisc = kGrG + 49152;
constexpr uint32_t kGrZero = kGrAX + 16384;      // a tile of zeros
// tensor-memory columns; D5 lies over D3 and D3s (the small part pairs of D3), which are read before it starts
constexpr uint32_t cDa = 0, cD6 = 128, cD3 = 256, cD3s = 320, cD5 = 256, cD4 = 384;

struct GrMisc {
    GVec vec;
    float be[64], lam[64], da[64], dc[64];
    float rs[4][128];      // row sums of a column group
    float cs[4][64];       // column sums of a lane quadrant
    float dot[4][128];     // per column group: q . dq's, and k . dk's state terms
    float dot2[4][64];     // k . (e^{c_last - c} U G^T)
    float sg[16];
    uint64_t bar;
    uint32_t tslot;
};
constexpr size_t kGrSmem = 1024 + kGrMisc + sizeof(GrMisc);
static_assert(kGrSmem <= 232448, "shared memory per CTA");

struct GradArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k;
    const __nv_bfloat16* dO;
    const float* beta;
    const GVec* vec;
    const float* S;
    const float* U;
    const float* G;
    const float* dX;
    void* dq;
    void* dk;
    float* dg;
    float* dbeta;
    int slots;
};

__device__ __forceinline__ void ld8(const float* p, bool in, float* x) {
    const float4 a = in ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b = in ? __ldg(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// parts of 8 values into a tile's row, the parts `stride` bytes apart
template <int P>
__device__ __forceinline__ void put8(unsigned char* tile, uint32_t stride, int r, int col, const float* x) {
    uint4 w[P];
    split8<P>(x, w);
#pragma unroll
    for (int p = 0; p < P; ++p) *reinterpret_cast<uint4*>(tile + p * stride + sw128(r, col)) = w[p];
}

// Sums over the warp of 16 values a lane: lanes 2m and 2m + 1 return the sum of x[m].
__device__ __forceinline__ float lane_sums16(float (&x)[16], int lane) {
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const bool up = lane & (2 * w);
#pragma unroll
        for (int m = 0; m < w; ++m) {
            const float send = up ? x[m] : x[m + w], keep = up ? x[m + w] : x[m];
            x[m] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * w);
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

template <typename Tout>
__global__ void __launch_bounds__(kGrThreads, 1) k_gt_grad(GDims d, GradArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    GrMisc& m = *reinterpret_cast<GrMisc*>(sm + kGrMisc);
    const int slot = blockIdx.x, hk = blockIdx.y, rep = d.H / d.Hk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = seq_of_slot(d, slot, kGC);
    const SeqAt s = seq_at(d, b, kGC);
    const int t0 = (slot - s.slot0) * kGC, n = min(kGC, s.len - t0), t = s.start + t0;
    if (n <= 0) return;
    const int dk = d.dk, dv = d.dv, nsl = (dv + 63) / 64, nblk = (dk + 63) / 64;

    // one slice of a value head's operands, on its way through registers: 8 columns a task
    struct Slice {
        float S[2][8], G[2][8], U[8], dX[8];
        uint4 dO;
    } x;
    const int r8 = tid >> 3, g8 = (tid & 7) * 8;   // rows r8 and r8 + 64 of S and G, row r8 of the others
    const auto fetch = [&](int h, int sl) {
        const size_t rec = (size_t)h * a.slots + slot;
        const int col = sl * 64 + g8;
        const bool in = col < dv;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const size_t at = (rec * dk + r8 + 64 * k) * dv + col;
            ld8(a.S + at, in && r8 + 64 * k < dk, x.S[k]);
            ld8(a.G + at, in && r8 + 64 * k < dk, x.G[k]);
        }
        const size_t at = (rec * kGC + r8) * dv + col;
        ld8(a.U + at, in, x.U);
        ld8(a.dX + at, in, x.dX);
        x.dO = in && r8 < n ? __ldg(reinterpret_cast<const uint4*>(a.dO + at3(d.dos, s.batch, h, t + r8) + col))
                            : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch(hk * rep, 0);
    if (tid == 0) {
        mbar_init(&m.bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&m.tslot, 512);
        tmem_relinquish();
    }
    for (int e = tid; e < 1024; e += kGrThreads) {   // [Q; K]: 64 rows of 8 chunks, per 64 dk
        const int r = e >> 4, ch = e & 15;
        const bool in = r < n && ch * 8 < dk;
        unsigned char* to = sm + kGrQK + (ch >> 3) * 16384 + sw128(r, (ch & 7) * 8);
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(to) =
            in ? __ldg(reinterpret_cast<const uint4*>(a.q + at3(d.qs, s.batch, hk, t + r) + ch * 8)) : z;
        *reinterpret_cast<uint4*>(to + 8192) =
            in ? __ldg(reinterpret_cast<const uint4*>(a.k + at3(d.ks, s.batch, hk, t + r) + ch * 8)) : z;
        *reinterpret_cast<uint4*>(sm + kGrZero + (e >> 9) * 16384 + (e & 511) * 16) = z;
    }
    uint32_t phase = 0;
    bool ok = true;
    const auto done = [&]() {   // every product so far
        ok = ok && __syncthreads_and(mbar_wait(&m.bar, phase, kWaitLimit));
        phase ^= 1;
        tc_fence_after();
    };
    const int qd = warp & 3, cg = warp >> 2, row = 32 * qd + lane, i = row & 63;
    const bool top = row < 64;
    const uint32_t lq = 32 * qd;
    float acc[32];   // this lane's dq (top) or dk, columns 32 cg .. 32 cg + 31
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
    uint32_t tb = 0;

    for (int h = hk * rep; h < (hk + 1) * rep && ok; ++h) {
        float sg = 0.f;   // <S, G>
        if (h > hk * rep) fetch(h, 0);
        for (int e = tid; e < (int)(sizeof(GVec) / 4); e += kGrThreads)
            reinterpret_cast<float*>(&m.vec)[e] = reinterpret_cast<const float*>(a.vec + (size_t)h * a.slots + slot)[e];
        if (tid < 64) m.be[tid] = tid < n ? a.beta[at3(d.bs, s.batch, h, t + tid)] : 0.f;
        for (int sl = 0; sl < nsl && ok; ++sl) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sg = fmaf(x.S[k][e], x.G[k][e], sg);
                put8<3>(sm + kGrS, 16384, r8 + 64 * k, g8, x.S[k]);
                put8<3>(sm + kGrG, 16384, r8 + 64 * k, g8, x.G[k]);
            }
            put8<3>(sm + kGrU, 8192, r8, g8, x.U);
            put8<3>(sm + kGrAX + 8192, 16384, r8, g8, x.dX);
            *reinterpret_cast<uint4*>(sm + kGrAX + sw128(r8, g8)) = x.dO;
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            tb = m.tslot;
            if (sl + 1 < nsl) fetch(h, sl + 1);
            if (tid == 0) {
                const uint64_t ax = sdesc_sw128(smem_u32(sm + kGrAX)), us = sdesc_sw128(smem_u32(sm + kGrU)),
                               ss = sdesc_sw128(smem_u32(sm + kGrS)), gs = sdesc_sw128(smem_u32(sm + kGrG)),
                               qk = sdesc_sw128(smem_u32(sm + kGrQK));
                if (sl == 0) {
#pragma unroll 1
                    for (int blk = 0; blk < nblk; ++blk)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD4, qk + blk * 1024 + ks * 2, qk + 512 + blk * 1024 + ks * 2,
                                       idesc_f16(128, 64, false, false, true), blk + ks > 0);
                }
                // The accumulators cut off what falls below their last bit, at every instruction: the
                // small part pairs go first (and, for dbeta's D3, into columns of their own), so that
                // few of them meet a large sum.
#pragma unroll
                for (int o = NP - 1; o >= 0; --o)   // pairs (p, y) of order o = p + y
#pragma unroll
                    for (int p = 0; p <= o; ++p)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + (o ? cD3s : cD3), ax + p * 1024 + ks * 2, us + (o - p) * 512 + ks * 2,
                                       idesc_f16(128, 64, false, false, true),
                                       sl > 0 || !((o == NP - 1 || o == 0) && p == 0 && ks == 0));
#pragma unroll
                for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                    for (int p = 0; p <= o; ++p)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cDa, ax + p * 1024 + ks * 2, ss + (o - p) * 1024 + ks * 2,
                                       idesc_f16(128, 128, false, false, true), sl > 0 || !(o == NP - 1 && p == 0 && ks == 0));
#pragma unroll
                for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                    for (int p = 0; p <= o; ++p)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD6, us + p * 512 - 512 + ks * 2, gs + (o - p) * 1024 + ks * 2,
                                       idesc_f16(128, 128, false, false, true), sl > 0 || !(o == NP - 1 && p == 0 && ks == 0));
                mma_commit(&m.bar);
            }
            done();
        }
        if (!ok) break;
        // ---- the chunk's pairs (i, j): columns j = 16 cg .. 16 cg + 15 of this lane's row
        {
            float y[16], z[16], w[16], col[16];
            tmem_ld16(taddr(tb, lq, cD3 + 16 * cg), y);
            tmem_ld16(taddr(tb, lq, cD3s + 16 * cg), w);
            tmem_ld16(taddr(tb, lq, cD4 + 16 * cg), z);
            tmem_ld_wait();
            loaded16(y);
            loaded16(w);
            loaded16(z);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] += w[e];
            const float chi = m.vec.chi[i], clo = m.vec.clo[i], al = m.vec.al[i];
            float rsum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = 16 * cg + e;
                if (!top && j == i) {
                    m.da[i] = i < n ? y[e] / al : 0.f;
                    m.lam[i] = z[e];
                }
                const float D = (top ? j <= i : j < i) && i < n ? decay2(chi, clo, m.vec.chi[j], m.vec.clo[j]) : 0.f;
                w[e] = (top ? j <= i : j < i) && i < n ? (top ? y[e] : -al * y[e]) * D : 0.f;
                col[e] = (top ? j <= i : j < i) && i < n ? w[e] * z[e] : 0.f;
                rsum += col[e];
            }
            put8<2>(sm + kGrS, 16384, row, 16 * cg, w);
            put8<2>(sm + kGrS, 16384, row, 16 * cg + 8, w + 8);
            m.rs[cg][row] = rsum;
            const float c = lane_sums16(col, lane);
            if ((lane & 1) == 0) m.cs[qd][16 * cg + (lane >> 1)] = c;
            sg = warp_sum(sg);
            if (lane == 0) m.sg[warp] = sg;
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (tid == 0) {
            const uint32_t p5 = smem_u32(sm + kGrS), z0 = smem_u32(sm + kGrZero), kq = smem_u32(sm + kGrQK);
            const uint64_t kb = sdesc_sw128(kq + 8192, 16384), qb = sdesc_sw128(kq, 16384);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint64_t a0 = sdesc_sw128(p5 + p * 16384);
                const uint64_t at = sdesc_sw128(z0, p5 + p * 16384 + 8192 - z0);   // [0 | dAD], rows are K indices
                const uint64_t pt = sdesc_sw128(z0, p5 + p * 16384 - z0);          // [0 | dPD]
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ss(tb + cD5, a0 + ks * 2, kb + ks * 128, idesc_f16(128, 128, false, true, true), p + ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ss(tb + cD5, at + ks * 128, kb + ks * 128, idesc_f16(128, 128, true, true, true), 1u);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ss(tb + cD5, pt + ks * 128, qb + ks * 128, idesc_f16(128, 128, true, true, true), 1u);
            }
            mma_commit(&m.bar);
        }
        if (tid < 64) {
            float c = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) c += m.rs[e][tid] + m.rs[e][64 + tid] - m.cs[e][tid];
            m.dc[tid] = c;
        }
        done();
        if (!ok) break;
        // ---- dq, dk: columns 32 cg .. 32 cg + 31 of this lane's token
        {
            const float up = m.vec.up[i], rest = m.vec.rest[i], al = m.vec.al[i];
            const float sa = top ? up : -al * up;
            const float dl = top ? 0.f : 2.f * m.da[i] * dalpha_dlambda_of(m.be[i], m.lam[i], d.euler);
            float dot = 0.f, dot2 = 0.f;
#pragma unroll
            for (int e0 = 0; e0 < 32; e0 += 16) {
                const int c = 32 * cg + e0;
                float da[16], d5[16], d6[16];
                tmem_ld16(taddr(tb, lq, cDa + c), da);
                tmem_ld16(taddr(tb, lq, cD5 + c), d5);
                if (!top) tmem_ld16(taddr(tb, lq, cD6 + c), d6);
                tmem_ld_wait();
                loaded16(da);
                loaded16(d5);
                if (!top) loaded16(d6);
#pragma unroll
                for (int e8 = 0; e8 < 16; e8 += 8) {
                    const uint4 w4 = *reinterpret_cast<const uint4*>(sm + kGrQK + (c >> 6) * 16384 + sw128(row, (c & 63) + e8));
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(&w4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float xk = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
                        const float st = sa * da[e8 + e];
                        float g = st + d5[e8 + e];
                        dot = fmaf(st, xk, dot);
                        if (!top) {
                            const float u = rest * d6[e8 + e];
                            g += fmaf(dl, xk, u);
                            dot2 = fmaf(u, xk, dot2);
                        }
                        acc[e0 + e8 + e] += g;
                    }
                }
            }
            m.dot[cg][row] = dot;
            if (!top) m.dot2[cg][i] = dot2;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {   // dc_i, then its sums to the chunk's end (two tokens a lane)
            float c[2], o2[2], tot = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * lane + e;
                float v = m.dc[j];
                o2[e] = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v += m.dot[k][j] + m.dot[k][64 + j];
                    o2[e] += m.dot2[k][j];
                }
                c[e] = j < n ? v - o2[e] : 0.f;
                tot += j < n ? o2[e] : 0.f;
            }
            tot = warp_sum(tot);
            float g = lane < 16 ? m.sg[lane] : 0.f;
            g = warp_sum(g);
            const float end = fmaf(m.vec.up[63], g, tot);   // everything that decays with the whole chunk
            if (2 * lane == n - 1) c[0] += end;
            if (2 * lane + 1 == n - 1) c[1] += end;
            float sum = c[0] + c[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_down_sync(0xffffffffu, sum, o);
                if (lane + o < 32) sum += y;
            }
            const size_t at = ((size_t)(d.packed ? 0 : b) * d.H + h) * d.L + t;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = 2 * lane + e;
                if (j < n) {
                    a.dg[at + j] = e ? sum - c[0] : sum;
                    a.dbeta[at + j] = m.da[j] * dalpha_dbeta_of(m.be[j], m.lam[j], d.euler);
                }
            }
        }
        __syncthreads();   // the head's vectors and sums are read
    }
    if (!ok) {
        if (tid == 0) {
            atomicOr(&g_gb_status, 1u);
            mbar_wait(&m.bar, phase ^ 1u, kWaitLimit);   // (products still in flight end before their tensor memory is freed)
        }
    } else if (i < n) {
        Tout* p = top ? (Tout*)a.dq + at3(d.dqs, s.batch, hk, t + i) : (Tout*)a.dk + at3(d.dks, s.batch, hk, t + i);
#pragma unroll
        for (int e = 0; e < 32; e += 16)
            if (32 * cg + e < dk) st16(p + 32 * cg + e, acc + e);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(m.tslot, 512);
}

struct BwdTcWs {
    unsigned char* img;
    GVec* vec;
    float *S, *U, *G, *dX;
};

size_t carve(const GDims& d, void* base, BwdTcWs* w) {
    const size_t n = (size_t)d.H * d.slots(kGC);
    char* p = (char*)base;
    const auto take = [&](size_t bytes) {
        char* r = p;
        p += align256(bytes);
        return r;
    };
    w->img = (unsigned char*)take(n * NP * 16384);
    w->vec = (GVec*)take(n * sizeof(GVec));
    w->S = (float*)take(n * d.dk * d.dv * 4);
    w->U = (float*)take(n * kGC * d.dv * 4);
    w->G = (float*)take(n * d.dk * d.dv * 4);
    w->dX = (float*)take(n * kGC * d.dv * 4);
    return (size_t)(p - (char*)base);
}

template <int N, typename Tout>
cudaError_t rscan(const GDims& d, const RscanArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mo,
                  cudaStream_t st) {
    constexpr size_t bytes = RscanSmem<N>::bytes;
    cudaError_t e = smem_attr(k_gt_rscan<N, Tout>, bytes);
    if (e != cudaSuccess) return e;
    k_gt_rscan<N, Tout><<<dim3((unsigned)d.BH(), (d.dv + N - 1) / N), kRsThreads, bytes, st>>>(d, a, mq, mk, mo);
    prof_mark("gated_rscan_tc", st);
    return cudaGetLastError();
}

template <typename Tout>
cudaError_t bwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                float* dbeta, float* dS0, void* ws, cudaStream_t st) {
    BwdTcWs w;
    carve(d, ws, &w);
    const int slots = d.slots(kGC), nb = d.packed ? 1 : d.B;
    CUtensorMap mq, mk, mo;
    bool narrow = false;
    cudaError_t e = strided_rows_map(&mq, q, d.dk, d.L, d.Hk, nb, d.qs);
    if (e == cudaSuccess) e = strided_rows_map(&mk, k, d.dk, d.L, d.Hk, nb, d.ks);
    if (e == cudaSuccess) e = strided_rows_map(&mo, dO, d.dv, d.L, d.H, nb, d.dos);
    if (e == cudaSuccess) e = narrow_slices(d, &narrow);
    if (e == cudaSuccess) e = smem_attr(k_gt_grad<Tout>, kGrSmem);
    if (e == cudaSuccess) e = launch_gated_prep_tc(d, q, k, g, beta, kFloorAlpha, w.img, w.vec, st);
    if (e == cudaSuccess) e = launch_gated_record_tc(d, q, k, v, S0, w.img, w.vec, w.S, w.U, st);
    if (e != cudaSuccess) return e;
    const RscanArgs ra{w.img, w.vec, dS_final, dS0, dv, w.G, w.dX, slots};
    e = narrow ? rscan<32, Tout>(d, ra, mq, mk, mo, st) : rscan<64, Tout>(d, ra, mq, mk, mo, st);
    if (e != cudaSuccess) return e;
    using B = __nv_bfloat16;
    const GradArgs ga{(const B*)q, (const B*)k, (const B*)dO, beta, w.vec, w.S, w.U, w.G, w.dX, dq, dk, dg, dbeta, slots};
    k_gt_grad<Tout><<<dim3(slots, d.Hk), kGrThreads, kGrSmem, st>>>(d, ga);
    prof_mark("gated_grad_tc", st);
    return cudaGetLastError();
}

}  // namespace

size_t gated_tc_bwd_ws_bytes(const GDims& d) {
    BwdTcWs w;
    return carve(d, nullptr, &w);
}

cudaError_t launch_gated_bwd_tc(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, const void* dO, const float* dS_final,
                                void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* ws,
                                cudaStream_t st) {
    return d.out_bf16 ? bwd<__nv_bfloat16>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, ws, st)
                      : bwd<float>(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, ws, st);
}

cudaError_t gated_bwd_tc_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_gb_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_gb_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

// gated_tc.cu -- the gated delta rule's forward on the tcgen05 tensor cores (bf16 tokens).
//
// The chunk form of gated_simt.cu with 64-token chunks, in two kernels:
//   k_gt_prep, every chunk at once: T = (I + strict_lower(alpha_i D_ij k_i.k_j))^{-1} and
//     P T (P = lower(D_ij q_i.k_j)), so that U and P U come from one product, as bf16 parts;
//   k_gt_scan, the chunks of a sequence one after another, one CTA for N columns of a head's
//     state, which it keeps in fp32 registers.
#include "common.cuh"
#include "gated_tc.cuh"
#include "launch.h"

namespace efla {

namespace {

__device__ unsigned int g_gt2_status = 0;   // bit 0: a bounded wait expired; kStatusBounds (debug builds): a write was skipped

// ------------------------------------------------------------------ preparation
// One chunk of a value head per CTA of 128 threads:
//   1. the chunk's K and Q rows by TMA into [K; Q] tiles (128 rows);
//   2. one product [K; Q] K^T: lanes 0..63 G = K K^T (its diagonal: lambda), 64..127 Q K^T;
//   3. from the decays: A (fp32, shared memory), and P as bf16 parts in rows 64..127 of the image;
//   4. T = (I + A)^{-1} in place of A (blocked substitution, split tf32: about fp32 accuracy),
//      its parts into rows 0..63 of the image;
//   5. one product [T; P] T, whose lanes 64..127 (P T) replace P's parts;
//   6. the [T; P T] image, NP parts of 128 rows in the operand layout, out by bulk copy.
// Bound by its chain of short dependent steps, not by data: what counts is how many chunks an
// SM has in flight.  The image lies over the dead tiles and T over A, so that four chunks fit.
struct PrepArgs {
    const float* g;
    const float* beta;
    unsigned char* img;   // [H][slots][NP][128 rows x 128 bytes]
    GVec* vec;            // [H][slots]
    int slots;
    float floor_alpha;    // |alpha| below this is taken as it (0: as it is)
};

template <int NP>
struct PrepSmem {
    static constexpr uint32_t IMG = 0;             // the tiles first; the inverse's scratch in its rows 0..63
    static constexpr uint32_t A = NP * 16384;      // [64][kLdA] fp32
    static constexpr uint32_t VEC = A + 64 * kLdA * 4;
    static constexpr uint32_t BAR = VEC + sizeof(GVec);
    static constexpr size_t bytes = 1024 + BAR + 64;
};

template <int NP>
__global__ void __launch_bounds__(128, 4) k_gt_prep(GDims d, PrepArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                    const __grid_constant__ CUtensorMap tm_k) {
    using M = PrepSmem<NP>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const int slot = blockIdx.x, h = blockIdx.y, hk = h / (d.H / d.Hk), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = seq_of_slot(d, slot, kGC);
    const SeqAt s = seq_at(d, b, kGC);
    const int t0 = (slot - s.slot0) * kGC, n = min(kGC, s.len - t0), t = s.start + t0;
    if (n <= 0) return;
    uint64_t* bar = (uint64_t*)(sm + M::BAR);
    uint32_t* tslot = (uint32_t*)(bar + 3);
    GVec* vec = (GVec*)(sm + M::VEC);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&bar[0], 4u * 8192u);
        for (int blk = 0; blk < 2; ++blk) {
            tma_load_4d(sm + blk * 16384, &tm_k, 64 * blk, t, hk, s.batch, &bar[0]);
            tma_load_4d(sm + blk * 16384 + 8192, &tm_q, 64 * blk, t, hk, s.batch, &bar[0]);
        }
    }
    if (warp == 0) {
        tmem_alloc(tslot, 64);
        tmem_relinquish();
    }
    if (warp == 1) {   // sums of the log decays (two tokens a lane), in fp64 until they are two floats
        const int i0 = 2 * lane;
        const double x0 = i0 < n ? (double)log_decay(a.g[at3(d.gs, s.batch, h, t + i0)]) * kLog2e : 0.0;
        const double x1 = i0 + 1 < n ? (double)log_decay(a.g[at3(d.gs, s.batch, h, t + i0 + 1)]) * kLog2e : 0.0;
        double c1 = x0 + x1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, c1, o);
            if (lane >= o) c1 += y;
        }
        const double last = __shfl_sync(0xffffffffu, c1, 31);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const double c = e ? c1 : c1 - x1;
            const float hi = (float)c;
            vec->chi[i0 + e] = hi;
            vec->clo[i0 + e] = (float)(c - (double)hi);
            vec->up[i0 + e] = exp2_fast(hi);
            vec->rest[i0 + e] = exp2_fast((float)(last - c));
        }
    }
    const float beta = tid < n ? a.beta[at3(d.bs, s.batch, h, t + tid)] : 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    if (tid == 0) {
        if (mbar_wait(&bar[0], 0, kWaitLimit)) {
            tc_fence_after();
            const uint64_t x = sdesc_sw128(smem_u32(sm));
#pragma unroll 1
            for (int blk = 0; blk < (d.dk + 63) / 64; ++blk)   // (zeros past dk)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma_f16_ss(tb, x + blk * 1024 + ks * 2, x + blk * 1024 + ks * 2, idesc_f16(128, 64, false, false, true),
                               blk + ks > 0);
            mma_commit(&bar[1]);
        } else {
            atomicOr(&g_gt2_status, 1u);
            mbar_wait(&bar[0], 0, kWaitLimit);   // let the copies land
        }
    }
    bool ok = __syncthreads_and(mbar_wait(&bar[1], 0, kWaitLimit));
    tc_fence_after();
    float* T = (float*)(sm + M::A);
    unsigned char* img = sm + M::IMG;
    if (ok) {
        const int i = tid & 63;   // this lane's token; lanes 0..63 hold A's rows, 64..127 P's
        const int cols = 32 * (warp & 1) + 32;   // columns that the warp's rows reach
        float v[64];
#pragma unroll
        for (int c = 0; c < 64; c += 16)
            tmem_ld16(taddr(tb, warp * 32, c), *reinterpret_cast<float(*)[16]>(v + c));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 64; c += 16) loaded16(v + c);
        const float chi = vec->chi[i], clo = vec->clo[i];
        float scale = 1.f;
        if (tid < 64) {
            float lam = 0.f;
#pragma unroll
            for (int j = 0; j < 64; ++j) lam = j == i ? v[j] : lam;
            scale = i < n ? alpha_of(beta, lam, d.euler) : 0.f;
            if (i < n && fabsf(scale) < a.floor_alpha) scale = a.floor_alpha;
            vec->al[i] = scale;
        }
        const int diag = tid < 64 ? i : i + 1;   // columns below this are kept
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
            if (j < cols) {
                const float4 h4 = *reinterpret_cast<const float4*>(vec->chi + j), l4 = *reinterpret_cast<const float4*>(vec->clo + j);
                v[j] = j < diag && i < n ? scale * decay2(chi, clo, h4.x, l4.x) * v[j] : 0.f;
                v[j + 1] = j + 1 < diag && i < n ? scale * decay2(chi, clo, h4.y, l4.y) * v[j + 1] : 0.f;
                v[j + 2] = j + 2 < diag && i < n ? scale * decay2(chi, clo, h4.z, l4.z) * v[j + 2] : 0.f;
                v[j + 3] = j + 3 < diag && i < n ? scale * decay2(chi, clo, h4.w, l4.w) * v[j + 3] : 0.f;
            } else {
                v[j] = v[j + 1] = v[j + 2] = v[j + 3] = 0.f;
            }
        }
        // 64 values as parts into a row of the image
        const auto put_row = [&](int r, const float* x) {
#pragma unroll
            for (int j = 0; j < 64; j += 8) {
                uint4 w[NP];
                split8<NP>(x + j, w);
#pragma unroll
                for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(img + p * 16384 + sw128(r, j)) = w[p];
            }
        };
        if (tid < 64) {
#pragma unroll
            for (int j = 0; j < 64; j += 4)
                *reinterpret_cast<float4*>(T + i * kLdA + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        } else {
            put_row(64 + i, v);
        }
        tc_fence_before();
        group_sync(1);
        unit_lower_inverse64(T, T, (float*)img, 1, tid);
        {   // T's parts, 32 columns a thread (zero above its 16x16 diagonal blocks)
            const int r = tid >> 1, h0 = 32 * (tid & 1);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                float x[8];
                const bool in = h0 + j < 16 * (r / 16 + 1);
                const float4 x0 = in ? *reinterpret_cast<const float4*>(T + r * kLd + h0 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 x1 = in ? *reinterpret_cast<const float4*>(T + r * kLd + h0 + j + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                x[0] = x0.x; x[1] = x0.y; x[2] = x0.z; x[3] = x0.w;
                x[4] = x1.x; x[5] = x1.y; x[6] = x1.z; x[7] = x1.w;
                uint4 w[NP];
                split8<NP>(x, w);
#pragma unroll
                for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(img + p * 16384 + sw128(r, h0 + j)) = w[p];
            }
        }
        fence_async_smem();
        tc_fence_before();
        group_sync(1);
        if (tid == 0) {   // [T; P] T, the part pairs p + x < NP (B: T's rows are K indices)
            tc_fence_after();
            const uint64_t da = sdesc_sw128(smem_u32(img));
#pragma unroll
            for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                for (int x = NP - 1 - p; x >= 0; --x)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(tb, da + p * 1024 + ks * 2, da + x * 1024 + ks * 128, idesc_f16(128, 64, false, true, true),
                                   !(p == NP - 1 && x == 0 && ks == 0));
            mma_commit(&bar[2]);
        }
        ok = group_sync_and(1, mbar_wait(&bar[2], 0, kWaitLimit));
        tc_fence_after();
        if (tid >= 64 && ok) {
#pragma unroll
            for (int c = 0; c < 64; c += 16)
                tmem_ld16(taddr(tb, warp * 32, c), *reinterpret_cast<float(*)[16]>(v + c));
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; c += 16) loaded16(v + c);
            put_row(64 + i, v);
            tc_fence_before();
        }
        fence_async_smem();
    }
    if (!ok) {
        atomicOr(&g_gt2_status, 1u);
        mbar_wait(&bar[1], 0, kWaitLimit);   // (products still in flight end before their tensor memory is freed)
        mbar_wait(&bar[2], 0, kWaitLimit);
    }
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && ok) {
        const size_t rec = (size_t)h * a.slots + slot, all = (size_t)d.H * a.slots;
        if (dbg_in(a.img + rec * NP * 16384, NP * 16384, a.img, all * NP * 16384, &g_gt2_status))
            bulk_s2g(a.img + rec * NP * 16384, img, NP * 16384);
        if (dbg_in(a.vec + rec, sizeof(GVec), a.vec, all * sizeof(GVec), &g_gt2_status))
            bulk_s2g(a.vec + rec, vec, sizeof(GVec));
        bulk_commit();
        bulk_wait_read();
    }
    if (warp == 0) tmem_dealloc(tb, 64);
}

// ------------------------------------------------------------------ forward scan
// Per chunk, with S [dk][N] (fp32 registers: 8 warps, thread = row x N/2 columns):
//   S as parts -> shared memory;  D1 = [K; Q] S           (lanes 0..63 K S, 64..127 Q S)
//   X = alpha (V - e^c K S)  as parts;  D2 = [T; P T] X    (U, P U)
//   o = e^c Q S + P U  (the warps of lanes 64..127)
//   U e^{c_last - c} as parts;  D3 = K^T (..);  S = e^{c_last} S + D3
// A ninth warp issues the copies (one chunk ahead) and the products.
constexpr int kScThreads = 288;

template <int NP, int N>
struct ScanSmem {
    static constexpr int TPS = NP == 2 ? 2 : 1;                      // stages of the [T; P T] image
    static constexpr uint32_t KQ = 0;                                // 2 stages x 2 blocks of 64 dk x [K rows | Q rows]
    static constexpr uint32_t TP = 65536;
    static constexpr uint32_t V = TP + TPS * NP * 16384;             // 2 stages
    // part p, column j of an operand is column p N + j: blocks of 64 columns, one after another
    static constexpr int BLK = (NP * N + 63) / 64;
    static constexpr uint32_t S = V + 2 * 8192;                      // BLK x [128 rows][64]
    static constexpr uint32_t X = S + BLK * 16384;                   // BLK x [64 rows][64]
    static constexpr uint32_t VEC = X + BLK * 8192;                  // 2 stages
    static constexpr uint32_t BAR = VEC + 2 * sizeof(GVec);
    static constexpr size_t bytes = 1024 + BAR + 128;
};
static_assert(ScanSmem<2, 64>::bytes <= 232448 && ScanSmem<3, 64>::bytes <= 232448, "shared memory per CTA");

struct ScanArgs {
    const unsigned char* img;
    const GVec* vec;
    const float* S0;
    void* o;
    float* S_final;
    int slots;
    float* rec_S;   // [H][slots][dk][dv]
    float* rec_U;   // [H][slots][64][dv]
};

// REC: the backward's pass, which writes no o but records every chunk's entering state and U (fp32).
template <int NP, int N, typename Tout, bool REC>
__global__ void __launch_bounds__(kScThreads, 1) k_gt_scan(GDims d, ScanArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                           const __grid_constant__ CUtensorMap tm_k,
                                                           const __grid_constant__ CUtensorMap tm_v) {
    using M = ScanSmem<NP, N>;
    constexpr int NC = N / 2;   // columns a thread
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t* full = (uint64_t*)(sm + M::BAR);   // [2] K, Q, V, vectors
    uint64_t* full_tp = full + 2;                // [2]
    uint64_t* s_ready = full + 4;
    uint64_t* x_ready = full + 5;
    uint64_t* u_ready = full + 6;
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
        for (int i = 0; i < 4; ++i) mbar_init(full + i, 1);
        mbar_init(s_ready, 8);   // warps
        mbar_init(x_ready, 4);
        mbar_init(u_ready, 8);
        mbar_init(d1, 1);
        mbar_init(d2, 1);
        mbar_init(d3, 1);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot, t1 = tb, t2 = tb + 256, t3 = tb;   // D3 over D1: every warp has read D1 by then

    if (warp == 8) {
        if (lane == 0 && nch > 0) {
            // ---------------- copies and products
            int issued = 0, issued_tp = 0;   // chunks whose copies are under way
            const auto load = [&](int c) {
                unsigned char* kq = sm + M::KQ + (c & 1) * 32768;
                uint64_t* f = &full[c & 1];
                const int t = s.start + c * kGC;
                mbar_arrive_expect_tx(f, 5u * 8192u + (uint32_t)sizeof(GVec));
                for (int blk = 0; blk < 2; ++blk) {
                    tma_load_4d(kq + blk * 16384, &tm_k, 64 * blk, t, hk, s.batch, f);
                    tma_load_4d(kq + blk * 16384 + 8192, &tm_q, 64 * blk, t, hk, s.batch, f);
                }
                tma_load_4d(sm + M::V + (c & 1) * 8192, &tm_v, c0, t, h, s.batch, f);
                bulk_g2s(sm + M::VEC + (c & 1) * sizeof(GVec), a.vec + rec0 + c, sizeof(GVec), f);
                issued = c + 1;
            };
            const auto load_tp = [&](int c) {
                uint64_t* f = &full_tp[c % M::TPS];
                mbar_arrive_expect_tx(f, NP * 16384u);
                bulk_g2s(sm + M::TP + (c % M::TPS) * NP * 16384, a.img + (rec0 + c) * NP * 16384, NP * 16384u, f);
                issued_tp = c + 1;
            };
            // The products take the operands' parts side by side along N (D keeps a column group for
            // each part of B; the epilogues add them): an instruction costs about 43 cycles up to
            // N = 64, 60 at 128 and 91 at 192, so NP parts in one cost less than NP instructions.
            const int nblk = (d.dk + 63) / 64;
            const uint32_t id_kt = idesc_f16(128, NP * N, true, true, true);   // A, B MN-major
            const uint64_t dS = sdesc_sw128(smem_u32(sm + M::S), 16384), dX = sdesc_sw128(smem_u32(sm + M::X), 8192);
            load(0);
            load_tp(0);
            bool ok = true;
            for (int c = 0; c < nch && ok; ++c) {
                const uint32_t ph = c & 1;
                unsigned char* kq = sm + M::KQ + (c & 1) * 32768;
                ok = mbar_wait(s_ready, ph, kWaitLimit);
                if (!ok) break;
                ok = mbar_wait(&full[c & 1], (c >> 1) & 1, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                {
                    const uint64_t a0 = sdesc_sw128(smem_u32(kq));
#pragma unroll 1
                    for (int blk = 0; blk < nblk; ++blk)   // (64 dk at a time, zeros past dk: no branch per instruction)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(t1, a0 + blk * 1024 + ks * 2, dS + blk * 512 + ks * 128,
                                       idesc_f16(128, NP * N, false, true, true), blk + ks > 0);
                }
                mma_commit(d1);
                if (c + 1 < nch) {   // (the stage's last readers were chunk c - 1's)
                    load(c + 1);
                    if (M::TPS == 2) load_tp(c + 1);
                }
                ok = mbar_wait(&full_tp[c % M::TPS], (c / M::TPS) & 1, kWaitLimit) && mbar_wait(x_ready, ph, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                {
                    const uint64_t a0 = sdesc_sw128(smem_u32(sm + M::TP + (c % M::TPS) * NP * 16384));
#pragma unroll
                    for (int p = 0; p < NP; ++p)   // with the part pairs p + x < NP
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(t2, a0 + p * 1024 + ks * 2, dX + ks * 128,
                                       idesc_f16(128, (NP - p) * N, false, true, true), p + ks > 0);
                }
                mma_commit(d2);
                ok = mbar_wait(u_ready, ph, kWaitLimit);
                if (!ok) break;
                tc_fence_after();
                if (M::TPS == 1 && c + 1 < nch) load_tp(c + 1);   // (D2 is done: u_ready came from it)
                {
                    const uint64_t a0 = sdesc_sw128(smem_u32(kq), 16384);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_f16_ss(t3, a0 + ks * 128, dX + ks * 128, id_kt, ks > 0);
                }
                mma_commit(d3);
            }
            if (!ok) {   // a wait gave up: the copies under way land before the CTA ends
                atomicOr(&g_gt2_status, 1u);
                for (int c = issued > 1 ? issued - 2 : 0; c < issued; ++c) mbar_wait(&full[c & 1], (c >> 1) & 1, kWaitLimit);
                for (int c = issued_tp > M::TPS ? issued_tp - M::TPS : 0; c < issued_tp; ++c)
                    mbar_wait(&full_tp[c % M::TPS], (c / M::TPS) & 1, kWaitLimit);
            }
        }
    } else {
        // ---------------- the state and the epilogues
        const int row = 32 * (warp & 3) + lane, half = warp >> 2, cc = half * NC;   // columns cc .. cc + NC - 1 of the slice
        const int i = row & 63;                                                      // token of lanes 0..63 and of 64..127
        const bool top = row < 64;
        const int nv = min(max(d.dv - c0 - cc, 0), NC);                              // columns of these that exist
        const size_t sb = ((size_t)blockIdx.x * d.dk + row) * d.dv + c0 + cc;
        const uint32_t lq = 32 * (warp & 3);
        // 8 values of `r`, column cc + e of the slice, as parts into an operand of 64-column blocks
        const auto put = [&](uint32_t base, uint32_t blk, int r, int e, const float2* x) {
            uint4 w[NP];
            split8<NP>(x, w);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int j = p * N + cc + e;
                *reinterpret_cast<uint4*>(sm + base + (j >> 6) * blk + sw128(r, j & 63)) = w[p];
            }
        };
        const auto arrive = [&](uint64_t* bar) {   // a warp's shared-memory writes and tensor-memory reads are done
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // (the warp leaves together if a wait gives up)
        const auto wait = [&](uint64_t* bar, uint32_t ph) { return __all_sync(0xffffffffu, mbar_wait(bar, ph, kWaitLimit)) != 0; };
        float2 S[NC / 2];
#pragma unroll
        for (int e = 0; e < NC; e += 4) {
            const float4 x = a.S0 && row < d.dk && e < nv ? *reinterpret_cast<const float4*>(a.S0 + sb + e)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
            S[e / 2] = make_float2(x.x, x.y);
            S[e / 2 + 1] = make_float2(x.z, x.w);
        }
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            const uint32_t ph = c & 1;
            const int n = min(kGC, s.len - c * kGC);
            const GVec* vec = (const GVec*)(sm + M::VEC + (c & 1) * sizeof(GVec));
#pragma unroll
            for (int e = 0; e < NC; e += 8) put(M::S, 16384, row, e, S + e / 2);
            if (d.packed && n < kGC) {   // rows past the sequence are another's: zero its keys (0 x NaN is not 0)
                ok = wait(&full[c & 1], (c >> 1) & 1);
                unsigned char* kq = sm + M::KQ + (c & 1) * 32768;
                for (int e = tid; e < (kGC - n) * 16; e += 256)
                    *reinterpret_cast<uint4*>(kq + (e & 1) * 16384 + (n + (e >> 4)) * 128 + ((e >> 1) & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            arrive(s_ready);
            if (REC && row < d.dk) {
                float* rs = a.rec_S + ((rec0 + c) * d.dk + row) * d.dv + c0 + cc;
#pragma unroll
                for (int e = 0; e < NC; e += 16)
                    if (e < nv) st16(rs + e, S + e / 2);
            }
            ok = ok && wait(&full[c & 1], (c >> 1) & 1);
            if (!ok) break;
            const float up = vec->up[i], last = vec->up[63];
            if (top) {
                // X = alpha V - (alpha e^c) K S; rows past the end are zero whatever lies there
                const bool live = i < n;
                const float2 al = both(vec->al[i]), au = both(-vec->al[i] * up), rest = both(vec->rest[i]);
                const unsigned char* vt = sm + M::V + (c & 1) * 8192;
                float2 v[NC / 2];
#pragma unroll
                for (int e = 0; e < NC; e += 8) {
                    const uint4 w = *reinterpret_cast<const uint4*>(vt + sw128(i, cc + e));
                    v[e / 2] = mul2(al, bf16x2(w.x));
                    v[e / 2 + 1] = mul2(al, bf16x2(w.y));
                    v[e / 2 + 2] = mul2(al, bf16x2(w.z));
                    v[e / 2 + 3] = mul2(al, bf16x2(w.w));
                }
                if (!(ok = wait(d1, ph))) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < NC; e += 16) {
                    float2 y[8];
                    tmem_sum16<NP>(taddr(t1, lq, cc + e), N, y);
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        y[m] = fma2(au, y[m], v[e / 2 + m]);
                        if (!live) y[m] = both(0.f);
                    }
                    put(M::X, 8192, i, e, y);
                    put(M::X, 8192, i, e + 8, y + 4);
                }
                arrive(x_ready);
                if (!(ok = wait(d2, ph))) break;
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < NC; e += 16) {
                    float2 y[8];
                    tmem_sum16<NP>(taddr(t2, lq, cc + e), N, y);
                    if (REC) {
#pragma unroll
                        for (int m = 0; m < 8; ++m) v[e / 2 + m] = y[m];
                    }
#pragma unroll
                    for (int m = 0; m < 8; ++m) y[m] = mul2(rest, y[m]);
                    put(M::X, 8192, i, e, y);
                    put(M::X, 8192, i, e + 8, y + 4);
                }
                arrive(u_ready);
                if (REC) {
                    float* ru = a.rec_U + ((rec0 + c) * kGC + i) * d.dv + c0 + cc;
#pragma unroll
                    for (int e = 0; e < NC; e += 16)
                        if (e < nv) st16(ru + e, v + e / 2);
                }
            } else {
                if (!(ok = wait(d1, ph))) break;
                tc_fence_after();
                float2 qs[NC / 2];
#pragma unroll
                for (int e = 0; e < NC; e += 16) tmem_sum16<NP>(taddr(t1, lq, cc + e), N, *reinterpret_cast<float2(*)[8]>(qs + e / 2));
                arrive(u_ready);
                if (!(ok = wait(d2, ph))) break;
                tc_fence_after();
                if (!REC) {
                    Tout* op = (Tout*)a.o + at3(d.os, s.batch, h, s.start + c * kGC + i) + c0 + cc;
#pragma unroll
                    for (int e = 0; e < NC; e += 16) {
                        float2 y[8];
                        tmem_sum16<NP>(taddr(t2, lq, cc + e), N, y);
#pragma unroll
                        for (int m = 0; m < 8; ++m) y[m] = fma2(both(up), qs[e / 2 + m], y[m]);
                        if (i < n && e < nv) st16(op + e, y);
                    }
                }
            }
            if (!(ok = wait(d3, ph))) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < NC; e += 16) {
                float2 y[8];
                tmem_sum16<NP>(taddr(t3, lq, cc + e), N, y);
#pragma unroll
                for (int m = 0; m < 8; ++m) S[e / 2 + m] = fma2(both(last), S[e / 2 + m], y[m]);
            }
        }
        if (!ok) atomicOr(&g_gt2_status, 1u);
        if (a.S_final && row < d.dk) {
#pragma unroll
            for (int e = 0; e < NC; e += 4)
                if (e < nv) *reinterpret_cast<float4*>(a.S_final + sb + e) =
                        make_float4(S[e / 2].x, S[e / 2].y, S[e / 2 + 1].x, S[e / 2 + 1].y);
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tb, 512);
}

struct TcWs {
    unsigned char* img;
    GVec* vec;
};

size_t carve(const GDims& d, int np, void* base, TcWs* w) {
    const size_t n = (size_t)d.H * d.slots(kGC);
    char* p = (char*)base;
    w->img = (unsigned char*)p;
    p += align256(n * np * 16384);
    w->vec = (GVec*)p;
    p += align256(n * sizeof(GVec));
    return (size_t)(p - (char*)base);
}

struct Maps {
    CUtensorMap q, k, v;
};

cudaError_t make_maps(const GDims& d, const void* q, const void* k, const void* v, Maps* m) {
    const int nb = d.packed ? 1 : d.B;
    cudaError_t e = strided_rows_map(&m->q, q, d.dk, d.L, d.Hk, nb, d.qs);
    if (e == cudaSuccess) e = strided_rows_map(&m->k, k, d.dk, d.L, d.Hk, nb, d.ks);
    if (e == cudaSuccess) e = strided_rows_map(&m->v, v, d.dv, d.L, d.H, nb, d.vs);
    return e;
}

template <int NP, int N, typename Tout, bool REC = false>
cudaError_t scan(const GDims& d, const ScanArgs& a, const Maps& m, cudaStream_t st) {
    constexpr size_t bytes = ScanSmem<NP, N>::bytes;
    cudaError_t e = smem_attr(k_gt_scan<NP, N, Tout, REC>, bytes);
    if (e != cudaSuccess) return e;
    k_gt_scan<NP, N, Tout, REC><<<dim3((unsigned)d.BH(), (d.dv + N - 1) / N), kScThreads, bytes, st>>>(d, a, m.q, m.k, m.v);
    prof_mark(REC ? "gated_record_tc" : "gated_scan_tc", st);
    return cudaGetLastError();
}

template <int NP>
cudaError_t prep(const GDims& d, const PrepArgs& a, const Maps& m, cudaStream_t st) {
    cudaError_t e = smem_attr(k_gt_prep<NP>, PrepSmem<NP>::bytes);
    if (e != cudaSuccess) return e;
    k_gt_prep<NP><<<dim3(a.slots, d.H), 128, PrepSmem<NP>::bytes, st>>>(d, a, m.q, m.k);
    prof_mark("gated_prep_tc", st);
    return cudaGetLastError();
}

template <int NP, typename Tout>
cudaError_t fwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, void* o, float* S_final, void* ws, cudaStream_t st) {
    TcWs w;
    carve(d, NP, ws, &w);
    Maps m{};
    const int slots = d.slots(kGC);
    bool narrow = false;
    cudaError_t e = make_maps(d, q, k, v, &m);
    if (e == cudaSuccess) e = narrow_slices(d, &narrow);
    if (e == cudaSuccess) e = prep<NP>(d, PrepArgs{g, beta, w.img, w.vec, slots, 0.f}, m, st);
    if (e != cudaSuccess) return e;
    const ScanArgs a{w.img, w.vec, S0, o, S_final, slots, nullptr, nullptr};
    return narrow ? scan<NP, 32, Tout>(d, a, m, st) : scan<NP, 64, Tout>(d, a, m, st);
}

}  // namespace

bool gated_tc_supported(const GDims& d) { return d.in_bf16 && d.L > 0; }
size_t gated_tc_fwd_ws_bytes(const GDims& d) {
    TcWs w;
    return carve(d, 3, nullptr, &w);
}

// The outputs' type decides the operands' parts: three where an fp32 result leaves (the state, or
// o in fp32), two where only bf16 does.
cudaError_t launch_gated_fwd_tc(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, void* o, float* S_final, void* ws,
                                cudaStream_t st) {
    if (!d.out_bf16) return fwd<3, float>(d, q, k, v, g, beta, S0, o, S_final, ws, st);
    return S_final ? fwd<3, __nv_bfloat16>(d, q, k, v, g, beta, S0, o, S_final, ws, st)
                   : fwd<2, __nv_bfloat16>(d, q, k, v, g, beta, S0, o, S_final, ws, st);
}

cudaError_t launch_gated_prep_tc(const GDims& d, const void* q, const void* k, const float* g, const float* beta,
                                 float floor_alpha, unsigned char* img, GVec* vec, cudaStream_t st) {
    Maps m{};
    const int nb = d.packed ? 1 : d.B;
    cudaError_t e = strided_rows_map(&m.q, q, d.dk, d.L, d.Hk, nb, d.qs);
    if (e == cudaSuccess) e = strided_rows_map(&m.k, k, d.dk, d.L, d.Hk, nb, d.ks);
    if (e != cudaSuccess) return e;
    return prep<3>(d, PrepArgs{g, beta, img, vec, d.slots(kGC), floor_alpha}, m, st);
}

cudaError_t launch_gated_record_tc(const GDims& d, const void* q, const void* k, const void* v, const float* S0,
                                   const unsigned char* img, const GVec* vec, float* rec_S, float* rec_U,
                                   cudaStream_t st) {
    Maps m{};
    bool narrow = false;
    cudaError_t e = make_maps(d, q, k, v, &m);
    if (e == cudaSuccess) e = narrow_slices(d, &narrow);
    if (e != cudaSuccess) return e;
    const ScanArgs a{img, vec, S0, nullptr, nullptr, d.slots(kGC), rec_S, rec_U};
    return narrow ? scan<3, 32, float, true>(d, a, m, st) : scan<3, 64, float, true>(d, a, m, st);
}

cudaError_t gated_tc_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_gt2_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_gt2_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

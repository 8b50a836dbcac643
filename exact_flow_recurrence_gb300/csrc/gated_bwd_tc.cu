// gated_bwd_tc.cu -- the gated delta rule's backward on the tcgen05 tensor cores (bf16 tokens).
//
// The formulas of gated_simt.cu's head comment with 64-token chunks, in four kernels:
//   k_gt_prep (gated_tc.cu)  T, P T, the residuals' inverse, decays of every chunk, three bf16 parts
//   k_gt_scan (gated_tc.cu)  recording pass: S entering every chunk and its residuals R
//   k_gt_rscan               the chunks backwards: G (the gradient of the state that leaves the
//                            chunk) and dX; dv = alpha dX; dS0
//   k_gt_grad                every chunk at once: dq, dk, dg, dbeta
// Every computed operand enters as three bf16 parts (about fp32 accuracy), whatever the outputs' type.
//
// The two scans need nothing of each other and run side by side where their CTAs find SMs (B7 H8
// T6001 packed, dv 64: 56 CTAs each; the backward takes 0.26 ms, 0.40 ms one after the other).
// The records are the operands of the last kernel as it reads them (parts, swizzled), so that it
// copies and multiplies: 1.5 times the bytes of fp32, and no conversion between copy and product.
//
// dalpha needs the token's residual r_i = v_i - f_i S^T k_i, and everything else U_i = alpha_i r_i.
// R is what is recorded: dalpha_i = dX_i . r_i is the diagonal of dX R^T, alpha scales the columns of
// the other products with it, and a token with alpha = 0 (beta = 0) is one like any other.
#include "common.cuh"
#include "gated_tc.cuh"
#include "launch.h"

#include <initializer_list>

namespace efla {

namespace {

__device__ unsigned int g_gb_status = 0;   // bit 0: a bounded wait expired; kStatusBounds (debug builds): a write was skipped

// ------------------------------------------------------------------ reverse scan
// As k_gt_scan: one CTA for 64 columns of a head's G, two chains of 32 in fp32 registers.  Per
// chunk and chain:
//   D1 = [K; Q] G  (lanes 0..63: K G);   E = e^c dO as parts (the warps of lanes 64..127)
//   D2 = (P T)^T dO + T^T Y,  Y = e^{c_last - c} K G as parts;   dX = D2
//   D3 = Q^T E + K^T Z,  Z = -alpha e^c dX as parts;   G = e^{c_last} G + D3
// dv = alpha dX goes out here.  G's parts, and dX's from a buffer of their own, are copied out as
// they lie in shared memory (a warp of its own does: stored from registers, a row a lane, they
// would hold up the load-store unit for everyone).  Bound as k_gt_scan by its chain: 64 chunks in
// 264 us at B4 H16 L4096 d 128, the tensor pipe 52% and DRAM 38% busy.
struct Rs {
    using C = Chain<2>;
    static constexpr uint32_t K = 0;                      // 2 stages x 2 blocks of 64 dk
    static constexpr uint32_t Q = 32768;                  // 2 blocks
    static constexpr uint32_t DO = Q + 16384;
    static constexpr uint32_t TP = DO + 8192;             // [T; P T], NP parts
    static constexpr uint32_t G = TP + NP * 16384;        // 3 blocks of 128 rows
    static constexpr uint32_t X = G + 3 * 16384;          // 3 blocks of 64 rows: Y, then Z
    static constexpr uint32_t E = X + 3 * 8192;           // likewise
    static constexpr uint32_t R = E + 3 * 8192;           // dX, a tile of 64 rows a part
    static constexpr uint32_t VEC = R + 3 * 8192;         // 2 stages of up, rest, al
    static constexpr uint32_t BAR = VEC + 2 * 768;
    static constexpr int bars = 12 + 2 * 9;
    static constexpr size_t bytes = 1024 + BAR + bars * 8 + 16;
    static constexpr int warps = 20;                      // 16 epilogue, 2 products, copies in, copies out
};
static_assert(Rs::bytes <= 232448, "shared memory per CTA");
static_assert(offsetof(GVec, chi) == 768, "up, rest, al come first");

struct RscanArgs {
    const unsigned char* img;
    const GVec* vec;
    const float* dS_final;
    float* dS0;
    void* dv;
    unsigned char* rec_G;    // [H][slots][slices][kRecS]
    unsigned char* rec_dX;   // [H][slots][slices][kRecT]
    int slots;
};

template <typename Tout>
__global__ void __launch_bounds__(Rs::warps * 32, 1) k_gt_rscan(GDims d, RscanArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                                const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_do) {
    using M = Rs;
    using C = Rs::C;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = (uint64_t*)(sm + M::BAR);
    uint64_t* full = bars;            // [2] K, vectors
    uint64_t* freed = bars + 2;       // [2] by both chains
    uint64_t* full_tp = bars + 4;     // [2] T, P T
    uint64_t* freed_tp = bars + 6;    // [2] by both chains' products
    uint64_t* full_qd = bars + 8;     // Q, dO
    uint64_t* freed_qd = bars + 9;    // by both chains' products
    uint64_t* g_free = bars + 10;     // G's, dX's parts have been copied out
    uint64_t* r_free = bars + 11;
    uint64_t* chain0 = bars + 12;     // per chain: g_ready, y_ready, z_ready, e_ready, d1, d2, d3, turn, r_ready (dX)
    uint32_t* tslot = (uint32_t*)(bars + M::bars);
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), c0 = blockIdx.y * 64;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SeqAt s = seq_at(d, b, kGC);
    const int nch = (s.len + kGC - 1) / kGC;
    const size_t rec0 = (size_t)h * a.slots + s.slot0;
    if (tid == 0) {
        for (int i = 0; i < 12; ++i) {
            const bool two = i == 2 || i == 3 || i == 6 || i == 7 || i == 9;
            mbar_init(&bars[i], two ? 2 : 1);
        }
        for (int g = 0; g < 2; ++g) {
            uint64_t* q = chain0 + 9 * g;
            mbar_init(q, 8);   // warps
            for (int i = 1; i < 4; ++i) mbar_init(q + i, 4);
            for (int i = 4; i < 8; ++i) mbar_init(q + i, 1);
            mbar_init(q + 8, 4);
        }
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    // This kernel reads nothing that the recording pass writes (and the preparation was complete
    // before that pass let it begin), so the two run side by side on the SMs that there are.
    griddep_launch_dependents();

    if (warp >= 16) {
        bool ok = true;
        if (warp >= 18 && lane == 0 && nch > 0) {
            if (warp == 18) {
                // ---------------- copies in (it counts the chunks from the sequence's end)
                int n_k = 0, n_tp[2] = {0, 0}, n_qd = 0;
                const auto load = [&](int it) {
                    const int c = nch - 1 - it;
                    uint64_t* f = &full[it & 1];
                    mbar_arrive_expect_tx(f, 2u * 8192u + 768u);
                    for (int blk = 0; blk < 2; ++blk)
                        tma_load_4d(sm + M::K + (it & 1) * 16384 + blk * 8192, &tm_k, 64 * blk, s.start + c * kGC, hk, s.batch, f);
                    bulk_g2s(sm + M::VEC + (it & 1) * 768, a.vec + rec0 + c, 768, f);
                    n_k = it + 1;
                };
                const auto load_qd = [&](int it) {
                    const int t = s.start + (nch - 1 - it) * kGC;
                    mbar_arrive_expect_tx(full_qd, 3u * 8192u);
                    for (int blk = 0; blk < 2; ++blk) tma_load_4d(sm + M::Q + blk * 8192, &tm_q, 64 * blk, t, hk, s.batch, full_qd);
                    tma_load_4d(sm + M::DO, &tm_do, c0, t, h, s.batch, full_qd);
                    n_qd = it + 1;
                };
                const auto load_tp = [&](int it, int what) {   // T's rows or P T's of every part
                    const unsigned char* from = a.img + (rec0 + nch - 1 - it) * NP * 16384 + what * 8192;
                    mbar_arrive_expect_tx(&full_tp[what], NP * 8192u);
                    for (int p = 0; p < NP; ++p)
                        bulk_g2s(sm + M::TP + p * 16384 + what * 8192, from + p * 16384, 8192u, &full_tp[what]);
                    n_tp[what] = it + 1;
                };
                load(0);
                load_qd(0);
                load_tp(0, 1);
                load_tp(0, 0);
                if (nch > 1) load(1);
                for (int it = 0; it + 1 < nch && ok; ++it) {   // in the order in which the products let go
                    ok = mbar_wait(&freed_tp[1], it & 1, kWaitLimit);
                    if (ok) load_tp(it + 1, 1);
                    ok = ok && mbar_wait(&freed_tp[0], it & 1, kWaitLimit);
                    if (ok) load_tp(it + 1, 0);
                    ok = ok && mbar_wait(freed_qd, it & 1, kWaitLimit);
                    if (ok) load_qd(it + 1);
                    if (ok && it + 2 < nch) {
                        ok = mbar_wait(&freed[it & 1], (it >> 1) & 1, kWaitLimit);
                        if (ok) load(it + 2);
                    }
                }
                if (!ok) {   // a wait gave up: the copies under way land before the CTA ends
                    for (int i = 0; i < 2; ++i) {
                        if (n_k > i) mbar_wait(&full[(n_k - 1 - i) & 1], ((n_k - 1 - i) >> 1) & 1, kWaitLimit);
                        mbar_wait(&full_tp[i], (n_tp[i] - 1) & 1, kWaitLimit);
                    }
                    mbar_wait(full_qd, (n_qd - 1) & 1, kWaitLimit);
                }
            } else {
                // ---------------- copies out
                for (int it = 0; it < nch; ++it) {
                    const uint32_t ph = it & 1;
                    const size_t rec = (rec0 + nch - 1 - it) * gridDim.y + blockIdx.y;
                    ok = mbar_wait(chain0, ph, kWaitLimit) && mbar_wait(chain0 + 9, ph, kWaitLimit);
                    if (!ok) break;
                    if (dbg_in(a.rec_G + rec * kRecS, kRecS, a.rec_G, records(d, a.slots, kRecS), &g_gb_status))
                        bulk_s2g(a.rec_G + rec * kRecS, sm + M::G, kRecS);
                    bulk_commit();
                    bulk_wait_read();   // (and the dX of the chunk before)
                    mbar_arrive(g_free);
                    if (it > 0) mbar_arrive(r_free);
                    ok = mbar_wait(chain0 + 8, ph, kWaitLimit) && mbar_wait(chain0 + 17, ph, kWaitLimit);
                    if (!ok) break;
                    if (dbg_in(a.rec_dX + rec * kRecT, kRecT, a.rec_dX, records(d, a.slots, kRecT), &g_gb_status))
                        bulk_s2g(a.rec_dX + rec * kRecT, sm + M::R, kRecT);
                    bulk_commit();
                }
                bulk_wait_read();
            }
        } else if (warp < 18) {
                // ---------------- a chain's products
                const int g = warp - 16;
                uint64_t* q = chain0 + 9 * g;
                const uint32_t t1 = tb + g * 256, t2 = t1 + 96, t3 = t1;   // D3 over D1, which is read by then
                const int nblk = (d.dk + 63) / 64;
                const bool one = elect_one();
                const uint64_t dG = sdesc_sw128(smem_u32(sm + M::G + g * 16384), C::lbo(g, 16384));
                const uint64_t dX = sdesc_sw128(smem_u32(sm + M::X + g * 8192), C::lbo(g, 8192));
                const uint64_t dE = sdesc_sw128(smem_u32(sm + M::E + g * 8192), C::lbo(g, 8192));
                // T^T and (P T)^T: the image's rows are K indices and its 64 columns the product's rows 0..63; rows
                // 64..127 are the same columns again (a stride of 0), for the warps there to write dX from
                const uint64_t dT = sdesc_sw128(smem_u32(sm + M::TP), 0);
                const uint64_t qm = sdesc_sw128(smem_u32(sm + M::Q), 8192);
                const uint64_t dDO = sdesc_sw128(smem_u32(sm + M::DO)) + g * 4;   // 32 columns in
                constexpr uint32_t kk = idesc_f16(128, NP * 32, false, true, true), m1 = idesc_f16(128, 32, true, true, true),
                                   m3 = idesc_f16(128, NP * 32, true, true, true);
                for (int it = 0; it < nch; ++it) {
                    const uint32_t ph = it & 1;
                    const uint32_t kt = smem_u32(sm + M::K + (it & 1) * 16384);
                    const uint64_t ka = sdesc_sw128(kt), km = sdesc_sw128(kt, 8192);   // (64 rows: 64..127 read what follows)
                    if (!(ok = warp_wait(q, ph) && warp_wait(&full[it & 1], (it >> 1) & 1))) break;
                    if (it > 0 && one) mbar_arrive(&freed[(it - 1) & 1]);
                    if (g == 1) ok = warp_wait(chain0 + 7, ph);   // the chains take turns: see Chain
                    else if (it > 0) ok = warp_wait(chain0 + 16, ph ^ 1u);
                    if (!ok) break;
                    if (one) {
#pragma unroll 1
                        for (int blk = 0; blk < nblk; ++blk)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ss(t1, ka + blk * 512 + ks * 2, dG + blk * 512 + ks * 128, kk, blk + ks > 0);
                        mma_commit(q + 4);
                    }
                    if (!(ok = warp_wait(full_qd, ph) && warp_wait(&full_tp[1], ph))) break;
                    if (one) {
                        // what does not wait for K G: (P T)^T dO (rows 64..127 of the image, 8 KB in), the small parts
                        // first (the accumulator cuts off, it does not round)
#pragma unroll
                        for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ss(t2, dT + p * 1024 + 512 + ks * 128, dDO + ks * 128, m1, p < NP - 1 || ks > 0);
                        mma_commit(&freed_tp[1]);
                    }
                    if (!(ok = warp_wait(&full_tp[0], ph) && warp_wait(q + 1, ph))) break;
                    if (one) {
                        // T^T Y, into column groups of its own
#pragma unroll
                        for (int p = 0; p < NP; ++p)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ss(t2 + 32, dT + p * 1024 + ks * 128, dX + ks * 128,
                                           idesc_f16(128, (NP - p) * 32, true, true, true), p + ks > 0);
                        mma_commit(q + 5);
                        mma_commit(&freed_tp[0]);
                        mbar_arrive(q + 7);
                    }
                    if (!(ok = warp_wait(q + 3, ph))) break;   // (long since)
                    if (one) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)   // Q^T E
                            mma_f16_ss(t3, qm + ks * 128, dE + ks * 128, m3, ks > 0);
                        mma_commit(freed_qd);   // (dO too: its products are over, and E came from it)
                        }
                    if (!(ok = warp_wait(q + 2, ph))) break;
                    if (one) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) mma_f16_ss(t3, km + ks * 128, dX + ks * 128, m3, 1u);
                        mma_commit(q + 6);
                    }
                }
        }
        if (!ok && lane == 0) atomicOr(&g_gb_status, 1u);
    } else {
        const int g = warp >> 3, row = 32 * (warp & 3) + lane, cc = ((warp >> 2) & 1) * 16;
        const int i = row & 63, col = c0 + g * 32 + cc;
        const bool top = row < 64, in = col < d.dv;
        uint64_t* q = chain0 + 9 * g;
        const uint32_t t1 = taddr(tb, 32 * (warp & 3), g * 256 + cc), t2 = t1 + 96, t3 = t1;
        const size_t sb = ((size_t)blockIdx.x * d.dk + row) * d.dv + col;
        float2 G[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float4 x = a.dS_final && row < d.dk && in ? *reinterpret_cast<const float4*>(a.dS_final + sb + 2 * e)
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
            G[e] = make_float2(x.x, x.y);
            G[e + 1] = make_float2(x.z, x.w);
        }
        bool ok = true;
        for (int it = 0; it < nch; ++it) {
            const uint32_t ph = it & 1;
            const int c = nch - 1 - it, n = min(kGC, s.len - c * kGC);
            const float* vec = (const float*)(sm + M::VEC + (it & 1) * 768);
            const unsigned char* dt = sm + M::DO;
            if (it > 0 && !(ok = warp_wait(g_free, ph ^ 1u))) break;
            C::put(sm + M::G, 16384, g, row, cc, G);
            if (d.packed && n < kGC) {   // rows past the sequence are another's: zero them (0 x NaN is not 0)
                if (!(ok = warp_wait(&full[it & 1], (it >> 1) & 1) && warp_wait(full_qd, ph))) break;
                for (int e = tid & 255; e < (kGC - n) * 40; e += 256) {   // five tiles of 64 rows of eight 16-byte chunks
                    const int tile = e % 5, r = n + e / 40, ch = (e / 5) & 7;
                    unsigned char* to = tile < 2 ? sm + M::K + (it & 1) * 16384 + tile * 8192 : sm + M::Q + (tile - 2) * 8192;
                    *reinterpret_cast<uint4*>(to + r * 128 + ch * 16) = make_uint4(0u, 0u, 0u, 0u);   // (dO follows Q)
                }
            }
            warp_arrive(q, lane);
            if (!(ok = warp_wait(&full[it & 1], (it >> 1) & 1))) break;
            const float up = vec[i], last = vec[63];
            const bool live = i < n;
            float2 y[8];
            if (top) {
                const float rest = vec[64 + i], al = vec[128 + i];
                if (!(ok = warp_wait(q + 4, ph))) break;
                tmem_sum<NP>(t1, 32, y);
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = live ? mul2(both(rest), y[m]) : both(0.f);
                C::put(sm + M::X, 8192, g, i, cc, y);
                warp_arrive(q + 1, lane);
                if (!(ok = warp_wait(q + 5, ph))) break;
                tmem_sum<NP + 1>(t2, 32, y);
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = mul2(both(-al * up), y[m]);
                C::put(sm + M::X, 8192, g, i, cc, y);
                warp_arrive(q + 2, lane);
            } else {
                if (!(ok = warp_wait(full_qd, ph))) break;
                const uint4 w0 = *reinterpret_cast<const uint4*>(dt + sw128(i, g * 32 + cc));
                const uint4 w1 = *reinterpret_cast<const uint4*>(dt + sw128(i, g * 32 + cc + 8));
                const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int m = 0; m < 8; ++m) y[m] = live ? mul2(both(up), bf16x2(w[m])) : both(0.f);
                C::put(sm + M::E, 8192, g, i, cc, y);
                warp_arrive(q + 3, lane);
                // dX once more: its record, and dv = alpha dX
                const float al = vec[128 + i];
                if (!(ok = warp_wait(q + 5, ph))) break;
                tmem_sum<NP + 1>(t2, 32, y);
                if (it > 0 && !(ok = warp_wait(r_free, ph ^ 1u))) break;
                put_parts(sm + M::R, i, g * 32 + cc, y);
                warp_arrive(q + 8, lane);
                if (live && in) {
                    Tout* vp = (Tout*)a.dv + at3(d.dvs, s.batch, h, s.start + c * kGC + i) + col;
#pragma unroll
                    for (int m = 0; m < 8; ++m) y[m] = mul2(both(al), y[m]);
                    if (dbg_in(vp, 16 * sizeof(Tout), a.dv, extent(d, d.dvs, d.H, d.dv) * sizeof(Tout), &g_gb_status)) st_row(vp, y);
                }
            }
            if (!(ok = warp_wait(q + 6, ph))) break;
            tmem_sum<NP>(t3, 32, y);
#pragma unroll
            for (int m = 0; m < 8; ++m) G[m] = fma2(both(last), G[m], y[m]);
        }
        if (!ok && lane == 0) atomicOr(&g_gb_status, 1u);
        if (a.dS0 && row < d.dk && in &&
            dbg_in(a.dS0 + sb, 64, a.dS0, (size_t)d.B * d.H * d.dk * d.dv * 4, &g_gb_status))
            st_row(a.dS0 + sb, G);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 16) tmem_dealloc(tb, 512);
    griddep_wait();   // the recording pass ends before this kernel does: what waits for this one waits for both
}

// ------------------------------------------------------------------ gradients of a chunk
// One chunk of a key head at a time, its value heads one after another, the value columns in
// slices of 64; a persistent CTA an SM.  With (dX, R, S, G as three parts)
//   Da = [dO; dX] S^T    D6 = [.; R] G^T    D3 = [dO; dX] R^T    D4 = [Q; K] K^T
//   (lanes 0..63 the first row block, 64..127 the second; every D with M = 128)
//   dPD = lower(D3 alpha_j D)  and  dAD = -strict_lower(alpha_i D3 alpha_j D)  from lanes 0..63 and 64..127
//   D5 = [dPD; dAD] K + [0; dAD^T] K + [0; dPD^T] Q
//   dQ = e^c Da + D5 (lanes 0..63);  dK = -alpha e^c Da + alpha e^{c_last - c} D6 + D5 (lanes 64..127)
// so that a lane is a token: decays scale lanes, and the dot products with q and k that dg needs
// are sums within a thread.
//
// The recorded parts come by bulk copy as the products read them, each kind into a buffer of its
// own that is filled again as soon as its products are done: [dO; dX_0], [0; dX_1], [0; dX_2], R, S,
// G; dO, q and k by TMA.  Warps: 8 epilogue (a lane a token; <S, G> in the products' shadow), one
// that issues products, one that copies.  The epilogue of the pairs runs while the last slice's
// products do.  4096 chunks of two slices: 394 us at B4 H16 L4096, 1.3 GB of records: a head's
// products, pairs, last products and epilogue follow one another, because its accumulators take all
// of the tensor memory and its operands (222 KB) all of shared memory, so only the copies of the next
// head run ahead.  (Of the 394, alpha on the pairs' columns takes 22 and the third part of [dPD; dAD] 17.)
constexpr int kGrWarps = 10;
constexpr uint32_t kGrQK = 0;                    // 2 blocks of 64 dk x [Q rows | K rows]
constexpr uint32_t kGrAX = 32768;                // dO | dX_0 | 0 | dX_1 | 0 | dX_2, tiles of 64 rows
constexpr uint32_t kGrR = kGrAX + 49152;         // R_0 | R_1 | R_2 (as an A operand, the tile before fills rows 0..63)
constexpr uint32_t kGrS = kGrR + 24576;          // 3 blocks of 128 rows: Chain<2>
constexpr uint32_t kGrG = kGrS + 49152;          // likewise
constexpr uint32_t kGrP5 = kGrS;                 // [dPD; dAD], a block of 128 rows a part, in S's place
constexpr uint32_t kGrMisc = kGrG + 49152;
constexpr uint32_t kGrZero = kGrAX + 16384;      // a tile of zeros
// tensor-memory columns; D5 lies over D3 and D3s (the small part pairs of D3), which are read before it starts
constexpr uint32_t cDa = 0, cD6 = 128, cD3 = 256, cD3s = 320, cD5 = 256, cD4 = 384;

struct GrMisc {
    GVec vec;
    float be[64], lam[64], da[64], dc[64];
    float rs[2][128];      // row sums of a column group
    float cs[4][64];       // column sums of a lane quadrant
    float dot[2][128];     // per column group: q . dq's, and k . dk's state terms
    float dot2[2][64];     // k . (alpha e^{c_last - c} R G^T)
    float sg[2][8];        // by the head's parity
    uint64_t f_vec, f_qk, f_ax, f_r, f_s, f_g;   // copies have landed
    uint64_t e_ax, e_r, e_s, e_g;      // products (and <S, G>) have read
    uint64_t d3, d5, p5;               // products; [dPD; dAD]
    uint64_t qk, end;                  // [Q; K] is fit for the products; the epilogue has read everything of the head
    uint32_t tslot;
};
constexpr size_t kGrSmem = 1024 + kGrMisc + sizeof(GrMisc);
static_assert(kGrSmem <= 232448, "shared memory per CTA");
static_assert(sizeof(GVec) % 16 == 0 && kGrMisc % 1024 == 0, "the vectors are copied in place");

struct GradArgs {
    const float* beta;
    const GVec* vec;
    const unsigned char* S;
    const unsigned char* R;
    const unsigned char* G;
    const unsigned char* dX;
    void* dq;
    void* dk;
    float* dg;
    float* dbeta;
    float* acc;    // [CTAs][128][128]: sums over a key head's value heads (null when there is one)
    int slots;
};

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

// The sum of the three parts of 8 columns (chunk j of 16 bytes of half-row g) of a row of S or G.
__device__ __forceinline__ void parts8(const unsigned char* base, int r, int g, int j, float2 (&x)[4]) {
    const uint4 a = *reinterpret_cast<const uint4*>(base + g * 16384 + sw128(r, 8 * j));
    const uint4 b = *reinterpret_cast<const uint4*>(base + g * 16384 + sw128(r, 32 + 8 * j));
    const uint4 c = *reinterpret_cast<const uint4*>(base + 32768 + sw128(r, 32 * g + 8 * j));
    x[0] = add2(bf16x2(a.x), add2(bf16x2(b.x), bf16x2(c.x)));
    x[1] = add2(bf16x2(a.y), add2(bf16x2(b.y), bf16x2(c.y)));
    x[2] = add2(bf16x2(a.z), add2(bf16x2(b.z), bf16x2(c.z)));
    x[3] = add2(bf16x2(a.w), add2(bf16x2(b.w), bf16x2(c.w)));
}

// This thread's share (of 256) of <S, G> over a slice.
__device__ __forceinline__ float inner256(const unsigned char* S, const unsigned char* G, int id) {
    float2 w = both(0.f);
#pragma unroll 2
    for (int e = id; e < 1024; e += 256) {   // rows of eight 8-column chunks
        float2 u[4], v[4];
        parts8(S, e >> 3, (e >> 2) & 1, e & 3, u);
        parts8(G, e >> 3, (e >> 2) & 1, e & 3, v);
#pragma unroll
        for (int x = 0; x < 4; ++x) w = fma2(u[x], v[x], w);
    }
    return w.x + w.y;
}

// Descriptor advance (16-byte units) to part p of column group g in blocks of `blk` bytes: Chain<2>.
__host__ __device__ constexpr uint32_t at_part(int g, int p, uint32_t blk) { return Chain<2>::part(g, p, blk) >> 4; }

template <typename Tout>
__global__ void __launch_bounds__(kGrWarps * 32, 1) k_gt_grad(GDims d, GradArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                              const __grid_constant__ CUtensorMap tm_k,
                                                              const __grid_constant__ CUtensorMap tm_do) {
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    GrMisc& m = *reinterpret_cast<GrMisc*>(sm + kGrMisc);
    const int rep = d.H / d.Hk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dk = d.dk, nsl = (d.dv + 63) / 64, nblk = (dk + 63) / 64;
    const long long items = (long long)a.slots * d.Hk;   // key head fastest: neighbours share a sequence's tokens
    if (tid == 0) {
        for (uint64_t* p : {&m.f_vec, &m.f_qk, &m.f_ax, &m.f_r, &m.f_s, &m.f_g, &m.e_ax, &m.e_r, &m.d3, &m.d5})
            mbar_init(p, 1);
        for (uint64_t* p : {&m.e_s, &m.e_g}) mbar_init(p, 1 + 8);
        for (uint64_t* p : {&m.qk, &m.p5, &m.end}) mbar_init(p, 8);
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&m.tslot, 512);
        tmem_relinquish();
    }
    for (int e = tid; e < 1024; e += kGrWarps * 32)
        *reinterpret_cast<uint4*>(sm + kGrZero + (e >> 9) * 16384 + (e & 511) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = m.tslot;
    griddep_wait();   // the records are complete
    bool ok = true;

    // every role walks the same chunks, value heads and slices; `sc` counts slices, `hc` heads
    uint32_t sc = 0, hc = 0;
    const auto place = [&](long long x, int& hk, int& slot, int& b, SeqAt& s, int& t0) {
        hk = (int)(x % d.Hk);
        slot = (int)(x / d.Hk);
        return chunk_at(d, slot, kGC, b, s, t0);
    };
    if (warp == 9) {
        // ---------------- copies in
        if (lane == 0) {
            uint32_t kc = 0;   // chunks
            const auto ahead = [&](int h, int slot, int sl, int t, int batch) {
                const size_t rec = ((size_t)h * a.slots + slot) * nsl + sl;
                tma_prefetch_4d(&tm_do, 64 * sl, t, h, batch);
                bulk_prefetch_l2(a.dX + rec * kRecT, kRecT);
                bulk_prefetch_l2(a.R + rec * kRecT, kRecT);
                bulk_prefetch_l2(a.S + rec * kRecS, kRecS);
                bulk_prefetch_l2(a.G + rec * kRecS, kRecS);
            };
            for (long long x = blockIdx.x; x < items && ok; x += gridDim.x) {
                int hk, slot, b, t0;
                SeqAt s;
                if (place(x, hk, slot, b, s, t0) <= 0) continue;
                const int t = s.start + t0;
                for (int h = hk * rep; h < (hk + 1) * rep && ok; ++h, ++hc) {
                    for (int sl = 0; sl < nsl && ok; ++sl, ++sc) {
                        const size_t rec = ((size_t)h * a.slots + slot) * nsl + sl;
                        const uint32_t ph = (sc & 1) ^ 1;   // (the first use of a buffer waits for nothing)
                        const auto next = [&](uint64_t* empty, uint64_t* full, uint32_t bytes) {
                            ok = ok && mbar_wait(empty, ph, kWaitLimit);
                            if (ok) mbar_arrive_expect_tx(full, bytes);
                            return ok;
                        };
                        if (!next(&m.e_ax, &m.f_ax, kRecT + 8192)) break;
                        tma_load_4d(sm + kGrAX, &tm_do, 64 * sl, t, h, s.batch, &m.f_ax);
                        for (int p = 0; p < 3; ++p)
                            bulk_g2s(sm + kGrAX + p * 16384 + 8192, a.dX + rec * kRecT + p * 8192, 8192, &m.f_ax);
                        if (!next(&m.e_r, &m.f_r, kRecT)) break;
                        bulk_g2s(sm + kGrR, a.R + rec * kRecT, kRecT, &m.f_r);
                        if (!next(&m.e_s, &m.f_s, kRecS)) break;
                        bulk_g2s(sm + kGrS, a.S + rec * kRecS, kRecS, &m.f_s);
                        if (!next(&m.e_g, &m.f_g, kRecS)) break;
                        bulk_g2s(sm + kGrG, a.G + rec * kRecS, kRecS, &m.f_g);
                        // what the buffers take next comes into L2 meanwhile
                        if (sl + 1 < nsl) {
                            ahead(h, slot, sl + 1, t, s.batch);
                        } else if (h + 1 < (hk + 1) * rep) {
                            ahead(h + 1, slot, 0, t, s.batch);
                        } else {
                            int hk2, slot2, b2, t2;
                            SeqAt s2;
                            if (x + gridDim.x < items && place(x + gridDim.x, hk2, slot2, b2, s2, t2) > 0) {
                                ahead(hk2 * rep, slot2, 0, s2.start + t2, s2.batch);
                                for (int blk = 0; blk < nblk; ++blk) {
                                    tma_prefetch_4d(&tm_q, 64 * blk, s2.start + t2, hk2, s2.batch);
                                    tma_prefetch_4d(&tm_k, 64 * blk, s2.start + t2, hk2, s2.batch);
                                }
                            }
                        }
                        if (sl > 0) continue;
                        // (after what can go ahead of the end of the head before)
                        if (hc > 0) ok = mbar_wait(&m.end, (hc - 1) & 1, kWaitLimit);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&m.f_vec, (uint32_t)sizeof(GVec));
                        bulk_g2s(&m.vec, a.vec + (size_t)h * a.slots + slot, sizeof(GVec), &m.f_vec);
                        if (h == hk * rep) {
                            mbar_arrive_expect_tx(&m.f_qk, 4 * 8192);
                            for (int blk = 0; blk < 2; ++blk) {
                                tma_load_4d(sm + kGrQK + blk * 16384, &tm_q, 64 * blk, t, hk, s.batch, &m.f_qk);
                                tma_load_4d(sm + kGrQK + blk * 16384 + 8192, &tm_k, 64 * blk, t, hk, s.batch, &m.f_qk);
                            }
                            ++kc;
                        }
                    }
                }
            }
            if (!ok) {   // what is under way lands before the CTA ends
                for (uint64_t* p : {&m.f_ax, &m.f_r, &m.f_s, &m.f_g}) mbar_wait(p, sc & 1, kWaitLimit);
                if (kc) mbar_wait(&m.f_qk, (kc - 1) & 1, kWaitLimit);
                mbar_wait(&m.f_vec, hc & 1, kWaitLimit);
            }
        }
    } else if (warp == 8) {
        // ---------------- products
        const bool one = elect_one();
        const uint64_t ax = sdesc_sw128(smem_u32(sm + kGrAX)), rs = sdesc_sw128(smem_u32(sm + kGrR)),
                       ss = sdesc_sw128(smem_u32(sm + kGrS)), gs = sdesc_sw128(smem_u32(sm + kGrG)),
                       qk = sdesc_sw128(smem_u32(sm + kGrQK));
        const uint32_t p5 = smem_u32(sm + kGrP5), z0 = smem_u32(sm + kGrZero), kq = smem_u32(sm + kGrQK);
        const uint64_t kb = sdesc_sw128(kq + 8192, 16384), qb = sdesc_sw128(kq, 16384);
        constexpr uint32_t n64 = idesc_f16(128, 64, false, false, true), n128 = idesc_f16(128, 128, false, false, true);
        uint32_t kc = 0;   // chunks
        for (long long x = blockIdx.x; x < items && ok; x += gridDim.x) {
            int hk, slot, b, t0;
            SeqAt s;
            if (place(x, hk, slot, b, s, t0) <= 0) continue;
            if (!(ok = warp_wait(&m.f_qk, kc++ & 1))) break;
            for (int h = hk * rep; h < (hk + 1) * rep && ok; ++h, ++hc) {
                // [Q; K] is fit, and the epilogue has read the accumulators of the head before
                if (!(ok = warp_wait(&m.qk, hc & 1))) break;
                if (one) {
#pragma unroll 1
                    for (int blk = 0; blk < nblk; ++blk)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD4, qk + blk * 1024 + ks * 2, qk + 512 + blk * 1024 + ks * 2, n64, blk + ks > 0);
                }
                for (int sl = 0; sl < nsl; ++sl, ++sc) {
                    const uint32_t ph = sc & 1, more = sl > 0;
                    if (!(ok = warp_wait(&m.f_ax, ph) && warp_wait(&m.f_r, ph))) break;
                    // The accumulators cut off what falls below their last bit, at every instruction: the small
                    // part pairs go first (and, for dbeta's D3, into columns of their own), so that few of them
                    // meet a large sum.
                    if (one) {
#pragma unroll
                        for (int o = NP - 1; o >= 0; --o)   // pairs (p, o - p) of order o
#pragma unroll
                            for (int p = 0; p <= o; ++p)
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_f16_ss(tb + (o ? cD3s : cD3), ax + p * 1024 + ks * 2, rs + (o - p) * 512 + ks * 2, n64,
                                               more | !((o == NP - 1 || o == 0) && p == 0 && ks == 0));
                        if (sl == nsl - 1) mma_commit(&m.d3);   // the pairs' epilogue can start
                    }
                    if (!(ok = warp_wait(&m.f_s, ph))) break;
                    if (one) {   // (S and G: 32 columns are two steps of K)
#pragma unroll
                        for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                            for (int p = 0; p <= o; ++p)
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_f16_ss(tb + cDa, ax + p * 1024 + ks * 2,
                                               ss + at_part(ks >> 1, o - p, 16384) + (ks & 1) * 2, n128,
                                               more | !(o == NP - 1 && p == 0 && ks == 0));
                        mma_commit(&m.e_ax);
                        if (sl < nsl - 1) mma_commit(&m.e_s);
                    }
                    if (!(ok = warp_wait(&m.f_g, ph))) break;
                    if (one) {
#pragma unroll
                        for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                            for (int p = 0; p <= o; ++p)
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    mma_f16_ss(tb + cD6, rs + p * 512 - 512 + ks * 2,
                                               gs + at_part(ks >> 1, o - p, 16384) + (ks & 1) * 2, n128,
                                               more | !(o == NP - 1 && p == 0 && ks == 0));
                        mma_commit(&m.e_r);
                        mma_commit(&m.e_g);
                    }
                }
                if (!ok || !(ok = warp_wait(&m.p5, hc & 1))) break;
                if (one) {
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p) {   // (q and k are one part)
                        const uint64_t a0 = sdesc_sw128(p5 + p * 16384);
                        const uint64_t at = sdesc_sw128(z0, p5 + p * 16384 + 8192 - z0);   // [0 | dAD], rows are K indices
                        const uint64_t pt = sdesc_sw128(z0, p5 + p * 16384 - z0);          // [0 | dPD]
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD5, a0 + ks * 2, kb + ks * 128, idesc_f16(128, 128, false, true, true), p < NP - 1 || ks > 0);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD5, at + ks * 128, kb + ks * 128, idesc_f16(128, 128, true, true, true), 1u);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(tb + cD5, pt + ks * 128, qb + ks * 128, idesc_f16(128, 128, true, true, true), 1u);
                    }
                    mma_commit(&m.d5);
                    mma_commit(&m.e_s);   // (S's buffer, which held [dPD; dAD])
                }
            }
        }
    } else {
        // ---------------- epilogues: this lane's token, columns 32 cg .. + 31 of the pairs, 64 cg .. + 63 of dq, dk
        const int qd = warp & 3, cg = warp >> 2, row = 32 * qd + lane, i = row & 63;
        const bool top = row < 64;
        const uint32_t lq = taddr(tb, 32 * qd, 0);
        float* my = a.acc ? a.acc + ((size_t)blockIdx.x * 128 + row) * 128 + 64 * cg : nullptr;
        uint32_t kc = 0;   // chunks
        for (long long x = blockIdx.x; x < items && ok; x += gridDim.x, ++kc) {
            int hk, slot, b, t0;
            SeqAt s;
            const int n = place(x, hk, slot, b, s, t0);
            if (n <= 0) {
                --kc;
                continue;
            }
            const int t = s.start + t0;
            for (int h = hk * rep; h < (hk + 1) * rep && ok; ++h, ++hc) {
                const GVec& vec = m.vec;
                const float be = i < n ? __ldg(a.beta + at3(d.bs, s.batch, h, t + i)) : 0.f;
                if (h == hk * rep) {
                    ok = warp_wait(&m.f_qk, kc & 1);
                    if (d.packed && n < kGC)   // rows past the sequence are another's: zero them (0 x NaN is not 0)
                        for (int e = tid; e < (kGC - n) * 32; e += 256)
                            *reinterpret_cast<uint4*>(sm + kGrQK + (e & 3) * 8192 + (n + (e >> 5)) * 128 + ((e >> 2) & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                }
                warp_arrive(&m.qk, lane);
                ok = ok && warp_wait(&m.f_vec, hc & 1);
                // ---- <S, G>, slice by slice (the last one's after the pairs)
                float sg = 0.f;
                const auto inner = [&]() {
                    ok = ok && warp_wait(&m.f_s, sc & 1) && warp_wait(&m.f_g, sc & 1);
                    sg += inner256(sm + kGrS, sm + kGrG, tid);
                    ++sc;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.e_g);
                };
                for (int sl = 0; sl + 1 < nsl; ++sl) {
                    inner();
                    if (lane == 0) mbar_arrive(&m.e_s);   // (the last slice's S buffer goes on to [dPD; dAD])
                }
                // ---- the chunk's pairs (i, j): columns j = 32 cg .. 32 cg + 31 of this lane's row
                ok = ok && warp_wait(&m.d3, hc & 1);
                const float al = vec.al[i], sw = top ? 1.f : -al;
                const int diag = top ? i + 1 : i;                       // columns below this are kept
                const bool some = 32 * cg < 32 * (qd & 1) + 32;         // the warp's rows reach these columns
                float2 w5[16];
                float rsum = 0.f;
                if (some) {
                    const float chi = vec.chi[i], clo = vec.clo[i];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j0 = 32 * cg + 16 * k;
                        float y[16], y2[16], z[16];
                        tmem_ld16(lq + cD3 + j0, y);
                        tmem_ld16(lq + cD3s + j0, y2);
                        tmem_ld16(lq + cD4 + j0, z);
                        float g[16];   // alpha_j times the decays, while the loads are under way
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 h4 = *reinterpret_cast<const float4*>(vec.chi + j0 + e);
                            const float4 l4 = *reinterpret_cast<const float4*>(vec.clo + j0 + e);
                            const float4 a4 = *reinterpret_cast<const float4*>(vec.al + j0 + e);
                            g[e] = a4.x * decay2(chi, clo, h4.x, l4.x);
                            g[e + 1] = a4.y * decay2(chi, clo, h4.y, l4.y);
                            g[e + 2] = a4.z * decay2(chi, clo, h4.z, l4.z);
                            g[e + 3] = a4.w * decay2(chi, clo, h4.w, l4.w);
                        }
                        tmem_ld_wait();
                        loaded16(y);
                        loaded16(y2);
                        loaded16(z);
                        float dg = 0.f, lam = 0.f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const bool keep = j0 + e < diag && i < n;
                            y[e] += y2[e];
                            if (j0 + e == i) {
                                dg = y[e];
                                lam = z[e];
                            }
                            const float w = keep ? sw * y[e] * g[e] : 0.f;
                            (e & 1 ? w5[8 * k + e / 2].y : w5[8 * k + e / 2].x) = w;
                            z[e] = keep && j0 + e < i ? w * z[e] : 0.f;   // (a token's own pair does not decay)
                            rsum += z[e];
                        }
                        if (!top && (i & ~15) == j0) {   // the diagonal: dalpha, and lambda
                            m.da[i] = i < n ? dg : 0.f;
                            m.lam[i] = lam;
                        }
                        const float cs = lane_sums16(z, lane);
                        if ((lane & 1) == 0) m.cs[qd][j0 + (lane >> 1)] = cs;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) w5[k] = both(0.f);
                    if (lane < 32) m.cs[qd][32 * cg + lane] = 0.f;
                }
                m.rs[cg][row] = rsum;
                inner();
                sg = warp_sum(sg);
                if (lane == 0) m.sg[hc & 1][warp] = sg;
                // (S's buffer: the last slice's products have read it, and so has <S, G>)
                ok = ok && warp_wait(&m.e_r, (nsl * (hc + 1) - 1) & 1);   // D6 follows Da
                if (!(ok = group_sync_and(1, ok, 256))) break;                  // (the warps leave together if a wait gave up)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4 w[NP];
                    split8<NP>(w5 + 4 * k, w);
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        *reinterpret_cast<uint4*>(sm + kGrP5 + p * 16384 + sw128(row, 32 * cg + 8 * k)) = w[p];
                }
                warp_arrive(&m.p5, lane);
                if (lane == 0) mbar_arrive(&m.e_s);   // with the products' own arrival after D5: the buffer is free
                if (tid < 64) {
                    float c = 0.f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) c += m.rs[e][tid] + m.rs[e][64 + tid];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c -= m.cs[e][tid];
                    m.dc[tid] = c;
                    m.be[tid] = be;
                }
                const float up = vec.up[i], rest = vec.rest[i];
                const float2 sa = both(top ? up : -al * up), rs2 = both(al * rest);
                const float2 dl = both(top ? 0.f : 2.f * dlambda_of(m.da[i], be, m.lam[i], d.euler));
                float2 dot = both(0.f), dot2 = both(0.f);
                Tout* out = top ? (Tout*)a.dq + at3(d.dqs, s.batch, hk, t + i) : (Tout*)a.dk + at3(d.dks, s.batch, hk, t + i);
                ok = warp_wait(&m.d5, hc & 1);
                // ---- dq, dk: columns 64 cg .. 64 cg + 63 of this lane's token
#pragma unroll 1
                for (int e0 = 0; e0 < 64; e0 += 16) {
                    const int c = 64 * cg + e0;
                    if (c >= dk) break;
                    float da[16], y[16], d6[16];
                    tmem_ld16(lq + cDa + c, da);
                    tmem_ld16(lq + cD5 + c, y);
                    if (!top) tmem_ld16(lq + cD6 + c, d6);
                    uint4* const q0 = reinterpret_cast<uint4*>(sm + kGrQK + (c >> 6) * 16384 + sw128(row, c & 63));
                    uint4* const q1 = reinterpret_cast<uint4*>(sm + kGrQK + (c >> 6) * 16384 + sw128(row, (c & 63) + 8));
                    const uint4 w0 = *q0, w1 = *q1;
                    const uint32_t wk[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                    tmem_ld_wait();
                    loaded16(da);
                    loaded16(y);
                    if (!top) loaded16(d6);
                    float2 o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 xk = bf16x2(wk[e]), st = mul2(sa, make_float2(da[2 * e], da[2 * e + 1]));
                        dot = fma2(st, xk, dot);
                        o[e] = add2(make_float2(y[2 * e], y[2 * e + 1]), st);
                        if (!top) {
                            const float2 u = mul2(rs2, make_float2(d6[2 * e], d6[2 * e + 1]));
                            dot2 = fma2(u, xk, dot2);
                            o[e] = add2(o[e], fma2(dl, xk, u));
                        }
                    }
                    if (my) {   // several value heads: their sum, in fp32
                        if (h > hk * rep) {
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float4 v = *reinterpret_cast<const float4*>(my + e0 + 2 * e);
                                o[e] = add2(o[e], make_float2(v.x, v.y));
                                o[e + 1] = add2(o[e + 1], make_float2(v.z, v.w));
                            }
                        }
                        if (h + 1 < (hk + 1) * rep) st_row(my + e0, o);
                    }
                    if (h + 1 == (hk + 1) * rep) {
                        if constexpr (sizeof(Tout) == 2) {   // (in place of the q or k just read)
                            uint4 v[1];
                            split8<1>(o, v);
                            *q0 = v[0];
                            split8<1>(o + 4, v);
                            *q1 = v[0];
                        } else if (i < n && dbg_in(out + c, 64, top ? a.dq : a.dk,
                                                   extent(d, top ? d.dqs : d.dks, d.Hk, dk) * 4, &g_gb_status)) {
                            st_row(out + c, o);
                        }
                    }
                }
                m.dot[cg][row] = dot.x + dot.y;
                if (!top) m.dot2[cg][i] = dot2.x + dot2.y;
                tc_fence_before();
                if (!(ok = group_sync_and(1, ok, 256))) break;
                if (sizeof(Tout) == 2 && h + 1 == (hk + 1) * rep) {   // whole rows, 16 bytes a lane
                    Tout* const pq = (Tout*)a.dq + at3(d.dqs, s.batch, hk, t);
                    Tout* const pk = (Tout*)a.dk + at3(d.dks, s.batch, hk, t);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = e * 16 + (tid >> 4), ch = tid & 15, j = r & 63;
                        Tout* const to = (e < 4 ? pq + j * d.dqs[2] : pk + j * d.dks[2]) + ch * 8;
                        if (j < n && ch * 8 < dk &&
                            dbg_in(to, 16, e < 4 ? a.dq : a.dk, extent(d, e < 4 ? d.dqs : d.dks, d.Hk, dk) * 2, &g_gb_status))
                            *reinterpret_cast<uint4*>(to) =
                                *reinterpret_cast<const uint4*>(sm + kGrQK + (ch >> 3) * 16384 + sw128(r, (ch & 7) * 8));
                    }
                }
                const float up63 = vec.up[63];
                warp_arrive(&m.end, lane);   // (what warp 0 still reads, the next head writes only after it has come along)
                if (warp == 0) {   // dc_i, then its sums to the chunk's end (two tokens a lane)
                    float c[2], o2[2], tot = 0.f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * lane + e;
                        float v = m.dc[j];
                        o2[e] = 0.f;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            v += m.dot[k][j] + m.dot[k][64 + j];
                            o2[e] += m.dot2[k][j];
                        }
                        if (j >= n - 1) o2[e] = 0.f;   // (the chunk's last token does not decay inside it)
                        c[e] = j < n ? v - o2[e] : 0.f;
                        tot += o2[e];
                    }
                    tot = warp_sum(tot);
                    const float g = warp_sum(lane < 8 ? m.sg[hc & 1][lane] : 0.f);
                    const float end = fmaf(up63, g, tot);   // everything that decays with the whole chunk
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
                        const size_t all = (size_t)(d.packed ? 1 : d.B) * d.H * d.L * 4;
                        if (j < n && dbg_in(a.dg + at + j, 4, a.dg, all, &g_gb_status)) {   // (dbeta: the same places)
                            a.dg[at + j] = e ? sum - c[0] : sum;
                            a.dbeta[at + j] = m.da[j] * dalpha_dbeta_of(m.be[j], m.lam[j], d.euler);
                        }
                    }
                }
            }
        }
        tc_fence_before();
    }
    if (!ok && lane == 0) atomicOr(&g_gb_status, 1u);
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tb, 512);
}

struct BwdTcWs {
    unsigned char *img, *img_r;
    GVec* vec;
    unsigned char *S, *R, *G, *dX;
    float* acc;
};

constexpr int kGrCtas = 152;   // CTAs of the gradient kernel: one an SM

size_t carve(const GDims& d, void* base, BwdTcWs* w) {
    const size_t n = (size_t)d.H * d.slots(kGC), nsl = (d.dv + 63) / 64;
    char* p = (char*)base;
    const auto take = [&](size_t bytes) {
        char* r = p;
        p += align256(bytes);
        return (unsigned char*)r;
    };
    w->img = take(n * NP * 16384);
    w->img_r = take(n * NP * 8192);
    w->vec = (GVec*)take(n * sizeof(GVec));
    w->S = take(n * nsl * kRecS);
    w->R = take(n * nsl * kRecT);
    w->G = take(n * nsl * kRecS);
    w->dX = take(n * nsl * kRecT);
    w->acc = d.H > d.Hk ? (float*)take((size_t)kGrCtas * 128 * 128 * 4) : nullptr;
    return (size_t)(p - (char*)base);
}

template <typename Tout>
cudaError_t bwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dg,
                float* dbeta, float* dS0, void* ws, cudaStream_t st) {
    BwdTcWs w;
    carve(d, ws, &w);
    const int slots = d.slots(kGC), nb = d.packed ? 1 : d.B;
    CUtensorMap mq, mk, mo;
    cudaError_t e = strided_rows_map(&mq, q, d.dk, d.L, d.Hk, nb, d.qs);
    if (e == cudaSuccess) e = strided_rows_map(&mk, k, d.dk, d.L, d.Hk, nb, d.ks);
    if (e == cudaSuccess) e = strided_rows_map(&mo, dO, d.dv, d.L, d.H, nb, d.dos);
    if (e == cudaSuccess) e = smem_attr(k_gt_rscan<Tout>, Rs::bytes);
    if (e == cudaSuccess) e = smem_attr(k_gt_grad<Tout>, kGrSmem);
    if (e == cudaSuccess) e = launch_gated_prep_tc(d, q, k, g, beta, w.img, w.img_r, w.vec, st);
    if (e == cudaSuccess) e = launch_gated_record_tc(d, q, k, v, S0, w.img_r, w.vec, w.S, w.R, st);
    if (e != cudaSuccess) return e;
    const RscanArgs ra{w.img, w.vec, dS_final, dS0, dv, w.G, w.dX, slots};
    e = launch_early(k_gt_rscan<Tout>, dim3((unsigned)d.BH(), (d.dv + 63) / 64), Rs::warps * 32, Rs::bytes, st, d, ra,
                     mq, mk, mo);
    prof_mark("gated_rscan_tc", st);
    if (e != cudaSuccess) return e;
    const GradArgs ga{beta, w.vec, w.S, w.R, w.G, w.dX, dq, dk, dg, dbeta, w.acc, slots};
    const long long items = (long long)slots * d.Hk;
    e = launch_early(k_gt_grad<Tout>, dim3((unsigned)(items < kGrCtas ? items : kGrCtas)), kGrWarps * 32, kGrSmem, st, d,
                     ga, mq, mk, mo);
    prof_mark("gated_grad_tc", st);
    return e;
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

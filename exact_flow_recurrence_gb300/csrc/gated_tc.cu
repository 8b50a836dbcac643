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
//   3. from the decays: A (fp32, shared memory), and P, which stays in registers meanwhile;
//   4. T = (I + A)^{-1} in place of A (blocked substitution, split tf32: about fp32 accuracy),
//      its bf16 parts on their way out by bulk copy; then P's parts in place of A and T;
//   5. one product P T, whose parts replace P's and go out too: the [T; P T] image, NP parts of
//      128 rows in the operand layout.
// The backward also wants the tokens' residuals r = U / alpha, where alpha is zero too.  With A =
// diag(alpha) N they are r = (I + N diag(alpha))^{-1} (V - e^c K S), and that inverse is
// I - N T diag(alpha): N's parts fill the other 64 rows of the product of step 5, and no quotient
// by alpha is formed.  It goes out as an image of its own.  N needs room: three chunks an SM, 4096
// chunks in 121 us.
// Bound by its chain of short dependent steps, not by data: what counts is how many chunks an
// SM has in flight.  P's parts lie over A and T, and both over the dead tiles, so that four
// chunks fit (as many as the registers allow).  With three of them an SM a chunk took 11 us from its
// start: 2.2 us until its tiles were there, 2 us the first product, decays and A, 3.2 us the inverse,
// 1.8 us T's parts, P T and its parts, 1.8 us the copies out.  4096 chunks: 101 us, 15% of the DRAM rate (three
// chunks an SM: 113 us).
constexpr uint32_t kPolls = 1u << 22;   // of a chunk's flag, at 32 ns or more each

struct PrepArgs {
    const float* g;
    const float* beta;
    unsigned char* img;   // [H][slots][NP][128 rows x 128 bytes]
    GVec* vec;            // [H][slots]
    int slots;
    unsigned char* img_r;   // BWD: [H][slots][NP][64 rows x 128 bytes], the residuals' inverse
};

template <bool BWD>
struct PrepSmem {
    static constexpr uint32_t P = 0;               // P's tiles of 64 rows (BWD: [P; N], 128 rows); [64][kLdA] fp32 before
    static constexpr uint32_t PB = BWD ? 16384 : 8192;   // (and the K, Q tiles first): bytes of a part
    static constexpr uint32_t T = NP * PB;         // NP tiles; the inverse's scratch before
    static constexpr uint32_t VEC = T + NP * 8192;
    static constexpr uint32_t BAR = VEC + sizeof(GVec);
    static constexpr size_t bytes = 1024 + BAR + 64;
};

// One chunk, by four warps (named barrier `bid`) whose bars[0..2] count phases `ph` and whose 64 columns
// of tensor memory are at *tslot (valid after the first barrier).  `flag`: set once the results are in global memory.
template <bool BWD>
__device__ bool prep_chunk(const GDims& d, const PrepArgs& a, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                           unsigned char* sm, int bid, int tid, int slot, int h, const SeqAt& s, uint32_t ph,
                           const uint32_t* tslot, int* flag) {
    using M = PrepSmem<BWD>;
    const int hk = h / (d.H / d.Hk), warp = tid >> 5, lane = tid & 31;
    const int t0 = (slot - s.slot0) * kGC, n = min(kGC, s.len - t0), t = s.start + t0;
    uint64_t* bar = (uint64_t*)(sm + M::BAR);
    GVec* vec = (GVec*)(sm + M::VEC);
    if (tid == 0) {
        mbar_arrive_expect_tx(&bar[0], 4u * 8192u);
        for (int blk = 0; blk < 2; ++blk) {
            tma_load_4d(sm + blk * 16384, tm_k, 64 * blk, t, hk, s.batch, &bar[0]);
            tma_load_4d(sm + blk * 16384 + 8192, tm_q, 64 * blk, t, hk, s.batch, &bar[0]);
        }
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
    group_sync(bid);
    if (!flag) griddep_launch_dependents();   // (the scan's CTAs come as SMs run empty)
    tc_fence_after();
    const uint32_t tb = *tslot;
    if (warp == 0) {
        if (warp_wait(&bar[0], ph)) {
            const uint64_t x = sdesc_sw128(smem_u32(sm));
            if (elect_one()) {
#pragma unroll 1
                for (int blk = 0; blk < (d.dk + 63) / 64; ++blk)   // (zeros past dk)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(tb, x + blk * 1024 + ks * 2, x + blk * 1024 + ks * 2, idesc_f16(128, 64, false, false, true),
                                   blk + ks > 0);
                mma_commit(&bar[1]);
            }
        } else if (lane == 0) {
            atomicOr(&g_gt2_status, 1u);
            mbar_wait(&bar[0], ph, kWaitLimit);   // let the copies land
        }
        __syncwarp();
    }
    const size_t rec = (size_t)h * a.slots + slot, all = (size_t)d.H * a.slots;
    unsigned char* const out = a.img + rec * NP * 16384;
    const bool out_ok = dbg_in(out, NP * 16384, a.img, all * NP * 16384, &g_gt2_status);
    bool ok = group_sync_and(bid, mbar_wait(&bar[1], ph, kWaitLimit));
    tc_fence_after();
    float* T = (float*)(sm + M::P);
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
            vec->al[i] = scale;
        }
        const float row = BWD ? 1.f : scale;     // BWD: N first, alpha as A is stored
        const int diag = tid < 64 ? i : i + 1;   // columns below this are kept
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
            if (j < cols) {
                const float4 h4 = *reinterpret_cast<const float4*>(vec->chi + j), l4 = *reinterpret_cast<const float4*>(vec->clo + j);
                v[j] = j < diag && i < n ? row * decay2(chi, clo, h4.x, l4.x) * v[j] : 0.f;
                v[j + 1] = j + 1 < diag && i < n ? row * decay2(chi, clo, h4.y, l4.y) * v[j + 1] : 0.f;
                v[j + 2] = j + 2 < diag && i < n ? row * decay2(chi, clo, h4.z, l4.z) * v[j + 2] : 0.f;
                v[j + 3] = j + 3 < diag && i < n ? row * decay2(chi, clo, h4.w, l4.w) * v[j + 3] : 0.f;
            } else {
                v[j] = v[j + 1] = v[j + 2] = v[j + 3] = 0.f;
            }
        }
        // 64 values as parts into row r of P's tiles
        const auto put_row = [&](int r, const float* x) {
#pragma unroll
            for (int j = 0; j < 64; j += 8) {
                uint4 w[NP];
                split8<NP>(x + j, w);
#pragma unroll
                for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(sm + M::P + p * M::PB + sw128(r, j)) = w[p];
            }
        };
        if (tid < 64) {
            const float al = BWD ? scale : 1.f;
#pragma unroll
            for (int j = 0; j < 64; j += 4)
                *reinterpret_cast<float4*>(T + i * kLdA + j) = make_float4(al * v[j], al * v[j + 1], al * v[j + 2], al * v[j + 3]);
        }
        tc_fence_before();
        group_sync(bid);
        unit_lower_inverse64(T, T, (float*)(sm + M::T), bid, tid);
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
                for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(sm + M::T + p * 8192 + sw128(r, h0 + j)) = w[p];
            }
        }
        fence_async_smem();
        group_sync(bid);
        if (tid == 0 && out_ok)
            for (int p = 0; p < NP; ++p) bulk_s2g(out + p * 16384, sm + M::T + p * 8192, 8192);
        if (BWD || tid >= 64) put_row(BWD ? tid ^ 64 : i, v);   // BWD: P's rows, then N's
        fence_async_smem();
        tc_fence_before();
        group_sync(bid);
        if (warp == 0 && elect_one()) {   // P T (BWD: N T too), the part pairs p + x < NP (B: T's rows are K indices;
            tc_fence_after();             // else rows 64..127 of A are what follows P's tiles, and not used)
            const uint64_t da = sdesc_sw128(smem_u32(sm + M::P)), db = sdesc_sw128(smem_u32(sm + M::T));
#pragma unroll
            for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                for (int x = NP - 1 - p; x >= 0; --x)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_f16_ss(tb, da + p * (M::PB >> 4) + ks * 2, db + x * 512 + ks * 128, idesc_f16(128, 64, false, true, true),
                                   !(p == NP - 1 && x == 0 && ks == 0));
            mma_commit(&bar[2]);
        }
        ok = group_sync_and(bid, mbar_wait(&bar[2], ph, kWaitLimit));
        tc_fence_after();
        if ((BWD || tid < 64) && ok) {
#pragma unroll
            for (int c = 0; c < 64; c += 16)
                tmem_ld16(taddr(tb, warp * 32, c), *reinterpret_cast<float(*)[16]>(v + c));
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 64; c += 16) loaded16(v + c);
            if (BWD && tid >= 64) {   // I - N T diag(alpha)
#pragma unroll
                for (int j = 0; j < 64; ++j) v[j] = fmaf(-vec->al[j], v[j], j == i ? 1.f : 0.f);
            }
            put_row(tid, v);
            tc_fence_before();
        }
        fence_async_smem();
    }
    if (!ok) {
        atomicOr(&g_gt2_status, 1u);
        mbar_wait(&bar[1], ph, kWaitLimit);   // (products still in flight end before their tensor memory is freed)
        mbar_wait(&bar[2], ph, kWaitLimit);
    }
    group_sync(bid);
    tc_fence_after();
    if (tid == 0 && ok) {
        if (out_ok)
            for (int p = 0; p < NP; ++p) bulk_s2g(out + p * 16384 + 8192, sm + M::P + p * M::PB, 8192);
        if constexpr (BWD) {
            unsigned char* const out_r = a.img_r + rec * NP * 8192;
            if (dbg_in(out_r, NP * 8192, a.img_r, all * NP * 8192, &g_gt2_status))
                for (int p = 0; p < NP; ++p) bulk_s2g(out_r + p * 8192, sm + M::P + p * M::PB + 8192, 8192);
        }
        if (dbg_in(a.vec + rec, sizeof(GVec), a.vec, all * sizeof(GVec), &g_gt2_status))
            bulk_s2g(a.vec + rec, vec, sizeof(GVec));
    }
    if (tid == 0) {   // (T's parts are on their way even if a wait has given up since)
        bulk_commit();
        if (flag && ok) {
            bulk_wait_all();
            fence_proxy_async_global();
            st_release_gpu(flag, 1);
        } else {
            bulk_wait_read();
        }
    }
    return ok;
}

template <bool BWD>
__global__ void __launch_bounds__(128, BWD ? 3 : 4) k_gt_prep(GDims d, PrepArgs a, const __grid_constant__ CUtensorMap tm_q,
                                                    const __grid_constant__ CUtensorMap tm_k) {
    using M = PrepSmem<BWD>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const int slot = blockIdx.x, tid = threadIdx.x;
    int b, t0;
    SeqAt s;
    if (chunk_at(d, slot, kGC, b, s, t0) <= 0) return;
    uint64_t* bar = (uint64_t*)(sm + M::BAR);
    uint32_t* tslot = (uint32_t*)(bar + 3);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    if (tid < 32) {
        tmem_alloc(tslot, 64);
        tmem_relinquish();
    }
    prep_chunk<BWD>(d, a, &tm_q, &tm_k, sm, 1, tid, slot, blockIdx.y, s, 0, tslot, nullptr);
    if (tid < 32) tmem_dealloc(*tslot, 64);
}

// ------------------------------------------------------------------ forward scan
// Per chunk and chain, with S [dk][32] in fp32 registers (8 warps, thread = row x 16 columns):
//   S as parts -> shared memory;  D1 = [K; Q] S           (lanes 0..63 K S, 64..127 Q S)
//   X = alpha (V - e^c K S)  as parts;  D2 = [T; P T] X    (U, P U)
//   o = e^c Q S + P U  (the warps of lanes 64..127)
//   U e^{c_last - c} as parts;  D3 = K^T (..);  S = e^{c_last} S + D3
// Each chain has a warp that issues its products; one more copies the chunks in, one ahead.
//
// REC is the backward's recording pass: no queries and no o; the parts of every chunk's entering
// S, and of its residuals R, go out as they lie in shared memory (a warp of its own copies them).
// Its second product is R = (I + N diag(alpha))^{-1} (V - e^c K S), and U = alpha R.  The inverse
// fills both halves of that product, so that the warps of lanes 64..127, which have no queries
// here, can write R's record while the others go on with the chain.
//
// Bound by the latency of the chain of three products and three epilogues a chunk, not by data
// (10 to 30% of the DRAM rate) nor by the tensor pipe (33 to 45% busy).  A chunk of a single chain
// takes about 2.1 us: 0.6 us of products (D1, D2, D3: 8, 12 and 4 instructions of 43 to 50 cycles),
// three times 0.11 us from a commit to the wait that sees it, and three epilogues of 0.3 to 0.4 us
// each (tensor memory to registers, parts to shared memory, the proxy fence).  Twice the epilogue
// warps with half the columns each change nothing: it is fixed latencies.  Two chains of a CTA
// overlap: 3.2 us a chunk for both.  Measured (d 128): B8 H8 L2048 (32 chunks) 102 us; B1 H16
// L16384 (one chain a CTA, 256 chunks) 545 us; the recording pass at B4 H16 L4096 (64 chunks)
// 212 us.  CTAs start in the order of the sequences: packed prompts that do not fit at once take
// longer when a long one comes late (13 of them, 16384 tokens: 226 us longest first, 295 shortest first).
template <int NCH, bool REC>
struct ScanSmem {
    using C = Chain<NCH>;
    static constexpr uint32_t KQB = REC ? 8192 : 16384;              // a 64-dk block: K rows (and Q rows)
    static constexpr uint32_t TPB = 16384;                           // an image part: T rows, P T rows (REC: the inverse twice)
    static constexpr uint32_t KQ = 0;                                // 2 stages x 2 blocks
    static constexpr uint32_t TP = 4 * KQB;
    static constexpr uint32_t V = TP + NP * TPB;                     // 2 stages
    static constexpr uint32_t S = V + 2 * 8192;                      // blocks of 128 rows
    static constexpr uint32_t X = S + C::blocks * 16384;             // blocks of 64 rows
    static constexpr uint32_t R = X + C::blocks * 8192;              // REC: a tile of 64 rows a part
    static constexpr uint32_t VEC = R + (REC ? C::blocks * 8192 : 0);   // 2 stages
    static constexpr uint32_t BAR = VEC + 2 * sizeof(GVec);
    static constexpr int bars = 4 + 2 + 1 + 1 + 9 * NCH;   // (per chain: 7, and its turn)
    static constexpr size_t bytes = 1024 + BAR + bars * 8 + 16;
    // a chain's epilogue warps: a thread has one row and CW of the 32 columns (8 columns: the same times)
    static constexpr int CW = 16;
    static constexpr int EW = 4 * 32 / CW;
    static constexpr int MW = NCH * EW;                      // first product warp
    static constexpr int IW = MW + NCH;                      // copies in, and (REC) out
    static constexpr int warps = IW + 1 + (REC ? 1 : 0);
};
static_assert(ScanSmem<2, false>::bytes <= 232448 && ScanSmem<2, true>::bytes <= 232448, "shared memory per CTA");

struct ScanArgs {
    const unsigned char* img;   // (REC: the residuals' inverse)
    const GVec* vec;
    const float* S0;
    void* o;
    float* S_final;
    int slots;
    unsigned char* rec_S;   // [H][slots][slices][kRecS]
    unsigned char* rec_R;   // [H][slots][slices][kRecT]
    const int* flags;       // [H][slots], or null: set as the chunks' preparations are complete
};

// bx: sequence and value head; by: slice (of `slices`)
template <int NCH, typename Tout, bool REC>
__device__ void scan_cta(const GDims& d, const ScanArgs& a, const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                         const CUtensorMap& tm_v, int bx, int by, int slices) {
    using M = ScanSmem<NCH, REC>;
    using C = Chain<NCH>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = (uint64_t*)(sm + M::BAR);
    uint64_t* full = bars;               // [2] K, Q, V, vectors
    uint64_t* freed = bars + 2;          // [2] by every chain
    uint64_t* full_tp = bars + 4;        // the image
    uint64_t* freed_tp = full_tp + 1;    // by every chain
    uint64_t* s_free = freed_tp + 1;     // REC: S's and R's parts have been copied out
    uint64_t* r_free = s_free + 1;
    uint64_t* chain0 = r_free + 1;       // per chain: s_ready, x_ready, u_ready, r_ready (REC: R's parts), d1, d2, d3, turn
    uint32_t* tslot = (uint32_t*)(bars + M::bars);
    const int b = bx / d.H, h = bx % d.H, hk = h / (d.H / d.Hk), c0 = by * 32 * NCH;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const SeqAt s = seq_at(d, b, kGC);
    const int nch = (s.len + kGC - 1) / kGC;
    const size_t rec0 = (size_t)h * a.slots + s.slot0;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&freed[i], NCH);
        }
        mbar_init(full_tp, 1);
        mbar_init(freed_tp, NCH);
        mbar_init(s_free, 1);
        mbar_init(r_free, 1);
        for (int g = 0; g < NCH; ++g) {
            uint64_t* q = chain0 + 9 * g;
            mbar_init(q + 0, M::EW);                        // s_ready (warps)
            mbar_init(q + 1, M::EW / 2);                    // x_ready
            mbar_init(q + 2, REC ? M::EW / 2 : M::EW);      // u_ready
            mbar_init(q + 3, M::EW / 2);                    // r_ready
            for (int i = 4; i < 8; ++i) mbar_init(q + i, 1);
        }
        fence_mbar_init();
    }
    if (warp == M::MW) {
        tmem_alloc(tslot, NCH * 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = *tslot;
    if (!a.flags) griddep_wait();               // the preparation is complete
    if (REC) griddep_launch_dependents();       // the reverse scan needs it too, but nothing of this kernel's

    if (warp >= M::MW) {
        bool ok = true;
        if (warp >= M::IW && lane == 0 && nch > 0) {
            if (warp == M::IW) {
                // ---------------- copies in
                int n_kq = 0, n_tp = 0;   // chunks whose copies are under way
                const auto prepared = [&](int c) {   // (chunk 0 with patience: its preparation starts as this does)
                    if (!a.flags) return true;
                    const int* f = a.flags + rec0 + c;
                    uint32_t n = 0;
                    while (ld_acquire_gpu(f) == 0 && ++n < kPolls) __nanosleep(32);
                    fence_proxy_async_global();
                    return n < kPolls;
                };
                const auto load = [&](int c) {
                    unsigned char* kq = sm + M::KQ + (c & 1) * 2 * M::KQB;
                    uint64_t* f = &full[c & 1];
                    const int t = s.start + c * kGC;
                    mbar_arrive_expect_tx(f, (REC ? 3u : 5u) * 8192u + (uint32_t)sizeof(GVec));
                    for (int blk = 0; blk < 2; ++blk) {
                        tma_load_4d(kq + blk * M::KQB, &tm_k, 64 * blk, t, hk, s.batch, f);
                        if (!REC) tma_load_4d(kq + blk * M::KQB + 8192, &tm_q, 64 * blk, t, hk, s.batch, f);
                    }
                    tma_load_4d(sm + M::V + (c & 1) * 8192, &tm_v, c0, t, h, s.batch, f);
                    bulk_g2s(sm + M::VEC + (c & 1) * sizeof(GVec), a.vec + rec0 + c, sizeof(GVec), f);
                    n_kq = c + 1;
                };
                const auto load_tp = [&](int c) {
                    unsigned char* to = sm + M::TP;
                    const unsigned char* from = a.img + (rec0 + c) * NP * (REC ? 8192 : 16384);
                    mbar_arrive_expect_tx(full_tp, NP * M::TPB);
                    if (REC) {
                        for (int p = 0; p < 2 * NP; ++p) bulk_g2s(to + p * 8192, from + p / 2 * 8192, 8192, full_tp);
                    } else {
                        bulk_g2s(to, from, NP * M::TPB, full_tp);
                    }
                    n_tp = c + 1;
                };
                ok = prepared(0);
                if (ok) {
                    load(0);
                    load_tp(0);
                }
                if (ok && nch > 1 && (ok = prepared(1))) load(1);
                for (int c = 0; c + 1 < nch && ok; ++c) {
                    ok = mbar_wait(freed_tp, c & 1, kWaitLimit);   // the image's place is free once every chain has chunk c's D2
                    if (ok) load_tp(c + 1);
                    if (ok && c + 2 < nch) {
                        ok = mbar_wait(&freed[c & 1], (c >> 1) & 1, kWaitLimit);
                        ok = ok && prepared(c + 2);
                        if (!ok) break;
                        load(c + 2);
                    }
                }
                if (!ok) {   // a wait gave up: the copies under way land before the CTA ends
                    for (int i = 0; i < 2; ++i)
                        if (n_kq > i) mbar_wait(&full[(n_kq - 1 - i) & 1], ((n_kq - 1 - i) >> 1) & 1, kWaitLimit);
                    if (n_tp > 0) mbar_wait(full_tp, (n_tp - 1) & 1, kWaitLimit);
                }
            } else if (REC && warp == M::IW + 1) {
                // ---------------- copies out
                for (int c = 0; c < nch; ++c) {
                    const uint32_t ph = c & 1;
                    for (int g = 0; g < NCH; ++g) ok = ok && mbar_wait(chain0 + 9 * g, ph, kWaitLimit);
                    if (!ok) break;
                    unsigned char* const to_S = a.rec_S + ((rec0 + c) * slices + by) * kRecS;
                    if (dbg_in(to_S, kRecS, a.rec_S, records(d, a.slots, kRecS), &g_gt2_status)) bulk_s2g(to_S, sm + M::S, kRecS);
                    bulk_commit();
                    bulk_wait_read();   // (and the R of the chunk before)
                    mbar_arrive(s_free);
                    if (c > 0) mbar_arrive(r_free);
                    for (int g = 0; g < NCH; ++g) ok = ok && mbar_wait(chain0 + 9 * g + 3, ph, kWaitLimit);
                    if (!ok) break;
                    unsigned char* const to_R = a.rec_R + ((rec0 + c) * slices + by) * kRecT;
                    if (dbg_in(to_R, kRecT, a.rec_R, records(d, a.slots, kRecT), &g_gt2_status)) bulk_s2g(to_R, sm + M::R, kRecT);
                    bulk_commit();
                }
                bulk_wait_read();
            }
        } else if (warp < M::IW) {
                // ---------------- a chain's products
                const int g = warp - M::MW;
                uint64_t* q = chain0 + 9 * g;
                const uint32_t t1 = tb + g * 256, t2 = t1 + 128, t3 = t1;   // D3 over D1, which is read by then
                const int nblk = (d.dk + 63) / 64;
                const bool one = elect_one();
                const uint64_t dS = sdesc_sw128(smem_u32(sm + M::S + g * 16384), C::lbo(g, 16384));
                const uint64_t dX = sdesc_sw128(smem_u32(sm + M::X + g * 8192), C::lbo(g, 8192));
                const uint64_t ta = sdesc_sw128(smem_u32(sm + M::TP));
                for (int c = 0; c < nch; ++c) {
                    const uint32_t ph = c & 1;
                    const uint32_t kq = smem_u32(sm + M::KQ + (c & 1) * 2 * M::KQB);
                    const uint64_t ka = sdesc_sw128(kq), km = sdesc_sw128(kq, M::KQB);
                    if (!(ok = warp_wait(q, ph) && warp_wait(&full[c & 1], (c >> 1) & 1))) break;
                    if (c > 0 && one) mbar_arrive(&freed[(c - 1) & 1]);   // the chunk before: every product and epilogue is over
                    if (NCH == 2) {   // (the other chain has issued its second product: of this chunk, of the one before)
                        if (g == 1) ok = warp_wait(chain0 + 7, ph);
                        else if (c > 0) ok = warp_wait(chain0 + 16, ph ^ 1u);
                        if (!ok) break;
                    }
                    if (one) {
#pragma unroll 1
                        for (int blk = 0; blk < nblk; ++blk)   // (64 dk at a time, zeros past dk: no branch per instruction)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ss(t1, ka + blk * (M::KQB >> 4) + ks * 2, dS + blk * 512 + ks * 128,
                                           idesc_f16(128, NP * 32, false, true, true), blk + ks > 0);
                        mma_commit(q + 4);
                    }
                    if (!(ok = warp_wait(full_tp, ph) && warp_wait(q + 1, ph))) break;
                    if (one) {
#pragma unroll
                        for (int p = 0; p < NP; ++p)   // with the part pairs p + x < NP
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ss(t2, ta + p * (M::TPB >> 4) + ks * 2, dX + ks * 128,
                                           idesc_f16(128, (NP - p) * 32, false, true, true), p + ks > 0);
                        mma_commit(q + 5);
                        mma_commit(freed_tp);   // (the next image is a long load: as early as can be)
                        if (NCH == 2) mbar_arrive(q + 7);
                    }
                    if (!(ok = warp_wait(q + 2, ph))) break;
                    if (one) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_f16_ss(t3, km + ks * 128, dX + ks * 128, idesc_f16(128, NP * 32, true, true, true), ks > 0);
                        mma_commit(q + 6);
                    }
                }
        }
        if (!ok && lane == 0) atomicOr(&g_gt2_status, 1u);
    } else {
        // ---------------- the state and the epilogues
        constexpr int CW = M::CW;
        const int g = warp / M::EW, row = 32 * (warp & 3) + lane, cc = (warp % M::EW >> 2) * CW;   // CW columns from cc of the chain
        const int i = row & 63, col = c0 + g * 32 + cc;                                            // token of the lane; first column
        const bool top = row < 64, in = col < d.dv;
        uint64_t* q = chain0 + 9 * g;
        const uint32_t lq = taddr(tb, 32 * (warp & 3), g * 256 + cc), t1 = lq, t2 = lq + 128, t3 = lq;
        const size_t sb = ((size_t)bx * d.dk + row) * d.dv + col;
        float2 S[CW / 2];
#pragma unroll
        for (int e = 0; e < CW / 2; e += 2) {
            const float4 x = a.S0 && row < d.dk && in ? *reinterpret_cast<const float4*>(a.S0 + sb + 2 * e)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
            S[e] = make_float2(x.x, x.y);
            S[e + 1] = make_float2(x.z, x.w);
        }
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const uint32_t ph = c & 1;
            const int n = min(kGC, s.len - c * kGC);
            const GVec* vec = (const GVec*)(sm + M::VEC + (c & 1) * sizeof(GVec));
            if (REC && c > 0 && !(ok = warp_wait(s_free, ph ^ 1u))) break;
            C::put(sm + M::S, 16384, g, row, cc, S);
            if (d.packed && n < kGC) {   // rows past the sequence are another's: zero its keys (0 x NaN is not 0)
                if (!(ok = warp_wait(&full[c & 1], (c >> 1) & 1))) break;
                unsigned char* kq = sm + M::KQ + (c & 1) * 2 * M::KQB;
                for (int e = tid % (32 * M::EW); e < (kGC - n) * 16; e += 32 * M::EW)   // (every chain: the same zeros)
                    *reinterpret_cast<uint4*>(kq + (e & 1) * M::KQB + (n + (e >> 4)) * 128 + ((e >> 1) & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            warp_arrive(q, lane);
            if (!(ok = warp_wait(&full[c & 1], (c >> 1) & 1))) break;
            const float up = vec->up[i], last = vec->up[63];
            if (top) {
                // X = alpha V - (alpha e^c) K S (REC: without alpha, which R takes on its way to U); rows past the
                // end are zero whatever lies there
                const bool live = i < n;
                const float xa = REC ? 1.f : vec->al[i], ua = REC ? vec->al[i] * vec->rest[i] : vec->rest[i];
                const float2 al = both(xa), au = both(-xa * up);
                const unsigned char* vt = sm + M::V + (c & 1) * 8192;
                uint4 vw[CW / 8];
#pragma unroll
                for (int e = 0; e < CW / 8; ++e) vw[e] = *reinterpret_cast<const uint4*>(vt + sw128(i, g * 32 + cc + 8 * e));
                if (!(ok = warp_wait(q + 4, ph))) break;
                float2 y[CW / 2];
                tmem_sum<NP>(t1, 32, y);
#pragma unroll
                for (int m = 0; m < CW / 2; ++m) {
                    y[m] = fma2(au, y[m], mul2(al, bf16x2(reinterpret_cast<const uint32_t*>(vw)[m])));
                    if (!live) y[m] = both(0.f);
                }
                C::put(sm + M::X, 8192, g, i, cc, y);
                warp_arrive(q + 1, lane);
                if (!(ok = warp_wait(q + 5, ph))) break;
                tmem_sum<NP>(t2, 32, y);
#pragma unroll
                for (int m = 0; m < CW / 2; ++m) y[m] = mul2(both(ua), y[m]);
                C::put(sm + M::X, 8192, g, i, cc, y);
                warp_arrive(q + 2, lane);
            } else if (REC) {   // R once more: its record
                if (!(ok = warp_wait(q + 5, ph))) break;
                float2 R[CW / 2];
                tmem_sum<NP>(t2, 32, R);
                if (c > 0 && !(ok = warp_wait(r_free, ph ^ 1u))) break;
                put_parts(sm + M::R, i, g * 32 + cc, R);
                warp_arrive(q + 3, lane);
            } else {
                if (!(ok = warp_wait(q + 4, ph))) break;
                float2 y[CW / 2], z[CW / 2];
                tmem_sum<NP>(t1, 32, y);
                warp_arrive(q + 2, lane);
                if (!(ok = warp_wait(q + 5, ph))) break;
                tmem_sum<NP>(t2, 32, z);
#pragma unroll
                for (int m = 0; m < CW / 2; ++m) z[m] = fma2(both(up), y[m], z[m]);
                if (i < n && in) {
                    Tout* op = (Tout*)a.o + at3(d.os, s.batch, h, s.start + c * kGC + i) + col;
                    if (dbg_in(op, CW * sizeof(Tout), a.o, extent(d, d.os, d.H, d.dv) * sizeof(Tout), &g_gt2_status)) st_row(op, z);
                }
            }
            if (!(ok = warp_wait(q + 6, ph))) break;
            float2 y[CW / 2];
            tmem_sum<NP>(t3, 32, y);
#pragma unroll
            for (int m = 0; m < CW / 2; ++m) S[m] = fma2(both(last), S[m], y[m]);
        }
        if (!ok && lane == 0) atomicOr(&g_gt2_status, 1u);
        if (a.S_final && row < d.dk && in &&
            dbg_in(a.S_final + sb, CW * 4, a.S_final, (size_t)d.B * d.H * d.dk * d.dv * 4, &g_gt2_status))
            st_row(a.S_final + sb, S);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == M::MW) tmem_dealloc(tb, NCH * 256);
}

template <int NCH, typename Tout, bool REC>
__global__ void __launch_bounds__((ScanSmem<NCH, REC>::warps * 32), 1)
    k_gt_scan(GDims d, ScanArgs a, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v) {
    scan_cta<NCH, Tout, REC>(d, a, tm_q, tm_k, tm_v, blockIdx.x, blockIdx.y, gridDim.y);
}

// ------------------------------------------------------------------ few heads, many chunks
// The scan's CTAs and, on the other SMs, the chunks' preparation, in one cooperative launch (all CTAs run
// at once, which makes waiting for their flags safe).  Three groups of four warps a preparing CTA take the
// chunks in the order in which the scans come to them.
struct LongSmem {
    static constexpr int groups = 3, threads = 128 * groups;
    static constexpr size_t group = PrepSmem<false>::bytes / 1024 * 1024 + 1024;
    static constexpr size_t scan = ScanSmem<1, false>::bytes;
    static constexpr size_t bytes = groups * group > scan ? groups * group : scan;
};

template <typename Tout>
__global__ void __launch_bounds__(LongSmem::threads, 1)
    k_gt_long(GDims d, PrepArgs p, ScanArgs a, int* flags, int slices, const __grid_constant__ CUtensorMap tm_q,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    static_assert(ScanSmem<1, false>::warps * 32 <= LongSmem::threads, "the scan's warps");
    const int bh = d.B * d.H, nscan = bh * slices;
    if ((int)blockIdx.x < nscan) {
        scan_cta<1, Tout, false>(d, a, tm_q, tm_k, tm_v, blockIdx.x % bh, blockIdx.x / bh, slices);
        return;
    }
    using M = PrepSmem<false>;
    extern __shared__ unsigned char raw[];
    const int gid = threadIdx.x >> 7, tid = threadIdx.x & 127;
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023) + gid * LongSmem::group;
    uint64_t* bar = (uint64_t*)(sm + M::BAR);
    uint32_t* tslot = (uint32_t*)(bar + 3);
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    uint32_t* const base = (uint32_t*)(sm - gid * LongSmem::group + M::BAR) + 8;   // (past the first group's barriers and slot)
    if (threadIdx.x < 32) {   // for all groups (no allocation may follow the relinquishing)
        tmem_alloc(base, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) *tslot = *base + gid * 64;
    const long long items = (long long)((d.L + kGC - 1) / kGC) * bh;
    bool ok = true;
    uint32_t ph = 0;
    for (long long x = (long long)(blockIdx.x - nscan) * LongSmem::groups + gid; x < items && ok;
         x += (long long)(gridDim.x - nscan) * LongSmem::groups) {
        const int c = (int)(x / bh), b = (int)(x % bh) / d.H, h = (int)(x % bh) % d.H;
        const SeqAt s = seq_at(d, b, kGC);
        if (c * kGC >= s.len) continue;
        const int slot = s.slot0 + c;
        ok = prep_chunk<false>(d, p, &tm_q, &tm_k, sm, 1 + gid, tid, slot, h, s, ph, tslot, flags + (size_t)h * p.slots + slot);
        ph ^= 1;
        group_sync(1 + gid);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x < 32) tmem_dealloc(*base, 256);
}

struct TcWs {
    unsigned char* img;
    GVec* vec;
};

size_t carve(const GDims& d, void* base, TcWs* w) {
    const size_t n = (size_t)d.H * d.slots(kGC);
    char* p = (char*)base;
    w->img = (unsigned char*)p;
    p += align256(n * NP * 16384);
    w->vec = (GVec*)p;
    p += align256(n * sizeof(GVec));
    p += align256(n * sizeof(int));
    return (size_t)(p - (char*)base);
}

// Flags of the joint launch, behind the images and vectors.
int* flags_of(const GDims& d, const TcWs& w) { return (int*)((char*)w.vec + align256((size_t)d.H * d.slots(kGC) * sizeof(GVec))); }

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

template <int NCH, typename Tout, bool REC = false>
cudaError_t scan(const GDims& d, const ScanArgs& a, const Maps& m, cudaStream_t st) {
    using M = ScanSmem<NCH, REC>;
    const auto k = k_gt_scan<NCH, Tout, REC>;
    cudaError_t e = smem_attr(k, M::bytes);
    if (e != cudaSuccess) return e;
    e = launch_early(k, dim3((unsigned)d.BH(), (d.dv + 32 * NCH - 1) / (32 * NCH)), M::warps * 32, M::bytes, st, d, a,
                     m.q, m.k, m.v);
    prof_mark(REC ? "gated_record_tc" : "gated_scan_tc", st);
    return e;
}

template <bool BWD>
cudaError_t prep(const GDims& d, const PrepArgs& a, const Maps& m, cudaStream_t st) {
    cudaError_t e = smem_attr(k_gt_prep<BWD>, PrepSmem<BWD>::bytes);
    if (e != cudaSuccess) return e;
    k_gt_prep<BWD><<<dim3(a.slots, d.H), 128, PrepSmem<BWD>::bytes, st>>>(d, a, m.q, m.k);
    prof_mark("gated_prep_tc", st);
    return cudaGetLastError();
}

// Whether preparation and scan go in one launch (*nsm: its CTAs, else 0).  Two kernels: the preparation takes
// 4 us a chunk and SM on all of them, then the scan starts.  One: it starts with the first chunk, 9 us
// later than it could (the flags, the launch, a chunk's preparation on its own), and the rest costs nothing
// as long as the scan leaves a third of the SMs.  In us, d 128, two kernels, one:
//   H 8 L 4096 (512 chunks of a head)  161, 155      H 16 L 4096 (1024)  174, 156
//   H 25 L 1024 (400)                   52,  54      H 25 L 2048 (800)    94,  90
//   H 16 L 16384 (4096)                684, 563
cudaError_t long_form(const GDims& d, bool narrow, int* nsm) {
    int dev = 0, n = 0;
    const long long scan = d.BH() * ((d.dv + 31) / 32);
    *nsm = 0;
    if (!narrow || (long long)d.H * d.slots(kGC) < 640) return cudaSuccess;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && 3 * scan <= 2 * n) *nsm = n;
    return e;
}

template <typename Tout>
cudaError_t fwd(const GDims& d, const void* q, const void* k, const void* v, const float* g, const float* beta,
                const float* S0, void* o, float* S_final, void* ws, cudaStream_t st) {
    TcWs w;
    carve(d, ws, &w);
    Maps m{};
    const int slots = d.slots(kGC);
    bool narrow = false;
    cudaError_t e = make_maps(d, q, k, v, &m);
    if (e == cudaSuccess) e = narrow_slices(d, &narrow);
    int nsm = 0;
    if (e == cudaSuccess) e = long_form(d, narrow, &nsm);
    if (e == cudaSuccess && nsm) {
        const auto k = k_gt_long<Tout>;
        if ((e = smem_attr(k, LongSmem::bytes)) != cudaSuccess) return e;
        int* flags = flags_of(d, w);
        if ((e = cudaMemsetAsync(flags, 0, (size_t)d.H * slots * sizeof(int), st)) != cudaSuccess) return e;
        cudaLaunchAttribute coop{};
        coop.id = cudaLaunchAttributeCooperative;
        coop.val.cooperative = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(nsm);
        cfg.blockDim = dim3(LongSmem::threads);
        cfg.dynamicSmemBytes = LongSmem::bytes;
        cfg.stream = st;
        cfg.attrs = &coop;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, k, d, PrepArgs{g, beta, w.img, w.vec, slots, nullptr},
                               ScanArgs{w.img, w.vec, S0, o, S_final, slots, nullptr, nullptr, flags}, flags, (d.dv + 31) / 32,
                               m.q, m.k, m.v);
        prof_mark("gated_long_tc", st);
        return e;
    }
    if (e == cudaSuccess) e = prep<false>(d, PrepArgs{g, beta, w.img, w.vec, slots, nullptr}, m, st);
    if (e != cudaSuccess) return e;
    const ScanArgs a{w.img, w.vec, S0, o, S_final, slots, nullptr, nullptr, nullptr};
    return narrow ? scan<1, Tout>(d, a, m, st) : scan<2, Tout>(d, a, m, st);
}

}  // namespace

bool gated_tc_supported(const GDims& d) { return d.in_bf16 && d.L > 0; }
size_t gated_tc_fwd_ws_bytes(const GDims& d) {
    TcWs w;
    return carve(d, nullptr, &w);
}

cudaError_t launch_gated_fwd_tc(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, void* o, float* S_final, void* ws,
                                cudaStream_t st) {
    return d.out_bf16 ? fwd<__nv_bfloat16>(d, q, k, v, g, beta, S0, o, S_final, ws, st)
                      : fwd<float>(d, q, k, v, g, beta, S0, o, S_final, ws, st);
}

cudaError_t launch_gated_prep_tc(const GDims& d, const void* q, const void* k, const float* g, const float* beta,
                                 unsigned char* img, unsigned char* img_r, GVec* vec, cudaStream_t st) {
    Maps m{};
    const int nb = d.packed ? 1 : d.B;
    cudaError_t e = strided_rows_map(&m.q, q, d.dk, d.L, d.Hk, nb, d.qs);
    if (e == cudaSuccess) e = strided_rows_map(&m.k, k, d.dk, d.L, d.Hk, nb, d.ks);
    if (e != cudaSuccess) return e;
    return prep<true>(d, PrepArgs{g, beta, img, vec, d.slots(kGC), img_r}, m, st);
}

cudaError_t launch_gated_record_tc(const GDims& d, const void* q, const void* k, const void* v, const float* S0,
                                   const unsigned char* img_r, const GVec* vec, unsigned char* rec_S, unsigned char* rec_R,
                                   cudaStream_t st) {
    Maps m{};
    const cudaError_t e = make_maps(d, q, k, v, &m);
    if (e != cudaSuccess) return e;
    return scan<2, float, true>(d, ScanArgs{img_r, vec, S0, nullptr, nullptr, d.slots(kGC), rec_S, rec_R, nullptr}, m, st);
}

cudaError_t gated_tc_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_gt2_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_gt2_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

// gated_step.cu -- one new token of the gated delta rule for a batch of sequences, on a cache
// of fp32 states updated in place.
//
// For each sequence and value head, f = e^{g}:
//   lambda = ||k||^2, alpha (beta, or the exact flow's);   r = v - f S^T k
//   S <- f S + alpha k r^T;   o = S_new^T q = f S^T q + alpha (k . q) r
// Bound by HBM: the state crosses it twice (2 dk dv 4 bytes a head), everything else is
// 2 (dk + dv) elements.  One pass: a thread keeps its rows of the state in registers between
// the read (whose column sums S^T k and S^T q need no decay yet) and the write.
//
// With a state for every SM and dv = 64 or 128 (k_gated_step_ring): one CTA an SM takes every
// gridDim.x-th state; a producer thread bulk-copies states and their q, k, v rows into three
// stages of shared memory, eight warps update the stage before and store from registers, so that
// two states an SM are on their way in at any time and cost no registers.  Else (k_gated_step) a
// CTA owns 16 columns of one state, so that a few states still use every SM.  dk = dv = 128, states
// that fit L2: 151 states 6.5 us (16 columns a CTA), 152 states 4.6 us (ring).  4096 states (B256 H16,
// 537 MB both ways): 90.8 us, 5.95 TB/s, 0.88 of a plain copy's rate; 16 states: 3.9 us, a launch.
#include "gated_seq.cuh"
#include "launch.h"
#include "tc_common.cuh"

namespace efla {

namespace {


struct GStepArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    float* S;
    const int* slots;
    int nslots;
    void* o;
};

// The state of sequence b (its place in the cache), or -1 where the caller's index is outside.
__device__ __forceinline__ long long state_of(const GStepArgs& a, int b) {
    if (!a.slots) return b;
    const int s = __ldg(a.slots + b);
    return s >= 0 && s < a.nslots ? s : -1;
}


// A CTA of 256 threads owns DV columns of one head's state.  Any dk <= 128, dv a multiple of DV.
template <typename Tin, typename Tout, int DV>
__global__ void __launch_bounds__(256) k_gated_step(GDims d, GStepArgs a) {
    constexpr int C4 = DV / 4, RP = 256 / C4, RT = 128 / RP;
    __shared__ float qs[128], ks[128], vs[DV], rs[DV];
    __shared__ float red_k[RP][DV + 4], red_q[RP][DV + 4];   // rows stay 16-byte aligned
    __shared__ float s_alpha, s_kq;
    const int b = blockIdx.x / d.H, h = blockIdx.x % d.H, hk = h / (d.H / d.Hk), col0 = blockIdx.y * DV;
    const int tid = threadIdx.x, c4 = tid % C4, g0 = tid / C4, dk = d.dk, dv = d.dv;
    Tout* op = (Tout*)a.o + at3(d.os, b, h, 0) + col0;
    const long long sl = state_of(a, b);
    if (sl < 0) {
        if (tid < DV) st_elem(op + tid, 0.f);
        return;
    }
    float* Sh = a.S + (sl * d.H + h) * (long long)dk * dv + col0;
    float4 s[RT];   // the state first: it is the long latency
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const int r = g0 + m * RP;
        s[m] = r < dk ? *reinterpret_cast<const float4*>(Sh + (size_t)r * dv + 4 * c4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float f = expf(a.g[at3(d.gs, b, h, 0)]);
    if (tid < 128) {
        const Tin* qp = (const Tin*)a.q + at3(d.qs, b, hk, 0);
        const Tin* kp = (const Tin*)a.k + at3(d.ks, b, hk, 0);
        qs[tid] = tid < dk ? ld_elem(qp + tid) : 0.f;
        ks[tid] = tid < dk ? ld_elem(kp + tid) : 0.f;
    } else if (tid - 128 < DV) {
        vs[tid - 128] = ld_elem((const Tin*)a.v + at3(d.vs, b, h, 0) + col0 + tid - 128);
    }
    __syncthreads();
    if (tid < 32) {
        float l = 0.f, kq = 0.f;
#pragma unroll
        for (int i = tid; i < 128; i += 32) {
            l = fmaf(ks[i], ks[i], l);
            kq = fmaf(ks[i], qs[i], kq);
        }
        l = warp_sum(l);
        kq = warp_sum(kq);
        if (tid == 0) {
            s_alpha = alpha_of(a.beta[at3(d.bs, b, h, 0)], l, d.euler);
            s_kq = kq;
        }
    }
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const float kr = ks[g0 + m * RP], qr = qs[g0 + m * RP];
        pk.x = fmaf(s[m].x, kr, pk.x); pk.y = fmaf(s[m].y, kr, pk.y);
        pk.z = fmaf(s[m].z, kr, pk.z); pk.w = fmaf(s[m].w, kr, pk.w);
        pq.x = fmaf(s[m].x, qr, pq.x); pq.y = fmaf(s[m].y, qr, pq.y);
        pq.z = fmaf(s[m].z, qr, pq.z); pq.w = fmaf(s[m].w, qr, pq.w);
    }
    *reinterpret_cast<float4*>(&red_k[g0][4 * c4]) = pk;
    *reinterpret_cast<float4*>(&red_q[g0][4 * c4]) = pq;
    __syncthreads();
    const float alpha = s_alpha;
    if (tid < DV) {
        float sk = 0.f, sq = 0.f;
#pragma unroll 8
        for (int x = 0; x < RP; ++x) {
            sk += red_k[x][tid];
            sq += red_q[x][tid];
        }
        const float r = fmaf(-f, sk, vs[tid]);
        rs[tid] = r;
        st_elem(op + tid, fmaf(alpha * s_kq, r, f * sq));
    }
    __syncthreads();
    const float4 rr = *reinterpret_cast<const float4*>(rs + 4 * c4);
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const int r = g0 + m * RP;
        if (r < dk) {
            const float ak = alpha * ks[r];
            *reinterpret_cast<float4*>(Sh + (size_t)r * dv + 4 * c4) =
                make_float4(fmaf(ak, rr.x, f * s[m].x), fmaf(ak, rr.y, f * s[m].y), fmaf(ak, rr.z, f * s[m].z),
                            fmaf(ak, rr.w, f * s[m].w));
        }
    }
}

__device__ unsigned int g_gs_status = 0;   // bit 0: a bounded wait expired; kStatusBounds (debug builds): a write was skipped

constexpr int kRsCons = 256;
constexpr int kRsStages = 3;
constexpr uint32_t kRsState = 65536;                      // most bytes of a state
constexpr uint32_t kRsStage = kRsState + 3 * 512;         // and its q, k, v rows
constexpr uint32_t kRsRed = kRsStages * kRsStage;         // column sums [8][128] x 2
constexpr uint32_t kRsR = kRsRed + 8192;                  // r [128]
constexpr uint32_t kRsMisc = kRsR + 512;                  // alpha, k.q, f
constexpr uint32_t kRsBar = kRsMisc + 16;                 // full[3], done[3]
constexpr size_t kRsSmem = 128 + kRsBar + 2 * kRsStages * 8;
static_assert(kRsSmem <= 232448, "shared memory per CTA");

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// Consumer thread (warp w, lane l) owns four adjacent columns of rows w R + l / (DV / 4), + 8 R, ...
// (R = 128 / DV rows a warp): a warp reads and writes whole 512-byte spans.
template <typename Tin, typename Tout, int DV>
__global__ void __launch_bounds__(kRsCons + 32, 1) k_gated_step_ring(GDims d, GStepArgs a) {
    constexpr int R = 128 / DV, RT = 16 / R, C4 = DV / 4;   // rows a warp takes at once, and per thread
    extern __shared__ unsigned char raw[];
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 127) & ~(uintptr_t)127);
    uint64_t* full = (uint64_t*)(sm + kRsBar);
    uint64_t* done = full + kRsStages;
    float* red_k = (float*)(sm + kRsRed);
    float* red_q = red_k + 8 * 128;
    float* rs = (float*)(sm + kRsR);
    float* misc = (float*)(sm + kRsMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, dk = d.dk;
    const int BH = d.B * d.H, G = gridDim.x;
    const uint32_t bytes = (uint32_t)dk * DV * 4, kb = dk * sizeof(Tin), vb = DV * sizeof(Tin);
    if (tid == 0) {
        for (int s = 0; s < kRsStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], kRsCons / 32);
        }
        fence_mbar_init();
    }
    __syncthreads();
    if (warp == kRsCons / 32) {
        if (lane == 0) {
            const auto issue = [&](int s, int x) {
                const int b = x / d.H, h = x % d.H, hk = h / (d.H / d.Hk);
                const long long sl = state_of(a, b);
                unsigned char* st = sm + s * kRsStage;
                if (sl < 0) {   // no state: the consumers only write zeros
                    mbar_arrive(&full[s]);
                    return;
                }
                mbar_arrive_expect_tx(&full[s], bytes + 2 * kb + vb);
                bulk_g2s(st, a.S + (sl * d.H + h) * (long long)dk * DV, bytes, &full[s]);
                bulk_g2s(st + kRsState, (const Tin*)a.q + at3(d.qs, b, hk, 0), kb, &full[s]);
                bulk_g2s(st + kRsState + 512, (const Tin*)a.k + at3(d.ks, b, hk, 0), kb, &full[s]);
                bulk_g2s(st + kRsState + 1024, (const Tin*)a.v + at3(d.vs, b, h, 0), vb, &full[s]);
            };
            int issued = 0;
            for (long long x = blockIdx.x; issued < kRsStages && x < BH; x += G) issue(issued++, (int)x);
            int it = 0;
            for (long long x = blockIdx.x; x < BH; x += G, ++it) {
                const int s = it % kRsStages;
                if (!mbar_wait(&done[s], (uint32_t)(it / kRsStages) & 1u, kWaitLimit)) {
                    atomicOr(&g_gs_status, 1u);
                    break;
                }
                if (x + (long long)kRsStages * G < BH) {
                    issue(s, (int)(x + (long long)kRsStages * G));
                    ++issued;
                }
            }
            for (int j = it; j < issued; ++j)   // (an abandoned run: what was issued lands before the exit)
                mbar_wait(&full[j % kRsStages], (uint32_t)(j / kRsStages) & 1u, kWaitLimit);
        }
        return;
    }
    const int r0 = warp * R + lane / C4, c4 = (lane % C4) * 4;
    int it = 0;
    for (long long x = blockIdx.x; x < BH; x += G, ++it) {
        const int b = (int)x / d.H, h = (int)x % d.H, s = it % kRsStages;
        const long long sl = state_of(a, b);
        const float be = tid == 0 ? a.beta[at3(d.bs, b, h, 0)] : 0.f;   // in flight with the wait
        const float f = expf(a.g[at3(d.gs, b, h, 0)]);
        if (!group_sync_and(1, mbar_wait(&full[s], (uint32_t)(it / kRsStages) & 1u, kWaitLimit), kRsCons)) {
            if (tid == 0) atomicOr(&g_gs_status, 1u);
            break;
        }
        Tout* op = (Tout*)a.o + at3(d.os, b, h, 0);
        if (sl < 0) {
            if (lane == 0) mbar_arrive(&done[s]);
            if (tid < DV) st_elem(op + tid, 0.f);
            continue;
        }
        const float* St = (const float*)(sm + s * kRsStage);
        const Tin* qv = (const Tin*)(sm + s * kRsStage + kRsState);
        const Tin* kv = (const Tin*)(sm + s * kRsStage + kRsState + 512);
        const Tin* vv = (const Tin*)(sm + s * kRsStage + kRsState + 1024);
        if (warp == 0) {   // lambda = ||k||^2 -> alpha, and k.q
            float l = 0.f, kq = 0.f;
            for (int i = lane; i < dk; i += 32) {
                const float ki = widen(kv[i]);
                l = fmaf(ki, ki, l);
                kq = fmaf(ki, widen(qv[i]), kq);
            }
            l = warp_sum(l);
            kq = warp_sum(kq);
            if (lane == 0) {
                misc[0] = alpha_of(be, l, d.euler);
                misc[1] = kq;
            }
        }
        float4 sv[RT], pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
        float kr[RT];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const int r = r0 + 8 * R * m;
            const bool in = r < dk;
            sv[m] = in ? *reinterpret_cast<const float4*>(St + r * DV + c4) : make_float4(0.f, 0.f, 0.f, 0.f);
            kr[m] = in ? widen(kv[r]) : 0.f;
            const float qr = in ? widen(qv[r]) : 0.f;
            pk.x = fmaf(sv[m].x, kr[m], pk.x); pk.y = fmaf(sv[m].y, kr[m], pk.y);
            pk.z = fmaf(sv[m].z, kr[m], pk.z); pk.w = fmaf(sv[m].w, kr[m], pk.w);
            pq.x = fmaf(sv[m].x, qr, pq.x); pq.y = fmaf(sv[m].y, qr, pq.y);
            pq.z = fmaf(sv[m].z, qr, pq.z); pq.w = fmaf(sv[m].w, qr, pq.w);
        }
        const float vt = tid < DV ? widen(vv[tid]) : 0.f;
        if (R == 2) {   // the warp's two rows together
            pk.x += __shfl_xor_sync(0xffffffffu, pk.x, 16); pk.y += __shfl_xor_sync(0xffffffffu, pk.y, 16);
            pk.z += __shfl_xor_sync(0xffffffffu, pk.z, 16); pk.w += __shfl_xor_sync(0xffffffffu, pk.w, 16);
            pq.x += __shfl_xor_sync(0xffffffffu, pq.x, 16); pq.y += __shfl_xor_sync(0xffffffffu, pq.y, 16);
            pq.z += __shfl_xor_sync(0xffffffffu, pq.z, 16); pq.w += __shfl_xor_sync(0xffffffffu, pq.w, 16);
        }
        if (lane < C4) {
            *reinterpret_cast<float4*>(red_k + warp * 128 + c4) = pk;
            *reinterpret_cast<float4*>(red_q + warp * 128 + c4) = pq;
        }
        group_sync(1, kRsCons);
        if (lane == 0) mbar_arrive(&done[s]);   // (every warp has read the stage, warp 0's k and q included)
        const float alpha = misc[0];   // (read before the next barrier: warp 0 rewrites it for the next state)
        if (tid < DV) {
            float sk = 0.f, sq = 0.f;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                sk += red_k[g * 128 + tid];
                sq += red_q[g * 128 + tid];
            }
            const float r = fmaf(-f, sk, vt);
            rs[tid] = r;
            st_elem(op + tid, fmaf(alpha * misc[1], r, f * sq));
        }
        group_sync(1, kRsCons);
        const float4 rr = *reinterpret_cast<const float4*>(rs + c4);
        float* Sg = a.S + (sl * d.H + h) * (long long)dk * DV;
        const bool wr = dbg_in(Sg, bytes, a.S, (size_t)a.nslots * d.H * bytes, &g_gs_status);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const int r = r0 + 8 * R * m;
            const float ak = alpha * kr[m];
            if (wr && r < dk)
                __stcs(reinterpret_cast<float4*>(Sg + r * DV + c4),
                       make_float4(fmaf(ak, rr.x, f * sv[m].x), fmaf(ak, rr.y, f * sv[m].y), fmaf(ak, rr.z, f * sv[m].z),
                                   fmaf(ak, rr.w, f * sv[m].w)));
        }
    }
}

// q, k, v rows that bulk copies can read
template <typename Tin>
bool wide_rows(const GDims& d, const GStepArgs& a) {
    const auto ok = [](const void* p, const long long (&s)[3]) {
        return ((uintptr_t)p & 15u) == 0 && s[0] * sizeof(Tin) % 16 == 0 && s[1] * sizeof(Tin) % 16 == 0;
    };
    return ok(a.q, d.qs) && ok(a.k, d.ks) && ok(a.v, d.vs);
}

template <typename Tin, typename Tout, int DV>
cudaError_t ring(const GDims& d, const GStepArgs& a, int nsm, cudaStream_t st) {
    const cudaError_t e = cudaFuncSetAttribute(k_gated_step_ring<Tin, Tout, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)kRsSmem);
    if (e != cudaSuccess) return e;
    k_gated_step_ring<Tin, Tout, DV><<<nsm, kRsCons + 32, kRsSmem, st>>>(d, a);
    prof_mark("gated_decode_step", st);
    return cudaGetLastError();
}

template <typename Tin, typename Tout>
cudaError_t dispatch(const GDims& d, const GStepArgs& a, cudaStream_t st) {
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (d.BH() >= nsm && wide_rows<Tin>(d, a)) {
        if (d.dv == 128) return ring<Tin, Tout, 128>(d, a, nsm, st);
        if (d.dv == 64) return ring<Tin, Tout, 64>(d, a, nsm, st);
    }
    // 16 columns a CTA (256 threads hold 128 x 16 of a state in two float4 each)
    const unsigned n = (unsigned)d.BH();
    k_gated_step<Tin, Tout, 16><<<dim3(n, d.dv / 16), 256, 0, st>>>(d, a);
    prof_mark("gated_decode_step", st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_step(const GDims& d, const void* q, const void* k, const void* v, const float* g,
                              const float* beta, float* S, const int* slots, int nslots, void* o, cudaStream_t st) {
    const GStepArgs a{q, k, v, g, beta, S, slots, nslots, o};
    using B = __nv_bfloat16;
    if (d.in_bf16) return d.out_bf16 ? dispatch<B, B>(d, a, st) : dispatch<B, float>(d, a, st);
    return d.out_bf16 ? dispatch<float, B>(d, a, st) : dispatch<float, float>(d, a, st);
}

cudaError_t gated_step_status_read_clear(unsigned int* status) {
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_gs_status, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    return *status ? cudaMemcpyToSymbol(g_gs_status, &zero, sizeof(unsigned int)) : cudaSuccess;
}

}  // namespace efla

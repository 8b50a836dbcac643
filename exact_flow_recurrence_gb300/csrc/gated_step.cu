// gated_step.cu -- one new token of the gated delta rule for a batch of sequences, on a cache
// of fp32 states updated in place.
//
// For each sequence and value head, f = e^{g}:
//   lambda = ||k||^2, alpha (beta, or the exact flow's);   r = v - f S^T k
//   S <- f S + alpha k r^T;   o = S_new^T q = f S^T q + alpha (k . q) r
// Bound by HBM: the state crosses it twice (2 dk dv 4 bytes a head), everything else is
// 2 (dk + dv) elements.  One pass: a thread keeps its rows of the state in registers between
// the read (whose column sums S^T k and S^T q need no decay yet) and the write.
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

template <typename Tin, typename Tout>
cudaError_t dispatch(const GDims& d, const GStepArgs& a, cudaStream_t st) {
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

}  // namespace efla

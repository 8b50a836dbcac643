// gated_seq.cuh -- where a sequence of a gated call lies, and the parts every gated kernel shares.
#pragma once

#include "common.cuh"
#include "gated.h"

namespace efla {

// Where sequence b's tokens are: the first one on the token axis, how many, its first chunk
// slot, and the index to use with batch strides.  Packed offsets are device data that the
// host cannot check: they are clamped to [0, L] and to a non-negative length here, so that no
// value of theirs leads outside the arrays.
struct SeqAt {
    int start, len, slot0, batch;
};

__device__ __forceinline__ int clamp_off(const GDims& d, int b) { return min(max(__ldg(d.offsets + b), 0), d.L); }

__device__ __forceinline__ SeqAt seq_at(const GDims& d, int b, int C) {
    SeqAt s;
    if (d.packed) {
        s.start = clamp_off(d, b);
        s.len = max(clamp_off(d, b + 1) - s.start, 0);
        s.slot0 = s.start / C + b;
        s.batch = 0;
    } else {
        s.start = 0;
        s.len = d.L;
        s.slot0 = b * ((d.L + C - 1) / C);
        s.batch = b;
    }
    return s;
}

// The sequence that chunk slot `slot` belongs to (slot0(b) <= slot < slot0(b + 1)); slots before the first
// sequence's (packed tokens may start past 0) count as sequence 0's, in front of its first chunk.
__device__ __forceinline__ int seq_of_slot(const GDims& d, int slot, int C) {
    if (!d.packed) return slot / ((d.L + C - 1) / C);
    int lo = 0, hi = d.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (clamp_off(d, mid) / C + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The tokens of chunk slot `slot`: the sequence b and its place s, the chunk's first token t0 in it, and how
// many there are (none: the slot holds no chunk).
__device__ __forceinline__ int chunk_at(const GDims& d, int slot, int C, int& b, SeqAt& s, int& t0) {
    b = seq_of_slot(d, slot, C);
    s = seq_at(d, b, C);
    t0 = (slot - s.slot0) * C;
    return t0 < 0 ? 0 : min(C, s.len - t0);
}

__device__ __forceinline__ long long at3(const long long (&s)[3], int b, int h, int t) {
    return b * s[0] + h * s[1] + t * s[2];
}

// da dalpha/dlambda.  Away from x = beta lambda = 0 it is da (x e^{-x} + expm1(-x)) / lambda^2, and lambda
// divides each factor by itself: its square, and the derivative alone, leave fp32's range for keys of
// ||k|| = 1e10 and more, where the product does not.
__device__ __forceinline__ float dlambda_of(float da, float beta, float lambda, int euler) {
    const float x = beta * lambda;
    if (euler || fabsf(x) < 0.5f) return da * dalpha_dlambda_of(beta, lambda, euler);
    return da / lambda * ((x * expf(-x) + expm1f(-x)) / lambda);
}

// Sums of log decays inside a chunk.  A decay below e^-128 is zero in fp32, so g is taken as at
// least -128 there: an infinite one (a state reset) then leaves no inf - inf behind.  The sums
// c_i are kept as two floats (hi + lo), since e^{c_i - c_j} needs the difference's absolute
// error small where c itself may be thousands.
__device__ __forceinline__ float log_decay(float g) { return g < -128.f ? -128.f : g; }
// The tensor-core kernels keep c in units of log 2.  ex2.approx: 2^-22 of the result.
constexpr double kLog2e = 1.4426950408889634;
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float decay2(float hi_i, float lo_i, float hi_j, float lo_j) {
    return exp2_fast((hi_i - hi_j) + (lo_i - lo_j));
}
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j) {
    return expf((hi_i - hi_j) + (lo_i - lo_j));
}

}  // namespace efla

// mix.cuh -- parts that the short convolution's and the selective scan's kernels share.
#pragma once

#include "common.cuh"
#include "mix.h"
#include "packed2.cuh"

namespace efla {

// A sequence's place: tokens start .. end-1 of its axis.  Offsets are device data that the host cannot
// check: they are clamped here, so that no value of theirs leads outside the arrays.
struct Seq {
    int b, start, end;
};

__device__ __forceinline__ int offset_at(const Axes& a, int b) { return min(max(__ldg(a.offsets + b), 0), a.L); }

__device__ __forceinline__ Seq seq_at(const Axes& a, int b) {
    if (!a.packed) return Seq{b, 0, a.L};
    const int s = offset_at(a, b);
    return Seq{b, s, max(offset_at(a, b + 1), s)};
}

// The last sequence of this axis that begins at token t or before it (the first one where none does): t lies
// in it, or outside every sequence.
__device__ __forceinline__ Seq seq_of(const Axes& a, int axis, int t) {
    if (!a.packed) return Seq{axis, 0, a.L};
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offset_at(a, mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return seq_at(a, lo);
}

// The next token from t on, before t1, that lies in a sequence, and that sequence in s (t1 if there is none).
__device__ __forceinline__ int next_inside(const Axes& a, Seq& s, int t, int t1) {
    while (t >= s.end && s.b + 1 < a.B && a.packed) s = seq_at(a, s.b + 1);
    if (t >= s.end) return t1;
    return min(max(t, s.start), t1);
}

// ------------------------------------------------------------------- VEC neighbouring elements
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* x) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
};
template <>
struct Vec<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float* x) const {
        x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float* x) {
        const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
        v = make_uint2(*reinterpret_cast<const uint32_t*>(&h[0]), *reinterpret_cast<const uint32_t*>(&h[1]));
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = v; }
};
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = (T)0.f; }
    __device__ __forceinline__ void get(float* x) const { x[0] = (float)v; }
    __device__ __forceinline__ void set(const float* x) { v = (T)x[0]; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
};

// ------------------------------------------------------------------- functions
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2eF = 1.4426950408889634f;
// 1 / (1 + e^{-x}): within (1.3 |x| + 8) 2^-24 of the result (|x| 2^-24 from the rounded exponent, where e^{-x} is large)
__device__ __forceinline__ float sigmoid_of(float x) { return rcp(1.f + ex2(-kLog2eF * x)); }
__device__ __forceinline__ float silu_of(float x) { return x * sigmoid_of(x); }
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 e = mul2(x, both(-kLog2eF)), s = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
    return make_float2(rcp(s.x), rcp(s.y));
}

inline bool aligned_rows(const void* p, const long long (&s)[2], int rows, int tokens, int bytes, int es) {
    return (uintptr_t)p % bytes == 0 && (rows < 2 || s[0] * es % bytes == 0) && (tokens < 2 || s[1] * es % bytes == 0);
}

}  // namespace efla

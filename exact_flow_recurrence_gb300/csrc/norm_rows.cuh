// norm_rows.cuh -- rows of a norm: their elements, the sums over a row's warps, and the rings that rows
// arrive in.
#pragma once

#include "common.cuh"
#include "packed2.cuh"
#include "tc_common.cuh"

namespace efla {

// VEC neighbouring elements as stored, and as fp32
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = __ldg(reinterpret_cast<const float4*>(p)); }
    __device__ __forceinline__ void get(float* x) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    __device__ __forceinline__ void set(const float* x) { v = make_float4(x[0], x[1], x[2], x[3]); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* x) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float* x) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v = *reinterpret_cast<const uint4*>(h);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
};
template <typename T>
struct Pack<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void get(float* x) const { x[0] = (float)v; }
    __device__ __forceinline__ void set(const float* x) { v = (T)x[0]; }
    __device__ __forceinline__ void store(T* p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = (T)0.f; }
};

// VEC weights from column c (fp32 or bf16)
template <int VEC>
__device__ __forceinline__ void weights(const void* w, int c, int bf16, float* x) {
    if (VEC == 1) {
        x[0] = bf16 ? __bfloat162float(((const __nv_bfloat16*)w)[c]) : __ldg((const float*)w + c);
    } else if (bf16) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>((const __nv_bfloat16*)w + c + i));
            x[i] = __uint_as_float(v.x << 16);
            x[(i + 1) % VEC] = __uint_as_float(v.x & 0xffff0000u);
            x[(i + 2) % VEC] = __uint_as_float(v.y << 16);
            x[(i + 3) % VEC] = __uint_as_float(v.y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>((const float*)w + c + i));
            x[i] = v.x;
            x[(i + 1) % VEC] = v.y;
            x[(i + 2) % VEC] = v.z;
            x[(i + 3) % VEC] = v.w;
        }
    }
}

// Sums over the W warps of a row (of s.x alone, or of both); `red` has room for W pairs and is not
// in use by an earlier sum that a warp of this row may still be reading.
template <int W, bool TWO>
__device__ __forceinline__ float2 row_sum(float2 s, float2* red, int bar, int warp_in_row) {
    s.x = warp_sum(s.x);
    if (TWO) s.y = warp_sum(s.y);
    if (W == 1) return s;
    if ((threadIdx.x & 31) == 0) red[warp_in_row] = s;
    group_sync(bar, 32 * W);
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        r.x += red[i].x;
        if (TWO) r.y += red[i].y;
    }
    return r;
}

// Threads a CTA: what the registers of 16 elements a thread allow.
template <int W, int SP, bool BWD>
struct Cta {
    static constexpr int threads = BWD || W > 8 || SP > 16 ? 512 : 768;
};
constexpr int kStages = 6;       // most stages of a ring
constexpr size_t kRing = 160 * 1024;

// One row group's ring: `arrays` rows a stage, each `bytes` long.
struct Ring {
    unsigned char* buf;
    uint64_t* full;   // [stages]
    uint32_t bytes;
    int stages, arrays, stage, phase;
    __device__ __forceinline__ unsigned char* row(int which) const { return buf + (size_t)(stage * arrays + which) * bytes; }
    // one thread: copies for the row after next use of stage `to`
    __device__ __forceinline__ void issue(int to, const void* x, const void* g, const void* h = nullptr) const {
        mbar_arrive_expect_tx(&full[to], bytes * arrays);
        bulk_g2s(buf + (size_t)to * arrays * bytes, x, bytes, &full[to]);
        if (arrays >= 2) bulk_g2s(buf + (size_t)(to * arrays + 1) * bytes, g, bytes, &full[to]);
        if (arrays == 3) bulk_g2s(buf + (size_t)(to * arrays + 2) * bytes, h, bytes, &full[to]);
    }
    __device__ __forceinline__ bool wait() const { return mbar_wait(&full[stage], phase, kWaitLimit); }
    __device__ __forceinline__ void next() {
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

}  // namespace efla

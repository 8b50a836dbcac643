// gated_tc.cuh -- pieces shared by the gated delta rule's tensor-core kernels: operands as sums
// of bf16 parts, the per-chunk record of the preparation, tensor maps of strided arrays.
//
// Precision.  The inputs q, k, v, dO are bf16 and enter the tensor cores as they are; every
// operand that is computed (the state, the chunk's corrected values, T and P T) enters as the
// sum of three bf16 parts, x = x_0 + x_1 + x_2, each the rounding of what the earlier ones left,
// and a product of two such operands takes the part pairs a + b < 3.  All products accumulate
// in fp32.  Three parts carry the 24 bits of an fp32 value: against the fp64 recurrence the
// outputs and the carried state come out within 5e-7 of their norm, where two parts leave 4e-6
// and one bf16 or fp16 operand 3e-3 or 3e-4.  Parts keep fp32's exponent range, so there is
// no range to check and no second path, and what a call returns does not depend on what else it
// returns.
#pragma once

#include <utility>

#include "gated_seq.cuh"
#include "packed2.cuh"
#include "tc_common.cuh"

namespace efla {

constexpr int kGC = 64;   // tokens a chunk of the tensor-core kernels
constexpr int NP = 3;     // bf16 parts of a computed operand
constexpr uint32_t kRecS = 3 * 16384, kRecT = 3 * 8192;   // bytes of a recorded slice of S or G, of R or dX

// Elements from the first to the last of a strided [batch][heads][token][width] array, and the bytes
// of all records of a kind (debug builds' bounds).
__device__ __forceinline__ size_t extent(const GDims& d, const long long (&s)[3], int heads, int width) {
    return (d.packed ? 0 : (d.B - 1) * s[0]) + (heads - 1) * s[1] + (d.L - 1) * s[2] + width;
}
__device__ __forceinline__ size_t records(const GDims& d, int slots, size_t bytes) {
    return (size_t)d.H * slots * ((d.dv + 63) / 64) * bytes;
}

// What the preparation leaves of a chunk and value head besides the T, P T image: five vectors.
struct GVec {
    float up[64];     // e^{c_i}
    float rest[64];   // e^{c_last - c_i}
    float al[64];     // alpha_i (0 past the sequence's end)
    float chi[64];    // c_i / log 2 = chi + clo
    float clo[64];
};

// To follow a wait for tensor-memory loads: the loaded values may be used from here on.  (The
// wait names no registers, so arithmetic on them could otherwise be scheduled before it.)
__device__ __forceinline__ void loaded8(float* v) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void loaded16(float* v) {
    loaded8(v);
    loaded8(v + 8);
}
template <int N>
__device__ __forceinline__ void loaded(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8) loaded8(v + i);
}

// 8 values -> N 16-byte chunks of bf16 parts
template <int N>
__device__ __forceinline__ void split8(const float2* x, uint4 (&w)[N]) {
    float2 r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = x[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
        uint32_t* o = reinterpret_cast<uint32_t*>(&w[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(r[i].x, r[i].y);
            o[i] = *reinterpret_cast<const uint32_t*>(&h);
            if (p + 1 < N) r[i] = sub2(r[i], bf16x2(o[i]));
        }
    }
}
template <int N>
__device__ __forceinline__ void split8(const float* x, uint4 (&w)[N]) {
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = make_float2(x[2 * i], x[2 * i + 1]);
    split8<N>(y, w);
}

// A scan CTA runs NCH chains of 32 state columns each: their products and epilogues are
// independent, so that one chain's products run while the other's epilogue does.
// Left to themselves the two fall into step and wait for the same things together; so they take
// turns: chain 1 starts a chunk when chain 0 has issued the chunk's second product, and chain 0
// the next one when chain 1 has.  A computed
// operand of 32 columns lies in blocks of 128-byte rows (64 columns; R rows, BLK = 128 R bytes):
//   block g < NCH   chain g's part 0 | part 1        block NCH   chain 0's part 2 | chain 1's
// so that its parts are neighbours along N and one product takes them all (D keeps a column
// group for each; the epilogues add them).  An instruction costs about 43 cycles up to N = 64
// and 50 at N = 96: three parts in one cost little more than one.
template <int NCH>
struct Chain {
    static constexpr int blocks = NCH + 1;
    // byte offset of part p's first column, and the stride to the block that holds part 2
    __host__ __device__ static constexpr uint32_t part(int g, int p, uint32_t blk) {
        return p < 2 ? g * blk + p * 64 : NCH * blk + g * 64;
    }
    __host__ __device__ static constexpr uint32_t lbo(int g, uint32_t blk) { return (NCH - g) * blk + g * 64; }
    // 2 W2 values of row r, columns from cc of chain g
    template <int W2>
    static __device__ __forceinline__ void put(unsigned char* base, uint32_t blk, int g, int r, int cc, const float2 (&x)[W2]);
};

// 2 W2 columns of this warp's lanes of an accumulator, summed over G column groups `gap` apart (the
// last ones first: they hold the small parts' products; two at a time, for the registers' sake:
// with all but a few KB of L1 taken by shared memory, a spilled register costs a trip to L2).
template <int G, int W2>
__device__ __forceinline__ void tmem_sum(uint32_t t, int gap, float2 (&y)[W2]) {
#pragma unroll
    for (int p = G - 1; p >= 0; p -= 2) {
        float x[2][2 * W2];
        tmem_ld16(t + p * gap, x[0]);
        if (p > 0) tmem_ld16(t + (p - 1) * gap, x[1]);
        tmem_ld_wait();
        loaded(x[0]);
        if (p > 0) loaded(x[1]);
#pragma unroll
        for (int m = 0; m < W2; ++m) {
            float2 z = make_float2(x[0][2 * m], x[0][2 * m + 1]);
            if (p < G - 1) z = add2(y[m], z);
            if (p > 0) z = add2(z, make_float2(x[1][2 * m], x[1][2 * m + 1]));
            y[m] = z;
        }
    }
}

template <int NCH>
template <int W2>
__device__ __forceinline__ void Chain<NCH>::put(unsigned char* base, uint32_t blk, int g, int r, int cc,
                                                    const float2 (&x)[W2]) {
#pragma unroll
    for (int e = 0; e < 2 * W2; e += 8) {
        uint4 w[NP];
        split8<NP>(x + e / 2, w);
#pragma unroll
        for (int p = 0; p < NP; ++p)
            *reinterpret_cast<uint4*>(base + (p < 2 ? g : NCH) * blk + sw128(r, (p < 2 ? p : g) * 32 + cc + e)) = w[p];
    }
}

// 2 W2 values of row r, from column col of a slice's 64, as parts in tiles of 64 rows one after another
// (the records of R and dX).
template <int W2>
__device__ __forceinline__ void put_parts(unsigned char* base, int r, int col, const float2 (&x)[W2]) {
#pragma unroll
    for (int e = 0; e < 2 * W2; e += 8) {
        uint4 w[NP];
        split8<NP>(x + e / 2, w);
#pragma unroll
        for (int p = 0; p < NP; ++p) *reinterpret_cast<uint4*>(base + p * 8192 + sw128(r, col + e)) = w[p];
    }
}

// A warp's shared-memory writes and tensor-memory reads are done.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    fence_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}
// (the warp leaves together if a wait gives up)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t ph) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, ph, kWaitLimit)) != 0;
    tc_fence_after();
    return ok;
}

// 2 W2 values to 16-byte aligned memory
template <int W2>
__device__ __forceinline__ void st_row(float* p, const float2 (&x)[W2]) {
#pragma unroll
    for (int i = 0; i < W2; i += 2) *reinterpret_cast<float4*>(p + 2 * i) = make_float4(x[i].x, x[i].y, x[i + 1].x, x[i + 1].y);
}
template <int W2>
__device__ __forceinline__ void st_row(__nv_bfloat16* p, const float2 (&x)[W2]) {
#pragma unroll
    for (int i = 0; i < W2; i += 4) {
        uint4 w[1];
        split8<1>(x + i, w);
        *reinterpret_cast<uint4*>(p + 2 * i) = w[0];
    }
}

// Tensor map of a strided bf16 [batch][head][token][d] array: boxes of 64 tokens x 64 columns
// with the 128-byte swizzle; elements outside read as zero.
inline cudaError_t strided_rows_map(CUtensorMap* m, const void* base, int d, int L, int heads, int batch,
                                    const long long (&s)[3]) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
    }
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)heads, (cuuint64_t)batch};
    // a dimension of one element has no stride of its own
    const auto bytes = [&](int n, long long st) { return (cuuint64_t)(n > 1 ? st * 2 : 256); };
    const cuuint64_t strides[3] = {bytes(L, s[2]), bytes(heads, s[1]), bytes(batch, s[0])};
    const cuuint32_t box[4] = {64, 64, 1, 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    const CUresult r = encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename K>
inline cudaError_t smem_attr(K k, size_t bytes) {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

// Launch that may begin before the kernel ahead of it in the stream ends: from when all of that
// one's CTAs have called griddep_launch_dependents (they hold their tensor memory by then, so that
// none of them waits for columns that an early CTA has taken).  The kernel itself says what it
// waits for.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*k)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A&&... args) {
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, std::forward<A>(args)...);
}

// Whether slices of 32 state columns (instead of 64) still find an SM each: a chain that shares its
// CTA with no other takes 2.1 us a chunk, two take 3.3 us, but twice the CTAs that do not all run
// at once take twice the time.  L 4096, d 128: 38 heads, the last that fit narrow slices, 206 us;
// 39 heads in wide ones 254 us.
inline cudaError_t narrow_slices(const GDims& d, bool* narrow) {
    int dev = 0, nsm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    *narrow = 2 * d.BH() * ((d.dv + 63) / 64) <= nsm;
    return e;
}

// The backward's parts of gated_tc.cu: the preparation, with the image of the residuals' inverse, and
// the pass that records every chunk's S and residuals R as parts, in the operand layout
// ([H][slots][slices of 64 columns][kRecS or kRecT bytes]).
cudaError_t launch_gated_prep_tc(const GDims& d, const void* q, const void* k, const float* g, const float* beta,
                                 unsigned char* img, unsigned char* img_r, GVec* vec, cudaStream_t st);
cudaError_t launch_gated_record_tc(const GDims& d, const void* q, const void* k, const void* v, const float* S0,
                                   const unsigned char* img_r, const GVec* vec, unsigned char* rec_S, unsigned char* rec_R,
                                   cudaStream_t st);

}  // namespace efla

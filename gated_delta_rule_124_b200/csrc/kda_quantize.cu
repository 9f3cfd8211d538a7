// A matrix to 8 bits with a scale per block of 128 columns of a row, or per
// 128 x 128 block, in the orientation that the 8-bit product reads: the matrix
// itself or its transpose.
//
// Elements are read once and written once as one byte: bound by HBM.  A CTA of
// 256 threads takes a 128 x 128 tile of x, a row's 128 columns in 16 lanes,
// eight rows a thread, all loads issued at once and kept as they came (bf16
// pairs), so that several CTAs fit on an SM; a block's maximum is a shuffle
// over those lanes, and over the CTA for a 128 x 128 block.  For the transpose
// the tile goes to shared memory by asynchronous copies, and a thread takes two
// neighbouring columns of 32 rows from there, so that it reads whole words
// without bank conflicts, once for the maximum and once more for the codes (so
// that six CTAs fit on an SM instead of three); the codes go through shared
// memory too, so that eight lanes write 128 bytes of a row of the result.
//
// Measured on a B200 (of the copy rate of 6.53 TB/s), calls in a graph, bf16: 12288 x
// 4096 by 128 x 128 blocks 26.4 us (87 %; 27.6 with ordinary stores; 28.7 a call, one
// after another from Python), fp32 39.6 (97 %); 4099 x 4096 transposed 11.4 us (68 %;
// 14.4 with codes written by columns and three CTAs per SM; 12.3 from Python), fp32
// 17.4 (74 %).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_fp8.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Two neighbouring elements and what is done with them.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
    uint32_t v;
    __device__ float lo() const { return __uint_as_float(v << 16); }
    __device__ float hi() const { return __uint_as_float(v & 0xFFFF0000u); }
};
template <>
struct Two<float> {
    float2 v;
    __device__ float lo() const { return v.x; }
    __device__ float hi() const { return v.y; }
};
// Running maxima of the magnitudes of both (a NaN is passed over).
__device__ __forceinline__ void max_abs(float2& m, Two<__nv_bfloat16> x) {
    m.x = fmaxf(m.x, fabsf(x.lo()));
    m.y = fmaxf(m.y, fabsf(x.hi()));
}
__device__ __forceinline__ void max_abs(float2& m, Two<float> x) {
    m.x = fmaxf(m.x, fabsf(x.v.x));
    m.y = fmaxf(m.y, fabsf(x.v.y));
}

// Eight elements of a row as they lie in memory.
template <typename T>
struct Row8 {
    Two<T> p[4];
    __device__ float max_abs8() const {
        float2 m = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) max_abs(m, p[i]);
        return fmaxf(m.x, m.y);
    }
    __device__ uint2 codes(float f) const {
        return make_uint2(
            fp8x4(p[0].lo() * f, p[0].hi() * f, p[1].lo() * f, p[1].hi() * f),
            fp8x4(p[2].lo() * f, p[2].hi() * f, p[3].lo() * f, p[3].hi() * f));
    }
};
__device__ __forceinline__ void load(Row8<__nv_bfloat16>& r, const __nv_bfloat16* p) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    r.p[0].v = u.x; r.p[1].v = u.y; r.p[2].v = u.z; r.p[3].v = u.w;
}
__device__ __forceinline__ void load(Row8<float>& r, const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    r.p[0].v = make_float2(a.x, a.y); r.p[1].v = make_float2(a.z, a.w);
    r.p[2].v = make_float2(b.x, b.y); r.p[3].v = make_float2(b.z, b.w);
}
__device__ __forceinline__ void set(Row8<__nv_bfloat16>& r, const __nv_bfloat16 (&e)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r.p[i].v = static_cast<uint32_t>(__bfloat16_as_ushort(e[2 * i + 1])) << 16 |
                   __bfloat16_as_ushort(e[2 * i]);
}
__device__ __forceinline__ void set(Row8<float>& r, const float (&e)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i].v = make_float2(e[2 * i], e[2 * i + 1]);
}

// Elements [c, c + 8) of row r, zeros outside the matrix.
template <typename T>
__device__ __forceinline__ Row8<T> row8(const T* x, int rows, int cols, bool vec, int r, int c) {
    Row8<T> v;
    const T* p = x + (size_t)r * cols + c;
    if (vec && r < rows && c < cols) {
        load(v, p);
    } else {
        T e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = r < rows && c + j < cols ? p[j] : from_f32<T>(0.f);
        set(v, e);
    }
    return v;
}

// Codes past L1 (they stay in L2 for the product that reads them).
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 v) {
    asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y)
                 : "memory");
}
__device__ __forceinline__ void store_codes(uint8_t* p, uint4 v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ float cta_max(float m, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
    __syncthreads();
    m = buf[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, buf[i]);
    return m;
}

template <typename T, bool kRowBlocks, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2)
    quantize_kernel(const T* __restrict__ x, int rows, int cols, int pitch,
                    uint8_t* __restrict__ y8, float* __restrict__ scale) {
    __shared__ float s_max[kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int KB = (cols + 127) / 128, RB = (rows + 127) / 128;
    const int kb = blockIdx.x % KB, rb = blockIdx.x / KB, c = kb * 128 + tx * 8;
    Row8<T> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = row8(x, rows, cols, kVec, rb * 128 + ty + 16 * i, c);
    float amax = 0.f;
    if (!kRowBlocks) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, v[i].max_abs8());
        amax = cta_max(amax, s_max);
        if (threadIdx.x == 0) scale[(size_t)kb * RB + rb] = fp8_scale(amax);
    }
    float f = fp8_factor(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = rb * 128 + ty + 16 * i;
        if (kRowBlocks) {
            amax = max16(v[i].max_abs8());
            f = fp8_factor(amax);
            if (tx == 0 && r < rows) scale[(size_t)kb * rows + r] = fp8_scale(amax);
        }
        if (r < rows && c < pitch) store_codes(y8 + (size_t)r * pitch + c, v[i].codes(f));
    }
}

// x [rows, cols] -> y8 [cols, pitch], pitch >= rows; blocks along x's rows.
template <typename T, bool kRowBlocks, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 3)
    quantize_t_kernel(const T* __restrict__ x, int rows, int cols, int pitch,
                      uint8_t* __restrict__ y8, float* __restrict__ scale) {
    extern __shared__ __align__(16) uint8_t q_smem[];
    T* tile = reinterpret_cast<T*>(q_smem);  // [128][128]
    __shared__ float s_col[4][128], s_max[kThreads / 32];
    const int CB = (cols + 127) / 128;
    const int cb = blockIdx.x % CB, kb = blockIdx.x / CB;  // column and row block of x
    if (kVec) {
        constexpr int PER = 16 / sizeof(T), CHUNKS = 128 / PER;  // 16-byte copies of a row
#pragma unroll
        for (int e = threadIdx.x; e < 128 * CHUNKS; e += kThreads) {
            const int r = e / CHUNKS, c = e % CHUNKS * PER;
            T* dst = tile + r * 128 + c;
            if (kb * 128 + r < rows && cb * 128 + c < cols)
                sm100::cp_async16(dst, x + (size_t)(kb * 128 + r) * cols + cb * 128 + c);
            else
                *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
        }
        sm100::cp_async_commit();
        sm100::cp_async_wait_all();
    } else {
#pragma unroll 8
        for (int e = threadIdx.x; e < 128 * 128; e += kThreads) {
            const int r = kb * 128 + e / 128, c = cb * 128 + e % 128;
            tile[e] = r < rows && c < cols ? x[(size_t)r * cols + c] : from_f32<T>(0.f);
        }
    }
    __syncthreads();
    // two columns of 32 rows
    const int pair = threadIdx.x & 63, rg = threadIdx.x >> 6;
    const int c = cb * 128 + 2 * pair;
    const T* mine = tile + rg * 32 * 128 + 2 * pair;
    float2 m = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int r = 0; r < 32; ++r) max_abs(m, *reinterpret_cast<const Two<T>*>(mine + r * 128));
    float f0, f1;
    if (kRowBlocks) {
        s_col[rg][2 * pair] = m.x;
        s_col[rg][2 * pair + 1] = m.y;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m.x = fmaxf(m.x, s_col[i][2 * pair]);
            m.y = fmaxf(m.y, s_col[i][2 * pair + 1]);
        }
        f0 = fp8_factor(m.x);
        f1 = fp8_factor(m.y);
        if (rg == 0) {
            if (c < cols) scale[(size_t)kb * cols + c] = fp8_scale(m.x);
            if (c + 1 < cols) scale[(size_t)kb * cols + c + 1] = fp8_scale(m.y);
        }
    } else {
        const float all = cta_max(fmaxf(m.x, m.y), s_max);
        if (threadIdx.x == 0) scale[(size_t)kb * CB + cb] = fp8_scale(all);
        f0 = f1 = fp8_factor(all);
    }
    uint4 q[2][2];  // [column][half of the 32 rows]
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            Two<T> w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = *reinterpret_cast<const Two<T>*>(mine + (16 * half + 4 * k + j) * 128);
            q0[k] = fp8x4(w[0].lo() * f0, w[1].lo() * f0, w[2].lo() * f0, w[3].lo() * f0);
            q1[k] = fp8x4(w[0].hi() * f1, w[1].hi() * f1, w[2].hi() * f1, w[3].hi() * f1);
        }
        q[0][half] = make_uint4(q0[0], q0[1], q0[2], q0[3]);
        q[1][half] = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    }
    __syncthreads();  // x has been read: the codes take its place, [column][144 bytes]
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int half = 0; half < 2; ++half)
            *reinterpret_cast<uint4*>(q_smem + (2 * pair + e) * 144 + rg * 32 + half * 16) = q[e][half];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // eight lanes a row of the result
        const int e = threadIdx.x + i * kThreads, row = e >> 3, piece = e & 7;
        if (cb * 128 + row < cols && kb * 128 + piece * 16 < pitch)
            store_codes(y8 + (size_t)(cb * 128 + row) * pitch + kb * 128 + piece * 16,
                        *reinterpret_cast<const uint4*>(q_smem + row * 144 + piece * 16));
    }
}

template <typename T, bool kRowBlocks, bool kVec>
cudaError_t quantize_case(const void* x, int rows, int cols, bool transpose, void* y8,
                          float* scale, cudaStream_t st) {
    const long long tiles = (long long)blocks128(cols) * blocks128(rows);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(tiles);
    const T* X = static_cast<const T*>(x);
    uint8_t* Y = static_cast<uint8_t*>(y8);
    if (!transpose) {
        quantize_kernel<T, kRowBlocks, kVec>
            <<<grid, kThreads, 0, st>>>(X, rows, cols, fp8_pitch(cols), Y, scale);
        return cudaGetLastError();
    }
    constexpr int bytes = 128 * 128 * sizeof(T);
    const cudaError_t e = cudaFuncSetAttribute(quantize_t_kernel<T, kRowBlocks, kVec>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    quantize_t_kernel<T, kRowBlocks, kVec>
        <<<grid, kThreads, bytes, st>>>(X, rows, cols, fp8_pitch(rows), Y, scale);
    return cudaGetLastError();
}

// Rows of x start on a 16-byte boundary, and eight columns are all inside or
// all outside, when cols is a multiple of 8; other sizes load element by element.
template <typename T>
cudaError_t quantize_type(const void* x, int rows, int cols, bool row_blocks, bool transpose,
                          void* y8, float* scale, cudaStream_t st) {
    if (cols % 8 == 0)
        return row_blocks ? quantize_case<T, true, true>(x, rows, cols, transpose, y8, scale, st)
                          : quantize_case<T, false, true>(x, rows, cols, transpose, y8, scale, st);
    return row_blocks ? quantize_case<T, true, false>(x, rows, cols, transpose, y8, scale, st)
                      : quantize_case<T, false, false>(x, rows, cols, transpose, y8, scale, st);
}

}  // namespace

cudaError_t launch_quantize(const void* x, int rows, int cols, kda_dtype_t dt, bool row_blocks,
                            bool transpose, void* y8, float* scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    return dt == KDA_DTYPE_BF16
               ? quantize_type<__nv_bfloat16>(x, rows, cols, row_blocks, transpose, y8, scale, st)
               : quantize_type<float>(x, rows, cols, row_blocks, transpose, y8, scale, st);
}

}  // namespace kda

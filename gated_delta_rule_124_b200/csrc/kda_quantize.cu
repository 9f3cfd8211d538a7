// A matrix to 8 bits with a scale per block of 128 columns of a row, or per
// 128 x 128 block, in the orientation that the 8-bit product reads: the matrix
// itself or its transpose.
//
// Elements are read once and written once as one byte: bound by HBM.  A CTA of
// 256 threads takes a 128 x 128 tile of x, a row's 128 columns in 16 lanes,
// eight rows a thread, all loads issued at once; a block's maximum is a
// shuffle over those lanes, and over the CTA for a 128 x 128 block.  For the
// transpose the tile goes through shared memory, where a thread takes two
// neighbouring columns of 32 rows, so that it reads whole words without bank
// conflicts and writes whole 32-byte sectors of two rows of the result.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;  // vectors of eight elements: rows ty, ty + 16, ...

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

template <typename T>
__device__ __forceinline__ void load_row8(const T* x, int rows, int cols, bool vec, int r, int c,
                                          float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (r >= rows || c >= cols) return;
    const T* p = x + (size_t)r * cols + c;
    if (vec) {
        load_vec8(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c + j < cols) v[j] = to_f32(p[j]);
    }
}

template <typename T, bool kRowBlocks>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const T* __restrict__ x, int rows,
                                                            int cols, int pitch, bool vec,
                                                            uint8_t* __restrict__ y8,
                                                            float* __restrict__ scale) {
    __shared__ float s_max[kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int KB = (cols + 127) / 128, RB = (rows + 127) / 128;
    const int kb = blockIdx.x % KB, rb = blockIdx.x / KB, c = kb * 128 + tx * 8;
    float v[kPerThread][8];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
        load_row8(x, rows, cols, vec, rb * 128 + ty + 16 * i, c, v[i]);
    float amax = 0.f;
    if (!kRowBlocks) {
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) amax = fmaxf(amax, max_abs8(v[i]));
        amax = cta_max(amax, s_max);
        if (threadIdx.x == 0) scale[(size_t)kb * RB + rb] = fp8_scale(amax);
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int r = rb * 128 + ty + 16 * i;
        if (kRowBlocks) {
            amax = max16(max_abs8(v[i]));
            if (tx == 0 && r < rows) scale[(size_t)kb * rows + r] = fp8_scale(amax);
        }
        if (r < rows && c < pitch)
            *reinterpret_cast<uint2*>(y8 + (size_t)r * pitch + c) = quantize8(v[i], fp8_factor(amax));
    }
}

// x [rows, cols] -> y8 [cols, pitch], pitch >= rows; blocks along x's rows.
template <typename T, bool kRowBlocks>
__global__ void __launch_bounds__(kThreads) quantize_t_kernel(const T* __restrict__ x, int rows,
                                                              int cols, int pitch, bool vec,
                                                              uint8_t* __restrict__ y8,
                                                              float* __restrict__ scale) {
    extern __shared__ __align__(16) uint8_t q_smem[];
    T* tile = reinterpret_cast<T*>(q_smem);  // [128][128]
    __shared__ float s_col[4][128], s_max[kThreads / 32];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int CB = (cols + 127) / 128;
    const int cb = blockIdx.x % CB, kb = blockIdx.x / CB;  // column and row block of x
    float all = 0.f;
    float v[kPerThread][8];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
        load_row8(x, rows, cols, vec, kb * 128 + ty + 16 * i, cb * 128 + tx * 8, v[i]);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (!kRowBlocks) all = fmaxf(all, max_abs8(v[i]));
        store_vec8(tile + (ty + 16 * i) * 128 + tx * 8, v[i]);
    }
    if (!kRowBlocks) {
        all = cta_max(all, s_max);
        if (threadIdx.x == 0) scale[(size_t)kb * CB + cb] = fp8_scale(all);
    }
    __syncthreads();
    // two columns of 32 rows
    const int pair = threadIdx.x & 63, rg = threadIdx.x >> 6;
    const int c = cb * 128 + 2 * pair;
    float f[2];
    if (kRowBlocks) {
        float m0 = 0.f, m1 = 0.f;
#pragma unroll 8
        for (int r = 0; r < 32; ++r) {
            const T* p = tile + (rg * 32 + r) * 128 + 2 * pair;
            m0 = fmaxf(m0, fabsf(to_f32(p[0])));
            m1 = fmaxf(m1, fabsf(to_f32(p[1])));
        }
        s_col[rg][2 * pair] = m0;
        s_col[rg][2 * pair + 1] = m1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float m = s_col[0][2 * pair + j];
#pragma unroll
            for (int i = 1; i < 4; ++i) m = fmaxf(m, s_col[i][2 * pair + j]);
            f[j] = fp8_factor(m);
            if (rg == 0 && c + j < cols) scale[(size_t)kb * cols + c + j] = fp8_scale(m);
        }
    } else {
        f[0] = f[1] = fp8_factor(all);
    }
    uint32_t q0[8], q1[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const T* p = tile + (rg * 32 + 4 * k + j) * 128 + 2 * pair;
            a[j] = to_f32(p[0]) * f[0];
            b[j] = to_f32(p[1]) * f[1];
        }
        q0[k] = fp8x4(a[0], a[1], a[2], a[3]);
        q1[k] = fp8x4(b[0], b[1], b[2], b[3]);
    }
    const int r0 = kb * 128 + rg * 32;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (r0 + 16 * half >= pitch) continue;
        if (c < cols)
            *reinterpret_cast<uint4*>(y8 + (size_t)c * pitch + r0 + 16 * half) =
                make_uint4(q0[4 * half], q0[4 * half + 1], q0[4 * half + 2], q0[4 * half + 3]);
        if (c + 1 < cols)
            *reinterpret_cast<uint4*>(y8 + (size_t)(c + 1) * pitch + r0 + 16 * half) =
                make_uint4(q1[4 * half], q1[4 * half + 1], q1[4 * half + 2], q1[4 * half + 3]);
    }
}

template <typename T, bool kRowBlocks>
cudaError_t quantize_case(const void* x, int rows, int cols, bool transpose, void* y8,
                          float* scale, cudaStream_t st) {
    const long long tiles = (long long)blocks128(cols) * blocks128(rows);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned grid = static_cast<unsigned>(tiles);
    // rows of x start on a 16-byte boundary when cols is a multiple of 8
    const bool vec = cols % 8 == 0;
    const T* X = static_cast<const T*>(x);
    uint8_t* Y = static_cast<uint8_t*>(y8);
    if (!transpose) {
        quantize_kernel<T, kRowBlocks>
            <<<grid, kThreads, 0, st>>>(X, rows, cols, fp8_pitch(cols), vec, Y, scale);
        return cudaGetLastError();
    }
    constexpr int bytes = 128 * 128 * sizeof(T);
    const cudaError_t e = cudaFuncSetAttribute(quantize_t_kernel<T, kRowBlocks>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    quantize_t_kernel<T, kRowBlocks>
        <<<grid, kThreads, bytes, st>>>(X, rows, cols, fp8_pitch(rows), vec, Y, scale);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const void* x, int rows, int cols, kda_dtype_t dt, bool row_blocks,
                            bool transpose, void* y8, float* scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    if (dt == KDA_DTYPE_BF16)
        return row_blocks
                   ? quantize_case<__nv_bfloat16, true>(x, rows, cols, transpose, y8, scale, st)
                   : quantize_case<__nv_bfloat16, false>(x, rows, cols, transpose, y8, scale, st);
    return row_blocks ? quantize_case<float, true>(x, rows, cols, transpose, y8, scale, st)
                      : quantize_case<float, false>(x, rows, cols, transpose, y8, scale, st);
}

}  // namespace kda

// RMS norm with the residual's addition, and its backward.
//
//   s = x + residual (held in the inputs' type, the layer's running residual)
//   y = s / sqrt(mean(s^2) + eps) * w, in the inputs' type and/or in 8 bits
//       with a scale per row and block of 128 columns
//
// The norm is taken of the stored (rounded) s, so that a backward pass that
// reads s differentiates the function that was evaluated.  A row is read once
// and written once: the kernels are bound by HBM.  A row belongs to TPR
// threads, each with VPT vectors of eight elements (16 bytes of bf16) in
// registers; vector i of thread t is i TPR + t of the row, so that a block of
// 128 columns is 16 consecutive lanes and its maximum four shuffles.  CTAs
// walk over rows, keep w in registers and request the next row before they
// reduce the present one.
//
// Backward, with r = 1 / sqrt(mean(s^2) + eps):
//   dx = dsum + r (w dy - s r^2 mean(s w dy))      (also the residual's gradient)
//   dw = sum over rows of dy s r
// dw is summed per thread over the CTA's rows, then over the CTAs in a second
// kernel, in a fixed order.
//
// Measured on a B200 (of the copy rate of 6.53 TB/s), bf16, calls in a graph: 16391 x
// 4096 with a residual to 8 bits 74 us (98 %; 77 with loads marked as streaming; 82 a
// call, one after another from Python), 16 rows 3.2 (15); fp32 153 (87 %); backward of
// 8192 x 4096 47 us (88 %, 4 of it the second kernel; 51 from Python).  Few CTAs hold
// short rows' backward back: 16384 x 2048 60 us (69 %), 32768 x 1024 95 (43 %), 32768 x
// 512 83 (25 %).  Without the
// request of the next row ahead of the reduction a row's loads would wait for the
// row before.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_fp8.cuh"

namespace kda {
namespace {

// Row groups that sum their own dw: two CTAs for each of a B200's 148 SMs where a
// CTA has one row (D > 1024), one or half a one where it has two or four.
constexpr int kMaxParts = 296;

template <int TPR>
struct RowGroup {
    static constexpr int kThreads = TPR < 128 ? 128 : TPR;
    static constexpr int kRowsPerCta = kThreads / TPR;
    // CTAs of an SM (768 threads forward, 512 backward: the registers allow it)
    static constexpr int kForward = 768 / kThreads;
    static constexpr int kBackward = 512 / kThreads;
};

// Sum over the TPR threads of a row (every thread gets it).  `buf` holds one
// value per warp; consecutive calls alternate between two buffers, so that one
// barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (TPR == 32) return x;
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = x;
    __syncthreads();
    const float* mine = buf + warp / W * W;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += mine[i];
    return s;
}

// The same for two sums at once.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 x, float2* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
    }
    if (TPR == 32) return x;
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) buf[warp] = x;
    __syncthreads();
    const float2* mine = buf + warp / W * W;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s.x += mine[i].x;
        s.y += mine[i].y;
    }
    return s;
}

template <typename T>
__device__ __forceinline__ float stored(float x) { return to_f32(from_f32<T>(x)); }

// A row's vectors of this thread, zeros beyond the row or the last row.
template <typename T, int TPR, int VPT>
__device__ __forceinline__ void load_row(Vec8<T> (&v)[VPT], const T* p, long long row, int rows,
                                         int D, int t) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * 8;
        v[i].zero();
        if (row < rows && c < D) v[i].load(p + row * D + c);
    }
}

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(RowGroup<TPR>::kThreads, RowGroup<TPR>::kForward)
    add_rms_norm_kernel(const T* x, const T* residual, const float* __restrict__ w, int rows,
                        int D, int pitch, float eps, T* sum, T* y, uint8_t* y8, float* y8_scale) {
    using G = RowGroup<TPR>;
    __shared__ float s_part[2][G::kThreads / 32];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const long long step = (long long)gridDim.x * G::kRowsPerCta;
    long long base = (long long)blockIdx.x * G::kRowsPerCta;
    Vec8<T> xv[VPT], rv[VPT];
    load_row<T, TPR, VPT>(xv, x, base + sub, rows, D, t);
    if (residual) load_row<T, TPR, VPT>(rv, residual, base + sub, rows, D, t);
    float wv[VPT][8];
    {
        Vec8<float> q[VPT];
        load_row<float, TPR, VPT>(q, w, 0, 1, D, t);
#pragma unroll
        for (int i = 0; i < VPT; ++i) q[i].get(wv[i]);
    }
    for (int flip = 0; base < rows; base += step, flip ^= 1) {
        const long long row = base + sub;
        const bool live = row < rows;
        float v[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            xv[i].get(v[i]);
            if (residual) {
                float r8[8];
                rv[i].get(r8);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = stored<T>(v[i][j] + r8[j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        }
        load_row<T, TPR, VPT>(xv, x, row + step, rows, D, t);
        if (residual) load_row<T, TPR, VPT>(rv, residual, row + step, rows, D, t);
        if (sum) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = (i * TPR + t) * 8;
                if (live && c < D) store_vec8(sum + row * D + c, v[i]);
            }
        }
        const float r = 1.f / sqrtf(row_sum<TPR>(ss, s_part[flip]) / D + eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * r * wv[i][j];
            if (y && live && c < D) store_vec8(y + row * D + c, v[i]);
            if (y8) {
                const float amax = max16(max_abs8(v[i]));
                // (behind D zeros, in a row of NaN too)
                if (live && c < pitch)
                    *reinterpret_cast<uint2*>(y8 + row * pitch + c) =
                        c < D ? quantize8(v[i], fp8_factor(amax)) : make_uint2(0u, 0u);
                if (live && c < D && (t & 15) == 0)
                    y8_scale[(size_t)(c / 128) * rows + row] = fp8_scale(amax);
            }
        }
    }
}

template <typename T, int TPR, int VPT>
__global__ void __launch_bounds__(RowGroup<TPR>::kThreads, RowGroup<TPR>::kBackward)
    add_rms_norm_bwd_kernel(const T* __restrict__ s, const float* __restrict__ w,
                            const T* __restrict__ dy, const T* dsum, int rows, int D, float eps,
                            T* dx, float* __restrict__ parts) {
    using G = RowGroup<TPR>;
    __shared__ float2 s_part[2][G::kThreads / 32];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const long long step = (long long)gridDim.x * G::kRowsPerCta;
    long long base = (long long)blockIdx.x * G::kRowsPerCta;
    // (four vectors a thread leave no registers for the next row's)
    constexpr bool kAhead = VPT <= 2;
    Vec8<T> sv[VPT], dv[VPT], av[VPT];
    auto load_rows = [&](long long row) {
        load_row<T, TPR, VPT>(sv, s, row, rows, D, t);
        load_row<T, TPR, VPT>(dv, dy, row, rows, D, t);
        if (dsum) load_row<T, TPR, VPT>(av, dsum, row, rows, D, t);
    };
    if (kAhead) load_rows(base + sub);
    float dw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    for (int flip = 0; base < rows; base += step, flip ^= 1) {
        const long long row = base + sub;
        const bool live = row < rows;
        if (!kAhead) load_rows(row);
        float v[VPT][8], d[VPT][8], add[VPT][8];
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * 8;
            float wv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (c < D) {
                *reinterpret_cast<float4*>(wv) = *reinterpret_cast<const float4*>(w + c);
                *reinterpret_cast<float4*>(wv + 4) = *reinterpret_cast<const float4*>(w + c + 4);
            }
            sv[i].get(v[i]);
            dv[i].get(d[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) add[i][j] = 0.f;
            if (dsum) av[i].get(add[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(v[i][j], v[i][j], ss);
                sd = fmaf(v[i][j], wv[j] * d[i][j], sd);
            }
        }
        // (dsum may be dx: a row is written by the threads that read it)
        if (kAhead) load_rows(row + step);
        const float2 sums = row_sum<TPR>(make_float2(ss, sd), s_part[flip]);
        const float r = 1.f / sqrtf(sums.x / D + eps), m = r * r * (sums.y / D);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * 8;
            if (!live || c >= D) continue;
            float wv[8], out[8];
            *reinterpret_cast<float4*>(wv) = *reinterpret_cast<const float4*>(w + c);
            *reinterpret_cast<float4*>(wv + 4) = *reinterpret_cast<const float4*>(w + c + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(d[i][j], v[i][j] * r, dw[i][j]);
                out[j] = fmaf(r, wv[j] * d[i][j] - v[i][j] * m, add[i][j]);
            }
            store_vec8(dx + row * D + c, out);
        }
    }
    float* mine = parts + ((size_t)blockIdx.x * G::kRowsPerCta + sub) * D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c < D) store_vec8(mine + c, dw[i]);
    }
}

// dw[c] = sum over parts, 32 columns a CTA: 32 warps take every 32nd part, all
// loads of a warp in flight at once (the parts are in L2: bound by latency), then
// one warp adds their sums.
constexpr int kSumWarps = 32;
constexpr int kPartsPerWarp = (kMaxParts + kSumWarps - 1) / kSumWarps;
__global__ void __launch_bounds__(32 * kSumWarps) sum_parts_kernel(const float* __restrict__ parts,
                                                                   int n, int D,
                                                                   float* __restrict__ dw) {
    __shared__ float s_sum[kSumWarps][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v[kPartsPerWarp];
#pragma unroll
    for (int u = 0; u < kPartsPerWarp; ++u) {
        const int i = w + u * kSumWarps;
        v[u] = i < n && c < D ? parts[(size_t)i * D + c] : 0.f;
    }
    float acc = 0.f;
#pragma unroll
    for (int u = 0; u < kPartsPerWarp; ++u) acc += v[u];
    s_sum[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < D) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) x += s_sum[i][lane];
        dw[c] = x;
    }
}

// CTAs that walk over `rows` rows: as many as fit on the device, `per_sm` each.
cudaError_t walkers(int rows, int rows_per_cta, int per_sm, unsigned* grid) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long ctas = ((long long)rows + rows_per_cta - 1) / rows_per_cta;
    const long long most = (long long)sms * per_sm;
    *grid = static_cast<unsigned>(ctas < most ? ctas : most);
    return e;
}

template <typename T, int TPR, int VPT>
cudaError_t norm_case(const void* x, const void* residual, const float* w, int rows, int D,
                      float eps, void* sum, void* y, void* y8, float* y8_scale, cudaStream_t st) {
    using G = RowGroup<TPR>;
    unsigned grid = 0;
    const cudaError_t e = walkers(rows, G::kRowsPerCta, G::kForward, &grid);
    if (e != cudaSuccess) return e;
    add_rms_norm_kernel<T, TPR, VPT><<<grid, G::kThreads, 0, st>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), w, rows, D, fp8_pitch(D), eps,
        static_cast<T*>(sum), static_cast<T*>(y), static_cast<uint8_t*>(y8), y8_scale);
    return cudaGetLastError();
}

template <typename T, int TPR, int VPT>
cudaError_t norm_bwd_case(const void* s, const float* w, const void* dy, const void* dsum,
                          int rows, int D, float eps, void* dx, float* dw, void* ws,
                          cudaStream_t st) {
    using G = RowGroup<TPR>;
    constexpr int most = kMaxParts / G::kRowsPerCta;
    const long long ctas = ((long long)rows + G::kRowsPerCta - 1) / G::kRowsPerCta;
    const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
    float* parts = static_cast<float*>(ws);
    if (grid > 0)
        add_rms_norm_bwd_kernel<T, TPR, VPT><<<grid, G::kThreads, 0, st>>>(
            static_cast<const T*>(s), w, static_cast<const T*>(dy), static_cast<const T*>(dsum),
            rows, D, eps, static_cast<T*>(dx), parts);
    sum_parts_kernel<<<(D + 31) / 32, 32 * kSumWarps, 0, st>>>(
        parts, static_cast<int>(grid) * G::kRowsPerCta, D, dw);
    return cudaGetLastError();
}

// A row's threads and vectors by its length: two vectors a thread keep enough
// loads in flight without the registers that would lower the occupancy.
#define KDA_BY_ROW_LENGTH(CALL)       \
    if (D <= 512) return CALL(32, 2); \
    if (D <= 1024) return CALL(64, 2); \
    if (D <= 2048) return CALL(128, 2); \
    if (D <= 4096) return CALL(256, 2); \
    if (D <= 8192) return CALL(512, 2); \
    return CALL(512, 4);

template <typename T>
cudaError_t norm_dispatch(const void* x, const void* residual, const float* w, int rows, int D,
                          float eps, void* sum, void* y, void* y8, float* y8_scale,
                          cudaStream_t st) {
#define KDA_CALL(TPR, VPT) \
    norm_case<T, TPR, VPT>(x, residual, w, rows, D, eps, sum, y, y8, y8_scale, st)
    KDA_BY_ROW_LENGTH(KDA_CALL)
#undef KDA_CALL
}

template <typename T>
cudaError_t norm_bwd_dispatch(const void* s, const float* w, const void* dy, const void* dsum,
                              int rows, int D, float eps, void* dx, float* dw, void* ws,
                              cudaStream_t st) {
#define KDA_CALL(TPR, VPT) norm_bwd_case<T, TPR, VPT>(s, w, dy, dsum, rows, D, eps, dx, dw, ws, st)
    KDA_BY_ROW_LENGTH(KDA_CALL)
#undef KDA_CALL
}

}  // namespace

size_t rms_norm_bwd_workspace_bytes(int rows, int D) {
    const int parts = rows < kMaxParts ? (rows + 3) / 4 * 4 : kMaxParts;  // whole CTAs of <= 4 rows
    return align_up(sizeof(float) * (size_t)(parts > 0 ? parts : 4) * D);
}

cudaError_t launch_add_rms_norm(const void* x, const void* residual, const float* w, int rows,
                                int D, kda_dtype_t dt, float eps, void* sum, void* y, void* y8,
                                float* y8_scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    if (dt == KDA_DTYPE_BF16)
        return norm_dispatch<__nv_bfloat16>(x, residual, w, rows, D, eps, sum, y, y8, y8_scale, st);
    return norm_dispatch<float>(x, residual, w, rows, D, eps, sum, y, y8, y8_scale, st);
}

cudaError_t launch_add_rms_norm_bwd(const void* s, const float* w, const void* dy,
                                    const void* dsum, int rows, int D, kda_dtype_t dt, float eps,
                                    void* dx, float* dw, void* workspace, cudaStream_t st) {
    if (dt == KDA_DTYPE_BF16)
        return norm_bwd_dispatch<__nv_bfloat16>(s, w, dy, dsum, rows, D, eps, dx, dw, workspace, st);
    return norm_bwd_dispatch<float>(s, w, dy, dsum, rows, D, eps, dx, dw, workspace, st);
}

}  // namespace kda

// The 8-bit product of few rows (a decode step's tokens) and a weight of a round or
// two: out [M, N] = A B^T for M <= 16, as in kda_fp8_matmul.cu.
//
// B (a weight) is read once and nothing else is large: the call is bound by HBM,
// and at its few microseconds by latency.  So everything a CTA needs is requested
// at its start and waited for once: sixteen warps take 32 rows of B, a warp 16 of
// them and every eighth block of 128 columns, its rows' bytes of up to four
// blocks (4096 columns a round) straight into registers; A's rows and the scales
// go to shared memory by asynchronous copies before them (they are in L2 and
// arrive first).  The products are warp-level ones of f16 values (every e4m3
// number is one; fp32 accumulation), B's bytes converted once for all of A's
// rows: the e4m3 form of these products converts both operands for every eight
// rows of A, 2.4 us more for 16 rows.  Inside a block lane q of a row holds bytes
// [32 q, 32 q + 32) of A and B alike: the products take K in an order of their
// own, the same for both, and a lane loads whole 32-byte sectors.  A block's
// products are added to fp32 sums with its scales; the warps' sums are added in
// a fixed order.
//
// Measured on a B200, weights from HBM, calls in a graph: 4096 x 4096 with 8 rows 6.2
// us, with 16 8.3 (2.6 at the copy rate; 11.6 a call from Python); 12288 x 4096 with 8
// rows 15.0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kGroups = 2;                  // of 16 rows of B
constexpr int kWays = 8;                    // warps that share a group's blocks
constexpr int kThreads = 32 * kGroups * kWays;
constexpr int kRowsB = 16 * kGroups;
constexpr int kAhead = 4;                   // blocks of a warp a round
constexpr int kBlocks = kWays * kAhead;     // blocks of a round
constexpr int kPitchA = kBlocks * 128 + 16; // bytes of A's rows in shared memory (bank shift)

struct SmallArgs {
    const uint8_t* a8;
    const float* sa;
    const uint8_t* b8;
    const float* sb;
    void* out;
    int M, N, K, KB, NB, pitch, out_bf16;
};

// MT: groups of eight rows of A.
template <int MT>
struct SmallSmem {
    union {
        uint8_t a[MT * 8 * kPitchA];
        float part[kWays][kRowsB][MT * 8 + 1];
    };
    float sa[kBlocks][MT * 8];
    float sb[kBlocks][kRowsB];  // (one column where a scale covers 128 rows)
};

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sm100::smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

struct Bytes32 {
    uint32_t w[8];
};
// 32 bytes of a row of B from byte c on (nothing beyond the row's `pitch`).
template <bool kWide>
__device__ __forceinline__ void load32(Bytes32& r, const uint8_t* row, int c, int pitch) {
    if constexpr (kWide) {  // rows start on 32 bytes
        if (c < pitch)
            asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                           "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                         : "l"(row + c));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c + 16 * h >= pitch) continue;
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + c) + h);
            r.w[4 * h] = v.x; r.w[4 * h + 1] = v.y; r.w[4 * h + 2] = v.z; r.w[4 * h + 3] = v.w;
        }
    }
}
// Zeros in the place of bytes from K on (c: the first byte's column).
__device__ __forceinline__ uint32_t cut(uint32_t w, int c, int K) {
    const int left = K - c;
    return left <= 0 ? 0u : left < 4 ? w & ((1u << (8 * left)) - 1u) : w;
}
__device__ __forceinline__ void cut(Bytes32& r, int c, int K) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = cut(r.w[i], c + 4 * i, K);
}
__device__ __forceinline__ void cut(uint4& r, int c, int K) {
    r = make_uint4(cut(r.x, c, K), cut(r.y, c + 4, K), cut(r.z, c + 8, K), cut(r.w, c + 12, K));
}

// The four e4m3 values of a word as two pairs of f16 (a NaN stays one).
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int MT, bool kRowScales, bool kWide>
__global__ void __launch_bounds__(kThreads, 1) fp8_small_kernel(const SmallArgs a) {
    extern __shared__ __align__(16) uint8_t small_smem[];
    SmallSmem<MT>& sm = *reinterpret_cast<SmallSmem<MT>*>(small_smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int group = warp / kWays, way = warp % kWays;
    const int n0 = blockIdx.x * kRowsB, r0 = 16 * group + g;
    // rows beyond the last one read the last one again; they are not written
    const uint8_t* b0 = a.b8 + (size_t)min(n0 + r0, a.N - 1) * a.pitch;
    const uint8_t* b1 = a.b8 + (size_t)min(n0 + r0 + 8, a.N - 1) * a.pitch;
    float sum[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[t][i] = 0.f;

    for (int base = 0; base < a.KB; base += kBlocks) {
        const int blocks = min(kBlocks, a.KB - base);
        if (base > 0) __syncthreads();  // the last round's A has been read
        const int pieces = min(blocks * 128, a.pitch - base * 128) / 16;
        for (int m = warp; m < a.M; m += kThreads / 32)
            for (int j = lane; j < pieces; j += 32) {
                // (every CTA copies the same rows: each begins elsewhere)
                const int i = (j + blockIdx.x * 37) % pieces;
                sm100::cp_async16(sm.a + m * kPitchA + 16 * i,
                                  a.a8 + (size_t)m * a.pitch + base * 128 + 16 * i);
            }
        for (int e = threadIdx.x; e < blocks * a.M; e += kThreads) {
            const int kb = e / a.M, m = e % a.M;
            cp_async4(&sm.sa[kb][m], a.sa + (size_t)(base + kb) * a.M + m);
        }
        if (kRowScales) {
            for (int e = threadIdx.x; e < blocks * kRowsB; e += kThreads) {
                const int kb = e / kRowsB, r = e % kRowsB;
                if (n0 + r < a.N)
                    cp_async4(&sm.sb[kb][r], a.sb + (size_t)(base + kb) * a.NB + n0 + r);
            }
        } else if (threadIdx.x < blocks) {
            cp_async4(&sm.sb[threadIdx.x][0],
                      a.sb + (size_t)(base + threadIdx.x) * a.NB + n0 / 128);
        }
        sm100::cp_async_commit();
        Bytes32 x0[kAhead], x1[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int kb = base + way + u * kWays;
            if (kb < a.KB) {
                load32<kWide>(x0[u], b0, kb * 128 + 32 * q, a.pitch);
                load32<kWide>(x1[u], b1, kb * 128 + 32 * q, a.pitch);
            }
        }
        sm100::cp_async_wait_all();
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = way + u * kWays, c = (base + i) * 128 + 32 * q;
            if (i >= blocks) break;
            const bool last = (base + i + 1) * 128 > a.K;  // K ends inside the block
            if (last) {
                cut(x0[u], c, a.K);
                cut(x1[u], c, a.K);
            }
            const float f0 = sm.sb[i][kRowScales ? r0 : 0], f1 = sm.sb[i][kRowScales ? r0 + 8 : 0];
            float d[MT][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[t][e] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 of the lane's 32 bytes
                uint4 y[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    y[t] = *reinterpret_cast<const uint4*>(sm.a + (8 * t + g) * kPitchA + i * 128 +
                                                           32 * q + 16 * h);
                    if (last) cut(y[t], c + 16 * h, a.K);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t f[4];
                    to_f16(x0[u].w[4 * h + j], f[0], f[2]);
                    to_f16(x1[u].w[4 * h + j], f[1], f[3]);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const uint32_t w = j == 0 ? y[t].x : j == 1 ? y[t].y : j == 2 ? y[t].z : y[t].w;
                        uint32_t lo, hi;
                        to_f16(w, lo, hi);
                        mma_f16(d[t], f[0], f[1], f[2], f[3], lo, hi);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float s0 = sm.sa[i][8 * t + 2 * q], s1 = sm.sa[i][8 * t + 2 * q + 1];
                sum[t][0] = fmaf(d[t][0], f0 * s0, sum[t][0]);
                sum[t][1] = fmaf(d[t][1], f0 * s1, sum[t][1]);
                sum[t][2] = fmaf(d[t][2], f1 * s0, sum[t][2]);
                sum[t][3] = fmaf(d[t][3], f1 * s1, sum[t][3]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        sm.part[way][r0][8 * t + 2 * q] = sum[t][0];
        sm.part[way][r0][8 * t + 2 * q + 1] = sum[t][1];
        sm.part[way][r0 + 8][8 * t + 2 * q] = sum[t][2];
        sm.part[way][r0 + 8][8 * t + 2 * q + 1] = sum[t][3];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kRowsB * MT * 8; e += kThreads) {
        const int r = e % kRowsB, m = e / kRowsB;
        if (n0 + r >= a.N || m >= a.M) continue;
        float v = sm.part[0][r][m];
#pragma unroll
        for (int w = 1; w < kWays; ++w) v += sm.part[w][r][m];
        const size_t o = (size_t)m * a.N + n0 + r;
        if (a.out_bf16)
            static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
        else
            static_cast<float*>(a.out)[o] = v;
    }
}

template <int MT, bool kRowScales, bool kWide>
cudaError_t run(const SmallArgs& a, cudaStream_t st) {
    constexpr int bytes = sizeof(SmallSmem<MT>);
    const cudaError_t e =
        cudaFuncSetAttribute(fp8_small_kernel<MT, kRowScales, kWide>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const unsigned grid = (static_cast<unsigned>(a.N) + kRowsB - 1) / kRowsB;
    fp8_small_kernel<MT, kRowScales, kWide><<<grid, kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}
template <int MT>
cudaError_t run_mt(const SmallArgs& a, bool b_rows, cudaStream_t st) {
    const bool wide = a.pitch % 32 == 0 && reinterpret_cast<uintptr_t>(a.b8) % 32 == 0;
    if (b_rows) return wide ? run<MT, true, true>(a, st) : run<MT, true, false>(a, st);
    return wide ? run<MT, false, true>(a, st) : run<MT, false, false>(a, st);
}

}  // namespace

cudaError_t launch_fp8_small(const void* a8, const float* a_scale, const void* b8,
                             const float* b_scale, int M, int N, int K, bool b_rows,
                             kda_dtype_t out_dt, void* out, cudaStream_t st) {
    SmallArgs a;
    a.a8 = static_cast<const uint8_t*>(a8);
    a.sa = a_scale;
    a.b8 = static_cast<const uint8_t*>(b8);
    a.sb = b_scale;
    a.out = out;
    a.M = M;
    a.N = N;
    a.K = K;
    a.KB = blocks128(K);
    a.NB = b_rows ? N : blocks128(N);
    a.pitch = fp8_pitch(K);
    a.out_bf16 = out_dt == KDA_DTYPE_BF16;
    if (M <= 8) return run_mt<1>(a, b_rows, st);
    return run_mt<2>(a, b_rows, st);
}

}  // namespace kda

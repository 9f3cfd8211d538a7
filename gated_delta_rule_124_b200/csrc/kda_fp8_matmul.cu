// out = A B^T of two 8-bit matrices with a scale per block of 128 along K:
//   out[m, n] = sum_kb sa[kb, m] sb[kb, n] sum_{k in block kb} a8[m, k] b8[n, k]
// (sb per row of B, or per 128 rows).
//
// The inner sums are e4m3 products on the tensor cores (tcgen05,
// kind::f8f6f4, fp32 accumulation); the scales differ from block to block, so
// every block's 128 x BM partial product leaves tensor memory and is added to
// fp32 sums in registers with its scales.  One CTA per SM walks over output
// tiles:
//   warp 0      TMA loads of both operands' blocks (128-byte rows, the swizzled
//               K-major layout the products read), a ring of stages;
//   warp 1      the products of a block (four of K = 32) into one of the
//               tensor-memory buffers;
//   warps 2, 3  the block's scales into shared memory;
//   warps 4-11  out += scale * partial product, then the tile's output.
// B's rows (a weight's outputs) are the 128 lanes of tensor memory and A's rows
// (tokens) its columns: the column count BM then follows the number of tokens,
// from 16 in a decode step to 256, and a warp writes 32 neighbouring outputs of
// one token.  In the lanes' layout a column's scale is shared by a warp, so it
// is read from shared memory as a broadcast; with sb per 128 rows it is one
// number for the tile and is multiplied into the columns' scales beforehand.
//
// Large products are bound by the tensor cores and the partial products' way
// out of tensor memory, small ones by reading B once.  With few tiles the K
// blocks are split over a cluster of up to 8 CTAs, which add their partial
// tiles through distributed shared memory in a fixed order.
//
// Every wait is bounded; a tile whose waits gave up is written as NaN.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kRowsB = 128;                       // lanes of a tile
constexpr uint32_t kTileB = kRowsB * 128;         // bytes of B's block
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kScaleSlots = 4;
constexpr int kMaxSplit = 8;

template <int BM>
struct Plan {
    static constexpr int kBuffers = BM == 256 ? 2 : 4;       // of BM tensor-memory columns
    static constexpr int kColumns = kBuffers * BM < 32 ? 32 : kBuffers * BM;
    static constexpr uint32_t kStage = kTileB + BM * 128;
    static constexpr int kStages = BM == 256 ? 4 : BM == 128 ? 6 : BM == 64 ? 8 : 9;
    static constexpr uint32_t kSlot = (BM + kRowsB) * 4;     // column and row scales
    static constexpr uint32_t kSmem = 1024 + kStages * kStage + kScaleSlots * kSlot;
    static_assert(kSmem <= 232448 - 1024, "one CTA per SM");
    static_assert(kStages * kStage >= BM * kRowsB * 4, "a partial tile fits the stages");
};

struct MatmulArgs {
    const float* sa;  // [KB, M]
    const float* sb;  // [KB, N] or [KB, ceil(N / 128)]
    void* out;        // [M, N]
    int M, N, KB;
    int out_bf16;
    int ntn, tiles, split;
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, kWaitNs);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) { tmem_ld8(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }

// Two fp32 values a register pair.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
    return static_cast<uint64_t>(b) << 32 | a;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float peer_f32(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .u32 p;\n\t"
        "mapa.shared::cluster.u32 p, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [p];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

template <int N>
__device__ __forceinline__ void set_max_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Columns [m, m + NC) of one lane's row n of the output.  bf16: neighbouring
// lanes swap one of two columns' values, so that each writes two outputs of one
// token in one word (the second lane takes the odd column).
template <int NC>
__device__ __forceinline__ void write_columns(const MatmulArgs& a, const float (&v)[NC], int m,
                                              int n) {
    const size_t N = a.N;
    if (!a.out_bf16) {
        float* out = static_cast<float*>(a.out) + n;
        if (n < a.N) {
#pragma unroll
            for (int j = 0; j < NC; ++j)
                if (m + j < a.M) out[(size_t)(m + j) * N] = v[j];
        }
        return;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    if (a.N % 2 == 0) {
        const int odd = threadIdx.x & 1;
#pragma unroll
        for (int j = 0; j < NC; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
            const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(got, v[j + 1])
                                         : __floats2bfloat162_rn(v[j], got);
            if (n < a.N && m + j + odd < a.M)
                *reinterpret_cast<__nv_bfloat162*>(out + (size_t)(m + j + odd) * N + (n - odd)) = h;
        }
    } else if (n < a.N) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
            if (m + j < a.M) out[(size_t)(m + j) * N + n] = __float2bfloat16_rn(v[j]);
    }
}

template <int BM, bool kRowScales>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                      const MatmulArgs a) {
    using P = Plan<BM>;
    constexpr int ST = P::kStages, NB = P::kBuffers, NC = BM / 2;
    extern __shared__ uint8_t mm_smem[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], tfull[NB], tempty[NB],
        sfull[kScaleSlots], sempty[kScaleSlots];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    uint8_t* stages = mm_smem + ((1024u - (smem_u32(mm_smem) & 1023u)) & 1023u);
    float* slots = reinterpret_cast<float*>(stages + ST * P::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 1) {
        tmem_alloc(&s_tmem, P::kColumns);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 8);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sfull[i], 64);
            mbar_init(&sempty[i], 8);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* fail = &s_fail;

    // this CTA's tiles and K blocks
    const int rank = blockIdx.x % a.split;
    const int kb0 = static_cast<int>((long long)rank * a.KB / a.split);
    const int kb1 = static_cast<int>((long long)(rank + 1) * a.KB / a.split);
    const int first = blockIdx.x / a.split, step = gridDim.x / a.split;

    if (warp < 4) {
        if constexpr (BM == 256) set_max_regs_down<72>();
        if (warp == 0) {
            if (lane == 0) {
                int it = 0;
                for (int tile = first; tile < a.tiles && !*fail; tile += step) {
                    const int n0 = tile % a.ntn * kRowsB, m0 = tile / a.ntn * BM;
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % ST;
                        if (!wait(&empty[s], ((it / ST) & 1) ^ 1)) {
                            *fail = 1;
                            break;
                        }
                        uint8_t* st = stages + s * P::kStage;
                        mbar_arrive_expect_tx(&full[s], P::kStage);
                        tma_load_2d(st, &tmb, &full[s], kb * 128, n0);
                        tma_load_2d(st + kTileB, &tma, &full[s], kb * 128, m0);
                    }
                }
                // loads in flight land before the CTA may end (a no-op unless
                // a wait gave up: the products have waited for every load)
                for (int s = 0; s < ST && s < it; ++s)
                    wait(&full[s], ((it - 1 - s) / ST) & 1);
            }
        } else if (warp == 1) {
            if (lane == 0) {
                constexpr uint32_t id = idesc_e4m3_f32(kRowsB, BM);
                int it = 0;
                for (int tile = first; tile < a.tiles && !*fail; tile += step) {
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % ST, b = it % NB;
                        if (!wait(&full[s], (it / ST) & 1) ||
                            !wait(&tempty[b], ((it / NB) & 1) ^ 1)) {
                            *fail = 1;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sB = smem_u32(stages + s * P::kStage), sA = sB + kTileB;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(tmem + b * BM, sdesc_sw128(sB + k * 32, 16, 1024),
                                   sdesc_sw128(sA + k * 32, 16, 1024), id, k > 0);
                        mma_commit(&empty[s]);
                        mma_commit(&tfull[b]);
                    }
                }
                // no product is in flight when the tensor memory goes back
                if (it > 0) wait(&tfull[(it - 1) % NB], ((it - 1) / NB) & 1);
            }
        } else {
            // scales: 64 threads; four blocks' values are requested together
            constexpr int PER = (BM + 63) / 64;
            const int t = threadIdx.x - 64;
            int it = 0;
            for (int tile = first; tile < a.tiles && !*fail; tile += step) {
                const int nb = tile % a.ntn, n0 = nb * kRowsB, m0 = tile / a.ntn * BM;
                for (int kb = kb0; kb < kb1; kb += 4) {
                    float col[4][PER], row[4][2];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const bool on = kb + u < kb1;
                        float f = 1.f;
                        if (!kRowScales) f = on ? a.sb[(size_t)(kb + u) * a.ntn + nb] : 0.f;
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            const int m = m0 + t + 64 * i;
                            col[u][i] = on && t + 64 * i < BM && m < a.M
                                            ? a.sa[(size_t)(kb + u) * a.M + m] * f
                                            : 0.f;
                        }
                        if (kRowScales) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int n = n0 + t + 64 * i;
                                row[u][i] =
                                    on && n < a.N ? a.sb[(size_t)(kb + u) * a.N + n] : 0.f;
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (kb + u >= kb1) break;
                        const int i4 = it % kScaleSlots;
                        if (!wait(&sempty[i4], ((it / kScaleSlots) & 1) ^ 1)) {
                            *fail = 1;
                            break;
                        }
                        float* slot = slots + i4 * (BM + kRowsB);
#pragma unroll
                        for (int i = 0; i < PER; ++i)
                            if (t + 64 * i < BM) slot[t + 64 * i] = col[u][i];
                        if (kRowScales) {
                            slot[BM + t] = row[u][0];
                            slot[BM + t + 64] = row[u][1];
                        }
                        mbar_arrive(&sfull[i4]);
                        ++it;
                    }
                    if (*fail) break;
                }
            }
        }
        __syncwarp();
        if (a.split > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        if constexpr (BM == 256) set_max_regs_up<216>();
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(quarter) << 21);  // lane 32 quarter
        int it = 0;
        for (int tile = first; tile < a.tiles; tile += step) {
            const int n = tile % a.ntn * kRowsB + quarter * 32 + lane;
            const int m = tile / a.ntn * BM + wg * NC;
            uint64_t acc[NC / 2];
#pragma unroll
            for (int j = 0; j < NC / 2; ++j) acc[j] = 0ull;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it % NB, i4 = it % kScaleSlots;
                ok = __all_sync(0xffffffffu, wait(&tfull[b], (it / NB) & 1) &&
                                                 wait(&sfull[i4], (it / kScaleSlots) & 1));
                if (!ok) {
                    *fail = 1;
                    break;
                }
                tc_fence_after();
                const float* slot = slots + i4 * (BM + kRowsB);
                const uint64_t rs =
                    kRowScales ? pair(__float_as_uint(slot[BM + quarter * 32 + lane]),
                                      __float_as_uint(slot[BM + quarter * 32 + lane]))
                               : 0ull;
                constexpr int CH = NC < 16 ? NC : 16;  // columns a load
#pragma unroll
                for (int c = 0; c < NC; c += CH) {
                    uint32_t r[CH];
                    tmem_ld(tq + b * BM + wg * NC + c, r);
                    tmem_wait_ld();
                    if (c + CH == NC) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&tempty[b]);
                    }
#pragma unroll
                    for (int j = 0; j < CH; j += 4) {
                        const ulonglong2 s2 =
                            *reinterpret_cast<const ulonglong2*>(slot + wg * NC + c + j);
                        uint64_t s0 = s2.x, s1 = s2.y;
                        if (kRowScales) {
                            s0 = mul2(s0, rs);
                            s1 = mul2(s1, rs);
                        }
                        acc[(c + j) / 2] = fma2(pair(r[j], r[j + 1]), s0, acc[(c + j) / 2]);
                        acc[(c + j) / 2 + 1] =
                            fma2(pair(r[j + 2], r[j + 3]), s1, acc[(c + j) / 2 + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[i4]);
            }
            if (a.split == 1) {
                float v[NC];
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    v[j] = ok ? __uint_as_float(static_cast<uint32_t>(acc[j / 2] >> (j % 2 * 32)))
                              : __uint_as_float(0x7FFFFFFFu);
                write_columns<NC>(a, v, m, n);
            } else {
                // [column][lane]: every load of this CTA has been consumed
                float* part = reinterpret_cast<float*>(stages);
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    part[(wg * NC + j) * kRowsB + quarter * 32 + lane] =
                        ok ? __uint_as_float(static_cast<uint32_t>(acc[j / 2] >> (j % 2 * 32)))
                           : __uint_as_float(0x7FFFFFFFu);
            }
            if (!ok) break;
        }
        if (a.split > 1) {
            __syncwarp();
            cluster_sync();
            const int n0 = first % a.ntn * kRowsB, m0 = first / a.ntn * BM;
            const int per = BM / a.split;
            for (int e = threadIdx.x - 128; e < per * kRowsB; e += 256) {
                const int c = rank * per + e / kRowsB, l = e % kRowsB;
                const uint32_t addr = smem_u32(stages) + (c * kRowsB + l) * 4;
                float v = 0.f;
                for (int q = 0; q < a.split; ++q) v += peer_f32(addr, q);
                if (m0 + c < a.M && n0 + l < a.N) {
                    const size_t o = (size_t)(m0 + c) * a.N + n0 + l;
                    if (a.out_bf16)
                        static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
                    else
                        static_cast<float*>(a.out)[o] = v;
                }
            }
            __syncwarp();
            cluster_sync();  // no CTA leaves while others read its part
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, P::kColumns);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// Bytes [rows, K] with rows of fp8_pitch(K) bytes, in boxes of 128 bytes of
// `box` rows; zeros are read beyond K and beyond the last row.
bool map_bytes(CUtensorMap* m, const void* base, int rows, int K, int box) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)fp8_pitch(K)};
    cuuint32_t boxes[2] = {128, (cuuint32_t)box};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BM, bool kRowScales>
cudaError_t run(const void* a8, const void* b8, MatmulArgs a, int K, int sms, cudaStream_t st) {
    using P = Plan<BM>;
    CUtensorMap tma, tmb;
    if (!map_bytes(&tma, a8, a.M, K, BM) || !map_bytes(&tmb, b8, a.N, K, kRowsB))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(
        fp8_matmul_kernel<BM, kRowScales>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.split > 1 ? a.tiles * a.split : a.tiles < sms ? a.tiles : sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fp8_matmul_kernel<BM, kRowScales>, tma, tmb, a);
}

template <bool kRowScales>
cudaError_t run_bm(int bm, const void* a8, const void* b8, const MatmulArgs& a, int K, int sms,
                   cudaStream_t st) {
    switch (bm) {
        case 16: return run<16, kRowScales>(a8, b8, a, K, sms, st);
        case 32: return run<32, kRowScales>(a8, b8, a, K, sms, st);
        case 64: return run<64, kRowScales>(a8, b8, a, K, sms, st);
        case 128: return run<128, kRowScales>(a8, b8, a, K, sms, st);
        default: return run<256, kRowScales>(a8, b8, a, K, sms, st);
    }
}

// Columns of a tile and the split of K.
void choose(int M, int N, int KB, int sms, int* bm, int* split) {
    *bm = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
    const long long ntn = blocks128(N);
    while (*bm > 64 && ntn * ((M + *bm - 1) / *bm) * 2 <= sms) *bm /= 2;
    const long long tiles = ntn * ((M + *bm - 1) / *bm);
    int s = 1;
    while (s < kMaxSplit && tiles * s * 2 <= sms && KB >= 4 * s) s *= 2;
    *split = s;
}

cudaError_t matmul_with(int bm, int split, const void* a8, const float* a_scale, const void* b8,
                        const float* b_scale, int M, int N, int K, bool b_rows,
                        kda_dtype_t out_dt, void* out, int sms, cudaStream_t st) {
    MatmulArgs a{};
    a.sa = a_scale;
    a.sb = b_scale;
    a.out = out;
    a.M = M;
    a.N = N;
    a.KB = blocks128(K);
    a.out_bf16 = out_dt == KDA_DTYPE_BF16;
    a.ntn = blocks128(N);
    a.split = split;
    const long long tiles = (long long)a.ntn * (((long long)M + bm - 1) / bm);
    if (tiles * split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<int>(tiles);
    return b_rows ? run_bm<true>(bm, a8, b8, a, K, sms, st)
                  : run_bm<false>(bm, a8, b8, a, K, sms, st);
}

}  // namespace

bool fp8_matmul_available() { return encode_fn() != nullptr; }

cudaError_t launch_fp8_matmul(const void* a8, const float* a_scale, const void* b8,
                              const float* b_scale, int M, int N, int K, bool b_rows,
                              kda_dtype_t out_dt, void* out, cudaStream_t st) {
    if (M == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int bm = 0, split = 0;
    choose(M, N, blocks128(K), sms, &bm, &split);
    return matmul_with(bm, split, a8, a_scale, b8, b_scale, M, N, K, b_rows, out_dt, out, sms, st);
}

}  // namespace kda

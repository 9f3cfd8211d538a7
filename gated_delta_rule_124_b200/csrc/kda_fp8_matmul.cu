// out = A B^T of two 8-bit matrices with a scale per block of 128 along K:
//   out[m, n] = sum_kb sa[kb, m] sb[kb, n] sum_{k in block kb} a8[m, k] b8[n, k]
// (sb per row of B, or per 128 rows).
//
// The inner sums are e4m3 products on the tensor cores (tcgen05,
// kind::f8f6f4, fp32 accumulation); the scales differ from block to block, so
// every block's 128 x BN partial product leaves tensor memory and is added to
// fp32 sums in registers with its scales.  One CTA per SM walks over output
// tiles of 128 rows of A by BN rows of B:
//   warp 0      TMA loads of both operands' blocks (128-byte rows, the swizzled
//               K-major layout the products read), a ring of stages;
//   warps 1, 2  the products of a block (four of K = 32) into one of the four
//               tensor-memory buffers of 128 columns, in turn (the waits and
//               hand-overs of one issuing thread take longer than a product);
//   warp 3      the block's scales into the same stage (a product is issued when
//               both are there, so the warps below wait for the product alone);
//   warps 4-11  out += scale * partial product, then the tile's output.
// The output is stored from registers, whole 32-byte sectors where a thread has a
// row (through shared memory and TMA it took 2900 cycles a tile, the time of five
// blocks' products, in which the sums waited for their buffers).
// A 256-column tile is two products of 128 columns, each handed to its own four
// warps: with two buffers of 256 columns the way from a product through its
// sums back to the buffer (a commit, a wake-up, the reads and sums, an arrival)
// was longer than the next product, and both groups of sums competed for the
// same issue slots at the same time (1220 cycles a block; a product takes 512).
// With few tiles the K blocks are split over a cluster of up to 8 CTAs, which
// add their partial tiles through distributed shared memory in a fixed order.
//
// Measured on a B200 (calls in a graph; one after another from Python, under the
// power cap, in brackets): 8192 x 4096 x 4096 in bf16 129 to 136 us, about 2.05
// PFLOP/s (158), with a scale per row on both sides 4096 x 4096 x 4099 in fp32 110 to
// 120 us, about 1.2 PFLOP/s (130); a block's products and sums take 1000 cycles and
// the products alone 512.  Giving each half of a last, part-filled round of
// tiles to a CTA of its own gained nothing: a half takes a block as long.
//
// Every wait is bounded; a tile whose waits gave up, and every later one of its CTA,
// is written as NaN.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kRowsA = 128;                       // lanes of a tile
constexpr uint32_t kTileA = kRowsA * 128;         // bytes of A's block
constexpr int kBuffers = 4;                       // tensor-memory buffers of 128 columns
constexpr int kMaxSplit = 8;

template <int BN>
struct Plan {
    static constexpr int kHalves = BN / 128;                 // products of 128 columns a block
    static constexpr uint32_t kStage = kTileA + BN * 128;
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr uint32_t kSlot = (kRowsA + BN) * 4;     // row and column scales
    static constexpr uint32_t kSmem =
        1024 + kStages * (kStage + kSlot);
    static_assert(kSmem <= 232448 - 1024, "one CTA per SM");
    static constexpr int kPartPitch = BN + 8;                // floats of a partial tile's row
    static_assert(kStages * kStage >= kPartPitch * kRowsA * 4, "a partial tile fits the stages");
};

struct MatmulArgs {
    const float* sa;  // [KB, M]
    const float* sb;  // [KB, N] or [KB, ceil(N / 128)]
    void* out;        // [M, N]
    int M, N, KB, NB; // NB: columns of sb
    int out_bf16, out_wide;  // wide: out starts on 32 bytes
    int ntm, tiles, split;
    Fp8Withheld withheld;
};
// The block that this CTA's loads leave out (-1: none).
template <bool kTest>
__device__ __forceinline__ int withheld(const MatmulArgs& a) {
    return kTest && static_cast<int>(blockIdx.x) == a.withheld.cta ? a.withheld.block : -1;
}

// Bounded wait on a phase parity (some seconds at most; milliseconds in the kernels
// that test the limit).  A test before the loop and a plain loop of tests: the waits
// of the threads that issue the products are mostly for phases that are complete,
// and with only a loop (or one with a clock and a sleep in it) such a wait took 140
// to 250 cycles more.  The limit is a constant: as an argument of the launch it cost
// 0.6 % with a scale per row of B.
template <bool kTest>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    if (mbar_test_wait(bar, parity)) return true;
    for (int i = 0; i < (kTest ? 1 << 18 : 1 << 26); ++i)
        if (mbar_test_wait(bar, parity)) return true;
    return false;
}

// 32 lanes x 16 columns: thread t has lane t.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// 16 lanes x 32 columns: r[4 i + 2 h + j] of thread t is lane t / 4 + 8 h, column
// 8 i + 2 (t % 4) + j.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Waits for the loads before it; the values pass through, so that nothing reads
// them earlier.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]),
                          "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

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
__device__ __forceinline__ float4 peer_f32x4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .u32 p;\n\t"
        "mapa.shared::cluster.u32 p, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [p];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// Four neighbouring outputs from index o, `left` of the row's columns left.
__device__ __forceinline__ void write4(const MatmulArgs& a, const float (&v)[4], size_t o,
                                       int left) {
    if (a.out_bf16) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + o;
        if (a.N % 4 == 0) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(v[2], v[3]);
            *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                        *reinterpret_cast<const uint32_t*>(&hi));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) out[i] = __float2bfloat16_rn(v[i]);
        }
    } else {
        float* out = static_cast<float*>(a.out) + o;
        if (a.N % 4 == 0) {
            *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < left) out[i] = v[i];
        }
    }
}

template <int N>
__device__ __forceinline__ void set_max_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float half_of(uint64_t v, int j) {
    return __uint_as_float(static_cast<uint32_t>(v >> (32 * j)));
}

__device__ __forceinline__ void store32(const MatmulArgs& args, void* p, uint4 a, uint4 b) {
    if (!args.out_wide) {
        static_cast<uint4*>(p)[0] = a;
        static_cast<uint4*>(p)[1] = b;
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ uint4 words(uint64_t a, uint64_t b) {
    return make_uint4(static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32),
                      static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32));
}

// A warp's part of a tile, 32 rows (the lanes of its quarter of tensor memory) by
// NC columns of fp32 sums, in one of two layouts:
//   RowSums:  thread t has row t, so that a block's scale is one number per
//             thread; whole-lane loads read tensor memory at its full rate;
//   FragSums: thread t has the column pairs 8 i + 2 (t % 4) of rows t / 4 + 8 h,
//             for scales that differ by column: a thread needs a quarter of
//             them (a column's scale costs a shared-memory word per warp that
//             reads it, and whole rows' worth of them was the bound: 1100
//             cycles a block of 256 columns), at half the rate of the loads.
// add() adds a block: `src` its columns in tensor memory, `row` the scales of the
// 32 rows, `col` those of the columns (RowSums: the one of the 128); `release`
// is called when tensor memory has been read.  The loads of the next 32 columns
// are in flight during a chunk's sums.
// store() writes the part, whose first row and column are m and n, to the output.
__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(half_of(v, 0), half_of(v, 1));
    return *reinterpret_cast<const uint32_t*>(&x);
}

template <int NC>
struct RowSums {
    uint64_t acc[NC / 2];
    __device__ void fill(uint64_t v) {
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) acc[j] = v;
    }
    template <typename F>
    __device__ void add(uint32_t src, const float* row, const float* col, int lane, F release) {
        uint32_t r[2][16];
        tmem_ld16(src, r[0]);
        const uint32_t x = __float_as_uint(row[lane] * *col);
        const uint64_t scale = pair(x, x);
#pragma unroll
        for (int c = 0; c < NC / 16; ++c) {
            uint32_t(&p)[16] = r[c & 1];
            tmem_wait(p);
            if (c + 1 < NC / 16) tmem_ld16(src + (c + 1) * 16, r[(c + 1) & 1]);
            else release();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc[8 * c + j] = fma2(pair(p[2 * j], p[2 * j + 1]), scale, acc[8 * c + j]);
        }
    }
    // The sums as floats, the 32 rows `pitch` floats apart.
    __device__ void partial(float* part, int pitch, int lane) const {
#pragma unroll
        for (int j = 0; j < NC / 2; j += 2) {
            ulonglong2 v;
            v.x = acc[j];
            v.y = acc[j + 1];
            *reinterpret_cast<ulonglong2*>(part + lane * pitch + 2 * j) = v;
        }
    }
    __device__ void store(const MatmulArgs& a, int m, int n, int lane) const {
        if (m + lane >= a.M) return;
        const size_t o = (size_t)(m + lane) * a.N + n;
        const int left = a.N - n;  // columns of the output from n on
        if (a.out_bf16) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + o;
            if (a.N % 16 == 0) {  // rows, and 16 columns, are whole 32-byte pieces
#pragma unroll
                for (int j = 0; j < NC / 16; ++j) {
                    if (16 * j >= left) break;
                    const uint64_t* v = acc + 8 * j;
                    store32(a, out + 16 * j,
                            make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3])),
                            make_uint4(bf16_pair(v[4]), bf16_pair(v[5]), bf16_pair(v[6]), bf16_pair(v[7])));
                }
            } else {
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (j < left) out[j] = __float2bfloat16_rn(half_of(acc[j / 2], j % 2));
            }
        } else {
            float* out = static_cast<float*>(a.out) + o;
            if (a.N % 8 == 0) {
#pragma unroll
                for (int j = 0; j < NC / 8; ++j) {
                    if (8 * j >= left) break;
                    const uint64_t* v = acc + 4 * j;
                    store32(a, out + 8 * j, words(v[0], v[1]), words(v[2], v[3]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (j < left) out[j] = half_of(acc[j / 2], j % 2);
            }
        }
    }
};

template <int NC>
struct FragSums {
    uint64_t acc[NC / 8][4];
    __device__ void fill(uint64_t v) {
#pragma unroll
        for (int j = 0; j < NC / 8; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h) acc[j][h] = v;
    }
    template <typename F>
    __device__ void add(uint32_t src, const float* row, const float* col, int lane, F release) {
        const int g = lane >> 2, q = lane & 3;
        uint32_t r[2][2][16];
        tmem_ld_frag(src, r[0][0]);
        tmem_ld_frag(src + (16u << 16), r[0][1]);
        uint64_t rs[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t x = __float_as_uint(row[g + 8 * h]);
            rs[h] = pair(x, x);
        }
#pragma unroll
        for (int c = 0; c < NC / 32; ++c) {
            uint32_t(&p)[2][16] = r[c & 1];
            tmem_wait(p[0]);
            tmem_wait(p[1]);
            if (c + 1 < NC / 32) {
                tmem_ld_frag(src + (c + 1) * 32, r[(c + 1) & 1][0]);
                tmem_ld_frag(src + (c + 1) * 32 + (16u << 16), r[(c + 1) & 1][1]);
            } else {
                release();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t cs = *reinterpret_cast<const uint64_t*>(col + c * 32 + 8 * i + 2 * q);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t* x = p[h >> 1] + 4 * i + 2 * (h & 1);
                    acc[4 * c + i][h] = fma2(pair(x[0], x[1]), mul2(rs[h], cs), acc[4 * c + i][h]);
                }
            }
        }
    }
    __device__ void partial(float* part, int pitch, int lane) const {
        part += (lane >> 2) * pitch + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < NC / 8; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h)
                *reinterpret_cast<uint64_t*>(part + 8 * h * pitch + 8 * j) = acc[j][h];
    }
    __device__ void store(const MatmulArgs& a, int m, int n, int lane) const {
        n += 2 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int row = m + (lane >> 2) + 8 * h;
            if (row >= a.M) break;
            const size_t o = (size_t)row * a.N + n;
            const int left = a.N - n;
            __nv_bfloat16* half = static_cast<__nv_bfloat16*>(a.out) + o;
            float* full = static_cast<float*>(a.out) + o;
#pragma unroll
            for (int j = 0; j < NC / 8; ++j) {
                if (8 * j >= left) break;
                const uint64_t v = acc[j][h];
                if (a.N % 2 == 0) {  // pairs start on 4 or 8 bytes
                    if (a.out_bf16) *reinterpret_cast<uint32_t*>(half + 8 * j) = bf16_pair(v);
                    else *reinterpret_cast<uint64_t*>(full + 8 * j) = v;
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (8 * j + e >= left) break;
                    if (a.out_bf16) half[8 * j + e] = __float2bfloat16_rn(half_of(v, e));
                    else full[8 * j + e] = half_of(v, e);
                }
            }
        }
    }
};

template <int BN, bool kRowScales, bool kTest>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                      const MatmulArgs a) {
    using P = Plan<BN>;
    constexpr int ST = P::kStages, NB = kBuffers, NC = BN / 2, HV = P::kHalves;
    extern __shared__ uint8_t mm_smem[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], sempty[ST], tfull[NB], tempty[NB];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    uint8_t* stages = mm_smem + ((1024u - (smem_u32(mm_smem) & 1023u)) & 1023u);
    float* slots = reinterpret_cast<float*>(stages + ST * P::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 1) {
        tmem_alloc(&s_tmem, NB * 128);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1 + 32);    // the loads, the scales' warp
            mbar_init(&empty[i], HV);       // the products
            mbar_init(&sempty[i], 8);       // the warps that read the scales
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&tfull[i], 2);        // the product, and its issuing thread
            mbar_init(&tempty[i], 8 / HV);  // the warps that read it
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* fail = &s_fail;

    // this CTA's tiles (A's rows vary fastest) and K blocks
    const int rank = blockIdx.x % a.split;
    const int kb0 = static_cast<int>((long long)rank * a.KB / a.split);
    const int kb1 = static_cast<int>((long long)(rank + 1) * a.KB / a.split);
    const int first = blockIdx.x / a.split, step = gridDim.x / a.split;

    if (warp < 4) {
        if constexpr (BN == 256) set_max_regs_down<72>();
        if (warp == 0) {
            if (elect_one()) {
                int it = 0;
                const int left_out = withheld<kTest>(a);
                for (int tile = first; tile < a.tiles && !*fail; tile += step) {
                    const int m0 = tile % a.ntm * kRowsA, n0 = tile / a.ntm * BN;
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % ST;
                        if (!wait<kTest>(&empty[s], ((it / ST) & 1) ^ 1)) {
                            *fail = 1;
                            break;
                        }
                        if (it == left_out) continue;
                        uint8_t* st = stages + s * P::kStage;
                        mbar_arrive_expect_tx(&full[s], P::kStage);
                        tma_load_2d(st, &tma, &full[s], kb * 128, m0);
                        tma_load_2d(st + kTileA, &tmb, &full[s], kb * 128, n0);
                    }
                }
                // loads in flight land before the CTA may end (a no-op unless
                // a wait gave up: the products have waited for every load)
                for (int s = 0; s < ST && s < it; ++s)
                    wait<kTest>(&full[s], ((it - 1 - s) / ST) & 1);
            }
        } else if (warp < 3) {
            if (elect_one()) {
                // unit u is a block's 128 columns; this thread's: u % 2 == warp - 1
                constexpr uint32_t id = idesc_e4m3_f32(kRowsA, 128);
                int it = 0, last = -1;
                for (int tile = first; tile < a.tiles && !*fail; tile += step) {
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int h = HV == 2 ? warp - 1 : 0, u = it * HV + h;
                        if (HV == 1 && (u & 1) != warp - 1) continue;
                        const int s = it % ST, b = u % NB;
                        if (!wait<kTest>(&full[s], (it / ST) & 1)) {
                            *fail = 1;
                            break;
                        }
                        if (!wait<kTest>(&tempty[b], ((u / NB) & 1) ^ 1)) {
                            *fail = 1;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sA = smem_u32(stages + s * P::kStage);
                        const uint32_t sB = sA + kTileA + h * 16384;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8(tmem + b * 128, sdesc_sw128(sA + k * 32, 16, 1024),
                                   sdesc_sw128(sB + k * 32, 16, 1024), id, k > 0);
                        mma_commit(&tfull[b]);
                        mbar_arrive(&tfull[b]);  // (passes the scales on)
                        mma_commit(&empty[s]);
                        last = u;
                    }
                }
                // no product is in flight when the tensor memory goes back
                if (last >= 0) wait<kTest>(&tfull[last % NB], (last / NB) & 1);
            }
        } else {
            // scales: the values of the next blocks (across tiles) are requested
            // before those of the last ones are stored
            constexpr int PER = kRowScales ? BN / 32 : 1, GROUP = kRowScales ? 2 : 4;
            struct Values {
                float row[4], col[PER];
            };
            const int t = lane;
            int tile = first, kb = kb0;
            auto request = [&](Values (&v)[GROUP]) {
                int n = 0;
#pragma unroll
                for (int u = 0; u < GROUP; ++u) {
                    if (tile >= a.tiles) continue;
                    const int m0 = tile % a.ntm * kRowsA, nt = tile / a.ntm;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = m0 + t + 32 * i;
                        v[u].row[i] = m < a.M ? a.sa[(size_t)kb * a.M + m] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int n = kRowScales ? nt * BN + t + 32 * i : nt * (BN / 128) + t;
                        v[u].col[i] = n < a.NB && (kRowScales || t < BN / 128)
                                          ? a.sb[(size_t)kb * a.NB + n]
                                          : 0.f;
                    }
                    ++n;
                    if (++kb == kb1) {
                        kb = kb0;
                        tile += step;
                    }
                }
                return n;
            };
            Values now[GROUP], next[GROUP];
            int count = request(now), it = 0;
            while (count > 0 && !*fail) {
                const int more = request(next);
#pragma unroll
                for (int u = 0; u < GROUP; ++u) {
                    if (u >= count) break;
                    const int s = it % ST;
                    if (!wait<kTest>(&sempty[s], ((it / ST) & 1) ^ 1)) {
                        *fail = 1;
                        break;
                    }
                    float* slot = slots + s * (kRowsA + BN);
#pragma unroll
                    for (int i = 0; i < 4; ++i) slot[t + 32 * i] = now[u].row[i];
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (kRowScales || t < BN / 128) slot[kRowsA + t + 32 * i] = now[u].col[i];
                    mbar_arrive(&full[s]);
                    ++it;
                }
#pragma unroll
                for (int u = 0; u < GROUP; ++u) now[u] = next[u];
                count = more;
            }
        }
        __syncwarp();
        if (a.split > 1) {
            group_sync(1, kThreads);
            cluster_sync();
            cluster_sync();
        }
    } else {
        if constexpr (BN == 256) set_max_regs_up<216>();
        // this warp: lanes [32 quarter, + 32) and columns [NC wg, + NC)
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t tq = tmem + (static_cast<uint32_t>(quarter) << 21) + (HV == 1 ? wg * NC : 0);
        int it = 0;
        bool ok = true;
        for (int tile = first; tile < a.tiles; tile += step) {
            const int m = tile % a.ntm * kRowsA + quarter * 32;
            const int n = tile / a.ntm * BN + wg * NC;
            typename std::conditional<kRowScales, FragSums<NC>, RowSums<NC>>::type sums;
            sums.fill(0ull);
            for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                const int u = HV == 1 ? it : it * HV + wg, b = u % NB, s = it % ST;
                ok = __all_sync(0xffffffffu, wait<kTest>(&tfull[b], (u / NB) & 1));
                if (!ok) {
                    *fail = 1;
                    break;
                }
                tc_fence_after();
                const float* slot = slots + s * (kRowsA + BN);
                sums.add(tq + b * 128, slot + quarter * 32,
                         slot + kRowsA + (kRowScales ? wg * NC : wg * NC / 128), lane, [&] {
                             tc_fence_before();
                             __syncwarp();
                             if (lane == 0) mbar_arrive(&tempty[b]);
                         });
                __syncwarp();
                if (lane == 0) mbar_arrive(&sempty[s]);
            }
            // NaN instead of a sum that lacks blocks
            if (!ok) sums.fill(0x7FFFFFFF7FFFFFFFull);
            if (a.split > 1) {
                // [row][column], where the stages were, once every warp of the CTA
                // is done with them: with 256 rows of B a group's sums wait for
                // their own half's products only, and those of the other half may
                // be blocks behind, reading the same stages
                group_sync(1, kThreads);
                if (m < a.M)
                    sums.partial(reinterpret_cast<float*>(stages) + quarter * 32 * P::kPartPitch +
                                     wg * NC,
                                 P::kPartPitch, lane);
                break;
            }
            sums.store(a, m, n, lane);
        }
        if (a.split > 1) {
            __syncwarp();
            cluster_sync();
            const int m0 = first % a.ntm * kRowsA, n0 = first / a.ntm * BN;
            // this CTA's share of the tile, neighbouring columns in neighbouring lanes
            const int all = min(kRowsA, a.M - m0) * (BN / 4);
            const int e0 = all * rank / a.split, e1 = all * (rank + 1) / a.split;
            for (int e = e0 + threadIdx.x - 128; e < e1; e += 256) {
                const int l = e / (BN / 4), c = e % (BN / 4) * 4;
                if (n0 + c >= a.N) continue;
                const uint32_t addr = smem_u32(stages) + (l * P::kPartPitch + c) * 4;
                float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int p = 0; p < a.split; ++p) {
                    const float4 x = peer_f32x4(addr, p);
                    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
                }
                write4(a, v, (size_t)(m0 + l) * a.N + n0 + c, a.N - n0 - c);
            }
            __syncwarp();
            cluster_sync();  // no CTA leaves while others read its part
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, NB * 128);
}

// Up to 16 rows of A: the operands change places, so that the 128 lanes of a product
// are rows of B (a weight, read once: the call is bound by HBM) and its 16 columns
// the rows of A.  A CTA has 128 rows of B and a share of the K blocks, two CTAs an
// SM, each with five blocks' loads in flight; warp 0 loads, warp 1 issues the
// products, warps 2-5 take a row of B a thread through its blocks, the scales of the
// next four requested ahead.  16 x 12288 x 4096 15.2 us (7.7 at the copy rate; with
// the plan above 21.3), 16 x 8192 x 4096 12.3 (14.0); an SM takes in about 60 bytes
// a ns this way, with more stages or two blocks a stage no more.
constexpr int kFewThreads = 192;
constexpr int kFewRows = 16;                                // of A
constexpr uint32_t kFewStage = kTileA + kFewRows * 128;
constexpr int kFewStages = 5;
constexpr int kFewBuffers = 4;                              // of tensor memory
constexpr uint32_t kFewSmem = 1024 + kFewStages * kFewStage;
static_assert(kFewStages * kFewStage >= kFewRows * kRowsA * 4, "a partial tile fits the stages");

template <bool kRowScales, bool kTest>
__global__ void __launch_bounds__(kFewThreads)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx,
                   const MatmulArgs a) {
    constexpr int ST = kFewStages, NB = kFewBuffers, MP = kFewRows;
    extern __shared__ uint8_t mm_smem[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], tfull[NB], tempty[NB];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    uint8_t* stages = mm_smem + ((1024u - (smem_u32(mm_smem) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.split, n0 = blockIdx.x / a.split * kRowsA;
    const int kb0 = static_cast<int>((long long)rank * a.KB / a.split);
    const int kb1 = static_cast<int>((long long)(rank + 1) * a.KB / a.split);

    if (warp == 1) {
        tmem_alloc(&s_tmem, NB * MP);
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
            mbar_init(&tempty[i], 4);
        }
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* fail = &s_fail;
    float* part = reinterpret_cast<float*>(stages);  // [rows of A][128], once the stages are read

    if (warp == 0) {
        if (elect_one()) {
            int it = 0;
            const int left_out = withheld<kTest>(a);
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST;
                if (*fail || !wait<kTest>(&empty[s], ((it / ST) & 1) ^ 1)) {
                    *fail = 1;
                    break;
                }
                if (it == left_out) continue;
                uint8_t* st = stages + s * kFewStage;
                mbar_arrive_expect_tx(&full[s], kFewStage);
                tma_load_2d(st, &tmw, &full[s], kb * 128, n0);
                tma_load_2d(st + kTileA, &tmx, &full[s], kb * 128, 0);
            }
            // loads in flight land before the stages are written again (a no-op
            // unless a wait gave up: the products have waited for every load)
            for (int s = 0; s < ST && s < it; ++s) wait<kTest>(&full[s], ((it - 1 - s) / ST) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t id = idesc_e4m3_f32(kRowsA, MP);
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % ST, b = it % NB;
                if (!wait<kTest>(&full[s], (it / ST) & 1) || !wait<kTest>(&tempty[b], ((it / NB) & 1) ^ 1)) {
                    *fail = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t sA = smem_u32(stages + s * kFewStage);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_f8(tmem + b * MP, sdesc_sw128(sA + k * 32, 16, 1024),
                           sdesc_sw128(sA + kTileA + k * 32, 16, 1024), id, k > 0);
                mma_commit(&tfull[b]);
                mma_commit(&empty[s]);
            }
            // no product is in flight when the tensor memory goes back
            if (it > 0) wait<kTest>(&tfull[(it - 1) % NB], ((it - 1) / NB) & 1);
        }
    } else {
        const int quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t tq = tmem + (static_cast<uint32_t>(quarter) << 21);
        // a block's scales: lane m has row m's of A, every lane its row's of B
        const int nb = kRowScales ? n0 + row : n0 / 128;
        auto scale_a = [&](int kb) {
            return kb < kb1 && lane < a.M ? a.sa[(size_t)kb * a.M + lane] : 0.f;
        };
        auto scale_b = [&](int kb) {
            return kb < kb1 && nb < a.NB ? a.sb[(size_t)kb * a.NB + nb] : 0.f;
        };
        float xa[NB], xb[NB];
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            xa[u] = scale_a(kb0 + u);
            xb[u] = scale_b(kb0 + u);
        }
        float acc[MP];
#pragma unroll
        for (int m = 0; m < MP; ++m) acc[m] = 0.f;
        bool ok = true;
        for (int base = kb0; base < kb1 && ok; base += NB) {
#pragma unroll
            for (int u = 0; u < NB; ++u) {  // block u of these is in buffer u
                const int kb = base + u, it = kb - kb0;
                if (kb >= kb1 || !ok) break;
                ok = __all_sync(0xffffffffu, wait<kTest>(&tfull[u], (it / NB) & 1));
                if (!ok) {
                    *fail = 1;
                    break;
                }
                tc_fence_after();
                uint32_t r[16];
                tmem_ld16(tq + u * MP, r);
                tmem_wait(r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[u]);
#pragma unroll
                for (int m = 0; m < MP; ++m) {
                    const float s = __shfl_sync(0xffffffffu, xa[u], m) * xb[u];
                    acc[m] = fmaf(__uint_as_float(r[m]), s, acc[m]);
                }
                xa[u] = scale_a(kb + NB);
                xb[u] = scale_b(kb + NB);
            }
        }
        // NaN instead of a sum that lacks blocks
        if (!ok)
#pragma unroll
            for (int m = 0; m < MP; ++m) acc[m] = __int_as_float(0x7FFFFFFF);
        if (a.split == 1) {
            if (n0 + row < a.N) {
#pragma unroll
                for (int m = 0; m < MP; ++m) {
                    if (m >= a.M) break;
                    const size_t o = (size_t)m * a.N + n0 + row;
                    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(acc[m]);
                    else static_cast<float*>(a.out)[o] = acc[m];
                }
            }
        } else {
            // (after the loads and products of a CTA whose waits gave up, too)
            group_sync(1, kFewThreads);
#pragma unroll
            for (int m = 0; m < MP; ++m)
                if (m < a.M) part[m * kRowsA + row] = acc[m];
        }
    }
    __syncwarp();
    if (a.split > 1) {
        if (warp < 2) group_sync(1, kFewThreads);
        cluster_sync();
        // this CTA's share of the tile, neighbouring rows of B in neighbouring lanes
        const int all = a.M * (kRowsA / 4);
        const int e0 = all * rank / a.split, e1 = all * (rank + 1) / a.split;
        for (int e = e0 + threadIdx.x; e < e1; e += kFewThreads) {
            const int m = e / (kRowsA / 4), c = e % (kRowsA / 4) * 4;
            if (n0 + c >= a.N) continue;
            const uint32_t addr = smem_u32(part) + (m * kRowsA + c) * 4;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int p = 0; p < a.split; ++p) {
                const float4 x = peer_f32x4(addr, p);
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            }
            write4(a, v, (size_t)m * a.N + n0 + c, a.N - n0 - c);
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while others read its part
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, NB * MP);
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

// A launch of `ctas` CTAs in clusters of `split`.
template <typename F>
cudaError_t launch(F kernel, int ctas, int threads, uint32_t smem, int split, cudaStream_t st,
                   const CUtensorMap& m0, const CUtensorMap& m1, const MatmulArgs& a) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = split > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, m0, m1, a);
}

template <int BN, bool kRowScales>
cudaError_t run(const void* a8, const void* b8, MatmulArgs a, int K, int sms, cudaStream_t st) {
    using P = Plan<BN>;
    CUtensorMap tma, tmb;
    if (!map_bytes(&tma, a8, a.M, K, kRowsA) || !map_bytes(&tmb, b8, a.N, K, BN))
        return cudaErrorInvalidValue;
    const int ctas = a.split > 1 ? a.tiles * a.split : a.tiles < sms ? a.tiles : sms;
    auto kernel = a.withheld.cta < 0 ? fp8_matmul_kernel<BN, kRowScales, false>
                                     : fp8_matmul_kernel<BN, kRowScales, true>;
    return launch(kernel, ctas, kThreads, P::kSmem, a.split, st, tma, tmb, a);
}

// Rows of B per tile and the split of K: the pair with the least time by a model
// of B200 measurements (us, calls in a graph): a block takes 0.39 with 128 rows and
// 0.54 with 256 (all SMs busy), joining a cluster's partial tiles 4 and 7.  K = 4096, N = 4096,
// measured for 128, 256, 512, 1024 and 8192 rows of A: 128 rows of B split 4 ways
// 12.0 (16.7 unsplit), 2 ways 15.2 (16.9), unsplit 17.6; 256 rows unsplit 22.3
// (29.6 with 128) and 134 (174).  With a scale per row of B 0.53 and 0.83
// (4096 x 4096 x 4099: 110 with 256 rows, 124 with 128).
// Longer K, the best split with 128 and with 256 rows of B: 64 x 2048 x 14336 16.6 (4
// ways) and 15.7 (8), 64 x 6144 x 8192 19.3 (2) and 17.7 (4), 256 x 5120 x 6144 22.4
// (whole) and 20.4 (3), 128 x 7168 x 16384 33.7 (2) and 31.1 (4), 512 x 4096 x 14336
// 44.8 (whole) and 38.7 (2), 128 x 4096 x 14336 19.9 (4) and 24.0 (4); scales per row
// 1024 x 1024 x 16384 39.1 (2) and 33.4 (4), 512 x 4096 x 8192 36.1 (whole) and 34.9 (2).
// Of 32 shapes of 32 to 2048 rows of A, K = 4096 to 16384, 28 got the best of the plans
// below and four were 1 to 4 % off it (128 x 12288 x 8192: 31.0, best 29.8 whole with
// 128 rows).
// The CTAs of a cluster share one of the device's groups of SMs, whose sizes few
// numbers divide: 148 SMs hold 45 clusters of three, 33 of four and 15 of eight (the
// occupancy query's answers; 16 tiles split eight ways took two rounds, 15.6 for 64
// x 2048 x 4096 against 9.5 split four ways; 64 x 5120 x 4096 11.2 split three ways,
// 12.6 two).  Five to seven ways are left out: a tenth better for one shape in
// fifteen, up to 4 % worse than four or eight for others.
constexpr int kSplits[] = {1, 2, 3, 4, kMaxSplit};
int clusters(int sms, int split) {
    return sms * (split == 3 ? 45 : split == 4 ? 33 : split == 8 ? 15 : 148 / split) / 148;
}
void choose(int M, int N, int KB, bool b_rows, int sms, int* bn, int* split) {
    double best = 0.;
    for (int n = 128; n <= 256; n += 128) {
        const double block = b_rows ? (n == 128 ? 0.53 : 0.83) : (n == 128 ? 0.39 : 0.54);
        const double join = n == 128 ? 4. : 7.;
        const double tiles = ((M + kRowsA - 1) / kRowsA) * (double)((N + n - 1) / n);
        for (const int s : kSplits) {
            if (s > KB) break;
            const double rounds = std::ceil(tiles / clusters(sms, s));
            const double t = rounds * ((KB + s - 1) / s * block + (s > 1 ? join : 0.));
            if (best == 0. || t < best) {
                best = t;
                *bn = n;
                *split = s;
            }
        }
    }
}

// Shares of K: two CTAs an SM where there are few tiles (K = 4096, 16 rows: 32 tiles
// split 4 and 8 ways 9.3 and 9.4 us, unsplit 13.2; 64 tiles 11.8 split 4 ways, 13.7
// unsplit; 96 tiles 14.4 unsplit, 15.7 split 2 ways).
int few_split(int tiles, int KB, int sms) {
    if (KB < 24) return 1;
    if (tiles <= 2 * clusters(sms, 8)) return 8;
    if (tiles <= 2 * clusters(sms, 4)) return 4;
    return KB >= 64 && tiles <= 2 * clusters(sms, 2) ? 2 : 1;
}

template <bool kRowScales>
cudaError_t run_few(const void* a8, const void* b8, const MatmulArgs& a, int K, cudaStream_t st) {
    CUtensorMap tmw, tmx;
    if (!map_bytes(&tmw, b8, a.N, K, kRowsA) || !map_bytes(&tmx, a8, a.M, K, kFewRows))
        return cudaErrorInvalidValue;
    auto kernel = a.withheld.cta < 0 ? fp8_few_kernel<kRowScales, false>
                                     : fp8_few_kernel<kRowScales, true>;
    return launch(kernel, a.tiles * a.split, kFewThreads, kFewSmem, a.split, st, tmw, tmx, a);
}

// Which kernel a product takes.  bn: rows of B per tile of the first one; kFewRowsPlan:
// changed places; kNoStagesPlan: kda_fp8_small.cu.
constexpr int kFewRowsPlan = 0, kNoStagesPlan = -1;
void plan(int M, int N, int K, bool b_rows, int sms, int* bn, int* split) {
    // few rows: the kernel without stages while it takes a round or two (of 4096
    // columns by 32 rows of B an SM), then the one of changed places (us, 8 and 16
    // rows of A: 4096 x 4096 6.5 and 9.7 against 9.0 and 9.3, 4096 x 2048 4.7 and 6.5
    // against 8.0, 8192 x 4096 11.0 and 17.5 against 11.8, 12288 x 4096 15.4 and 24.9
    // against 14.4)
    *split = 1;
    const long long rounds =
        ((long long)N + 32 * sms - 1) / (32 * sms) * (((long long)K + 4095) / 4096);
    if (M <= 8 ? rounds <= 2 : M <= kFewRows && rounds <= 1) {
        *bn = kNoStagesPlan;
    } else if (M <= kFewRows) {
        *bn = kFewRowsPlan;
        *split = few_split(blocks128(N), blocks128(K), sms);
    } else {
        choose(M, N, blocks128(K), b_rows, sms, bn, split);
    }
}

cudaError_t matmul_with(int bn, int split, const void* a8, const float* a_scale, const void* b8,
                        const float* b_scale, int M, int N, int K, bool b_rows,
                        kda_dtype_t out_dt, void* out, const Fp8Withheld& withheld, int sms,
                        cudaStream_t st) {
    MatmulArgs a{};
    a.withheld = withheld;
    a.sa = a_scale;
    a.sb = b_scale;
    a.out = out;
    a.M = M;
    a.N = N;
    a.KB = blocks128(K);
    a.NB = b_rows ? N : blocks128(N);
    a.out_bf16 = out_dt == KDA_DTYPE_BF16;
    a.out_wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
    a.split = split;
    if (bn == kFewRowsPlan) {
        a.tiles = blocks128(N);
        if ((long long)a.tiles * a.split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        return b_rows ? run_few<true>(a8, b8, a, K, st) : run_few<false>(a8, b8, a, K, st);
    }
    a.ntm = static_cast<int>(((long long)M + kRowsA - 1) / kRowsA);
    const long long tiles = (long long)a.ntm * (((long long)N + bn - 1) / bn);
    if (tiles * split > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<int>(tiles);
    if (bn == 256)
        return b_rows ? run<256, true>(a8, b8, a, K, sms, st) : run<256, false>(a8, b8, a, K, sms, st);
    return b_rows ? run<128, true>(a8, b8, a, K, sms, st) : run<128, false>(a8, b8, a, K, sms, st);
}

}  // namespace

bool fp8_matmul_available() { return encode_fn() != nullptr; }

void fp8_matmul_plan(int M, int N, int K, bool b_rows, int sms, int* tile_rows, int* split) {
    plan(M, N, K, b_rows, sms, tile_rows, split);
}

cudaError_t launch_fp8_matmul(const void* a8, const float* a_scale, const void* b8,
                              const float* b_scale, int M, int N, int K, bool b_rows,
                              kda_dtype_t out_dt, void* out, cudaStream_t st,
                              const Fp8Withheld& withheld) {
    if (M == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int bn = 0, split = 1;
    plan(M, N, K, b_rows, sms, &bn, &split);
    if (bn == kNoStagesPlan && withheld.cta >= 0) return cudaErrorNotSupported;  // (no waits)
    if (bn == kNoStagesPlan)
        return launch_fp8_small(a8, a_scale, b8, b_scale, M, N, K, b_rows, out_dt, out, st);
    return matmul_with(bn, split, a8, a_scale, b8, b_scale, M, N, K, b_rows, out_dt, out, withheld, sms,
                       st);
}

}  // namespace kda

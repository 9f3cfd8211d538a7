// Gated linear recurrence: h_t = exp(g_t) h_{t-1} + x_t per (sequence, head,
// channel), its backward pass and its one-token step.
//
// The delta-rule operator without the key side (one state value per channel):
// every (token, channel) is an affine map h -> alpha h + x, and maps compose
// associatively, (alpha2, x2) o (alpha1, x1) = (alpha1 alpha2, alpha2 x1 + x2),
// so a long sequence splits over time.  A token is used once (a few flops per
// 8 bytes), so the kernels are bound by HBM: each element is read once and
// written once, and the state crosses tiles through a few bytes per channel.
//
// Forward: the packed tokens are cut into tiles of 64 (256 where lanes have one
// channel; regardless of sequence bounds) by 128 channels.  A 256-thread CTA holds
// one tile in registers: lane l of warp w holds channels [4 l, 4 l + 4) of rows
// [8 w, 8 w + 8), all loads issued at once.  Each warp composes its eight rows,
// the CTA's eight maps are composed through shared memory, and the tile's entry
// state comes from the tiles before it: each publishes its composed map, the last
// one of a group also that of the group, and, once it knows it, the group's exit
// state (a group is one tile, or several where there are few channels).  A tile's
// entry state is the exit state of the group before its own, passed through the
// maps of its own group's tiles in their order; the exit state of a group comes in
// the same way through the maps of groups.  So the state is computed by one
// formula whatever was published first, and results do not depend on the order
// of execution.  Then every warp runs the recurrence once more from its own entry
// state, in the order of the definition, and writes h.
// The first token of a sequence replaces the state by the initial one: a map that
// forgets the state before it is an exit state by itself.
//
// A published value is one 64-bit word per (tile, channel), written and read
// with single relaxed accesses, so that no fence is needed: {log2 of the gate
// product, state part}; two NaN patterns in the first half mark "not yet" and
// "exit state".  Gate products stay logarithms (their sum in fp32) until they
// meet a state: exp is split into two factors, so that a product beyond the
// fp32 range times a small state is still right.
//
// Tiles are taken by ticket in the order of the look-back (channels fastest),
// so a tile only ever waits for tiles that have started.  The waits are
// bounded all the same.
//
// Backward: with e the gradient that reaches the state from the right (the
// final state's gradient at a sequence's last token),
//     dh_t = dout_t + e_{t+1},  dx_t = dh_t,  e_t = alpha_t dh_t,
//     dg_t = e_t h_{t-1},  dh_0 = e at the first token:
// the same look-back runs from the right for e, and h_{t-1} is recomputed
// inside each tile from the tile's entry state, which the forward keeps (one
// fp32 row per 64 tokens).  x, g, dout in and dx, dg out, each once.
//
// Measured on a B200 (of the copy rate of 6.53 TB/s), bf16, calls in a graph: forward
// of 65536 x 4096 channels 414 us (79 %; 447 a call, one after another from Python; 576
// in fp32, 86 %), backward 667 (86 %; fp32 813); 4096 x 4096 33 and 53 (both 90, 96 from
// Python); 262144 x 128 93 and 130; a step of 256 x 4096 2.5 us (7).
// Against the copy rate the look-back costs most: without it the long forward
// took 350.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_common.cuh"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// A warp has R rows of a tile and a lane VEC channels; a tile has 8 R rows, a
// multiple of the kScanRows between entry states.
constexpr uint32_t kNotYet = 0xFFFFFFFFu;   // NaNs: no sum of logarithms is one
constexpr uint32_t kExit = 0xFFFFFFFEu;
constexpr int kDepth = 64;             // groups' maps a look-back passes at most

struct ScanArgs {
    const void* x;
    const float* g;
    const float* h0;        // initial states [N, C] or NULL
    const int32_t* cu;      // packed offsets or NULL
    int T, total, N, C;
    void* h;                // forward: [total, C], or NULL (entry states only)
    float* final_state;     // [N, C] or NULL
    float* entry;           // [tiles, C]: forward: out or NULL; backward: in
    const void* dout;       // backward
    const float* dfinal;    // [N, C] or NULL
    void* dx;
    float* dg;
    float* dh0;             // [N, C] or NULL
    uint32_t* status;
    uint32_t* ticket;       // starts at 0xFFFFFFFF; NULL: one tile per channel block
    uint64_t* words;        // [tiles, C] maps, then [groups, C]
    int tiles, ctiles;      // of the launched kernel's size
    int keep_status;        // a pass of the same call has set the status word
    int first_task;         // the tasks before it are never run (0; tests of the waits)
    unsigned long long wait_ns;  // limit of a wait for a word
};

// How x, g and dout are loaded (every element once): past L1, or with L1's and
// L2's ordinary policy, which is better for the backward pass where rows are long
// (65536 tokens, us, past L1 and ordinary: backward of 4096 channels 701 and 665,
// fp32 870 and 809, of 1024 198 and 206; forward of 4096 414 and 425, of 1024 138
// and 145).  Stores go past L1.
enum class Policy { kPastL1, kOrdinary };
constexpr int kLongRow = 2048;

// Four channels (VEC = 4) or one (VEC = 1) of a row; fp32 or bf16.
template <int VEC, typename T>
struct Raw;
template <>
struct Raw<4, float> {
    float4 v;
    __device__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    template <Policy P>
    __device__ void load(const float* p) {
        if (P == Policy::kOrdinary)
            v = __ldg(reinterpret_cast<const float4*>(p));
        else
            asm("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                : "l"(p));
    }
    __device__ void get(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
};
template <>
struct Raw<4, __nv_bfloat16> {
    uint2 v;
    __device__ void zero() { v = make_uint2(0u, 0u); }
    template <Policy P>
    __device__ void load(const __nv_bfloat16* p) {
        if (P == Policy::kOrdinary)
            v = __ldg(reinterpret_cast<const uint2*>(p));
        else
            asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                : "=r"(v.x), "=r"(v.y)
                : "l"(p));
    }
    __device__ void get(float (&o)[4]) const {
        o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xFFFF0000u);
        o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
};
template <typename T>
struct Raw<1, T> {
    T v;
    __device__ void zero() { v = from_f32<T>(0.f); }
    template <Policy>
    __device__ void load(const T* p) { v = *p; }
    __device__ void get(float (&o)[1]) const { o[0] = to_f32(v); }
};

__device__ __forceinline__ void put(float* p, const float (&o)[4]) {
    asm volatile("st.global.L1::no_allocate.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(o[0]),
                 "f"(o[1]), "f"(o[2]), "f"(o[3])
                 : "memory");
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&o)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(o[2], o[3]);
    asm volatile("st.global.L1::no_allocate.v2.u32 [%0], {%1, %2};" ::"l"(p),
                 "r"(*reinterpret_cast<const uint32_t*>(&a)),
                 "r"(*reinterpret_cast<const uint32_t*>(&b))
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void put(T* p, const float (&o)[1]) { *p = from_f32<T>(o[0]); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// exp(g), and its logarithm to base 2 added to G: 2^y (1 + r ln 2) with y + r =
// g log2(e) in two floats, so that the error stays that of ex2 (2 units in the
// last place).  g is held above -1e25 first (a NaN stays one): exp is 0 there all
// the same, and y, r and G stay finite.  So g = -inf is a gate of 0, which any
// state meets as in the definition, and G = -inf is left to the maps below.
__device__ __forceinline__ float gate(float g, float& G) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299e-8f;  // log2(e)
    constexpr float kLn2 = 0.693147182464599609375f;
    asm("max.NaN.f32 %0, %0, 0fE9045951;" : "+f"(g));
    const float y = g * kHi;
    const float r = fmaf(g, kHi, -y) + g * kLo;
    G += y;
    const float e = ex2(y);
    return fmaf(e, r * kLn2, e);
}

// A state times 2^G is (h e) e with e = 2^(G / 2), so that a product of gates
// beyond the fp32 range times a small state is still right (and 0 times a
// product that overflows is 0).
__device__ __forceinline__ float scaled(float h, float e) { return h == 0.f ? 0.f : (h * e) * e; }
// e of a map; negative for one that forgets the state before it (G = -inf).
__device__ __forceinline__ float half_gate(float G) {
    return G == -INFINITY ? -1.f : ex2(0.5f * G);
}
// The state after a map (e, b) applied to h.
__device__ __forceinline__ float applied(float e, float b, float h) {
    return e < 0.f ? b : b + scaled(h, e);
}

__device__ __forceinline__ void publish(uint64_t* w, float G, float b, bool exit_state) {
    const uint32_t lo = exit_state ? kExit : __float_as_uint(G);
    const uint64_t v = static_cast<uint64_t>(__float_as_uint(b)) << 32 | lo;
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(w), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t read_word(const uint64_t* w) {
    uint64_t v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(w) : "memory");
    return v;
}

// A word once it is there (for `exit_only`: once it is an exit state).
__device__ __forceinline__ uint64_t await_word(const uint64_t* w, uint64_t v, bool exit_only,
                                               const ScanArgs& a) {
    const auto ready = [&] {
        const uint32_t lo = static_cast<uint32_t>(v);
        return exit_only ? lo == kExit : lo != kNotYet;
    };
    if (ready()) return v;
    const uint64_t t0 = sm100::global_timer_ns();
    do {
        v = read_word(w);
        if (ready()) return v;
    } while (sm100::global_timer_ns() - t0 <= a.wait_ns);
    atomicOr(a.status, STATUS_TIMEOUT);
    return kExit;  // (a state of 0; the outputs of the call are unspecified)
}
__device__ __forceinline__ float map_G(uint64_t v) {
    return __uint_as_float(static_cast<uint32_t>(v));
}
__device__ __forceinline__ float map_b(uint64_t v) {
    return __uint_as_float(static_cast<uint32_t>(v >> 32));
}

// The exit state of group g: from the nearest group before or at it that has
// published its own (group 0 always does), through the maps of the groups between
// in their order.  Maps found on the way back are kept (in local memory); behind
// kDepth of them only an exit state will do.
__device__ float group_exit(const uint64_t* groups, size_t C, int g, const ScanArgs& a) {
    uint64_t kept[kDepth];
    int n = 0;
    const uint64_t* at = groups + (size_t)g * C;
    uint64_t next = read_word(at);
    float h = 0.f;
    for (; g >= 0; --g, at -= C) {
        uint64_t v = next;
        if (g > 0) next = read_word(at - C);
        v = await_word(at, v, n == kDepth || g == 0, a);
        if (static_cast<uint32_t>(v) == kExit) {
            h = map_b(v);
            break;
        }
        kept[n++] = v;
    }
    while (n > 0) {
        const uint64_t v = kept[--n];
        h = applied(half_gate(map_G(v)), map_b(v), h);
    }
    return h;
}

// Publishes a channel's map (G, b) of the tile at position pos (0: no tile is
// before it), and its group's where it closes one; returns the state that enters
// the tile (0 unless `needed`).
template <int kTiles>
__device__ float pass_tile(const ScanArgs& a, int ch, int pos, float G, float b, bool needed) {
    const size_t C = a.C;
    uint64_t* words = a.words + ch;
    uint64_t* groups = kTiles == 1 ? words : words + (size_t)a.tiles * C;
    const int in = pos % kTiles, g = pos / kTiles;
    uint64_t* own = words + (size_t)(pos - in) * C;  // the group's first tile
    const bool last = pos == a.tiles - 1, closes = in == kTiles - 1 && !last;
    if (!last && !closes) publish(words + (size_t)pos * C, G, b, false);
    // the maps of the group's tiles before this one, requested together
    uint64_t v[kTiles > 1 ? kTiles - 1 : 1];
    const bool all = needed || (closes && G != -INFINITY);
#pragma unroll
    for (int k = 0; k < kTiles - 1; ++k)
        if (all && k < in) v[k] = read_word(own + (size_t)k * C);
    float Gg = 0.f, bg = 0.f;
    bool known = true;
    if (closes) {
        if (G != -INFINITY) {  // (a map that forgets needs none of the others)
#pragma unroll
            for (int k = 0; k < kTiles - 1; ++k) {
                v[k] = await_word(own + (size_t)k * C, v[k], false, a);
                bg = applied(half_gate(map_G(v[k])), map_b(v[k]), bg);
                Gg += map_G(v[k]);
            }
        }
        bg = applied(half_gate(G), b, bg);
        Gg += G;
        known = g == 0 || Gg == -INFINITY;
        publish(groups + (size_t)g * C, Gg, bg, known);
    }
    float h = 0.f;
    if (g > 0 && (needed || !known)) h = group_exit(groups, C, g - 1, a);
    if (!known) publish(groups + (size_t)g * C, 0.f, applied(half_gate(Gg), bg, h), true);
    if (!needed) return 0.f;
#pragma unroll
    for (int k = 0; k < kTiles - 1; ++k) {
        if (k >= in) break;
        v[k] = await_word(own + (size_t)k * C, v[k], false, a);
        h = applied(half_gate(map_G(v[k])), map_b(v[k]), h);
    }
    return h;
}

// Where the tile's sequences begin and end: first_of[r] = the sequence whose first
// token is row r, last_of[r] = the one whose last token it is, -1 elsewhere.
// Reads of cu stay inside [0, N] and writes inside the tile whatever cu holds.
template <int kRows>
struct Bounds {
    int first_of[kRows], last_of[kRows];
    int lo;      // the last sequence whose first token is at or before the tile
    int plain;   // the tile lies inside one sequence, which goes on beyond both ends
};
// By every thread of the CTA; ends with a barrier.
template <int kRows>
__device__ __forceinline__ void find_bounds(const ScanArgs& a, int t0, Bounds<kRows>& s) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int lo = 0;
        if (!a.cu) {
            lo = a.T > 0 ? t0 / a.T : 0;
        } else {  // 32 offsets at a time
            int span = a.N;
            while (true) {
                const int step = span <= 32 ? 1 : (span + 31) / 32;
                const int idx = lo + lane * step;
                const bool le = idx < lo + span && idx < a.N && a.cu[idx] <= t0;
                const unsigned m = __ballot_sync(0xffffffffu, le);
                lo += (m ? 31 - __clz(static_cast<int>(m)) : 0) * step;
                if (step == 1) break;
                span = min(step, a.N - lo);
            }
        }
        if (lane == 0) {
            const int b = a.cu ? a.cu[lo] : lo * a.T;
            const int e = a.cu ? a.cu[lo + 1] : (lo + 1) * a.T;
            s.lo = lo;
            s.plain = b < t0 && e > t0 + kRows && t0 + kRows <= a.total;
        }
    }
    __syncthreads();
    if (s.plain) return;
    for (int r = threadIdx.x; r < kRows; r += kThreads) s.first_of[r] = s.last_of[r] = -1;
    __syncthreads();
    for (int i = s.lo + threadIdx.x; i < a.N; i += kThreads) {
        const int b = (a.cu ? a.cu[i] : i * a.T) - t0;
        if (b >= kRows) break;
        const int e = (a.cu ? a.cu[i + 1] : (i + 1) * a.T) - t0;
        if (e <= b) continue;  // an empty sequence has no token
        if (b >= 0) s.first_of[b] = i;
        if (e >= 1 && e <= kRows) s.last_of[e - 1] = i;
    }
    __syncthreads();
}

// Whether the offsets run from 0 to total without decreasing: the CTA of the
// first tile and channels sets the status word (it starts before every CTA
// that could report a timeout there, and such a report is seconds later); the
// second pass of a call adds to what the first one left there.
__device__ void report_status(const ScanArgs& a) {
    bool bad = false;
    if (a.cu) {
        for (int i = threadIdx.x; i < a.N; i += kThreads) bad |= a.cu[i] > a.cu[i + 1];
        if (threadIdx.x == 0) bad |= a.cu[0] != 0 || a.cu[a.N] != a.total;
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x != 0) return;
    if (!a.keep_status) *a.status = any ? STATUS_BAD_SEQLENS : 0u;
    else if (any) atomicOr(a.status, STATUS_BAD_SEQLENS);
}

// States of empty sequences: nothing changes them (channels [c0, c0 + n)).
__device__ void pass_empty(const ScanArgs& a, const float* from, float* to, int c0, int n) {
    if (!to) return;
    for (int i = threadIdx.x / 32; i < a.N; i += kWarps) {
        const int len = a.cu ? a.cu[i + 1] - a.cu[i] : a.T;
        if (len > 0) continue;
        for (int c = threadIdx.x & 31; c < n; c += 32) {
            const size_t k = (size_t)i * a.C + c0 + c;
            to[k] = from ? from[k] : 0.f;
        }
    }
}

// The tile this CTA works on, in the order in which tiles wait for one another.
__device__ __forceinline__ int next_tile(const ScanArgs& a) {
    if (!a.ticket) return blockIdx.x;
    __shared__ uint32_t s_ticket;
    if (threadIdx.x == 0) s_ticket = atomicAdd(a.ticket, 1u) + 1u;
    __syncthreads();
    return static_cast<int>(s_ticket) + a.first_task;
}

// A warp's rows of a tile in registers.  Lanes beyond the last channel load the
// last ones again (they store nothing); rows beyond the last token hold zeros,
// which change no state.
template <Policy P, int VEC, int R, typename U>
__device__ __forceinline__ void load_rows(Raw<VEC, U> (&v)[R], const U* p, size_t C, int rows) {
    if (rows >= R) {
#pragma unroll
        for (int r = 0; r < R; ++r) v[r].template load<P>(p + r * C);
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r].zero();
            if (r < rows) v[r].template load<P>(p + r * C);
        }
    }
}
template <int VEC>
__device__ __forceinline__ void state_of(const float* states, int seq, size_t C, int c,
                                         float (&v)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = states ? states[(size_t)seq * C + c + j] : 0.f;
}

// Shared memory of a tile: the warps' maps and, in the end, the states that
// enter the warps.
template <int VEC>
struct Maps {
    float G[kWarps][32 * VEC], e[kWarps][32 * VEC], b[kWarps][32 * VEC];
    __device__ void set(int w, int lane, const float (&g)[VEC], const float (&v)[VEC]) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            // (a NaN, or gates beyond fp32's range, are in v too; here they would
            // turn the -inf of a later sequence's start into NaN)
            const float sum = fminf(g[j], 1e30f);
            G[w][lane * VEC + j] = sum;
            e[w][lane * VEC + j] = half_gate(sum);
            b[w][lane * VEC + j] = v[j];
        }
    }
    __device__ float sum(int ch) const {
        float g = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) g += G[i][ch];
        return g;
    }
    // Walks a channel's state through the warps (from the last one if
    // kReverse); kKeep: leaves in b what enters each.  Returns what leaves.
    template <bool kReverse, bool kKeep>
    __device__ float walk(int ch, float h) {
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const int i = kReverse ? kWarps - 1 - k : k;
            const float bi = b[i][ch];
            if (kKeep) b[i][ch] = h;
            h = applied(e[i][ch], bi, h);
        }
        return h;
    }
};

// Tiles of a group: where few blocks of channels leave many tiles of one sequence on
// the device at once, groups keep the look-back short (bf16, us, forward / backward:
// 262144 x 128 in groups of six 93 / 129, without 244; 65536 x 512 in sixes 75 / 113,
// in threes 73 / 109; 200000 x 1024 in sixes 375 / 602, in threes 363 / 593, without
// 401 / 583; 65536 x 4096 in sixes 448, without 415).
constexpr int kLongGroup = 6, kShortGroup = 3;
inline int group_of(int vec, int ctiles, bool backward) {
    if (ctiles <= 2) return kLongGroup;
    return ctiles < (vec == 4 && !backward ? 16 : 8) ? kShortGroup : 1;
}

// A thread's gates between the two passes over its rows, where a lane has one
// channel (its 32 rows are more registers than there are: 100000 x 155 bf16 58 ->
// 54 us; with four channels they stay in registers, 415 us against 430).
template <int VEC, int R>
struct KeptGates {
    float v[VEC == 1 ? R : 1][VEC == 1 ? kThreads : 1];
};

// kBounds: sequences begin or end in the tile, or the tokens do.
template <int VEC, int R, int GROUP, typename T, bool kBounds>
__device__ __forceinline__ void fwd_tile(const ScanArgs& a, int tile, int c0, Maps<VEC>& s_maps,
                                         const Bounds<8 * R>& s_bounds, KeptGates<VEC, R>& s_gates,
                                         const Raw<VEC, T> (&xr)[R],
                                         const Raw<VEC, float> (&gr)[R], int c, bool mine) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, t0 = tile * 8 * R;
    const size_t C = a.C;
    // the map of this warp's rows
    float al[VEC == 1 ? 1 : R][VEC];  // (one channel: the present row's)
    {
        float G[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) G[j] = b[j] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            constexpr bool kKeep = VEC == 1;
            const int k = kKeep ? 0 : r;
            float gv[VEC], xv[VEC];
            gr[r].get(gv);
            xr[r].get(xv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) al[k][j] = gate(gv[j], G[j]);
            const int first = kBounds ? s_bounds.first_of[w * R + r] : -1;
            if (kBounds && first >= 0) {
                state_of<VEC>(a.h0, first, C, c, b);
#pragma unroll
                for (int j = 0; j < VEC; ++j) G[j] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[j] = fmaf(al[k][j], b[j], xv[j]);
            // from here on a first row's al is its state: initial_state is read
            // before this tile publishes anything, so that final_state may be
            // the same buffer
            if (kBounds && first >= 0) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) al[k][j] = b[j];
            }
            if (kKeep) s_gates.v[kKeep ? r : 0][kKeep ? threadIdx.x : 0] = al[0][0];
        }
        s_maps.set(w, lane, G, b);
    }
    __syncthreads();

    // one thread per channel: the tile's map out, its entry state in, every
    // warp's entry state
    if (threadIdx.x < 32 * VEC && c0 + threadIdx.x < a.C) {
        const int ch = threadIdx.x;
        float h = 0.f;
        // (the entry state is used unless a sequence starts with the tile)
        if (a.ticket)
            h = pass_tile<GROUP>(a, c0 + ch, tile, s_maps.sum(ch), s_maps.template walk<false, false>(ch, 0.f),
                          !(kBounds && s_bounds.first_of[0] >= 0));
        s_maps.template walk<false, true>(ch, h);
        if (a.entry) {  // the states before rows 0, kScanRows, ... of the tile
            constexpr int W = kScanRows / R < 1 ? 1 : kScanRows / R;
            const int n0 = t0 / kScanRows, n1 = (a.total - 1) / kScanRows;
#pragma unroll
            for (int i = 0; i < kWarps; i += W) {
                const int n = n0 + i * R / kScanRows;
                if (i == 0 || n <= n1) a.entry[(size_t)n * C + c0 + ch] = s_maps.b[i][ch];
            }
        }
    }
    if (!a.h && !a.final_state) return;
    __syncthreads();

    // the recurrence from this warp's entry state
    if (!mine) return;
    float h[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = s_maps.b[w][lane * VEC + j];
    T* out = static_cast<T*>(a.h) + (size_t)(t0 + w * R) * C + c;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (kBounds && t0 + w * R + r >= a.total) return;
        const int first = kBounds ? s_bounds.first_of[w * R + r] : -1;
        constexpr bool kKeep = VEC == 1;
        const int k = kKeep ? 0 : r;
        if (kKeep) al[0][0] = s_gates.v[kKeep ? r : 0][kKeep ? threadIdx.x : 0];
        float xv[VEC];
        xr[r].get(xv);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            h[j] = kBounds && first >= 0 ? al[k][j] : fmaf(al[k][j], h[j], xv[j]);
        if (a.h) put(out + r * C, h);
        const int last = kBounds ? s_bounds.last_of[w * R + r] : -1;
        if (kBounds && last >= 0 && a.final_state) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) a.final_state[(size_t)last * C + c + j] = h[j];
        }
    }
}

template <int VEC, int R, int GROUP, typename T>
__global__ void __launch_bounds__(kThreads, 3) scan_fwd_kernel(const ScanArgs a) {
    constexpr int CT = 32 * VEC;  // channels of a tile
    __shared__ __align__(16) Maps<VEC> s_maps;
    __shared__ KeptGates<VEC, R> s_gates;
    __shared__ Bounds<8 * R> s_bounds;
    const int task = next_tile(a), tile = task / a.ctiles, c0 = (task % a.ctiles) * CT;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (tile * 8 + w) * R, mine = c0 + lane * VEC < a.C;
    const int c = mine ? c0 + lane * VEC : a.C - VEC;
    Raw<VEC, T> xr[R];
    Raw<VEC, float> gr[R];
    load_rows<Policy::kPastL1>(xr, static_cast<const T*>(a.x) + (size_t)t * a.C + c, a.C,
                               a.total - t);
    load_rows<Policy::kPastL1>(gr, a.g + (size_t)t * a.C + c, a.C, a.total - t);
    find_bounds(a, tile * 8 * R, s_bounds);
    if (tile == 0) {
        if (c0 == 0) report_status(a);
        pass_empty(a, a.h0, a.final_state, c0, min(CT, a.C - c0));
    }
    if (s_bounds.plain)
        fwd_tile<VEC, R, GROUP, T, false>(a, tile, c0, s_maps, s_bounds, s_gates, xr, gr, c, mine);
    else
        fwd_tile<VEC, R, GROUP, T, true>(a, tile, c0, s_maps, s_bounds, s_gates, xr, gr, c, mine);
}

template <int VEC, int R, int GROUP, typename T, bool kBounds>
__device__ __forceinline__ void bwd_tile(const ScanArgs& a, int tile, int c0, Maps<VEC>& s_maps,
                                         Maps<VEC>& s_back, const Bounds<8 * R>& s_bounds,
                                         const Raw<VEC, T> (&xr)[R], const Raw<VEC, T> (&dr)[R],
                                         const Raw<VEC, float> (&gr)[R], int c, bool mine) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, t0 = tile * 8 * R;
    const size_t C = a.C;
    // the two maps of this warp's rows: of h, and of e from the right
    float al[R][VEC];
    {
        float G[VEC], Ge[VEC], b[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) G[j] = b[j] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float gv[VEC], xv[VEC];
            gr[r].get(gv);
            xr[r].get(xv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) al[r][j] = gate(gv[j], G[j]);
            const int first = kBounds ? s_bounds.first_of[w * R + r] : -1;
            if (kBounds && first >= 0) state_of<VEC>(a.h0, first, C, c, b);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[j] = fmaf(al[r][j], b[j], xv[j]);
        }
        bool starts = false, ends = false;
        if (kBounds) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                starts |= s_bounds.first_of[w * R + r] >= 0;
                ends |= s_bounds.last_of[w * R + r] >= 0;
            }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            Ge[j] = kBounds && ends ? -INFINITY : G[j];
            if (kBounds && starts) G[j] = -INFINITY;
        }
        s_maps.set(w, lane, G, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = 0.f;
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
            const int last = kBounds ? s_bounds.last_of[w * R + r] : -1;
            if (kBounds && last >= 0) state_of<VEC>(a.dfinal, last, C, c, b);
            float dv[VEC];
            dr[r].get(dv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) b[j] = al[r][j] * (dv[j] + b[j]);
        }
        s_back.set(w, lane, Ge, b);
    }
    __syncthreads();

    if (threadIdx.x < 32 * VEC && c0 + threadIdx.x < a.C) {
        const int ch = threadIdx.x;
        float e = 0.f;
        if (a.ticket)
            e = pass_tile<GROUP>(a, c0 + ch, a.tiles - 1 - tile, s_back.sum(ch),
                          s_back.template walk<true, false>(ch, 0.f),
                          !(kBounds && s_bounds.last_of[8 * R - 1] >= 0));
        s_back.template walk<true, true>(ch, e);
    } else if (threadIdx.x >= kThreads - 32 * VEC && c0 + threadIdx.x - (kThreads - 32 * VEC) < a.C) {
        // meanwhile (other warps): the states that enter the warps
        const int ch = threadIdx.x - (kThreads - 32 * VEC);
        s_maps.template walk<false, true>(ch, a.entry[(size_t)(t0 / kScanRows) * C + c0 + ch]);
    }
    __syncthreads();

    if (!mine) return;
    float hb[R][VEC], h[VEC], e[VEC];  // hb: the state before each row
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        h[j] = s_maps.b[w][lane * VEC + j];
        e[j] = s_back.b[w][lane * VEC + j];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int first = kBounds ? s_bounds.first_of[w * R + r] : -1;
        if (kBounds && first >= 0) state_of<VEC>(a.h0, first, C, c, h);
        float xv[VEC];
        xr[r].get(xv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            hb[r][j] = h[j];
            h[j] = fmaf(al[r][j], h[j], xv[j]);
        }
    }
    T* dx = static_cast<T*>(a.dx) + (size_t)(t0 + w * R) * C + c;
    float* dg = a.dg + (size_t)(t0 + w * R) * C + c;
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
        if (kBounds && t0 + w * R + r >= a.total) continue;
        const int last = kBounds ? s_bounds.last_of[w * R + r] : -1;
        if (kBounds && last >= 0) state_of<VEC>(a.dfinal, last, C, c, e);
        float dv[VEC], dgv[VEC];
        dr[r].get(dv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            dv[j] += e[j];
            e[j] = al[r][j] * dv[j];
            dgv[j] = e[j] * hb[r][j];
        }
        put(dx + r * C, dv);
        put(dg + r * C, dgv);
        const int first = kBounds ? s_bounds.first_of[w * R + r] : -1;
        if (kBounds && first >= 0 && a.dh0) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) a.dh0[(size_t)first * C + c + j] = e[j];
        }
    }
}

template <int VEC, int R, int GROUP, Policy P, typename T>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(const ScanArgs a) {
    constexpr int CT = 32 * VEC;
    __shared__ __align__(16) Maps<VEC> s_maps, s_back;
    __shared__ Bounds<8 * R> s_bounds;
    const int task = next_tile(a), tile = a.tiles - 1 - task / a.ctiles;
    const int c0 = (task % a.ctiles) * CT;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = (tile * 8 + w) * R, mine = c0 + lane * VEC < a.C;
    const int c = mine ? c0 + lane * VEC : a.C - VEC;
    Raw<VEC, T> xr[R], dr[R];
    Raw<VEC, float> gr[R];
    load_rows<P>(gr, a.g + (size_t)t * a.C + c, a.C, a.total - t);
    load_rows<P>(xr, static_cast<const T*>(a.x) + (size_t)t * a.C + c, a.C, a.total - t);
    load_rows<P>(dr, static_cast<const T*>(a.dout) + (size_t)t * a.C + c, a.C, a.total - t);
    find_bounds(a, tile * 8 * R, s_bounds);
    if (tile == a.tiles - 1) {
        if (c0 == 0) report_status(a);
        pass_empty(a, a.dfinal, a.dh0, c0, min(CT, a.C - c0));
    }
    if (s_bounds.plain)
        bwd_tile<VEC, R, GROUP, T, false>(a, tile, c0, s_maps, s_back, s_bounds, xr, dr, gr, c, mine);
    else
        bwd_tile<VEC, R, GROUP, T, true>(a, tile, c0, s_maps, s_back, s_bounds, xr, dr, gr, c, mine);
}

// One token per sequence: state = exp(g) state + x, h = the state in T.
template <int VEC, typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(const T* __restrict__ x,
                                                        const float* __restrict__ g,
                                                        const float* state_in, float* state_out,
                                                        T* __restrict__ h, long long n) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * VEC;
    if (i >= n) return;
    Raw<VEC, T> xr;
    Raw<VEC, float> gr, sr;
    xr.template load<Policy::kPastL1>(x + i);
    gr.template load<Policy::kPastL1>(g + i);
    sr.v = *reinterpret_cast<const decltype(sr.v)*>(state_in + i);  // (may be state_out)
    float xv[VEC], gv[VEC], s[VEC];
    xr.get(xv);
    gr.get(gv);
    sr.get(s);
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = fmaf(expf(gv[j]), s[j], xv[j]);
    put(state_out + i, s);
    put(h + i, s);
}

// The workspace of a scan: [0, 256) status word, then the ticket (256 bytes)
// and one 64-bit word per (tile, channel) and per (group of tiles, channel) --
// none of these when the tokens fit in one tile -- and, for a backward without
// entry states, those.
struct ScanSpace {
    uint32_t* status;
    uint32_t* ticket;
    uint64_t* words;
    float* entry;
    size_t total_bytes;
};
ScanSpace carve_scan(void* base, int total, int C, bool with_entry) {
    ScanSpace s{};
    char* p = static_cast<char*>(base);
    const size_t tiles = scan_tiles(total);
    s.status = reinterpret_cast<uint32_t*>(p);
    size_t off = kAlign;
    if (tiles > 1) {
        s.ticket = reinterpret_cast<uint32_t*>(p + off);
        s.words = reinterpret_cast<uint64_t*>(p + off + kAlign);
        off = align_up(off + kAlign + sizeof(uint64_t) * (tiles + tiles / kShortGroup) * C);
    }
    if (with_entry) {
        s.entry = reinterpret_cast<float*>(p + off);
        off = align_up(off + sizeof(float) * tiles * C);
    }
    s.total_bytes = off;
    return s;
}

template <int VEC, int R, int GROUP, typename T>
auto scan_kernel(bool backward) {
    return backward ? scan_bwd_kernel<VEC, R, GROUP, Policy::kPastL1, T>
                    : scan_fwd_kernel<VEC, R, GROUP, T>;
}

template <int VEC, int R, typename T>
cudaError_t run_scan(ScanArgs a, const ScanSpace& s, bool backward, bool withhold,
                     cudaStream_t st) {
    static_assert(8 * R % kScanRows == 0, "a tile begins at an entry state");
    a.status = s.status;
    a.tiles = a.total > 0 ? static_cast<int>(((long long)a.total + 8 * R - 1) / (8 * R)) : 1;
    a.ctiles = (a.C + 32 * VEC - 1) / (32 * VEC);
    const long long grid = (long long)a.tiles * a.ctiles;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const int group = group_of(VEC, a.ctiles, backward);
    if (withhold) {
        if (a.tiles < 2) return cudaErrorInvalidConfiguration;  // (no tile waits)
        a.first_task = a.ctiles;
        const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(uint32_t), st);
        if (e != cudaSuccess) return e;
    }
    if (a.tiles > 1) {
        a.ticket = s.ticket;
        a.words = s.words;
        const int words = group == 1 ? a.tiles : a.tiles + a.tiles / group;
        const cudaError_t e =
            cudaMemsetAsync(s.ticket, 0xFF, kAlign + sizeof(uint64_t) * a.C * (size_t)words, st);
        if (e != cudaSuccess) return e;
    }
    auto kernel = group == kLongGroup    ? scan_kernel<VEC, R, kLongGroup, T>(backward)
                  : group == kShortGroup ? scan_kernel<VEC, R, kShortGroup, T>(backward)
                                         : scan_kernel<VEC, R, 1, T>(backward);
    if constexpr (VEC == 4)
        if (backward && a.C >= kLongRow) kernel = scan_bwd_kernel<VEC, R, 1, Policy::kOrdinary, T>;
    kernel<<<static_cast<unsigned>(grid) - a.first_task, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch_scan(const ScanArgs& a, const ScanSpace& s, bool backward, bool withhold,
                          cudaStream_t st) {
    // rows of C channels start on a 16-byte (fp32) or 8-byte (bf16) boundary
    // when C is a multiple of 4; other sizes take one channel per lane, and
    // four times the rows (100000 x 155 bf16: 54 us, 93 with eight rows)
    if (a.C % 4 != 0) return run_scan<1, 32, T>(a, s, backward, withhold, st);
    return run_scan<4, 8, T>(a, s, backward, withhold, st);
}

cudaError_t dispatch_scan(const ScanArgs& a, const ScanSpace& s, bool backward, bool withhold,
                          kda_dtype_t dt, cudaStream_t st) {
    return dt == KDA_DTYPE_BF16 ? dispatch_scan<__nv_bfloat16>(a, s, backward, withhold, st)
                                : dispatch_scan<float>(a, s, backward, withhold, st);
}

}  // namespace

size_t scan_workspace_bytes(int total, int C, bool backward) {
    return carve_scan(nullptr, total, C, backward).total_bytes;
}

cudaError_t launch_scan_fwd(const void* x, const float* g, const float* h0, const int32_t* cu,
                            int T, int total, int N, int C, kda_dtype_t dt, void* h,
                            float* final_state, float* entry, void* workspace, cudaStream_t st,
                            const ScanTimeout& timeout) {
    ScanArgs a{};
    a.wait_ns = timeout.wait_ns;
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu; a.T = T; a.total = total; a.N = N; a.C = C;
    a.h = h; a.final_state = final_state; a.entry = entry;
    return dispatch_scan(a, carve_scan(workspace, total, C, false), false, timeout.withhold, dt, st);
}

cudaError_t launch_scan_bwd(const void* x, const float* g, const float* h0, const void* dout,
                            const float* dfinal, const float* entry, const int32_t* cu, int T,
                            int total, int N, int C, kda_dtype_t dt, void* dx, float* dg,
                            float* dh0, void* workspace, cudaStream_t st,
                            const ScanTimeout& timeout) {
    ScanArgs a{};
    a.wait_ns = timeout.wait_ns;
    a.x = x; a.g = g; a.h0 = h0; a.cu = cu; a.T = T; a.total = total; a.N = N; a.C = C;
    const ScanSpace s = carve_scan(workspace, total, C, entry == nullptr);
    if (!entry) {
        a.entry = s.entry;
        const cudaError_t e = dispatch_scan(a, s, false, timeout.withhold, dt, st);
        if (e != cudaSuccess) return e;
        a.keep_status = 1;
    }
    a.entry = entry ? const_cast<float*>(entry) : s.entry;
    a.dout = dout; a.dfinal = dfinal; a.dx = dx; a.dg = dg; a.dh0 = dh0;
    return dispatch_scan(a, s, true, timeout.withhold && entry, dt, st);
}

cudaError_t launch_scan_step(const void* x, const float* g, const float* state_in,
                             float* state_out, long long n, kda_dtype_t dt, void* h,
                             cudaStream_t st) {
    if (n == 0) return cudaSuccess;
    const bool vec = n % 4 == 0;
    const unsigned grid = static_cast<unsigned>((n + (vec ? 1023 : 255)) / (vec ? 1024 : 256));
    if (dt == KDA_DTYPE_BF16) {
        const __nv_bfloat16* X = static_cast<const __nv_bfloat16*>(x);
        __nv_bfloat16* Hh = static_cast<__nv_bfloat16*>(h);
        if (vec)
            scan_step_kernel<4, __nv_bfloat16><<<grid, 256, 0, st>>>(X, g, state_in, state_out, Hh, n);
        else
            scan_step_kernel<1, __nv_bfloat16><<<grid, 256, 0, st>>>(X, g, state_in, state_out, Hh, n);
    } else {
        const float* X = static_cast<const float*>(x);
        float* Hh = static_cast<float*>(h);
        if (vec)
            scan_step_kernel<4, float><<<grid, 256, 0, st>>>(X, g, state_in, state_out, Hh, n);
        else
            scan_step_kernel<1, float><<<grid, 256, 0, st>>>(X, g, state_in, state_out, Hh, n);
    }
    return cudaGetLastError();
}

}  // namespace kda

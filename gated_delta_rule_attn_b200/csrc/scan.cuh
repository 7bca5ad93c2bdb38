// scan.cuh — the gated linear recurrence with a vector state, one gate per
// channel, and its backward pass:
//     h_t = a_t h_{t-1} + u_t            (h_{-1} = h0)
// with a_t = g_t or sigmoid(g_t) and u_t = x_t or (1 - a_t) x_t (tied).
// Backward, with c_t the gradient that reaches h_t from token t + 1
// (c_{T-1} = dh_last):
//     G_t = dh_t + c_t,  c_{t-1} = a_t G_t,  dh0 = c_{-1},
//     dx_t = G_t [(1 - a_t) G_t],  da_t = G_t h_{t-1} [G_t (h_{t-1} - x_t)],
//     dg_t = da_t, or da_t a_t (1 - a_t) for a logit.
//
// Every token is an affine map of the state, s -> a s + u (backward, from the
// last token on: c -> a c + a dh), and maps compose: (A2, X2) after (A1, X1) is
// (A2 A1, A2 X1 + X2).  Both directions are bound by HBM, so the work is laid out for
// bytes in flight and few instructions an element:
//   - a lane holds two channels (packed fp32 pairs), a warp 64 channels; it takes its
//     tokens serially per channel, so there are no shuffles, and a sequence that starts
//     on the way is a branch the whole warp takes;
//   - its tokens come in steps of kScanR as TMA boxes into a ring of the warp's own slots
//     (rows that TMA cannot take: copies of single elements); outputs replace their inputs
//     in the slot and leave it by TMA.
// The warps divide the token axis (a walk) in one of three ways, by scan_plan:
//   kScanOut, alone   a warp takes the whole walk: short ones, and many channel blocks;
//   kScanTeam         the W warps of the K CTAs of a cluster take consecutive steps.
//                     Each composes its step's map, the CTA composes its warps' and
//                     writes the result into the shared memory of the cluster's CTAs, and
//                     every warp applies the maps before its step to the state that entered
//                     the round.  One pass over the data, one exchange a round;
//   kScanMap and then kScanOut, in segments   a first kernel composes the map of every
//                     segment but the last; the warps of the second apply the maps before
//                     theirs to the initial state and then take their segment.  Two passes
//                     over the gates and inputs, but no warp waits for another: for few
//                     channel blocks, where clusters would have to be large.
// Several sequences on one token axis (packed ones, or short dense ones) are walked
// as one: at a sequence's first token the map forgets the state before it
// (kScanReset), so the load does not depend on the lengths.
// The order of all sums is fixed: results are the same from run to run.
// Measured (bf16): forward B=2 T=8192 D=2048, fp32 gates, 56 us (4.8 TB/s of what it
// cannot do without); backward B=4 T=8192 D=4096 310 to 318 us (6.0 TB/s); T=32768 D=1024
// with tied logits 68 us forward and 95 us backward (3.0 and 4.2 TB/s).
#pragma once

#include <algorithm>
#include <climits>
#include <type_traits>

#include "rowvec.cuh"

namespace la {

struct ScanParams {
    int64_t B, T, D;
    const void *x, *g;
    int64_t x_row, g_row;
    const float *h0;
    void *h;
    int64_t h_row;
    float *h_last;
    // backward
    const void *hs, *dh;            // stored outputs, their gradient
    int64_t hs_row, dh_row;
    const float *dh_last;
    void *dx, *dg;
    int64_t dx_row, dg_row;
    float *dh0;
    const int64_t *cu_seqlens;
    int64_t max_seqlen;
    int logit, tied;
    int n;                          // sequences per walk
    int ncb;                        // channel blocks
    int nblk;                       // channel blocks of all walks
    int S, L;                       // segments per walk, tokens per segment (a multiple of kScanR)
    int W, NS, K;                   // warps per CTA, slots per warp, CTAs per cluster
    void *scratch;                  // S > 1: see ScanScratch
};
struct ScanTiles {
    CUtensorMap g, x, dh, hs, dx, dg, h;   // boxes of kScanR tokens
};

constexpr int kScanCB = 64;         // channels of a warp, two a lane (a team's warps share them)
constexpr int kScanR = 16;          // tokens a step
constexpr int kScanStages = 3;      // slots of a warp (more where warps are few)
constexpr int kScanMaxStages = 8;
constexpr int kScanW = 4;           // warps of a CTA (a team: up to twice as many)
enum : int { kScanOut = 0, kScanMap = 1, kScanTeam = 2 };

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Write a float4 at the address that `saddr` (own shared memory) has in CTA `rank`
// and count its bytes at that CTA's barrier: the data and its arrival are one
// message, with no fence (a release at cluster scope would also wait for the
// output's stores: 77 against 60 us at B=2, T=8192, D=2048).
__device__ __forceinline__ void st_async_f4(uint32_t saddr, uint32_t sbar, uint32_t rank, float4 v) {
    uint32_t remote, bar;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(saddr), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(sbar), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(remote), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar) : "memory");
}

// Scratch of a call whose walks are cut, for every segment and channel block: the
// segment's map as (A0, A1, X0, X1) per lane, and the state that the last sequence
// starting in it starts from (the second kernel may by then have written that
// sequence's end over it).
struct ScanScratch {
    static constexpr size_t kMap = 32 * 16, kBegin = 32 * 8;
    static size_t bytes(int64_t S, int64_t nblk) { return (size_t)S * (size_t)nblk * (kMap + kBegin); }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// a and r = 1 - a of a gate or of its logit l.  The exponential of a logit is taken of -|l|,
// so neither overflows nor cancels.  The larger of the two is good to 4 half steps of fp32,
// the smaller to 12 + 2.4 |l| of them (the exponential's documented 2 + 1.2 |l| steps and the
// quotient's; measured 3 at 0, 16 at 20, 64 at 87); from |l| = 87.34 on, where the exponential
// is flushed, it is 0.
template <bool LOGIT>
__device__ __forceinline__ void gate(float g, float &a, float &r) {
    if (!LOGIT) {
        a = g;
        r = 1.f - g;
    } else {
        const float e = ex2_approx(fabsf(g) * -1.4426950408889634f), big = rcp_approx(1.f + e), small = e * big;
        a = g >= 0.f ? big : small;
        r = g >= 0.f ? small : big;
    }
}
template <bool LOGIT>
__device__ __forceinline__ void gate(float2 g, float2 &a, float2 &r) {
    if (!LOGIT) {
        a = g;
        r = make_float2(1.f - g.x, 1.f - g.y);
    } else {
        const float2 e = make_float2(ex2_approx(fabsf(g.x) * -1.4426950408889634f), ex2_approx(fabsf(g.y) * -1.4426950408889634f));
        const float2 s = add2(e, make_float2(1.f, 1.f)), big = make_float2(rcp_approx(s.x), rcp_approx(s.y)), small = mul2(e, big);
        a = make_float2(g.x >= 0.f ? big.x : small.x, g.y >= 0.f ? big.y : small.y);
        r = make_float2(g.x >= 0.f ? small.x : big.x, g.y >= 0.f ? small.y : big.y);
    }
}

// Two channels' maps: gate products and offsets.
struct ScanMap {
    float2 A, X;
};
// The gate product of a map that forgets the state before it (a sequence starts
// inside).  A flag and not a zero, so that an infinity or a NaN of the sequence
// before does not reach the next one.  No product of gates has these bits: the
// hardware's products give one canonical NaN.
constexpr uint32_t kScanReset = 0x7fa5c31du;
__device__ __forceinline__ bool map_resets(const ScanMap &m) { return __float_as_uint(m.A.x) == kScanReset; }
__device__ __forceinline__ ScanMap map_load(const float4 *p) {
    const float4 v = *p;
    return ScanMap{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
__device__ __forceinline__ void map_apply(const ScanMap &m, float2 &h) {
    const float2 f = fma2(m.A, h, m.X);
    h = map_resets(m) ? m.X : f;
}
__device__ __forceinline__ ScanMap map_after(const ScanMap &m, const ScanMap &p) {   // m after p
    if (map_resets(m)) return m;
    return ScanMap{map_resets(p) ? p.A : mul2(m.A, p.A), fma2(m.A, p.X, m.X)};
}
// The product of two gates, or gate products, that is 0 only if one of them is: one that
// underflows keeps its sign and the smallest magnitude there is, so that a map made of many
// small gates passes an infinite state on as they do one after the other (0 would make it
// NaN).  A finite state is moved by at most 2^-149 times its size, as by any rounding there.
// Where factors are many the plain product is taken, and this one if that is 0.
__device__ __forceinline__ float mul_kept(float a, float b) {
    const float p = a * b;
    return p == 0.f && a != 0.f && b != 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}
__device__ __forceinline__ float2 mul2_kept(float2 a, float2 b) { return make_float2(mul_kept(a.x, b.x), mul_kept(a.y, b.y)); }
__device__ __forceinline__ bool any_zero(float2 a) { return a.x == 0.f || a.y == 0.f; }
__device__ __forceinline__ void scan_load(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c, int row) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(row) : "memory");
}
__device__ __forceinline__ void scan_store(const CUtensorMap *map, uint32_t src, int c, int row) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c), "r"(row) : "memory");
}

// A lane's two channels of a token in shared memory (rows of 64 channels).  VEC:
// neighbours; else 32 apart, so that single-element stores to global memory are dense.
template <typename T, bool VEC>
__device__ __forceinline__ uint32_t lane_off() {
    return (threadIdx.x & 31) * (uint32_t)sizeof(T) * (VEC ? 2 : 1);
}
template <typename T, bool VEC>
__device__ __forceinline__ float2 take_pair(uint32_t at) {
    float2 v;
    if constexpr (sizeof(T) == 4) {
        if constexpr (VEC) {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
        } else {
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v.x) : "r"(at) : "memory");
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v.y) : "r"(at + 128) : "memory");
        }
    } else if constexpr (VEC) {
        uint32_t r;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
        v = make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    } else {
        unsigned short lo, hi;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(lo) : "r"(at) : "memory");
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(hi) : "r"(at + 64) : "memory");
        v = make_float2(__uint_as_float((uint32_t)lo << 16), __uint_as_float((uint32_t)hi << 16));
    }
    return v;
}
template <typename T>
__device__ __forceinline__ void give_pair(uint32_t at, float2 v) {   // VEC only
    if constexpr (sizeof(T) == 4) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(pack_bf16x2(v.x, v.y)) : "memory");
}
// Two channels of an output token, to global memory.
template <typename T, bool VEC>
__device__ __forceinline__ void put_pair(T *p, float2 v, bool ok0, bool ok1) {
    if (ok0) p[0] = from_f32<T>(v.x);
    if (ok1) p[VEC ? 1 : 32] = from_f32<T>(v.y);
}

// Products with mul2_kept of what the plain product made 0: of the n gates at `at`, `down` apart,
// and of n maps' products.  Calls, so that they take no registers where they are not made
// (in line the forward teams spilled: 57.0 against 55.5 us at B=2, T=8192, D=2048).
template <typename TG, bool VEC, bool LOGIT>
__device__ __noinline__ float2 gates_kept(uint32_t at, int down, int n) {
    float2 A = make_float2(1.f, 1.f);
    for (; n > 0; --n, at += down) {
        float2 a, r;
        gate<LOGIT>(take_pair<TG, VEC>(at), a, r);
        A = mul2_kept(A, a);
    }
    return A;
}
__device__ __noinline__ float2 maps_kept(const float4 *maps, int n) {
    float2 A = map_load(maps).A;
    for (int w = 1; w < n; ++w) A = mul2_kept(A, map_load(maps + w * 32).A);
    return A;
}

// Rows that TMA cannot take: a warp copies the n <= R tokens of its own run, channel
// c0 + lane and the one 32 further, from `p` (this lane's element of the run's first
// place) to rows `at`, `at` + down, ...
template <typename T>
__device__ __forceinline__ void copy_run(const T *p, int64_t row, int n, uint32_t at, int down, bool ok0, bool ok1) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll 4
        for (int r = 0; r < n; ++r) {
            if (ok0) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(p) : "memory");
            if (ok1) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 128), "l"(p + 32) : "memory");
            p += row;
            at += down;
        }
    } else {
        for (int r0 = 0; r0 < n; r0 += 8) {
            unsigned short v[8][2];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                v[r][0] = v[r][1] = 0;
                if (ok0 && r0 + r < n) v[r][0] = __ldg(reinterpret_cast<const unsigned short *>(p));
                if (ok1 && r0 + r < n) v[r][1] = __ldg(reinterpret_cast<const unsigned short *>(p) + 32);
                p += row;
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r0 + r >= n) break;
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(v[r][0]) : "memory");
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 64), "h"(v[r][1]) : "memory");
                at += down;
            }
        }
    }
}

// The sequences of a walk, as places in the order in which it meets the tokens
// (BWD: the last token is place 0).  bound(i) is the first place of the walk's
// i-th sequence, bound(n) the end; id(i) that sequence's number.  Offsets are
// clamped into [0, T], so that no bad array moves an access out of the tensors.
template <bool BWD>
struct ScanSeqs {
    const int64_t *cu;
    int n, T, beg, end, first;
    __device__ __forceinline__ int offset(int j) const {
        if (!cu) return j * T;
        const int64_t v = __ldg(cu + j);
        return v < 0 ? 0 : v > T ? T : (int)v;
    }
    __device__ __forceinline__ ScanSeqs(const ScanParams &P, int walk) : cu(P.cu_seqlens), T((int)P.T) {
        first = walk * P.n;
        n = min(P.n, (int)P.B - first);
        beg = offset(0);
        end = max(beg, offset(n));
    }
    __device__ __forceinline__ int bound(int i) const { return BWD ? end - offset(n - i) : offset(i) - beg; }
    __device__ __forceinline__ int64_t id(int i) const { return first + (BWD ? n - 1 - i : i); }
    // The first i whose bound is not below t (n + 1: none), 32 bounds at a time.
    __device__ __forceinline__ int search(int t) const {
        const int lane = threadIdx.x & 31;
        int lo = 0, left = n + 1;              // the answer lies in [lo, lo + left]
        while (left > 32) {
            const int hop = (left + 31) / 32, i = lo + (lane + 1) * hop - 1;
            const int below = __popc(__ballot_sync(0xffffffffu, i <= n && bound(i) < t));
            lo += below * hop;
            left = min(hop - 1, max(n + 1 - lo, 0));
        }
        return lo + __popc(__ballot_sync(0xffffffffu, lane < left && bound(lo + lane) < t));
    }
    // What the R places from t on meet.  Bit r: a sequence (or the end) lies at place
    // t + r, 0 <= r <= R.  at: the first i whose bound is not below t (it only grows from
    // call to call), so at - 1 is the sequence of place t - 1.
    __device__ __forceinline__ uint32_t marks(int t, int R, int &at) const {
        const int total = end - beg;
        if (n == 1) {
            at = t > 0 ? 1 : 0;
            return (t == 0 ? 1u : 0u) | (total >= t && total - t <= R ? 1u << (total - t) : 0u);
        }
        const int lane = threadIdx.x & 31;
        for (;;) {
            const int i = at + lane;
            const uint32_t m = ~__ballot_sync(0xffffffffu, i <= n && bound(i) < t);
            at += m ? __ffs(m) - 1 : 32;
            if (m) break;
        }
        uint32_t bits = 0;
        for (int i = at + lane;; i += 32) {
            const int v = i <= n ? bound(i) : INT_MAX;
            bits |= v >= t && v - t <= R ? 1u << (v - t) : 0u;
            if (__ballot_sync(0xffffffffu, v > t + R)) break;
        }
        return __reduce_or_sync(0xffffffffu, bits);
    }
    // From the sequence before place t on, the one that place t belongs to.
    __device__ __forceinline__ int walk_to(int i, int t) const {
        while (i + 1 < n && bound(i + 1) <= t) ++i;
        return max(i, 0);
    }
};

template <typename TX, typename TG, bool BWD, bool TIED, bool MAP>
struct ScanShape {
    static constexpr bool kX = !BWD || (TIED && !MAP);        // x is read
    static constexpr bool kD = BWD, kH = BWD && !MAP;         // dh and the stored outputs are
    static constexpr int kBox = kScanR * kScanCB;
    static constexpr uint32_t kGB = kBox * sizeof(TG), kXB = kBox * sizeof(TX);
    static constexpr uint32_t kAtD = kGB, kAtH = kAtD + kXB, kAtX = kGB + (kD ? kXB : 0) + (kH ? kXB : 0);
    static constexpr uint32_t kSlot = kAtX + (kX ? kXB : 0);
};

template <typename TX, typename TG, bool BWD, bool VEC, bool LOGIT, bool TIED, int MODE>
__global__ void __launch_bounds__(kScanW * 32 * (MODE == kScanTeam ? 2 : 1)) scan_kernel(const __grid_constant__ ScanParams P, const __grid_constant__ ScanTiles M) {
    constexpr bool MAP = MODE == kScanMap, TEAM = MODE == kScanTeam;
    using Shape = ScanShape<TX, TG, BWD, TIED, MAP>;
    constexpr int R = kScanR, U = 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, NS = VEC ? P.NS : kScanStages;

    // this warp's segment and channel block
    const int W = P.W, K = TEAM ? P.K : 1, rank = TEAM && K > 1 ? (int)cluster_ctarank() : 0;
    const int64_t unit = TEAM ? blockIdx.x / K : (int64_t)blockIdx.x * W + warp;
    const int seg = (int)(unit / P.nblk), blk = (int)(unit - (int64_t)seg * P.nblk);
    if (MAP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (seg >= P.S - (MAP ? 1 : 0)) return;
    const int walk = blk / P.ncb, c0 = (blk - walk * P.ncb) * kScanCB, D = (int)P.D;
    const ScanSeqs<BWD> seqs(P, walk);
    const int total = seqs.end - seqs.beg;
    float4 *maps = reinterpret_cast<float4 *>(P.scratch) + blk * 32 + lane;                       // [S][nblk][32]
    float2 *begins = reinterpret_cast<float2 *>(reinterpret_cast<float4 *>(P.scratch) + (size_t)P.S * P.nblk * 32) + blk * 32 + lane;

    // this lane's channels
    const int ch0 = c0 + (VEC ? 2 * lane : lane), ch1 = VEC ? ch0 + 1 : ch0 + 32;
    const bool ok0 = ch0 < D, ok1 = ch1 < D;
    auto state = [&](const float *s, int i) {
        float2 v = make_float2(0.f, 0.f);
        if (s) {
            s += seqs.id(i) * D;
            if (ok0) v.x = s[ch0];
            if (ok1) v.y = s[ch1];
        }
        return v;
    };
    auto put_state = [&](float *s, int i, float2 v) {
        if (s) {
            s += seqs.id(i) * D;
            if (ok0) s[ch0] = v.x;
            if (ok1) s[ch1] = v.y;
        }
    };
    const float *s_in = BWD ? P.dh_last : P.h0;
    float *s_out = BWD ? P.dh0 : P.h_last;

    // The places [lo, hi) in steps of R from `origin` on, `hop` apart.  Place t of the walk is
    // token row0 + t, or row0 - t (BWD: the last token is place 0).  A slot holds its tokens
    // in their order in memory: place r of the step is row r, or R - 1 - r.
    const int first = seg * P.L, hi = TEAM ? total : min(total, first + P.L);
    int lo = first, start = -1;
    if (MAP) {
        // what lies before the last sequence that starts here does not matter
        start = (seqs.n == 1 ? (hi > 0 ? 1 : 0) : seqs.search(hi)) - 1;
        const int b = start >= 0 && start < seqs.n ? seqs.bound(start) : -1;
        if (b < first) start = -1;
        else lo = max(b, first);
    }
    const int hop = TEAM ? K * W * R : R;
    const int origin = TEAM ? (rank * W + warp) * R : first + (lo - first) / R * R;
    const int count = TEAM ? (total + hop - 1) / hop : hi > lo ? (hi - origin + R - 1) / R : 0;   // steps
    const int64_t row0 = (seqs.cu ? 0 : (int64_t)seqs.first * P.T) + (BWD ? seqs.end - 1 : seqs.beg);
    constexpr int kDir = BWD ? -1 : 1;
    // shared memory: the warps' slots; of a team two rounds of its warps' maps and of the
    // cluster's (a round's are written while a slow warp may still read those of the round
    // before); the barriers of the slots and of the cluster's maps
    const uint32_t ring = smem_u32(smem) + warp * NS * Shape::kSlot;
    float4 *wmap = reinterpret_cast<float4 *>(smem + W * NS * Shape::kSlot) + lane;   // [2][W][32]
    float4 *cmap = wmap + (TEAM ? 2 * W * 32 : 0);                                    // [2][K][32]
    uint64_t *bars = reinterpret_cast<uint64_t *>(cmap - lane + (TEAM ? 2 * K * 32 : 0));
    uint64_t *full = bars + warp * NS, *heard = bars + W * NS;
    if (VEC) {
        if (lane == 0) {
            for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
            if (TEAM && warp == 0) {
                mbar_init(&heard[0], 1);
                mbar_init(&heard[1], 1);
            }
            fence_barrier_init();
        }
        __syncwarp();
    }
    if (TEAM && K > 1) cluster_sync();         // every CTA of the cluster has its barriers
    // Called by the whole warp; the slot has been read by all lanes.
    auto fetch = [&](int k, int slot) {
        const uint32_t to = ring + slot * Shape::kSlot;
        const int t = origin + k * hop;
        if (k < count && t < hi) {
            if constexpr (VEC) {
                if (lane == 0) {
                    const int row = (int)(row0 + kDir * (int64_t)t) - (BWD ? R - 1 : 0);
                    mbar_arrive_expect_tx(&full[slot], Shape::kSlot);
                    scan_load(to, &M.g, &full[slot], c0, row);
                    if (Shape::kD) scan_load(to + Shape::kAtD, &M.dh, &full[slot], c0, row);
                    if (Shape::kH) scan_load(to + Shape::kAtH, &M.hs, &full[slot], c0, row - 1);
                    if (Shape::kX) scan_load(to + Shape::kAtX, &M.x, &full[slot], c0, row);
                }
            } else {
                const int n = min(R, hi - t);
                const int64_t row = row0 + kDir * (int64_t)t;
                auto copy = [&](auto *p, int64_t stride, int64_t at, uint32_t off, int rows) {
                    using T = std::remove_cv_t<std::remove_reference_t<decltype(*p)>>;
                    constexpr int kB = kScanCB * (int)sizeof(T);
                    copy_run<T>(p + at * stride + ch0, kDir * stride, rows,
                                to + off + (BWD ? R - 1 : 0) * kB + lane * (int)sizeof(T), kDir * kB, ok0, ok1);
                };
                copy(static_cast<const TG *>(P.g), P.g_row, row, 0u, n);
                if (Shape::kD) copy(static_cast<const TX *>(P.dh), P.dh_row, row, Shape::kAtD, n);
                // the walk's last place has no token before it
                if (Shape::kH) copy(static_cast<const TX *>(P.hs), P.hs_row, row - 1, Shape::kAtH, min(n, total - 1 - t));
                if (Shape::kX) copy(static_cast<const TX *>(P.x), P.x_row, row, Shape::kAtX, n);
            }
        }
        if (!VEC) asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // Every box (and message of a cluster) is waited for, so that none is on its way to a CTA that has left: if the limit
    // runs out (the error word is set then), by waits of the full limit from there on.
    int lost = 0;
    uint32_t phases = 0;                       // bit i: the parity of slot i's next arrival
    auto wait = [&](auto cluster, uint64_t *bar, uint32_t parity) {
        constexpr bool C = decltype(cluster)::value;
        if (!lost && mbar_wait<C>(bar, parity)) return;
        lost = lost < 2 && mbar_drain<C>(bar, parity) ? 1 : 2;
    };
    auto arrived = [&](int slot) {
        if constexpr (VEC) {
            wait(std::false_type{}, &full[slot], phases >> slot & 1u);
            phases ^= 1u << slot;
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(kScanStages - 1) : "memory");
            __syncwarp();
        }
    };
    for (int k = 0; k < NS; ++k) fetch(k, k);

    constexpr int kGR = kDir * kScanCB * (int)sizeof(TG), kXR = kDir * kScanCB * (int)sizeof(TX);   // from place to place
    const uint32_t og = (BWD ? R - 1 : 0) * kScanCB * (uint32_t)sizeof(TG) + lane_off<TG, VEC>();
    const uint32_t ox = (BWD ? R - 1 : 0) * kScanCB * (uint32_t)sizeof(TX) + lane_off<TX, VEC>();
    int slot = 0;

    // (a 1 that the compiler does not know, so that every gate passes through a product)
    float one;
    asm volatile("mov.f32 %0, 0f3F800000;" : "=f"(one));
    // The map m, whose gate product is 1, followed by those of the places [rb, r1) of the step in a
    // slot; `starts`: where sequences start, from the states that `from` gives.
    auto compose = [&](ScanMap &m, int slot, int rb, int r1, uint32_t starts, auto from) {
        const uint32_t ag = ring + slot * Shape::kSlot + og;
        const uint32_t au = ring + slot * Shape::kSlot + (BWD ? Shape::kAtD : Shape::kAtX) + ox;
        auto token = [&](float2 g, float2 u) {
            float2 a, n;
            gate<LOGIT>(g, a, n);
            if (BWD) m.X = mul2(a, add2(m.X, u));
            else m.X = fma2(a, m.X, TIED ? mul2(u, n) : u);
            m.A = mul2(m.A, a);
        };
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += U) {
            float2 g[U], u[U];
#pragma unroll
            for (int r = 0; r < U; ++r) {
                g[r] = take_pair<TG, VEC>(ag + (r0 + r) * kGR);
                u[r] = take_pair<TX, VEC>(au + (r0 + r) * kXR);
            }
            if (r1 - rb == R && !starts) {
#pragma unroll
                for (int r = 0; r < U; ++r) token(g[r], u[r]);
            } else {
#pragma unroll
                for (int r = 0; r < U; ++r) {
                    if (r0 + r >= rb && r0 + r < r1) {
                        if (starts >> (r0 + r) & 1) m.X = from(r0 + r);
                        token(g[r], u[r]);
                    }
                }
            }
        }
        // (a gate of 0, or gates of less than 2^-9 on average)
        if (!starts && any_zero(m.A)) m.A = gates_kept<TG, VEC, LOGIT>(ag + rb * kGR, kGR, r1 - rb);
    };
    const float2 zero = make_float2(0.f, 0.f), reset = make_float2(__uint_as_float(kScanReset), __uint_as_float(kScanReset));

    if constexpr (MAP) {
        const float2 s = start >= 0 ? state(s_in, start) : zero;
        ScanMap m{make_float2(one, one), s};
        for (int k = 0; k < count; ++k) {
            arrived(slot);
            const int t = origin + k * R;
            ScanMap step{make_float2(one, one), m.X};
            compose(step, slot, max(lo - t, 0), min(R, hi - t), 0u, [&](int) { return zero; });
            m = ScanMap{mul2_kept(m.A, step.A), step.X};
            __syncwarp();
            fetch(k + NS, slot);
            slot = slot + 1 == NS ? 0 : slot + 1;
        }
        if (start >= 0) m.A = reset;
        maps[(size_t)seg * P.nblk * 32] = make_float4(m.A.x, m.A.y, m.X.x, m.X.y);
        begins[(size_t)seg * P.nblk * 32] = s;
        if (!VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        if (!TEAM && P.S > 1) asm volatile("griddepcontrol.wait;" ::: "memory");   // the segments' maps
        // sequences without tokens pass their state on; bad offsets are reported
        const int worker = TEAM ? rank * W + warp : seg, workers = TEAM ? K * W : P.S;
        for (int i = worker * 32; i < seqs.n; i += workers * 32) {
            const int j = i + lane;
            const bool in = j < seqs.n;
            uint32_t none = __ballot_sync(0xffffffffu, in && seqs.bound(j + 1) <= seqs.bound(j));
            for (; none; none &= none - 1) {
                const int e = i + __ffs(none) - 1;
                put_state(s_out, e, state(s_in, e));
            }
            if (seqs.cu && c0 == 0 && in) {
                const int64_t s = seqs.cu[j], e = seqs.cu[j + 1];
                if (s < 0 || e < s || e > P.T || e - s > P.max_seqlen) raise_error(kErrSeqlen);
            }
        }
        if (count <= 0) return;
        // The state that enters the segment, or a team's round.  The walk's first place is the start
        // of a sequence, so the first map forgets what is before it.
        float2 h = zero, carry = zero, last = zero;
        const bool cut = !TEAM && seg + 1 < P.S;
        if (!TEAM) {
#pragma unroll 16
            for (int i = 0; i < seg; ++i) map_apply(map_load(maps + (size_t)i * P.nblk * 32), h);
            if (cut) last = begins[(size_t)seg * P.nblk * 32];
        }
        // The last sequence that starts in the segment (or a team's step): its state has been read
        // before another warp can write its end over it.
        int kept_start = cut ? (seqs.n == 1 ? 0 : seqs.search(hi) - 1) : -1;
        auto begin = [&](int i) { return i == kept_start ? last : state(s_in, i); };
        int at = seqs.n == 1 ? 0 : seqs.search(origin), q = 0;
        uint32_t parity = 0;
        for (int k = 0; k < count; ++k) {
            const int t = origin + k * hop, n = min(R, hi - t);    // a team's last round: n <= 0 for some
            const uint32_t marks = seqs.marks(t, R, at);
            const uint32_t starts = n > 0 ? marks & ((1u << n) - 1u) : 0u, ends = marks >> 1;
            if constexpr (TEAM) {
                kept_start = starts ? seqs.walk_to(at - 1, t + 31 - __clz(starts)) : -1;
                if (starts) last = state(s_in, kept_start);
                ScanMap m{make_float2(one, one), zero};
                if (n > 0) {
                    arrived(slot);
                    compose(m, slot, 0, n, starts, [&](int r) { return begin(seqs.walk_to(at - 1, t + r)); });
                    if (starts) m.A = reset;
                }
                // the outputs of the round before have left their slot by now
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                if (k > 0) fetch(k - 1 + NS, slot == 0 ? NS - 1 : slot - 1);
                const float4 *wm = wmap + q * W * 32;
                wmap[(q * W + warp) * 32] = make_float4(m.A.x, m.A.y, m.X.x, m.X.y);
                __syncthreads();
                if (K > 1) {
                    // the CTA's map into every CTA of the cluster, which as many warps send
                    if (threadIdx.x == 0) mbar_arrive_expect_tx(&heard[q], K * 512);
                    if (warp < K) {
                        ScanMap c = map_load(wm);
#pragma unroll 4
                        for (int w = 1; w < W; ++w) c = map_after(map_load(wm + w * 32), c);
                        if (any_zero(c.A)) c.A = maps_kept(wm, W);   // (a map that forgets has a NaN there)
                        st_async_f4(smem_u32(&cmap[(q * K + rank) * 32]), smem_u32(&heard[q]), (uint32_t)warp,
                                    make_float4(c.A.x, c.A.y, c.X.x, c.X.y));
                    }
                    wait(std::true_type{}, &heard[q], parity);   // the maps come from the cluster's CTAs
                    for (int i = 0; i < K; ++i) {
                        if (i == rank) h = carry;
                        map_apply(map_load(&cmap[(q * K + i) * 32]), carry);
                    }
#pragma unroll 4
                    for (int w = 0; w < warp; ++w) map_apply(map_load(wm + w * 32), h);
                } else {
#pragma unroll 4
                    for (int w = 0; w < W; ++w) {
                        if (w == warp) h = carry;
                        map_apply(map_load(wm + w * 32), carry);
                    }
                }
                q ^= 1;
                if (!q) parity ^= 1;
            } else {
                arrived(slot);
            }
            const uint32_t base = ring + slot * Shape::kSlot, ag = base + og;
            const uint32_t au = base + (BWD ? Shape::kAtD : Shape::kAtX) + ox, ah = base + Shape::kAtH + ox, ax = base + Shape::kAtX + ox;
            const bool whole = VEC && n == R;  // else outputs go to global memory directly
            const int64_t row = row0 + kDir * (int64_t)t;
            TX *o = static_cast<TX *>(BWD ? P.dx : P.h) + row * (BWD ? P.dx_row : P.h_row) + ch0;
            TG *o2 = BWD ? static_cast<TG *>(P.dg) + row * P.dg_row + ch0 : nullptr;
            const int64_t orow = kDir * (BWD ? P.dx_row : P.h_row), grow = kDir * P.dg_row;
            // the definition's arithmetic.  u: the input, or dh; hp: the state before; xv: the input
            auto token = [&](int r, float2 g, float2 u, float2 hp, float2 xv, bool in_slot) {
                float2 a, n1;
                gate<LOGIT>(g, a, n1);
                if constexpr (BWD) {
                    const float2 G = add2(u, h);
                    float2 dx = G;
                    h = mul2(a, G);
                    if (TIED) {
                        hp = add2(hp, make_float2(-xv.x, -xv.y));
                        dx = mul2(G, n1);
                    }
                    float2 dg = mul2(G, hp);
                    if (LOGIT) dg = mul2(dg, mul2(a, n1));
                    if (in_slot) {
                        give_pair<TX>(au + r * kXR, dx);
                        give_pair<TG>(ag + r * kGR, dg);
                    } else {
                        put_pair<TX, VEC>(o + r * orow, dx, ok0, ok1);
                        put_pair<TG, VEC>(o2 + r * grow, dg, ok0, ok1);
                    }
                } else {
                    if (TIED) u = mul2(u, n1);
                    h = fma2(a, h, u);
                    if (in_slot) give_pair<TX>(au + r * kXR, h);
                    else put_pair<TX, VEC>(o + r * orow, h, ok0, ok1);
                }
            };
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += U) {
                float2 g[U], u[U], hp[U], xv[U];
#pragma unroll
                for (int r = 0; r < U; ++r) {
                    g[r] = take_pair<TG, VEC>(ag + (r0 + r) * kGR);
                    u[r] = take_pair<TX, VEC>(au + (r0 + r) * kXR);
                    hp[r] = BWD ? take_pair<TX, VEC>(ah + (r0 + r) * kXR) : zero;
                    xv[r] = BWD && TIED ? take_pair<TX, VEC>(ax + (r0 + r) * kXR) : zero;
                }
                if (n == R && !starts && !ends) {
#pragma unroll
                    for (int r = 0; r < U; ++r) token(r0 + r, g[r], u[r], hp[r], xv[r], VEC);
                } else {
#pragma unroll
                    for (int r = 0; r < U; ++r) {
                        if (r0 + r < n) {
                            const int p = t + r0 + r;
                            const bool head = starts >> (r0 + r) & 1, tail = ends >> (r0 + r) & 1;
                            const int i = head || tail ? seqs.walk_to(at - 1, p) : 0;
                            if (head) h = begin(i);
                            if (BWD && tail) hp[r] = state(P.h0, i);
                            token(r0 + r, g[r], u[r], hp[r], xv[r], whole);
                            if (tail) put_state(s_out, i, h);
                        }
                    }
                }
            }
            if constexpr (VEC) {
                if (whole) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (whole) {
                        const int r = (int)row - (BWD ? R - 1 : 0);
                        scan_store(BWD ? &M.dx : &M.h, base + (BWD ? Shape::kAtD : Shape::kAtX), c0, r);
                        if (BWD) scan_store(&M.dg, base, c0, r);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    if (!TEAM) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the step before has left its slot
                }
                if (!TEAM && k > 0) fetch(k - 1 + NS, slot == 0 ? NS - 1 : slot - 1);
            } else {
                __syncwarp();
                fetch(k + NS, slot);
            }
            slot = slot + 1 == NS ? 0 : slot + 1;
        }
        if (VEC && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (!VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}

// One token per sequence: state <- a state + u in place (fp32), output rounded
// once.  A thread takes V channels of one sequence; HBM-bound on the state (4096
// sequences of 8192 channels: 80 us, 6.7 TB/s).
template <typename TX, typename TG, int V, bool LOGIT, bool TIED>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanParams P) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V;
    if (i >= P.D) return;
    for (int64_t n = blockIdx.y; n < P.B; n += gridDim.y) {
        RowVec<TX, V> xr;
        RowVec<TG, V> gr;
        float s[V];
        float *st = P.h_last + n * P.D + i;
        xr.load(static_cast<const TX *>(P.x) + n * P.x_row + i);
        gr.load(static_cast<const TG *>(P.g) + n * P.g_row + i);
        if (V == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(st);
            s[0] = q.x; s[V > 1 ? 1 : 0] = q.y; s[V > 2 ? 2 : 0] = q.z; s[V > 3 ? 3 : 0] = q.w;
        } else {
            s[0] = *st;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a, r;
            gate<LOGIT>(gr.get(v), a, r);
            const float xv = xr.get(v);
            s[v] = fmaf(a, s[v], TIED ? r * xv : xv);
        }
        RowVec<float, V>::store(st, s);
        RowVec<TX, V>::store(static_cast<TX *>(P.h) + n * P.h_row + i, s);
    }
}

cudaError_t allow_smem(const void *kernel, int bytes);   // la.cu

// How a call is cut: dense sequences each by themselves or, where they are short, all in
// one walk; packed ones in one walk.  How a walk is divided is said at the top.
// Measured when the borders were chosen (us; bf16 x, fp32 gates unless said):
//   64 blocks   fwd, B=2 T=8192 D=2048    team of 4 CTAs x 8 warps 59, of 4 x 4 76, two kernels 79
//   256 blocks  bwd, B=4 T=8192 D=4096    team of 1 CTA x 4 warps 314, a warp each 371, two kernels 413
//   32 blocks   bwd, packed, T=16384 D=2048   two kernels 117, team of 4 CTAs x 8 warps 179
//   16 blocks   fwd, T=32768 D=1024, bf16 logits   two kernels 74, team of 8 CTAs x 8 warps 154
// and around kScanFew in one run, B=1 T=16384 (two kernels / team of 4 CTAs):
//   blocks                    24         32         48         63         64
//   fwd                    62 / 80    78 / 80   114 / 97   148 / 98   147 / 99
//   bwd                    88 / 131  116 / 133  171 / 160  222 / 164  222 / 165
//   fwd, tied bf16 logits  54 / 111   65 / 111   92 / 150  121 / 154  122 / 154
//   bwd, tied bf16 logits  73 / 195   95 / 197  143 / 217  190 / 221  190 / 222
// Values favour the team from about 40 blocks on, tied logits (sigmoids beside the exchange)
// two kernels at 64 too, and so does T=2048 (by 2 to 7 us): one border for all is a compromise.
constexpr int kScanShort = 512;     // tokens: up to there one warp takes the walk
constexpr int kScanMany = 296;      // channel blocks (two for each SM): from there on too
constexpr int kScanFew = 64;        // channel blocks: below, two kernels
constexpr int64_t kScanMaxS = 512;  // segments: their maps are applied one after the other
struct ScanPlan {
    int n;                          // sequences per walk
    int64_t nblk, S, L;             // S > 1: two kernels
    int W, NS, K;                   // K > 0: teams
};
// `elem`: bytes that an element's tensors take in a slot of the output kernel.
inline ScanPlan scan_plan(const ScanParams &p, int elem, bool vec) {
    const int64_t ncb = (p.D + kScanCB - 1) / kScanCB;
    ScanPlan q{};
    const bool whole = p.cu_seqlens || (p.B > 1 && p.T < 4 * kScanR && p.B * p.T <= (1 << 30));
    q.n = whole ? (int)p.B : 1;
    q.nblk = whole ? ncb : ncb * p.B;
    const int64_t len = std::max<int64_t>(1, whole && !p.cu_seqlens ? p.B * p.T : p.T);
    const int slot = kScanR * kScanCB * elem;
    const int64_t warps = kScanW * std::min<int64_t>(4, (227 << 10) / (kScanW * kScanStages * slot + 2048)) * sm_count();
    q.W = kScanW;
    q.NS = kScanStages;
    int64_t S = 1;
    if (len > kScanShort && q.nblk < kScanMany) {
        if (vec && q.nblk >= kScanFew) {
            // as many CTAs as two an SM make.  (A tied backward pass of fp32 x takes 123 to 139 KB
            // a CTA, so there one fits and some of the CTAs wait for a second turn: B=2 T=8192
            // D=2048 188 us where the bytes take 123.)
            q.K = q.nblk * 4 <= 2 * sm_count() ? 4 : q.nblk * 2 <= 2 * sm_count() ? 2 : 1;
            q.W = elem <= 6 ? 2 * kScanW : kScanW;
            q.NS = 2;
        } else {
            S = std::max<int64_t>(1, std::min<int64_t>({warps / q.nblk, len / (4 * kScanR), kScanMaxS}));
        }
    } else if (vec) {
        // few warps: as many slots as the SM's share has room for
        const int64_t per_sm = (q.nblk + sm_count() - 1) / sm_count();
        if (per_sm < kScanW) {
            q.W = 1;
            q.NS = (int)std::min<int64_t>(kScanMaxStages, (200 << 10) / (per_sm * slot));
        }
    }
    q.L = ((len + S - 1) / S + kScanR - 1) / kScanR * kScanR;
    q.S = (len + q.L - 1) / q.L;
    return q;
}
inline int scan_elem(int ex, int eg, bool bwd, bool tied) { return bwd ? 2 * ex + eg + (tied ? ex : 0) : ex + eg; }
inline size_t scan_scratch(const ScanParams &p, int elem) {
    const ScanPlan q = scan_plan(p, elem, false);   // (tiles or not: not less than with them)
    return q.S > 1 ? ScanScratch::bytes(q.S, q.nblk) : 0;
}

// Boxes of kScanR tokens x 64 channels of a token tensor (la.cu).
bool make_map_2d(CUtensorMap *map, const void *base, int esize, int64_t D, int64_t tokens, int64_t row, int box_d, int box_t);
inline bool scan_tile(CUtensorMap *map, const void *base, int esize, int64_t D, int64_t tokens, int64_t row) {
    return !base || make_map_2d(map, base, esize, D, tokens, row, kScanCB, kScanR);
}

template <typename TX, typename TG, bool BWD, bool VEC, bool LOGIT, bool TIED>
cudaError_t launch_walk(ScanParams p, cudaStream_t st) {
    using Out = ScanShape<TX, TG, BWD, TIED, false>;
    ScanPlan plan = scan_plan(p, Out::kSlot / Out::kBox, VEC);
    p.n = plan.n;
    p.ncb = (int)((p.D + kScanCB - 1) / kScanCB);
    p.nblk = (int)plan.nblk;
    p.S = (int)plan.S;
    p.L = (int)plan.L;
    ScanTiles m{};
    if constexpr (VEC) {
        const int64_t tokens = (p.cu_seqlens ? 1 : p.B) * p.T;
        const int ex = sizeof(TX), eg = sizeof(TG);
        if (tokens > 0 &&
            !(scan_tile(&m.g, p.g, eg, p.D, tokens, p.g_row) && scan_tile(&m.x, p.x, ex, p.D, tokens, p.x_row) &&
              scan_tile(&m.dh, p.dh, ex, p.D, tokens, p.dh_row) && scan_tile(&m.hs, p.hs, ex, p.D, tokens, p.hs_row) &&
              scan_tile(&m.h, p.h, ex, p.D, tokens, p.h_row) && scan_tile(&m.dx, p.dx, ex, p.D, tokens, p.dx_row) &&
              scan_tile(&m.dg, p.dg, eg, p.D, tokens, p.dg_row)))
            return cudaErrorInvalidValue;
    }
    p.W = plan.W;
    p.NS = plan.NS;
    p.K = plan.K;
    auto launch = [&](auto kernel, int smem, int64_t ctas, int cluster, bool after) {
        cudaError_t e = allow_smem((const void *)kernel, smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(p.W * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute at[2]{};
        int n = 0;
        if (after) {
            at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[n++].val.programmaticStreamSerializationAllowed = 1;
        }
        if (cluster > 1) {
            at[n].id = cudaLaunchAttributeClusterDimension;
            at[n].val.clusterDim.x = (unsigned)cluster;
            at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
            ++n;
        }
        cfg.attrs = at;
        cfg.numAttrs = n;
        return cudaLaunchKernelEx(&cfg, kernel, (const ScanParams)p, (const ScanTiles)m);
    };
    if constexpr (VEC) {
        if (plan.K > 0)
            return launch(scan_kernel<TX, TG, BWD, true, LOGIT, TIED, kScanTeam>,
                          p.W * p.NS * (Out::kSlot + 8) + 2 * (p.W + p.K) * 512 + 16, plan.nblk * p.K, p.K, false);
    }
    if (plan.S > 1) {
        const cudaError_t e = launch(scan_kernel<TX, TG, BWD, VEC, LOGIT, TIED, kScanMap>,
                                     p.W * p.NS * (ScanShape<TX, TG, BWD, TIED, true>::kSlot + 8),
                                     (plan.nblk * (plan.S - 1) + p.W - 1) / p.W, 1, false);
        if (e != cudaSuccess) return e;
    }
    return launch(scan_kernel<TX, TG, BWD, VEC, LOGIT, TIED, kScanOut>, p.W * p.NS * (Out::kSlot + 8),
                  (plan.nblk * plan.S + p.W - 1) / p.W, 1, plan.S > 1);
}

template <typename TX, typename TG, int V, bool LOGIT, bool TIED>
cudaError_t launch_step(ScanParams p, cudaStream_t st) {
    // dense rows are one row: no thread is lost at the end of each
    if (p.x_row == p.D && p.g_row == p.D && p.h_row == p.D) {
        p.D *= p.B;
        p.B = 1;
    }
    const dim3 grid((unsigned)((p.D + 256 * V - 1) / (256 * V)), (unsigned)std::min<int64_t>(p.B, 65535));
    scan_step_kernel<TX, TG, V, LOGIT, TIED><<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

enum class ScanOp { kFwd, kBwd, kStep };

// TMA takes rows whose address and distance are multiples of 16 bytes (the distance
// below 2^40), on a token axis of less than 2^31 tokens.  The rows' lengths have to be
// multiples of 16 bytes too: a store's end is cut at those only.
inline bool scan_tma_ok(const void *p, int64_t row, int esize) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && row * esize % 16 == 0 && row * esize < (1ll << 40));
}

// The step: accesses of four channels where the channel count, every row stride and
// every pointer allow them, else of single elements.
template <ScanOp OP, typename TX, typename TG>
cudaError_t launch_scan(const ScanParams &p, cudaStream_t st) {
    const int ex = sizeof(TX), eg = sizeof(TG), form = 2 * p.logit + p.tied;
    if constexpr (OP == ScanOp::kStep) {
        const bool v4 = p.D % 4 == 0 && vec_ok(p.x, p.x_row, ex, 4) && vec_ok(p.g, p.g_row, eg, 4) &&
                        vec_ok(p.h, p.h_row, ex, 4) && vec_ok(p.h_last, p.D, 4, 4);
        switch (form + (v4 ? 4 : 0)) {
            case 0: return launch_step<TX, TG, 1, false, false>(p, st);
            case 1: return launch_step<TX, TG, 1, false, true>(p, st);
            case 2: return launch_step<TX, TG, 1, true, false>(p, st);
            case 3: return launch_step<TX, TG, 1, true, true>(p, st);
            case 4: return launch_step<TX, TG, 4, false, false>(p, st);
            case 5: return launch_step<TX, TG, 4, false, true>(p, st);
            case 6: return launch_step<TX, TG, 4, true, false>(p, st);
            default: return launch_step<TX, TG, 4, true, true>(p, st);
        }
    } else {
        constexpr bool B = OP == ScanOp::kBwd;
        const bool vec = (p.cu_seqlens ? 1 : p.B) * p.T < (1ll << 31) - 1 && p.D * ex % 16 == 0 && p.D * eg % 16 == 0 &&
                         scan_tma_ok(p.x, p.x_row, ex) &&
                         scan_tma_ok(p.g, p.g_row, eg) && scan_tma_ok(p.h, p.h_row, ex) &&
                         scan_tma_ok(p.hs, p.hs_row, ex) && scan_tma_ok(p.dh, p.dh_row, ex) &&
                         scan_tma_ok(p.dx, p.dx_row, ex) && scan_tma_ok(p.dg, p.dg_row, eg);
        switch (form + (vec ? 4 : 0)) {
            case 0: return launch_walk<TX, TG, B, false, false, false>(p, st);
            case 1: return launch_walk<TX, TG, B, false, false, true>(p, st);
            case 2: return launch_walk<TX, TG, B, false, true, false>(p, st);
            case 3: return launch_walk<TX, TG, B, false, true, true>(p, st);
            case 4: return launch_walk<TX, TG, B, true, false, false>(p, st);
            case 5: return launch_walk<TX, TG, B, true, false, true>(p, st);
            case 6: return launch_walk<TX, TG, B, true, true, false>(p, st);
            default: return launch_walk<TX, TG, B, true, true, true>(p, st);
        }
    }
}
}  // namespace la

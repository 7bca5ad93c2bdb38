// norm.cuh — layer norm and RMS norm of rows, forward and backward.
//     layer  xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//     rms    xh = x rstd,           rstd = 1 / sqrt(mean(x^2) + eps)
//     y = xh w + b
// Backward, with d = dy w:
//     dx = rstd (d - mean(d) - xh mean(d xh))      (rms: without mean(d))
//     dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bytes: the forward pass reads and writes every row once, the backward pass
// reads x and dy and writes dx once.  A row is held in registers by a team of
// threads: 16 elements a thread and up to 32 threads of one warp for rows of up to
// 512 (several teams a warp), else the whole CTA; forward, rows of more than 512 take
// 32 elements a thread, one warp up to 1024 and the CTA above.  CTAs walk over rows;
// each thread copies its own elements of the next rows into its own slots of shared
// memory (cp.async, no barrier), up to kNormStages rows ahead, so that enough bytes are
// in flight whatever the reduction of the current row waits for.  The variance is taken
// from the centred values, not from a difference of moments.  Measured, bf16 layer norm:
// forward 16384 x 4096 53 us (5.0 TB/s), backward 94 us (4.3 TB/s), backward of RMS
// rows 262144 x 128 41 us (4.9 TB/s).  With 8 to 16 warps an SM (the registers allow no
// more) what is left is the latency of a row's dependent steps: sums over lanes, barrier,
// sums over warps; schedulers issue in 54 to 65% of the cycles, DRAM is at 49 to 58%.
//
// The weight's gradients are summed without atomics, in an order that does not
// depend on timing: a thread adds its columns over the rows it meets (fp32), the
// teams of a CTA are added, each CTA writes one row of partial sums, and a second
// kernel adds those rows.
#pragma once

#include <algorithm>

#include "rowvec.cuh"

namespace la {

struct NormParams {
    int64_t R;
    int D;
    const void *x, *dy;
    int64_t x_row, dy_row;
    const float *w, *b;
    float eps;
    void *y;                     // forward: y; backward: dx
    int64_t y_row;
    float *mean, *rstd;          // forward: written (may be null); backward: read
    float *part;                 // backward: [CTAs][2][D] partial dw and db, or null
    int team;                    // threads per row
};

constexpr int kNormE = 16;                 // elements a thread holds
constexpr int kNormNarrow = 256;           // CTA of the narrow form
constexpr int kNormMaxD = 1024 * kNormE;

// The elements of one row after another on their way to the thread that uses them: NV
// accesses of V elements a row.  RING: slots in shared memory, NS rows deep; else
// (16-bit elements one by one, and rows too long for the shared memory) registers,
// one row ahead.
template <typename T, int V, int NV, int NS, bool RING>
struct NormFeed {
    static constexpr int kA = V * (int)sizeof(T);              // bytes of an access: 16 or 4
    static constexpr int kBytes = RING ? NS * NV * kA : 0;     // of a thread
    RowVec<T, V> reg[RING ? 1 : NV];
    uint32_t at;
    // `base`: shared memory of the CTA for this feed.
    __device__ __forceinline__ void init(uint32_t base) { at = base + threadIdx.x * kA; }
    __device__ __forceinline__ uint32_t addr(int slot, int i) const { return at + (uint32_t)(slot * NV + i) * blockDim.x * kA; }
    __device__ __forceinline__ void issue(int slot, int i, const T *p, bool ok) {
        if constexpr (RING) {
            if (ok) {
                if constexpr (kA == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(addr(slot, i)), "l"(p) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(addr(slot, i)), "l"(p) : "memory");
            }
        } else {
            if (ok) reg[i].load(p);
            else reg[i].zero();
        }
    }
    __device__ __forceinline__ RowVec<T, V> take(int slot, int i, bool ok) const {
        if constexpr (RING) {
            RowVec<T, V> v;
            if constexpr (kA == 16) {
                uint32_t a, b, c, d;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr(slot, i)) : "memory");
                if constexpr (sizeof(T) == 4)
                    v.r = make_float4(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c), __uint_as_float(d));
                else
                    v.r = make_uint4(a, b, c, d);
            } else {
                uint32_t a;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(a) : "r"(addr(slot, i)) : "memory");
                if constexpr (sizeof(T) == 4) v.r = __uint_as_float(a);
                else v.r = a;
            }
            if (!ok) v.zero();
            return v;
        } else {
            return reg[i];
        }
    }
};
template <bool RING>
__device__ __forceinline__ void norm_commit() {
    if (RING) asm volatile("cp.async.commit_group;" ::: "memory");
}
template <bool RING, int N>
__device__ __forceinline__ void norm_arrived() {
    if (RING) asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr int kNormStages = 4;
constexpr int kNormLong = 1024;            // threads of a CTA for the longest rows
// Rows ahead and whether they are in shared memory, for TENSORS tensors read by up to
// MAXT threads.  With kNormLong threads there are 64 registers a thread: the COLS fp32
// vectors that a row is multiplied with (and added) stay in shared memory, else in
// registers.
template <typename T, int V, int E, int MAXT, int TENSORS, int COLS>
struct NormRing {
    static constexpr bool kCols = MAXT == kNormLong;
    static constexpr int kRow = E * (int)sizeof(T) * TENSORS;       // of a thread
    static constexpr int kColBytes = kCols ? E * 4 * COLS : 0;      // of a thread
    static constexpr int kFit = ((224 << 10) / MAXT - kColBytes) / kRow;
    static constexpr bool kOn = V * sizeof(T) >= 4 && kFit >= 2;
    static constexpr int kNS = kOn ? (kFit < kNormStages ? kFit : kNormStages) : 1;
    static constexpr int kThread = kColBytes + (kOn ? kNS * kRow : 0);   // shared memory of a thread
};

// Pairs of scalar operations: the packed ones were slower here (backward of 16384 rows of
// 4096: 108 against 96 us), for the moves that bring the pairs together.
__device__ __forceinline__ float2 norm_mul(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 norm_add(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 norm_fma(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }
__device__ __forceinline__ float2 norm_both(float a) { return make_float2(a, a); }

// Sums of N values over the team, the same in each of its threads.  Narrow: lanes of one
// warp, `team` a power of two.  Wide: the CTA; `red` is [2][N][32], zeroed, and `par`
// flips from call to call, so one barrier a call is enough.
template <bool WIDE, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int team, float (*red)[N][32], int &par) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1)
        if (WIDE || m < team) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
        }
    if (WIDE) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) red[par][k][threadIdx.x >> 5] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = red[par][k][threadIdx.x & 31];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], m);
        }
        par ^= 1;
    }
}

template <typename T, int V, int E, bool LAYER, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_fwd_kernel(const NormParams P) {
    constexpr int NV = E / V, E2 = E / 2;
    using Ring = NormRing<T, V, E, MAXT, 1, 2>;
    constexpr bool RING = Ring::kOn, COLS = Ring::kCols;
    constexpr int NS = Ring::kNS;
    __shared__ __align__(16) float red[2][1][32];
    extern __shared__ __align__(16) uint8_t norm_sm[];
    int par = 0;
    const int team = P.team, tm = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (team - 1);
    const int teams = (int)blockDim.x / team, my = WIDE ? 0 : (int)threadIdx.x / team;
    const float inv = 1.f / (float)P.D;
    const bool full = team * E == P.D;       // no thread holds places past the row's end
    auto col = [&](int e) { return ((e / V) * team + tm) * V + e % V; };
    // weight and bias of the thread's columns
    float2 w[COLS ? 1 : E2], bb[COLS ? 1 : E2];
    float2 *cols = reinterpret_cast<float2 *>(norm_sm) + threadIdx.x;   // [w, b][E2][threads]
    const int ct = (int)blockDim.x;
#pragma unroll
    for (int k = 0; k < E2; ++k) {
        const int c0 = col(2 * k), c1 = col(2 * k + 1);
        const float2 wv = make_float2(P.w && c0 < P.D ? P.w[c0] : 1.f, P.w && c1 < P.D ? P.w[c1] : 1.f);
        const float2 bv = make_float2(P.b && c0 < P.D ? P.b[c0] : 0.f, P.b && c1 < P.D ? P.b[c1] : 0.f);
        if (COLS) {
            cols[k * ct] = wv;
            cols[(E2 + k) * ct] = bv;
        } else {
            w[COLS ? 0 : k] = wv;
            bb[COLS ? 0 : k] = bv;
        }
    }
    if (WIDE) {
        if (threadIdx.x < 64) red[threadIdx.x >> 5][0][threadIdx.x & 31] = 0.f;
        __syncthreads();
    }
    NormFeed<T, V, NV, NS, RING> fx;
    fx.init(smem_u32(norm_sm) + ct * Ring::kColBytes);
    auto fetch = [&](int64_t row, int slot) {
        const T *x = static_cast<const T *>(P.x) + row * P.x_row;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * team + tm) * V;
            fx.issue(slot, i, x + c, row < P.R && (full || c < P.D));
        }
        norm_commit<RING>();
    };
    int64_t base = (int64_t)blockIdx.x * teams;
    const int64_t stride = (int64_t)gridDim.x * teams;
    int64_t ahead = base + my;
    for (int k = 0; k < NS; ++k, ahead += stride) fetch(ahead, k);
    for (int slot = 0; base < P.R; base += stride, slot = slot + 1 == NS ? 0 : slot + 1, ahead += stride) {
        const int64_t row = base + my;
        float2 x[E2];
        norm_arrived<RING, NS - 1>();
        {
            RowVec<T, V> v[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = fx.take(slot, i, row < P.R && (full || (i * team + tm) * V < P.D));
#pragma unroll
            for (int k = 0; k < E2; ++k)
                x[k] = make_float2(v[2 * k / V].get(2 * k % V), v[(2 * k + 1) / V].get((2 * k + 1) % V));
        }
        fetch(ahead, slot);
        float mean = 0.f, s[1];
        float2 a = make_float2(0.f, 0.f);
        if (LAYER) {
#pragma unroll
            for (int k = 0; k < E2; ++k) a = norm_add(a, x[k]);
            s[0] = a.x + a.y;
            team_sum<WIDE>(s, team, red, par);
            mean = s[0] * inv;
#pragma unroll
            for (int k = 0; k < E2; ++k) {
                x[k] = norm_add(x[k], norm_both(-mean));
                if (!full) {
                    if (col(2 * k) >= P.D) x[k].x = 0.f;
                    if (col(2 * k + 1) >= P.D) x[k].y = 0.f;
                }
            }
            a = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < E2; ++k) a = norm_fma(x[k], x[k], a);
        s[0] = a.x + a.y;
        team_sum<WIDE>(s, team, red, par);
        const float rstd = rsqrtf(s[0] * inv + P.eps);
        if (row < P.R) {
            T *y = static_cast<T *>(P.y) + row * P.y_row;
            float o[E];
#pragma unroll
            for (int k = 0; k < E2; ++k) {
                const float2 we = COLS ? cols[k * ct] : w[COLS ? 0 : k], be = COLS ? cols[(E2 + k) * ct] : bb[COLS ? 0 : k];
                const float2 v = norm_fma(norm_mul(x[k], norm_both(rstd)), we, be);
                o[2 * k] = v.x;
                o[2 * k + 1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (full || c < P.D) RowVec<T, V>::store(y + c, o + i * V);
            }
            if (tm == 0) {
                if (LAYER && P.mean) P.mean[row] = mean;
                if (P.rstd) P.rstd[row] = rstd;
            }
        }
    }
}

template <typename T, int V, int E, bool LAYER, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_bwd_kernel(const NormParams P) {
    constexpr int NV = E / V, E2 = E / 2;
    using Ring = NormRing<T, V, E, MAXT, 2, 1>;
    constexpr bool RING = Ring::kOn, COLS = Ring::kCols;
    constexpr int NS = Ring::kNS;
    __shared__ __align__(16) float red[2][2][32];
    extern __shared__ __align__(16) uint8_t norm_sm[];
    float *acc_sm = reinterpret_cast<float *>(norm_sm);    // after the rows
    int par = 0;
    const int team = P.team, tm = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (team - 1);
    const int teams = (int)blockDim.x / team, my = WIDE ? 0 : (int)threadIdx.x / team;
    const float inv = 1.f / (float)P.D;
    const bool full = team * E == P.D;
    auto col = [&](int e) { return ((e / V) * team + tm) * V + e % V; };
    float2 w[COLS ? 1 : E2], dw[E2], db[E2];
    float2 *cols = reinterpret_cast<float2 *>(norm_sm) + threadIdx.x;   // [E2][threads]
    const int ct = (int)blockDim.x;
#pragma unroll
    for (int k = 0; k < E2; ++k) {
        const int c0 = col(2 * k), c1 = col(2 * k + 1);
        const float2 wv = make_float2(P.w && c0 < P.D ? P.w[c0] : 1.f, P.w && c1 < P.D ? P.w[c1] : 1.f);
        if (COLS) cols[k * ct] = wv;
        else w[COLS ? 0 : k] = wv;
        dw[k] = db[k] = make_float2(0.f, 0.f);
    }
    if (WIDE) {
        if (threadIdx.x < 64) red[threadIdx.x >> 5][0][threadIdx.x & 31] = red[threadIdx.x >> 5][1][threadIdx.x & 31] = 0.f;
        __syncthreads();
    }
    NormFeed<T, V, NV, NS, RING> fx, fy;
    fx.init(smem_u32(norm_sm) + ct * Ring::kColBytes);
    fy.init(smem_u32(norm_sm) + ct * (Ring::kColBytes + decltype(fx)::kBytes));
    auto fetch = [&](int64_t row, int slot) {
        const T *x = static_cast<const T *>(P.x) + row * P.x_row;
        const T *dy = static_cast<const T *>(P.dy) + row * P.dy_row;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * team + tm) * V;
            const bool ok = row < P.R && (full || c < P.D);
            fx.issue(slot, i, x + c, ok);
            fy.issue(slot, i, dy + c, ok);
        }
        norm_commit<RING>();
    };
    int64_t base = (int64_t)blockIdx.x * teams;
    const int64_t stride = (int64_t)gridDim.x * teams;
    int64_t ahead = base + my;
    for (int k = 0; k < NS; ++k, ahead += stride) fetch(ahead, k);
    // the row's statistics, one row ahead
    float nm = 0.f, nr = 0.f;
    auto stats = [&](int64_t row) {
        nm = LAYER && row < P.R ? __ldg(P.mean + row) : 0.f;
        nr = row < P.R ? __ldg(P.rstd + row) : 0.f;
    };
    stats(base + my);
    for (int slot = 0; base < P.R; base += stride, slot = slot + 1 == NS ? 0 : slot + 1, ahead += stride) {
        const int64_t row = base + my;
        const float mean = nm, rstd = nr;
        stats(row + stride);
        RowVec<T, V> cx[NV], cy[NV];
        norm_arrived<RING, NS - 1>();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool ok = row < P.R && (full || (i * team + tm) * V < P.D);
            cx[i] = fx.take(slot, i, ok);
            cy[i] = fy.take(slot, i, ok);
        }
        // places past the end have dy = 0, so they add nothing
        auto pair = [](const RowVec<T, V> *v, int k) {
            return make_float2(v[2 * k / V].get(2 * k % V), v[(2 * k + 1) / V].get((2 * k + 1) % V));
        };
        auto normal = [&](int k) {                 // xh
            const float2 x = pair(cx, k);
            return norm_mul(LAYER ? norm_add(x, norm_both(-mean)) : x, norm_both(rstd));
        };
        float2 a1 = make_float2(0.f, 0.f), a2 = a1;
#pragma unroll
        for (int k = 0; k < E2; ++k) {
            const float2 xh = normal(k), dy = pair(cy, k), d = norm_mul(dy, COLS ? cols[k * ct] : w[COLS ? 0 : k]);
            if (LAYER) a1 = norm_add(a1, d);
            a2 = norm_fma(d, xh, a2);
            dw[k] = norm_fma(dy, xh, dw[k]);
            db[k] = norm_add(db[k], dy);
        }
        fetch(ahead, slot);
        float s1, s2;
        if (LAYER) {
            float s[2] = {a1.x + a1.y, a2.x + a2.y};
            team_sum<WIDE>(s, team, red, par);
            s1 = s[0] * inv;
            s2 = s[1] * inv;
        } else {
            float s[1] = {a2.x + a2.y};
            team_sum<WIDE>(s, team, reinterpret_cast<float (*)[1][32]>(red), par);
            s1 = 0.f;
            s2 = s[0] * inv;
        }
        if (row < P.R) {
            T *dx = static_cast<T *>(P.y) + row * P.y_row;
            float o[E];
#pragma unroll
            for (int k = 0; k < E2; ++k) {
                const float2 xh = normal(k), d = norm_mul(pair(cy, k), COLS ? cols[k * ct] : w[COLS ? 0 : k]);
                float2 v = norm_fma(xh, norm_both(-s2), LAYER ? norm_add(d, norm_both(-s1)) : d);
                v = norm_mul(v, norm_both(rstd));
                o[2 * k] = v.x;
                o[2 * k + 1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (full || c < P.D) RowVec<T, V>::store(dx + c, o + i * V);
            }
        }
    }
    if (!P.part) return;
    float *part = P.part + (int64_t)blockIdx.x * 2 * P.D;
    if (WIDE) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = col(e);
            if (c < P.D) {
                part[c] = e & 1 ? dw[e / 2].y : dw[e / 2].x;
                part[P.D + c] = e & 1 ? db[e / 2].y : db[e / 2].x;
            }
        }
    } else {
        // teams of the warp, then the CTA's warps
        norm_arrived<RING, 0>();
        __syncthreads();                   // the slots become the sums' place
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ncol = team * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float a = e & 1 ? dw[e / 2].y : dw[e / 2].x, b = e & 1 ? db[e / 2].y : db[e / 2].x;
            for (int m = team; m < 32; m <<= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, m);
                b += __shfl_xor_sync(0xffffffffu, b, m);
            }
            if (lane < team) {
                acc_sm[(warp * 2) * ncol + col(e)] = a;
                acc_sm[(warp * 2 + 1) * ncol + col(e)] = b;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * ncol; i += blockDim.x) {
            const int which = i / ncol, c = i % ncol;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kNormNarrow / 32; ++k) s += acc_sm[(k * 2 + which) * ncol + c];
            if (c < P.D) part[(int64_t)which * P.D + c] = s;
        }
    }
}

// Column sums of the CTAs' partial rows: 32 columns x 32 threads a CTA, blockIdx.y
// 0 for dw and 1 for db (`out1` null: one of them only).
__global__ void __launch_bounds__(1024) norm_cols_kernel(const float *part, int64_t rows, int D, float *out0, float *out1) {
    __shared__ float sm[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float *out = blockIdx.y == 0 ? out0 : out1;
    const float *p = part + (int64_t)(blockIdx.y) * D;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (c < D && out)
#pragma unroll 8
        for (int64_t r = ry; r < rows; r += 32) s += p[r * 2 * D + c];
    sm[ry][cx] = s;
    __syncthreads();
    s = sm[cx][ry];                        // warp ry: the 32 sums of column ry
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    const int oc = blockIdx.x * 32 + ry;
    if (cx == 0 && oc < D && out) out[oc] = s;
}

cudaError_t allow_smem(const void *kernel, int bytes);   // la.cu

struct NormPlan {
    int team, threads, ctas, e;
    bool wide;
};
// Elements a thread, threads a row, CTA size and grid of a pass over R rows of D
// elements; `per_sm`: threads an SM holds of that kernel; `e`: elements of a thread.
inline NormPlan norm_plan(int64_t R, int D, int per_sm, int e) {
    NormPlan n{};
    n.e = e;
    const int need = (D + e - 1) / e;
    n.wide = need > 32;
    if (n.wide) {
        n.team = (need + 31) / 32 * 32;
        n.threads = n.team;
    } else {
        n.team = 1;
        while (n.team < need) n.team *= 2;
        n.threads = kNormNarrow;
    }
    const int64_t rows = n.threads / n.team;
    const int64_t resident = (int64_t)sm_count() * std::max(1, per_sm / n.threads);
    n.ctas = (int)std::min<int64_t>((R + rows - 1) / rows, resident);
    return n;
}
// The threads of an SM that the grids are made for.  They are what the 16-byte forms of bf16
// rows were fastest with, not what fits.  Fewer are resident, and the rest of the CTAs follow
// as those end: of the narrow forward pass (95 to 175 registers) one or two CTAs of the four;
// of the narrow backward pass one of the two where it takes more than 128 registers (all but
// bf16 in 16 bytes, 124).  Backward with kNormLong threads leaves 64 registers a thread and
// spills 116 to 680 bytes: 4096 x 16384 takes 146 us in bf16 and 249 in fp32, where the bytes
// take 61 and 123.
constexpr int kNormFwdPerSM = 1024, kNormFwdLongPerSM = 384, kNormBwdPerSM = 512;
// Forward: 32 elements a thread for rows of more than 512, so that few warps meet at the
// row's two barriers.
inline NormPlan norm_fwd_plan(int64_t R, int D) {
    return D > 512 ? norm_plan(R, D, kNormFwdLongPerSM, 2 * kNormE) : norm_plan(R, D, kNormFwdPerSM, kNormE);
}
inline NormPlan norm_bwd_plan(int64_t R, int D) { return norm_plan(R, D, kNormBwdPerSM, kNormE); }

inline size_t norm_bwd_workspace(int64_t R, int D) {
    return R > 0 ? (size_t)norm_bwd_plan(R, D).ctas * 2 * (size_t)D * sizeof(float) : 0;
}

template <bool BWD, typename T, int V, bool LAYER>
cudaError_t launch_norm_rows(NormParams p, const NormPlan &n, cudaStream_t st) {
    p.team = n.team;
    auto launch = [&](auto kernel, int thread_bytes) {
        size_t smem = (size_t)thread_bytes * n.threads;
        if (BWD && !n.wide && p.part) smem = std::max(smem, (size_t)(kNormNarrow / 32) * 2 * n.team * kNormE * sizeof(float));
        const cudaError_t e = allow_smem((const void *)kernel, (int)smem);
        if (e == cudaSuccess) kernel<<<n.ctas, n.threads, smem, st>>>(p);
        return e;
    };
    constexpr int E = kNormE;
    cudaError_t e;
    if constexpr (BWD) {
        if (!n.wide) e = launch(norm_bwd_kernel<T, V, E, LAYER, false, kNormNarrow>, NormRing<T, V, E, kNormNarrow, 2, 1>::kThread);
        else if (n.threads <= 512) e = launch(norm_bwd_kernel<T, V, E, LAYER, true, 512>, NormRing<T, V, E, 512, 2, 1>::kThread);
        else e = launch(norm_bwd_kernel<T, V, E, LAYER, true, kNormLong>, NormRing<T, V, E, kNormLong, 2, 1>::kThread);
    } else {
        if (n.e == E) e = launch(norm_fwd_kernel<T, V, E, LAYER, false, kNormNarrow>, NormRing<T, V, E, kNormNarrow, 1, 2>::kThread);
        else if (!n.wide) e = launch(norm_fwd_kernel<T, V, 2 * E, LAYER, false, kNormNarrow>, NormRing<T, V, 2 * E, kNormNarrow, 1, 2>::kThread);
        else e = launch(norm_fwd_kernel<T, V, 2 * E, LAYER, true, 512>, NormRing<T, V, 2 * E, 512, 1, 2>::kThread);
    }
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// 16-byte accesses where the row length, every row stride and every pointer allow
// them, else (bf16) 4-byte ones, else single elements.  Layer norm of 16384 bf16 rows,
// forward and backward: of 4096 elements 53 and 94 us, of 4098 183 and 309, of 4097 590 and
// 375 (single elements of bf16 come by plain loads, and the wide forms spill).
template <bool BWD, typename T>
cudaError_t launch_norm_typed(const NormParams &p, bool layer, const NormPlan &n, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T), V2 = 4 / sizeof(T);
    const int es = sizeof(T);
    auto ok = [&](int v) {
        return p.D % v == 0 && vec_ok(p.x, p.x_row, es, v) && vec_ok(p.dy, p.dy_row, es, v) && vec_ok(p.y, p.y_row, es, v);
    };
    if (ok(V)) return layer ? launch_norm_rows<BWD, T, V, true>(p, n, st) : launch_norm_rows<BWD, T, V, false>(p, n, st);
    if (V2 == 1 || ok(V2)) return layer ? launch_norm_rows<BWD, T, V2, true>(p, n, st) : launch_norm_rows<BWD, T, V2, false>(p, n, st);
    return layer ? launch_norm_rows<BWD, T, 1, true>(p, n, st) : launch_norm_rows<BWD, T, 1, false>(p, n, st);
}

inline cudaError_t launch_norm_fwd(const NormParams &p, bool bf16, bool layer, cudaStream_t st) {
    const NormPlan n = norm_fwd_plan(p.R, p.D);
    return bf16 ? launch_norm_typed<false, __nv_bfloat16>(p, layer, n, st) : launch_norm_typed<false, float>(p, layer, n, st);
}

// dw and db may each be null; `part` is null when both are.
inline cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, bool layer, float *dw, float *db, cudaStream_t st) {
    const NormPlan n = norm_bwd_plan(p.R, p.D);
    cudaError_t e = bf16 ? launch_norm_typed<true, __nv_bfloat16>(p, layer, n, st) : launch_norm_typed<true, float>(p, layer, n, st);
    if (e != cudaSuccess || !p.part) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.D + 31) / 32), db ? 2u : 1u);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_cols_kernel, (const float *)p.part, (int64_t)n.ctas, p.D, dw, db);
}

}  // namespace la

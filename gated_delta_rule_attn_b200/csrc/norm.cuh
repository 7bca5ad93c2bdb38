// norm.cuh — layer norm and RMS norm of rows, forward and backward.
//     layer  xh = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//     rms    xh = x rstd,           rstd = 1 / sqrt(mean(x^2) + eps)
//     y = xh w + b
// Backward, with d = dy w:
//     dx = rstd (d - mean(d) - xh mean(d xh))      (rms: without mean(d))
//     dw = sum over rows of dy xh,  db = sum over rows of dy
//
// HBM-bound: the forward pass reads and writes every row once, the backward pass
// reads x and dy and writes dx once.  A row is held in registers by a team of
// threads, 16 elements a thread: up to 32 threads of one warp for rows of up to
// 512 (several teams a warp), else the whole CTA.  CTAs walk over rows with the
// next row's loads in flight while the current one is reduced.  The variance is
// taken from the centred values, not from a difference of moments.
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

// Sums of (a, b) over the team.  Narrow: lanes of one warp, `team` a power of two.
// Wide: the CTA; `red` is [2][32] and `par` flips from call to call, so one
// barrier a call is enough.
template <bool WIDE>
__device__ __forceinline__ void team_sum(float &a, float &b, int team, float2 (*red)[32], int &par) {
    if (!WIDE) {
        for (int m = team >> 1; m >= 1; m >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, m);
            b += __shfl_xor_sync(0xffffffffu, b, m);
        }
    } else {
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, m);
            b += __shfl_xor_sync(0xffffffffu, b, m);
        }
        if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const int nw = team >> 5, lane = threadIdx.x & 31;
        const float2 v = lane < nw ? red[par][lane] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, m);
            b += __shfl_xor_sync(0xffffffffu, b, m);
        }
        par ^= 1;
    }
}

// MAXT: largest CTA; with 1024 threads there are 64 registers a thread, and the
// weight and bias are read for every row (from L1) instead of being kept.
template <typename T, int V, bool LAYER, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const NormParams P) {
    constexpr int NV = kNormE / V;
    constexpr bool HOLD = MAXT < 1024;
    __shared__ float2 red[2][32];
    int par = 0;
    const int team = P.team, tm = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (team - 1);
    const int teams = (int)blockDim.x / team, my = WIDE ? 0 : (int)threadIdx.x / team;
    const float inv = 1.f / (float)P.D;
    float w[HOLD ? kNormE : 1], bb[HOLD ? kNormE : 1];
    if (HOLD) {
#pragma unroll
        for (int e = 0; e < kNormE; ++e) {
            const int c = ((e / V) * team + tm) * V + e % V;
            w[HOLD ? e : 0] = P.w && c < P.D ? P.w[c] : 1.f;
            bb[HOLD ? e : 0] = P.b && c < P.D ? P.b[c] : 0.f;
        }
    }
    RowVec<T, V> nx[NV];
    auto fetch = [&](int64_t row) {
        if (row < P.R) {
            const T *x = static_cast<const T *>(P.x) + row * P.x_row;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (c < P.D) nx[i].load(x + c);
                else nx[i].zero();
            }
        }
    };
    int64_t base = (int64_t)blockIdx.x * teams;
    const int64_t stride = (int64_t)gridDim.x * teams;
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i].zero();
    fetch(base + my);
    for (; base < P.R; base += stride) {
        const int64_t row = base + my;
        float x[kNormE];
#pragma unroll
        for (int e = 0; e < kNormE; ++e) x[e] = nx[e / V].get(e % V);
        fetch(row + stride);
        float mean = 0.f, s = 0.f, unused = 0.f;
        if (LAYER) {
#pragma unroll
            for (int e = 0; e < kNormE; ++e) s += x[e];
            team_sum<WIDE>(s, unused, team, red, par);
            mean = s * inv;
            s = 0.f;
        }
#pragma unroll
        for (int e = 0; e < kNormE; ++e) {
            if (LAYER) x[e] -= mean;
            if (((e / V) * team + tm) * V < P.D) s = fmaf(x[e], x[e], s);
        }
        team_sum<WIDE>(s, unused, team, red, par);
        const float rstd = rsqrtf(s * inv + P.eps);
        if (row < P.R) {
            T *y = static_cast<T *>(P.y) + row * P.y_row;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (c < P.D) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float we = HOLD ? w[HOLD ? i * V + v : 0] : P.w ? __ldg(P.w + c + v) : 1.f;
                        const float be = HOLD ? bb[HOLD ? i * V + v : 0] : P.b ? __ldg(P.b + c + v) : 0.f;
                        o[v] = fmaf(x[i * V + v] * rstd, we, be);
                    }
                    RowVec<T, V>::store(y + c, o);
                }
            }
            if (tm == 0) {
                if (LAYER && P.mean) P.mean[row] = mean;
                if (P.rstd) P.rstd[row] = rstd;
            }
        }
    }
}

template <typename T, int V, bool LAYER, bool WIDE, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormParams P) {
    constexpr int NV = kNormE / V;
    constexpr bool HOLD = MAXT < 1024;
    __shared__ float2 red[2][32];
    extern __shared__ float acc_sm[];
    int par = 0;
    const int team = P.team, tm = WIDE ? (int)threadIdx.x : (int)threadIdx.x & (team - 1);
    const int teams = (int)blockDim.x / team, my = WIDE ? 0 : (int)threadIdx.x / team;
    const float inv = 1.f / (float)P.D;
    float w[HOLD ? kNormE : 1];
    float dw[kNormE], db[kNormE];
#pragma unroll
    for (int e = 0; e < kNormE; ++e) {
        const int c = ((e / V) * team + tm) * V + e % V;
        if (HOLD) w[HOLD ? e : 0] = P.w && c < P.D ? P.w[c] : 1.f;
        dw[e] = db[e] = 0.f;
    }
    RowVec<T, V> nx[NV], ny[NV];
    float nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](int64_t row) {
        if (row < P.R) {
            const T *x = static_cast<const T *>(P.x) + row * P.x_row;
            const T *dy = static_cast<const T *>(P.dy) + row * P.dy_row;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (c < P.D) {
                    nx[i].load(x + c);
                    ny[i].load(dy + c);
                }
            }
            if (LAYER) nmean = __ldg(P.mean + row);
            nrstd = __ldg(P.rstd + row);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) { nx[i].zero(); ny[i].zero(); }
            nmean = nrstd = 0.f;
        }
    };
    int64_t base = (int64_t)blockIdx.x * teams;
    const int64_t stride = (int64_t)gridDim.x * teams;
#pragma unroll
    for (int i = 0; i < NV; ++i) { nx[i].zero(); ny[i].zero(); }
    fetch(base + my);
    for (; base < P.R; base += stride) {
        const int64_t row = base + my;
        const float mean = nmean, rstd = nrstd;
        RowVec<T, V> cx[NV], cy[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) { cx[i] = nx[i]; cy[i] = ny[i]; }
        fetch(row + stride);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * team + tm) * V;
            if (c < P.D) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int e = i * V + v;
                    const float xh = (LAYER ? cx[i].get(v) - mean : cx[i].get(v)) * rstd, dy = cy[i].get(v);
                    const float d = dy * (HOLD ? w[HOLD ? e : 0] : P.w ? __ldg(P.w + c + v) : 1.f);
                    s1 += d;
                    s2 = fmaf(d, xh, s2);
                    dw[e] = fmaf(dy, xh, dw[e]);
                    db[e] += dy;
                }
            }
        }
        team_sum<WIDE>(s1, s2, team, red, par);
        s1 = LAYER ? s1 * inv : 0.f;
        s2 *= inv;
        if (row < P.R) {
            T *dx = static_cast<T *>(P.y) + row * P.y_row;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * team + tm) * V;
                if (c < P.D) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int e = i * V + v;
                        const float xh = (LAYER ? cx[i].get(v) - mean : cx[i].get(v)) * rstd, dy = cy[i].get(v);
                        const float d = dy * (HOLD ? w[HOLD ? e : 0] : P.w ? __ldg(P.w + c + v) : 1.f);
                        o[v] = rstd * (d - s1 - xh * s2);
                    }
                    RowVec<T, V>::store(dx + c, o);
                }
            }
        }
    }
    if (!P.part) return;
    float *part = P.part + (int64_t)blockIdx.x * 2 * P.D;
    if (WIDE) {
#pragma unroll
        for (int e = 0; e < kNormE; ++e) {
            const int c = ((e / V) * team + tm) * V + e % V;
            if (c < P.D) {
                part[c] = dw[e];
                part[P.D + c] = db[e];
            }
        }
    } else {
        // teams of the warp, then the CTA's warps
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cols = team * kNormE;
#pragma unroll
        for (int e = 0; e < kNormE; ++e) {
            for (int m = team; m < 32; m <<= 1) {
                dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], m);
                db[e] += __shfl_xor_sync(0xffffffffu, db[e], m);
            }
            if (lane < team) {
                const int c = ((e / V) * team + tm) * V + e % V;
                acc_sm[(warp * 2) * cols + c] = dw[e];
                acc_sm[(warp * 2 + 1) * cols + c] = db[e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * cols; i += blockDim.x) {
            const int which = i / cols, c = i % cols;
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kNormNarrow / 32; ++k) s += acc_sm[(k * 2 + which) * cols + c];
            if (c < P.D) part[(int64_t)which * P.D + c] = s;
        }
    }
}

// Column sums of the CTAs' partial rows: 32 columns x 8 threads a CTA, blockIdx.y
// 0 for dw and 1 for db (`out1` null: one of them only).
__global__ void __launch_bounds__(256) norm_cols_kernel(const float *part, int64_t rows, int D, float *out0, float *out1) {
    __shared__ float sm[8][32];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float *out = blockIdx.y == 0 ? out0 : out1;
    const float *p = part + (int64_t)(blockIdx.y) * D;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (c < D && out)
#pragma unroll 8
        for (int64_t r = ry; r < rows; r += 8) s += p[r * 2 * D + c];
    sm[ry][cx] = s;
    __syncthreads();
    if (ry == 0 && c < D && out) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sm[k][cx];
        out[c] = s;
    }
}

struct NormPlan {
    int team, threads, ctas;
    bool wide;
};
// Threads a row, CTA size and grid of a pass over R rows of D elements;
// `per_sm`: threads an SM holds of that kernel.
inline NormPlan norm_plan(int64_t R, int D, int per_sm) {
    NormPlan n{};
    const int need = (D + kNormE - 1) / kNormE;
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
constexpr int kNormFwdPerSM = 1024, kNormBwdPerSM = 512;

inline size_t norm_bwd_workspace(int64_t R, int D) {
    return R > 0 ? (size_t)norm_plan(R, D, kNormBwdPerSM).ctas * 2 * (size_t)D * sizeof(float) : 0;
}

template <bool BWD, typename T, int V, bool LAYER>
cudaError_t launch_norm_rows(NormParams p, const NormPlan &n, cudaStream_t st) {
    p.team = n.team;
    const size_t smem = BWD && !n.wide && p.part ? (size_t)(kNormNarrow / 32) * 2 * n.team * kNormE * sizeof(float) : 0;
    if constexpr (BWD) {
        if (!n.wide) norm_bwd_kernel<T, V, LAYER, false, kNormNarrow><<<n.ctas, n.threads, smem, st>>>(p);
        else if (n.threads <= 512) norm_bwd_kernel<T, V, LAYER, true, 512><<<n.ctas, n.threads, 0, st>>>(p);
        else norm_bwd_kernel<T, V, LAYER, true, 1024><<<n.ctas, n.threads, 0, st>>>(p);
    } else {
        if (!n.wide) norm_fwd_kernel<T, V, LAYER, false, kNormNarrow><<<n.ctas, n.threads, 0, st>>>(p);
        else if (n.threads <= 512) norm_fwd_kernel<T, V, LAYER, true, 512><<<n.ctas, n.threads, 0, st>>>(p);
        else norm_fwd_kernel<T, V, LAYER, true, 1024><<<n.ctas, n.threads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

// 16-byte accesses where the row length, every row stride and every pointer allow
// them, else single elements.
template <bool BWD, typename T>
cudaError_t launch_norm_typed(const NormParams &p, bool layer, const NormPlan &n, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int es = sizeof(T);
    const bool vec = p.D % V == 0 && vec_ok(p.x, p.x_row, es, V) && vec_ok(p.dy, p.dy_row, es, V) &&
                     vec_ok(p.y, p.y_row, es, V);
    if (layer) return vec ? launch_norm_rows<BWD, T, V, true>(p, n, st) : launch_norm_rows<BWD, T, 1, true>(p, n, st);
    return vec ? launch_norm_rows<BWD, T, V, false>(p, n, st) : launch_norm_rows<BWD, T, 1, false>(p, n, st);
}

inline cudaError_t launch_norm_fwd(const NormParams &p, bool bf16, bool layer, cudaStream_t st) {
    const NormPlan n = norm_plan(p.R, p.D, kNormFwdPerSM);
    return bf16 ? launch_norm_typed<false, __nv_bfloat16>(p, layer, n, st) : launch_norm_typed<false, float>(p, layer, n, st);
}

// dw and db may each be null; `part` is null when both are.
inline cudaError_t launch_norm_bwd(const NormParams &p, bool bf16, bool layer, float *dw, float *db, cudaStream_t st) {
    const NormPlan n = norm_plan(p.R, p.D, kNormBwdPerSM);
    cudaError_t e = bf16 ? launch_norm_typed<true, __nv_bfloat16>(p, layer, n, st) : launch_norm_typed<true, float>(p, layer, n, st);
    if (e != cudaSuccess || !p.part) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.D + 31) / 32), db ? 2u : 1u);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_cols_kernel, (const float *)p.part, (int64_t)n.ctas, p.D, dw, db);
}

}  // namespace la

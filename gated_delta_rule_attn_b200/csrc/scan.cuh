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
// (A2 A1, A2 X1 + X2).  Both passes read and write HBM once and are bound by it,
// so the work is laid out for bytes in flight:
//   - a thread holds R tokens x V channels in registers, a CTA S such runs of
//     CG * V channels: S * R tokens;
//   - a cluster of K CTAs covers K * S * R consecutive tokens of one channel
//     block per step and walks the sequence in such steps, so few channels and a
//     long sequence still fill the GPU, with no second pass over the data and no
//     scratch in global memory;
//   - per step a thread composes its run, a warp its runs (shuffles), the CTA its
//     warps (shared memory) and the cluster its CTAs: every CTA writes its map
//     into the shared memory of the others and folds the K maps in order;
//   - knowing the state that enters its run, a thread repeats its R tokens
//     with the plain recurrence, so within a run the arithmetic is the
//     definition's, and writes the outputs;
//   - the next step's loads are issued before this step's exchange.
// The order of all sums is fixed: results are the same from run to run.  The
// only waits are the hardware's CTA and cluster barriers, which every thread of
// the cluster passes the same number of times.
#pragma once

#include <algorithm>

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
    int cg_log2;                    // log2 of channel groups per CTA
    int ncb;                        // channel blocks
    int K;                          // CTAs per cluster
};

constexpr int kScanThreads = 256;
constexpr int kScanMaxCluster = 16;
// channel groups per CTA, at most: 64 channels in groups of 4, 32 single ones
template <int V>
constexpr int kScanMaxCG = V == 4 ? 16 : 32;
// tokens a thread holds: enough loads in flight without spilling
template <int V>
constexpr int kScanRun = V == 4 ? 4 : 8;

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Write a float2 at the address that `saddr` (own shared memory) has in CTA `rank`.
__device__ __forceinline__ void st_cluster_f2(uint32_t saddr, uint32_t rank, float a, float b) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote), "f"(a), "f"(b) : "memory");
}

// sigmoid(l) and 1 - sigmoid(l), both to fp32 relative accuracy: the exponential
// is taken of -|l|, so neither overflows nor cancels.
__device__ __forceinline__ void sigmoid_pair(float l, float &a, float &r) {
    const float e = __expf(-fabsf(l));
    const float big = __fdividef(1.f, 1.f + e);
    const float small = e * big;
    a = l >= 0.f ? big : small;
    r = l >= 0.f ? small : big;
    if (l != l) a = r = l;
}

// A sigmoid kept in one register with full relative accuracy of both a and
// 1 - a: the smaller of the two, negative when it is 1 - a.
__device__ __forceinline__ float sig_pack(float l) {
    float a, r;
    sigmoid_pair(l, a, r);
    return l >= 0.f ? -r : a;
}
__device__ __forceinline__ float sig_a(float s) { return signbit(s) ? 1.f + s : s; }
__device__ __forceinline__ float sig_r(float s) { return signbit(s) ? -s : 1.f - s; }

template <int V>
struct ScanShared {
    static constexpr int kCB = kScanMaxCG<V> * V;
    float wA[2][kScanThreads / 32][kCB], wX[2][kScanThreads / 32][kCB];   // the warps' maps
    float2 slot[2][kScanMaxCluster][kCB];                                // the cluster's maps
    float cin[2][kCB];                                                   // state entering the CTA's tokens
};

// The state that enters every thread's run, from the run's map (A, X).
// `carry` is the state entering this step; with K > 1 it lives in a register of
// thread `tid` < CB for channel `tid`, with K == 1 in sm.cin[p].  Returns the
// state in `hin`; the caller runs its tokens and, with K == 1, the last run of
// the CTA stores the step's final state with scan_put_carry.
template <int V>
__device__ __forceinline__ void scan_exchange(ScanShared<V> &sm, int p, int K, uint32_t rank, int cg_log2,
                                              float (&A)[V], float (&X)[V], float &carry, float (&hin)[V]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int CG = 1 << cg_log2, cl = lane & (CG - 1);
    const int CB = CG * V;
    // maps of the warp's runs up to and including this one
    for (int off = CG; off < 32; off <<= 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float a1 = __shfl_up_sync(0xffffffffu, A[v], off);
            const float x1 = __shfl_up_sync(0xffffffffu, X[v], off);
            if (lane >= off) {
                X[v] = fmaf(A[v], x1, X[v]);
                A[v] *= a1;
            }
        }
    }
    if (lane >= 32 - CG) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sm.wA[p][warp][cl * V + v] = A[v];
            sm.wX[p][warp][cl * V + v] = X[v];
        }
    }
    // maps of the warp's runs before this one
    float Ae[V], Xe[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Ae[v] = __shfl_up_sync(0xffffffffu, A[v], CG & 31);
        Xe[v] = __shfl_up_sync(0xffffffffu, X[v], CG & 31);
        if (lane < CG) { Ae[v] = 1.f; Xe[v] = 0.f; }
    }
    __syncthreads();
    if (K > 1) {
        if (tid < CB) {
            float a = 1.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < kScanThreads / 32; ++w) {
                const float wa = sm.wA[p][w][tid];
                x = fmaf(wa, x, sm.wX[p][w][tid]);
                a *= wa;
            }
            const uint32_t s = smem_u32(&sm.slot[p][rank][tid]);
            for (int k = 0; k < K; ++k) st_cluster_f2(s, (uint32_t)k, a, x);
        }
        cluster_arrive();
        cluster_wait();
        if (tid < CB) {
            float h = carry;
            for (int k = 0; k < K; ++k) {
                if (k == (int)rank) sm.cin[p][tid] = h;
                const float2 m = sm.slot[p][k][tid];
                h = fmaf(m.x, h, m.y);
            }
            carry = h;
        }
        __syncthreads();
    }
#pragma unroll
    for (int v = 0; v < V; ++v) hin[v] = sm.cin[p][cl * V + v];
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) hin[v] = fmaf(sm.wA[p][w][cl * V + v], hin[v], sm.wX[p][w][cl * V + v]);
#pragma unroll
    for (int v = 0; v < V; ++v) hin[v] = fmaf(Ae[v], hin[v], Xe[v]);
}

template <typename TX, typename TG, int V, int R, bool LOGIT, bool TIED>
__global__ void __launch_bounds__(kScanThreads, 2) scan_fwd_kernel(const ScanParams P) {
    __shared__ ScanShared<V> sm;
    const int tid = threadIdx.x, lane = tid & 31;
    const int K = P.K;
    const uint32_t rank = K > 1 ? cluster_ctarank() : 0u;
    if (K > 1) cluster_arrive();   // every CTA of the cluster has started before its memory is written
    const int CG = 1 << P.cg_log2, cl = lane & (CG - 1), CB = CG * V;
    const int run = tid >> P.cg_log2, TT = (kScanThreads >> P.cg_log2) * R;
    const int64_t blk = blockIdx.x / K, b = blk / P.ncb, cb = blk % P.ncb;
    const SeqSpan sp = seq_span(P.cu_seqlens, b, P.T, P.max_seqlen, rank == 0 && cb == 0 && tid == 0);
    const int64_t c = cb * CB + cl * V;
    const bool cok = c < P.D;
    const TX *x = static_cast<const TX *>(P.x) + sp.row0 * P.x_row + c;
    const TG *g = static_cast<const TG *>(P.g) + sp.row0 * P.g_row + c;
    TX *h = static_cast<TX *>(P.h) + sp.row0 * P.h_row + c;

    // the state entering the sequence
    const int64_t cc = cb * CB + tid;
    float carry = 0.f;
    if (tid < CB) {
        if (P.h0 && cc < P.D) carry = P.h0[b * P.D + cc];
        sm.cin[0][tid] = carry;
    }
    if (K > 1) cluster_wait();

    RowVec<TX, V> xr[R];
    RowVec<TG, V> gr[R];
    const int64_t step = (int64_t)K * TT;
    const int64_t niter = (sp.len + step - 1) / step;
    int64_t t0 = (int64_t)rank * TT + run * R;
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (cok && t + r < sp.len) {
                xr[r].load(x + (t + r) * P.x_row);
                gr[r].load(g + (t + r) * P.g_row);
            }
    };
    fetch(t0);
    for (int64_t it = 0; it < niter; ++it, t0 += step) {
        const int p = (int)(it & 1);
        float a[R][V], u[R][V];
        float A[V], X[V], hv[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { A[v] = 1.f; X[v] = 0.f; }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool ok = cok && t0 + r < sp.len;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float av = gr[r].get(v), rv;
                if (LOGIT) sigmoid_pair(av, av, rv);
                else rv = 1.f - av;
                const float xv = xr[r].get(v);
                a[r][v] = ok ? av : 1.f;
                u[r][v] = ok ? (TIED ? rv * xv : xv) : 0.f;
                X[v] = fmaf(a[r][v], X[v], u[r][v]);
                A[v] *= a[r][v];
            }
        }
        fetch(t0 + step);
        scan_exchange<V>(sm, p, K, rank, P.cg_log2, A, X, carry, hv);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int v = 0; v < V; ++v) hv[v] = fmaf(a[r][v], hv[v], u[r][v]);
            if (cok && t0 + r < sp.len) RowVec<TX, V>::store(h + (t0 + r) * P.h_row, hv);
        }
        if (K == 1 && tid >= kScanThreads - CG) {
#pragma unroll
            for (int v = 0; v < V; ++v) sm.cin[p ^ 1][cl * V + v] = hv[v];
        }
    }
    if (P.h_last) {
        if (K == 1) {
            __syncthreads();
            if (tid < CB) carry = sm.cin[niter & 1][tid];
        }
        if (rank == 0 && tid < CB && cc < P.D) P.h_last[b * P.D + cc] = carry;
    }
}

template <typename TX, typename TG, int V, int R, bool LOGIT, bool TIED>
__global__ void __launch_bounds__(kScanThreads, 2) scan_bwd_kernel(const ScanParams P) {
    __shared__ ScanShared<V> sm;
    const int tid = threadIdx.x, lane = tid & 31;
    const int K = P.K;
    const uint32_t rank = K > 1 ? cluster_ctarank() : 0u;
    if (K > 1) cluster_arrive();
    const int CG = 1 << P.cg_log2, cl = lane & (CG - 1), CB = CG * V;
    const int run = tid >> P.cg_log2, TT = (kScanThreads >> P.cg_log2) * R;
    const int64_t blk = blockIdx.x / K, b = blk / P.ncb, cb = blk % P.ncb;
    const SeqSpan sp = seq_span(P.cu_seqlens, b, P.T, P.max_seqlen, rank == 0 && cb == 0 && tid == 0);
    const int64_t c = cb * CB + cl * V;
    const bool cok = c < P.D;
    // the walk goes from the last token to the first: place j is token len - 1 - j
    const int64_t last = sp.row0 + sp.len - 1;
    const TG *g = static_cast<const TG *>(P.g) + last * P.g_row + c;
    const TX *dh = static_cast<const TX *>(P.dh) + last * P.dh_row + c;
    const TX *hs = static_cast<const TX *>(P.hs) + (last - 1) * P.hs_row + c;
    const TX *x = TIED ? static_cast<const TX *>(P.x) + last * P.x_row + c : nullptr;
    TX *dx = static_cast<TX *>(P.dx) + last * P.dx_row + c;
    TG *dg = static_cast<TG *>(P.dg) + last * P.dg_row + c;

    const int64_t cc = cb * CB + tid;
    float carry = 0.f;
    if (tid < CB) {
        if (P.dh_last && cc < P.D) carry = P.dh_last[b * P.D + cc];
        sm.cin[0][tid] = carry;
    }
    if (K > 1) cluster_wait();

    RowVec<TG, V> gr[R];
    RowVec<TX, V> dr[R], hr[R], xr[TIED ? R : 1];
    const int64_t step = (int64_t)K * TT;
    const int64_t niter = (sp.len + step - 1) / step;
    int64_t j0 = (int64_t)rank * TT + run * R;
    auto fetch = [&](int64_t j) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (cok && j + r < sp.len) {
                gr[r].load(g - (j + r) * P.g_row);
                dr[r].load(dh - (j + r) * P.dh_row);
                if (j + r + 1 < sp.len) hr[r].load(hs - (j + r) * P.hs_row);
                if (TIED) xr[r].load(x - (j + r) * P.x_row);
            }
    };
    fetch(j0);
    for (int64_t it = 0; it < niter; ++it, j0 += step) {
        const int p = (int)(it & 1);
        float s[R][V];                       // the gate (LOGIT: packed, see sig_pack)
        RowVec<TX, V> dc[R], hc[R], xc[TIED ? R : 1];
        float A[V], X[V], cv[V];
#pragma unroll
        for (int v = 0; v < V; ++v) { A[v] = 1.f; X[v] = 0.f; }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool ok = cok && j0 + r < sp.len;
            if (!ok) dr[r].zero();
            dc[r] = dr[r];
            hc[r] = hr[r];
            if (TIED) xc[r] = xr[r];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float raw = gr[r].get(v);
                s[r][v] = ok ? (LOGIT ? sig_pack(raw) : raw) : (LOGIT ? -0.f : 1.f);
                const float a = LOGIT ? sig_a(s[r][v]) : s[r][v];
                X[v] = a * (X[v] + dc[r].get(v));
                A[v] *= a;
            }
        }
        fetch(j0 + step);
        scan_exchange<V>(sm, p, K, rank, P.cg_log2, A, X, carry, cv);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t j = j0 + r;
            const bool ok = cok && j < sp.len;
            float hp[V];
            if (ok && j + 1 == sp.len) {     // the first token: the state before it is h0
#pragma unroll
                for (int v = 0; v < V; ++v) hp[v] = P.h0 ? P.h0[b * P.D + c + v] : 0.f;
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) hp[v] = hc[r].get(v);
            }
            float dxv[V], dgv[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float a = LOGIT ? sig_a(s[r][v]) : s[r][v];
                const float q = LOGIT ? sig_r(s[r][v]) : 1.f - s[r][v];
                const float G = dc[r].get(v) + cv[v];
                cv[v] = a * G;
                dxv[v] = TIED ? q * G : G;
                const float da = G * (TIED ? hp[v] - xc[TIED ? r : 0].get(v) : hp[v]);
                dgv[v] = LOGIT ? da * (a * q) : da;
            }
            if (ok) {
                RowVec<TX, V>::store(dx - j * P.dx_row, dxv);
                RowVec<TG, V>::store(dg - j * P.dg_row, dgv);
            }
        }
        if (K == 1 && tid >= kScanThreads - CG) {
#pragma unroll
            for (int v = 0; v < V; ++v) sm.cin[p ^ 1][cl * V + v] = cv[v];
        }
    }
    if (P.dh0) {
        if (K == 1) {
            __syncthreads();
            if (tid < CB) carry = sm.cin[niter & 1][tid];
        }
        if (rank == 0 && tid < CB && cc < P.D) P.dh0[b * P.D + cc] = carry;
    }
}

// One token per sequence: state <- a state + u in place (fp32), output rounded
// once.  A thread takes V channels of one sequence; HBM-bound on the state.
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
            float a = gr.get(v), r;
            if (LOGIT) sigmoid_pair(a, a, r);
            else r = 1.f - a;
            const float xv = xr.get(v);
            s[v] = fmaf(a, s[v], TIED ? r * xv : xv);
        }
        RowVec<float, V>::store(st, s);
        RowVec<TX, V>::store(static_cast<TX *>(P.h) + n * P.h_row + i, s);
    }
}

enum class ScanOp { kFwd, kBwd, kStep };

template <ScanOp OP, typename TX, typename TG, int V, bool LOGIT, bool TIED>
cudaError_t launch_scan_typed(ScanParams p, cudaStream_t st) {
    if constexpr (OP == ScanOp::kStep) {
        // dense rows are one row: no thread is lost at the end of each
        if (p.x_row == p.D && p.g_row == p.D && p.h_row == p.D) {
            p.D *= p.B;
            p.B = 1;
        }
        const dim3 grid((unsigned)((p.D + 256 * V - 1) / (256 * V)), (unsigned)std::min<int64_t>(p.B, 65535));
        scan_step_kernel<TX, TG, V, LOGIT, TIED><<<grid, 256, 0, st>>>(p);
        return cudaGetLastError();
    } else {
        constexpr int R = kScanRun<V>;
        auto kernel = OP == ScanOp::kFwd ? scan_fwd_kernel<TX, TG, V, R, LOGIT, TIED>
                                         : scan_bwd_kernel<TX, TG, V, R, LOGIT, TIED>;
        const int64_t len = p.cu_seqlens ? p.max_seqlen : p.T;
        const int sms = sm_count();
        // Channels per CTA: as wide as the row accesses like, narrower while a
        // cluster of every width would leave SMs idle.
        int cg = V == 4 ? 4 : 5;
        auto blocks = [&](int l) { return (p.D + ((int64_t)V << l) - 1) / ((int64_t)V << l) * p.B; };
        auto tokens = [&](int l) { return (int64_t)(kScanThreads >> l) * R; };
        while (cg > 2 && blocks(cg) * kScanMaxCluster < 2 * sms && len > tokens(cg)) --cg;
        // CTAs along the sequence: until the GPU holds about four per SM, and no
        // more than the sequence has tokens for.
        int K = 1;
        while (K < kScanMaxCluster && blocks(cg) * K < 4 * sms && (int64_t)K * tokens(cg) < len) K *= 2;
        p.cg_log2 = cg;
        p.ncb = (int)(blocks(cg) / p.B);
        p.K = K;
        if (K > 8) {
            const cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(blocks(cg) * K));
        cfg.blockDim = dim3(kScanThreads);
        cfg.stream = st;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)K;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = K > 1 ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, kernel, (const ScanParams)p);
    }
}

template <ScanOp OP, typename TX, typename TG, int V>
cudaError_t launch_scan_forms(const ScanParams &p, bool logit, bool tied, cudaStream_t st) {
    if (logit) return tied ? launch_scan_typed<OP, TX, TG, V, true, true>(p, st)
                           : launch_scan_typed<OP, TX, TG, V, true, false>(p, st);
    return tied ? launch_scan_typed<OP, TX, TG, V, false, true>(p, st)
                : launch_scan_typed<OP, TX, TG, V, false, false>(p, st);
}

// Four channels per access where the channel count, every row stride and every
// pointer allow it, else one.
template <ScanOp OP, typename TX, typename TG>
cudaError_t launch_scan(const ScanParams &p, bool logit, bool tied, cudaStream_t st) {
    const int ex = sizeof(TX), eg = sizeof(TG);
    const bool v4 = p.D % 4 == 0 && vec_ok(p.x, p.x_row, ex, 4) && vec_ok(p.g, p.g_row, eg, 4) &&
                    vec_ok(p.h, p.h_row, ex, 4) && vec_ok(p.hs, p.hs_row, ex, 4) &&
                    vec_ok(p.dh, p.dh_row, ex, 4) && vec_ok(p.dx, p.dx_row, ex, 4) &&
                    vec_ok(p.dg, p.dg_row, eg, 4);
    return v4 ? launch_scan_forms<OP, TX, TG, 4>(p, logit, tied, st)
              : launch_scan_forms<OP, TX, TG, 1>(p, logit, tied, st);
}
}  // namespace la

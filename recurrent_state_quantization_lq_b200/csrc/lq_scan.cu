// The gated linear recurrence over vector states and its gradients.
//
// Per (sequence, head) unit and channel, alpha_t = exp(g_t):
//     h_t = alpha_t h_{t-1} + beta_t v_t,   out_t = h_t.
// A run of tokens maps the state before it to the state after it by
// h -> A h + H with A = prod alpha_t and H the run's own result from zero, and
// such maps compose: (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2).  The gradient
// X_t = alpha_t D_t, D_t = grad_out_t + X_{t+1}, runs the other way by
// X -> A X + E with the same A.  That is what lets a long sequence be split.
//
// A thread holds eight channels of a row (lq_vec8.cuh); row_lanes(d) adjacent
// lanes hold a row.
#include <cooperative_groups.h>

#include "lq_ops.h"
#include "lq_kernels.h"
#include "lq_vec8.cuh"

namespace cg = cooperative_groups;

namespace lq {

constexpr int kScanThreads = 256;
constexpr int kScanRun = 4;          // consecutive tokens a thread takes in the backward pass

int scan_checkpoint_tokens(int d) { return kScanThreads / row_lanes(d) * kScanRun; }

namespace {

// alpha = exp(g).  A gate near 1 acts over a thousand tokens, so its last bit
// counts: 1 + (Taylor's g + g^2/2 + ... + g^6/720) is rounded once, at the
// sum, where |g| <= 1/4 (remainder below 1.3e-8), and has no bias there.
__device__ __forceinline__ float gate_of(float g) {
    if (fabsf(g) <= 0.25f) {
        float p = fmaf(g, 1.0f / 720.0f, 1.0f / 120.0f);
        p = fmaf(g, p, 1.0f / 24.0f);
        p = fmaf(g, p, 1.0f / 6.0f);
        p = fmaf(g, p, 0.5f);
        p = fmaf(g, p, 1.0f);
        return fmaf(g, p, 1.0f);
    }
    return expf(g);
}

struct Unit {
    int u, b, h;     // unit, sequence, head
    int len;         // its tokens
};

__device__ __forceinline__ Unit unit_of(const lq_scan_args &a, int heads, int u) {
    Unit w;
    w.u = u;
    w.b = u / heads;
    w.h = u - w.b * heads;
    w.len = a.n_tokens;
    if (a.lengths != nullptr) w.len = min(max(__ldg(a.lengths + w.b), 0), a.n_tokens);
    return w;
}

__device__ __forceinline__ int64_t row_of(const lq_strides &s, const Unit &w, int t) {
    return (int64_t)t * s.token + (int64_t)w.b * s.seq + (int64_t)w.h * s.head;
}

// Eight gates of a token (scalar: one value).
template <bool CHAN, bool VEC>
struct Gates {
    float a[CHAN ? 8 : 1];
    __device__ __forceinline__ float operator[](int i) const { return a[CHAN ? i : 0]; }
    __device__ __forceinline__ void load(const float *p, int n) {   // log-gates, as they lie in memory
        if constexpr (CHAN) {
            Raw8<float> r;
            load8<VEC>(p, n, r);
            widen8(r, a);
        } else {
            a[0] = __ldg(p);
        }
    }
    __device__ __forceinline__ void exponentiate() {
#pragma unroll
        for (int i = 0; i < (CHAN ? 8 : 1); ++i) a[i] = gate_of(a[i]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (CHAN ? 8 : 1); ++i) a[i] = 0.0f;
    }
    __device__ __forceinline__ void one() {
#pragma unroll
        for (int i = 0; i < (CHAN ? 8 : 1); ++i) a[i] = 1.0f;
    }
};

// ------------------------------------------------------------------- forward

// Token after token, one row of lanes per unit.
template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kScanThreads) scan_rows_kernel(lq_scan_args a, int heads, int units, int d,
                                                                 int lanes, int every) {
    const int id = blockIdx.x * kScanThreads + threadIdx.x;
    const int u = id / lanes, c0 = (id % lanes) * 8;
    if (u >= units || c0 >= d) return;
    const Unit w = unit_of(a, heads, u);
    const int n = min(8, d - c0);
    const int64_t state = (int64_t)u * d + c0;
    float h[8] = {};
    if (a.h0 != nullptr) {
        Raw8<float> r;
        load8<VEC>(a.h0 + state, n, r);
        widen8(r, h);
    }
    for (int t = 0; t < w.len; ++t) {
        Raw8<InT> raw;
        load8<VEC>(static_cast<const InT *>(a.v) + row_of(a.v_stride, w, t) + c0, n, raw);
        Gates<CHAN, VEC> gate;
        gate.load(a.g + row_of(a.g_stride, w, t) + (CHAN ? c0 : 0), n);
        const float beta = a.beta != nullptr ? __ldg(a.beta + row_of(a.beta_stride, w, t)) : 1.0f;
        if (a.checkpoints != nullptr && t % every == 0)
            store8<VEC>(a.checkpoints + (int64_t)(t / every) * units * d + state, n, h);
        gate.exponentiate();
        float v[8];
        widen8(raw, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = fmaf(gate[i], h[i], beta * v[i]);
        if (a.out != nullptr) store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, h);
    }
    if (a.h_last != nullptr) store8<VEC>(a.h_last + state, n, h);
}

// A cluster of CTAs takes one unit: `ranks` CTAs x (rows of lanes) x R
// consecutive tokens at a time.  Each row runs its tokens from zero, the rows'
// maps are composed over the warp by shuffles, over the CTA's warps by one
// thread a channel and over the cluster through distributed shared memory;
// every CTA composes all of the cluster's maps, so each knows the state that
// the next tokens start from.  The row then runs its tokens, still in
// registers, again from their true start and stores them: every input is read
// and every output written once.
template <typename InT, bool CHAN>
struct ForwardRun {
    // 64 bytes of v a row at least in flight per thread, and no more registers than three CTAs an SM leave
    static constexpr int R = sizeof(InT) == 2 && !CHAN ? 8 : 4;
};

template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kScanThreads)
    scan_split_kernel(lq_scan_args a, int heads, int units, int d, int lanes, int every) {
    constexpr int NW = kScanThreads / 32, R = ForwardRun<InT, CHAN>::R, MAXD = 256;
    __shared__ float sA[NW][CHAN ? MAXD : 1], sH[NW][MAXD];   // the warps' maps, then the states before their tokens
    __shared__ float2 mine[2][MAXD];                          // this CTA's map (A, H), by the parity of the step
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int rows = kScanThreads / lanes, chunk = rows * R;
    const int c0 = (lane % lanes) * 8, row = tid / lanes;
    const Unit w = unit_of(a, heads, blockIdx.x / ranks);
    const bool on = c0 < d;
    const int n = on ? min(8, d - c0) : 0;
    float carry = 0.0f;              // thread c < d: the state before the step's tokens
    if (tid < d && a.h0 != nullptr) carry = a.h0[(int64_t)w.u * d + tid];

    int step = 0;
    for (int t0 = 0; t0 < w.len; t0 += ranks * chunk, ++step) {
        const int t_row = t0 + rank * chunk + row * R;
        Raw8<InT> rv[R];
        Gates<CHAN, VEC> gate[R];
        float beta[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            zero8(rv[i]);
            gate[i].zero();
            beta[i] = 1.0f;
            const int t = t_row + i;
            if (t < w.len && on) {
                load8<VEC>(static_cast<const InT *>(a.v) + row_of(a.v_stride, w, t) + c0, n, rv[i]);
                gate[i].load(a.g + row_of(a.g_stride, w, t) + (CHAN ? c0 : 0), n);
                if (a.beta != nullptr) beta[i] = __ldg(a.beta + row_of(a.beta_stride, w, t));
            }
        }
        Gates<CHAN, VEC> A;
        float H[8] = {};
        A.one();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[8];
            gate[i].exponentiate();
            widen8(rv[i], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) H[c] = fmaf(gate[i][c], H[c], beta[i] * v[c]);
#pragma unroll
            for (int c = 0; c < (CHAN ? 8 : 1); ++c) A.a[c] *= gate[i].a[c];
        }
        for (int o = lanes; o < 32; o *= 2) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float hp = __shfl_up_sync(0xffffffffu, H[c], o);
                if (lane >= o) H[c] = fmaf(A[c], hp, H[c]);
            }
#pragma unroll
            for (int c = 0; c < (CHAN ? 8 : 1); ++c) {
                const float ap = __shfl_up_sync(0xffffffffu, A.a[c], o);
                if (lane >= o) A.a[c] *= ap;
            }
        }
        if (on && lane >= 32 - lanes) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c0 + c < d) {
                    sH[warp][c0 + c] = H[c];
                    if (CHAN) sA[warp][c0 + c] = A[c];
                }
            if (!CHAN) sA[warp][0] = A.a[0];
        }
        __syncthreads();
        float pa[NW], ph[NW], ca = 1.0f, ch = 0.0f;
        if (tid < d) {
#pragma unroll
            for (int k = 0; k < NW; ++k) {           // the map of the warps before warp k
                pa[k] = ca;
                ph[k] = ch;
                const float ak = sA[k][CHAN ? tid : 0];
                ch = fmaf(ak, ch, sH[k][tid]);
                ca *= ak;
            }
        }
        float before = carry;
        if (ranks > 1) {
            if (tid < d) mine[step & 1][tid] = make_float2(ca, ch);
            // one barrier a step: the other parity's maps are written next, and
            // these only after every CTA has passed the next barrier
            cluster.sync();
            if (tid < d) {
                for (int r = 0; r < ranks; ++r) {
                    if (r == rank) before = carry;
                    const float2 m = cluster.map_shared_rank(&mine[step & 1][0], r)[tid];
                    carry = fmaf(m.x, carry, m.y);
                }
            }
        } else {
            carry = fmaf(ca, carry, ch);
        }
        if (tid < d) {
#pragma unroll
            for (int k = 0; k < NW; ++k) sH[k][tid] = fmaf(pa[k], before, ph[k]);
        }
        __syncthreads();
        float h[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {                // the map of the warp's rows before this one, then the warp's start
            const float hp = __shfl_up_sync(0xffffffffu, H[c], lanes), ap = __shfl_up_sync(0xffffffffu, A[c], lanes);
            const float hs = c0 + c < d ? sH[warp][c0 + c] : 0.0f;
            h[c] = lane >= lanes ? fmaf(ap, hs, hp) : hs;
        }
        if (a.checkpoints != nullptr && on && t_row % every == 0 && t_row < w.len)
            store8<VEC>(a.checkpoints + ((int64_t)(t_row / every) * units + w.u) * d + c0, n, h);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[8];
            widen8(rv[i], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) h[c] = fmaf(gate[i][c], h[c], beta[i] * v[c]);
            if (a.out != nullptr && on && t_row + i < w.len)
                store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t_row + i) + c0, n, h);
        }
        __syncthreads();                             // sH is read: the next step may write it
    }
    if (tid < d && rank == 0 && a.h_last != nullptr) a.h_last[(int64_t)w.u * d + tid] = carry;
    if (ranks > 1) cluster.sync();                   // no CTA leaves while another reads its map
}

// ------------------------------------------------------------------ backward

// One CTA per unit walks the sequence from its end, `chunk` tokens at a time:
// a row of lanes takes kScanRun consecutive tokens.  Each row runs its tokens
// forwards from zero (H) and backwards from zero (E); the rows' maps are
// composed over the warp by shuffles and over the CTA by one thread a channel,
// starting from the chunk's checkpoint (h) and from the tokens after it (X).
// Then every row knows the state before and the gradient after its tokens and
// runs them again.
template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kScanThreads)
    scan_backward_kernel(lq_scan_args a, lq_scan_grads g, int heads, int units, int d, int lanes) {
    constexpr int NW = kScanThreads / 32, R = kScanRun, MAXD = 256;
    __shared__ float sA[NW][CHAN ? MAXD : 1], sH[NW][MAXD], sE[NW][MAXD];   // the warps' maps
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int rows = kScanThreads / lanes, chunk = rows * R;
    const int c0 = (lane % lanes) * 8, row = tid / lanes;
    const Unit w = unit_of(a, heads, blockIdx.x);
    const bool on = c0 < d;
    const int n = on ? min(8, d - c0) : 0;
    float X = 0.0f;                  // thread c < d: the gradient that enters the chunk from its end
    if (tid < d && g.grad_last != nullptr) X = g.grad_last[(int64_t)w.u * d + tid];

    for (int t0 = (w.len + chunk - 1) / chunk * chunk - chunk; t0 >= 0; t0 -= chunk) {
        const int t_row = t0 + row * R;
        Raw8<InT> rv[R];
        Raw8<OutT> ry[R];
        Gates<CHAN, VEC> gate[R];
        float beta[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            zero8(rv[i]);
            zero8(ry[i]);
            gate[i].one();
            beta[i] = 1.0f;
            const int t = t_row + i;
            if (t < w.len && on) {
                load8<VEC>(static_cast<const InT *>(a.v) + row_of(a.v_stride, w, t) + c0, n, rv[i]);
                if (g.grad_out != nullptr)
                    load8<VEC>(static_cast<const OutT *>(g.grad_out) + row_of(g.grad_out_stride, w, t) + c0, n, ry[i]);
                gate[i].load(a.g + row_of(a.g_stride, w, t) + (CHAN ? c0 : 0), n);
                gate[i].exponentiate();
                if (a.beta != nullptr) beta[i] = __ldg(a.beta + row_of(a.beta_stride, w, t));
            }
        }
        // the row's map, then those of the rows before (A, H) and after (B, E) it in the warp
        Gates<CHAN, VEC> A, B;
        float H[8] = {}, E[8] = {};
        A.one();
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[8];
            widen8(rv[i], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) H[c] = fmaf(gate[i][c], H[c], beta[i] * v[c]);
#pragma unroll
            for (int c = 0; c < (CHAN ? 8 : 1); ++c) A.a[c] *= gate[i].a[c];
        }
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            float y[8];
            widen8(ry[i], y);
#pragma unroll
            for (int c = 0; c < 8; ++c) E[c] = gate[i][c] * (y[c] + E[c]);
        }
        B = A;
        for (int o = lanes; o < 32; o *= 2) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float hp = __shfl_up_sync(0xffffffffu, H[c], o), ep = __shfl_down_sync(0xffffffffu, E[c], o);
                if (lane >= o) H[c] = fmaf(A[c], hp, H[c]);
                if (lane + o < 32) E[c] = fmaf(B[c], ep, E[c]);
            }
#pragma unroll
            for (int c = 0; c < (CHAN ? 8 : 1); ++c) {
                const float ap = __shfl_up_sync(0xffffffffu, A.a[c], o), bp = __shfl_down_sync(0xffffffffu, B.a[c], o);
                if (lane >= o) A.a[c] *= ap;
                if (lane + o < 32) B.a[c] *= bp;
            }
        }
        if (on) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (lane >= 32 - lanes && c0 + c < d) {
                    sH[warp][c0 + c] = H[c];
                    if (CHAN) sA[warp][c0 + c] = A[c];
                }
                if (lane < lanes && c0 + c < d) sE[warp][c0 + c] = E[c];
            }
            if (!CHAN && lane >= 32 - lanes) sA[warp][0] = A.a[0];
        }
        __syncthreads();
        if (tid < d) {               // the maps become the state before, and the gradient after, each warp's tokens
            float h = a.checkpoints[((int64_t)(t0 / chunk) * units + w.u) * d + tid];
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const float hk = sH[k][tid];
                sH[k][tid] = h;
                h = fmaf(sA[k][CHAN ? tid : 0], h, hk);
            }
#pragma unroll
            for (int k = NW - 1; k >= 0; --k) {
                const float ek = sE[k][tid];
                sE[k][tid] = X;
                X = fmaf(sA[k][CHAN ? tid : 0], X, ek);
            }
        }
        __syncthreads();
        float h[8], x[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            // the row's neighbours' maps, then the warp's own start and end
            const float hp = __shfl_up_sync(0xffffffffu, H[c], lanes), ep = __shfl_down_sync(0xffffffffu, E[c], lanes);
            const float ap = __shfl_up_sync(0xffffffffu, A[c], lanes), bp = __shfl_down_sync(0xffffffffu, B[c], lanes);
            const float hs = c0 + c < d ? sH[warp][c0 + c] : 0.0f, xs = c0 + c < d ? sE[warp][c0 + c] : 0.0f;
            h[c] = lane >= lanes ? fmaf(ap, hs, hp) : hs;
            x[c] = lane + lanes < 32 ? fmaf(bp, xs, ep) : xs;
        }
        __syncthreads();             // sH and sE are read: the next chunk may write them
        float ah[R][8];              // alpha_t h_{t-1}
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float v[8];
            widen8(rv[i], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                ah[i][c] = gate[i][c] * h[c];
                h[c] = fmaf(beta[i], v[c], ah[i][c]);
            }
        }
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const int t = t_row + i;
            const bool live = t < w.len;
            float y[8], v[8], gv[8], gg[8], sum_g = 0.0f, sum_b = 0.0f;
            widen8(ry[i], y);
            widen8(rv[i], v);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float D = y[c] + x[c];
                x[c] = gate[i][c] * D;
                gv[c] = beta[i] * D;
                gg[c] = ah[i][c] * D;
                sum_g += gg[c];
                sum_b = fmaf(v[c], D, sum_b);
            }
            if (live && on && g.grad_v != nullptr)
                store8<VEC>(static_cast<InT *>(g.grad_v) + row_of(g.grad_v_stride, w, t) + c0, n, gv);
            if (CHAN && live && on && g.grad_g != nullptr)
                store8<VEC>(g.grad_g + row_of(g.grad_g_stride, w, t) + c0, n, gg);
            if (!on) sum_g = sum_b = 0.0f;     // lanes past d hold no channel
            for (int o = lanes / 2; o > 0; o /= 2) {
                if (!CHAN) sum_g += __shfl_xor_sync(0xffffffffu, sum_g, o);
                sum_b += __shfl_xor_sync(0xffffffffu, sum_b, o);
            }
            if (live && c0 == 0) {
                if (!CHAN && g.grad_g != nullptr) g.grad_g[row_of(g.grad_g_stride, w, t)] = sum_g;
                if (g.grad_beta != nullptr) g.grad_beta[row_of(g.grad_beta_stride, w, t)] = sum_b;
            }
        }
    }
    if (tid < d && g.grad_h0 != nullptr) g.grad_h0[(int64_t)w.u * d + tid] = X;
}

// ------------------------------------------------------------------ dispatch

// A kernel's types and variants, as one value.
template <typename In_, typename Out_, bool CHAN_, bool VEC_>
struct Variant {
    using In = In_;
    using Out = Out_;
    static constexpr bool CHAN = CHAN_, VEC = VEC_;
};

template <typename In, typename Out, typename F>
cudaError_t by_gate(const lq_scan_config &c, bool vec, F &&f) {
    if (c.gate == LQ_GATE_CHANNEL) return vec ? f(Variant<In, Out, true, true>()) : f(Variant<In, Out, true, false>());
    return vec ? f(Variant<In, Out, false, true>()) : f(Variant<In, Out, false, false>());
}

template <typename F>
cudaError_t by_variant(const lq_scan_config &c, bool vec, F &&f) {
    using B = __nv_bfloat16;
    const bool out_b = c.out_dtype == LQ_DTYPE_BF16;
    if (c.in_dtype == LQ_DTYPE_BF16) return out_b ? by_gate<B, B>(c, vec, f) : by_gate<B, float>(c, vec, f);
    return out_b ? by_gate<float, B>(c, vec, f) : by_gate<float, float>(c, vec, f);
}

}  // namespace

// A launch of `ranks` CTAs a unit as clusters.
template <typename... P, typename... V>
cudaError_t launch_clusters(void (*kernel)(P...), int units, int ranks, cudaStream_t s, const V &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units * (unsigned)ranks);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs that share a unit: as many as fill the device about twice over, up to
// the portable cluster size and to what the tokens keep busy.
int ranks_of(int units, long long tokens, int chunk) {
    int ranks = 1;
    while (ranks < 8 && (long long)units * ranks < 2 * sm_count() && (long long)ranks * chunk < tokens) ranks *= 2;
    return ranks;
}

cudaError_t launch_scan_forward(const lq_scan_config &c, const lq_scan_args &a, bool vec, cudaStream_t s) {
    const int units = c.batch * c.heads, lanes = row_lanes(c.d), every = scan_checkpoint_tokens(c.d);
    return by_variant(c, vec, [&](auto k) {
        using K = decltype(k);
        if (a.n_tokens <= 4) {
            const long long threads = (long long)units * lanes;
            scan_rows_kernel<typename K::In, typename K::Out, K::CHAN, K::VEC>
                <<<(unsigned)((threads + kScanThreads - 1) / kScanThreads), kScanThreads, 0, s>>>(
                    a, c.heads, units, c.d, lanes, every);
            return cudaGetLastError();
        }
        const int chunk = kScanThreads / lanes * ForwardRun<typename K::In, K::CHAN>::R;
        return launch_clusters(scan_split_kernel<typename K::In, typename K::Out, K::CHAN, K::VEC>, units,
                               ranks_of(units, a.n_tokens, chunk), s, a, c.heads, units, c.d, lanes, every);
    });
}

cudaError_t launch_scan_backward(const lq_scan_config &c, const lq_scan_args &a, const lq_scan_grads &g, bool vec,
                                 cudaStream_t s) {
    const int units = c.batch * c.heads;
    return by_variant(c, vec, [&](auto k) {
        using K = decltype(k);
        scan_backward_kernel<typename K::In, typename K::Out, K::CHAN, K::VEC>
            <<<units, kScanThreads, 0, s>>>(a, g, c.heads, units, c.d, row_lanes(c.d));
        return cudaGetLastError();
    });
}

}  // namespace lq

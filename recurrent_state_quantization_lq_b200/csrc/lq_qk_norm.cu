// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradients.
//
// For a row x of d channels, r = (sum x^2 (or mean x^2) + eps)^(-1/2):
//     xh = x r,  u = xh w,  y = s R(theta) u,
// with R a turn of the first rot_dim channels in pairs.  Backward, from dy:
//     dz = s R(-theta) dy,  dw = sum over rows of dz xh,  du = dz w,
//     dx = r (du - xh c),   c = sum xh du (L2) or its d-th part (RMS).
//
// Bound by memory: forward a row is read and written once, backward x and dy
// are read and dx written once.  A thread holds eight channels of a row and
// `lanes` adjacent threads hold a row (lq_vec8.cuh), so the sums are shuffles.
// The angles belong to a token and a channel, not to a head: a thread forms the
// cosines and sines of its channels once for a token and keeps them for the
// heads that it takes.  Neighbouring pairs lie in one thread; a half-rotation's
// partner lies in another thread of the row at the same place when rot_dim / 2
// is a multiple of eight channels (a shuffle), and otherwise anywhere (shared
// memory).
#include "lq_ops.h"
#include "lq_kernels.h"
#include "lq_vec8.cuh"

namespace lq {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;

// cos and sin of position * inv_freq: the angle is formed in FP64 and reduced
// to half a turn there, so a far position loses nothing; the FP32 functions
// then see at most pi.
__device__ __forceinline__ void angle_of(int position, double inv_freq, float *cosine, float *sine) {
    double turns = (double)position * inv_freq * 0.15915494309189535;   // 1 / (2 pi)
    turns -= rint(turns);
    sincospif((float)(2.0 * turns), sine, cosine);
}

// How a pair's two channels meet.
enum { ROT_NONE, ROT_NEIGHBOURS, ROT_SHUFFLE, ROT_SHARED };

// A thread's share of a row and, for the token it is at, its turns: channel i
// of the eight becomes cs[i] u_i + sn[i] u_partner.
template <int ROT>
struct Turns {
    float cs[ROT == ROT_NONE ? 1 : 8], sn[ROT == ROT_NONE ? 1 : 8];
    int partner;             // ROT_SHUFFLE: the partners' lane

    __device__ __forceinline__ void set(const lq_qk_norm_config &c, const lq_qk_norm_args &a, int64_t m, int c0, int lane) {
        if constexpr (ROT != ROT_NONE) {
            const int pos = __ldg(a.positions + m), half = c.rot_dim / 2;
            if (ROT == ROT_SHUFFLE) partner = c0 >= c.rot_dim ? lane : c0 < half ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = c0 + i;
                cs[i] = 1.0f;
                sn[i] = 0.0f;
                if (ROT == ROT_NEIGHBOURS && (i & 1)) {          // (the pair's first has the angle)
                    cs[i] = cs[i - 1];
                    sn[i] = -sn[i - 1];
                } else if (e < c.rot_dim) {
                    const bool first = ROT == ROT_NEIGHBOURS || (c.pairs == LQ_PAIRS_HALF ? e < half : (e & 1) == 0);
                    const int k = c.pairs == LQ_PAIRS_HALF ? (e < half ? e : e - half) : e / 2;
                    angle_of(pos, __ldg(a.inv_freq + k), &cs[i], &sn[i]);
                    if (first) sn[i] = -sn[i];
                }
            }
        }
    }
    // Turn u (BACK: by the opposite angles).  row: the warp's rows in shared memory, [row][dp].
    template <bool BACK>
    __device__ __forceinline__ void turn(const lq_qk_norm_config &c, float *row, int c0, float *u) const {
        if constexpr (ROT == ROT_NONE) return;
        float p[8];
        if constexpr (ROT == ROT_NEIGHBOURS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = u[i ^ 1];
        } else if constexpr (ROT == ROT_SHUFFLE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, u[i], partner);
        } else {
            const int half = c.rot_dim / 2;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) row[c0 + i] = u[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = c0 + i;
                const int at = e >= c.rot_dim ? e : c.pairs == LQ_PAIRS_HALF ? (e < half ? e + half : e - half) : e ^ 1;
                p[i] = row[at];
            }
        }
        if constexpr (ROT != ROT_NONE) {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = fmaf(BACK ? -sn[i] : sn[i], p[i], cs[i] * u[i]);
        }
    }
};

// The rows that a thread takes of a token's heads: row groups of the CTA share
// a token in `split` parts, part p taking heads p, p + split, ...
struct Share {
    int lanes, c0, n, lane;
    bool on;
    int64_t m;               // token
    int part;
};
__device__ __forceinline__ Share share_of(int d, int lanes, int split, int64_t group) {
    Share s;
    s.lanes = lanes;
    s.lane = threadIdx.x & 31;
    s.c0 = (threadIdx.x & (lanes - 1)) * 8;
    s.on = s.c0 < d;
    s.n = s.on ? min(8, d - s.c0) : 0;
    s.m = group / split;
    s.part = (int)(group % split);
    return s;
}

// One of q and k: a row's address and what its norm needs.
struct Heads {
    int n;                   // heads
    float scale;
    const float *weight;
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const T *p, const Share &s, Raw8<T> &r) {
    zero8(r);
    if (s.on) load8<VEC>(p, s.n, r);
}

__device__ __forceinline__ void load_weight(const float *w, const Share &s, float *x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w != nullptr && i < s.n ? __ldg(w + s.c0 + i) : 1.0f;
}

// r of a row whose eight channels are x.
__device__ __forceinline__ float scale_of(const lq_qk_norm_config &c, const float *x, int lanes) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
    for (int o = lanes / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return rsqrtf((c.norm == LQ_NORM_RMS ? s / (float)c.d : s) + c.eps);
}

constexpr int kAhead = 4;    // rows in flight per thread, forward

template <typename T, bool VEC, int ROT>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair out, int lanes, int split) {
    __shared__ float rows[ROT == ROT_SHARED ? kQkWarps * 32 * 8 : 1];
    const int64_t group = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) / lanes;
    Share s = share_of(c.d, lanes, split, group);
    const bool live = s.m < a.n_tokens;
    if (!live) s.m = a.n_tokens - 1, s.on = false;   // (the warp's shuffles want every lane)
    float *row = rows + (ROT == ROT_SHARED ? (threadIdx.x / lanes) * lanes * 8 : 0);
    Turns<ROT> turns;
    turns.set(c, a, s.m, s.c0, s.lane);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const bool is_q = which == 0;
        const int heads = is_q ? c.heads_q : c.heads_k;
        const float scale = is_q ? c.q_scale : 1.0f;
        const int64_t x_head = is_q ? a.q_head : a.k_head, y_head = is_q ? out.q_head : out.k_head;
        const T *x = static_cast<const T *>(is_q ? a.q : a.k) + s.m * (is_q ? a.q_token : a.k_token) + s.c0;
        T *y = static_cast<T *>(is_q ? out.q : out.k) + s.m * (is_q ? out.q_token : out.k_token) + s.c0;
        float w[8];
        load_weight(is_q ? a.weight_q : a.weight_k, s, w);
        for (int h0 = 0; h0 < heads; h0 += kAhead * split) {
            Raw8<T> raw[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int h = h0 + j * split + s.part;
                zero8(raw[j]);
                if (h < heads) load_row<T, VEC>(x + h * x_head, s, raw[j]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (h0 + j * split >= heads) break;      // (the same for every thread)
                const int h = h0 + j * split + s.part;
                float u[8];
                widen8(raw[j], u);
                const float r = scale_of(c, u, lanes);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] *= r * w[i];
                turns.template turn<false>(c, row, s.c0, u);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] *= scale;
                if (h < heads && s.on) store8<VEC>(y + h * y_head, s.n, u);
            }
        }
    }
}

template <typename T, bool VEC, int ROT>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_backward_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair gy, lq_qk_pair gx, float *partials,
                            int lanes, int split, int64_t groups) {
    __shared__ float rows[kQkThreads * 8];
    float *row = rows + (threadIdx.x / lanes) * lanes * 8;
    const int64_t first = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) / lanes;
    const int64_t all = (int64_t)gridDim.x * (kQkThreads / lanes);
    const int64_t rounds = (groups + all - 1) / all;
    float dw[2][8] = {};                  // this thread's part of the weight gradients, q and k
    for (int64_t round = 0; round < rounds; ++round) {
        Share s = share_of(c.d, lanes, split, first + round * all);
        const bool live = s.m < a.n_tokens;
        if (!live) s.m = a.n_tokens - 1, s.on = false;
        Turns<ROT> turns;
        turns.set(c, a, s.m, s.c0, s.lane);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const bool is_q = which == 0;
            const int heads = is_q ? c.heads_q : c.heads_k;
            const float scale = is_q ? c.q_scale : 1.0f;
            const T *x = static_cast<const T *>(is_q ? a.q : a.k) + s.m * (is_q ? a.q_token : a.k_token) + s.c0;
            const T *y = static_cast<const T *>(is_q ? gy.q : gy.k) + s.m * (is_q ? gy.q_token : gy.k_token) + s.c0;
            T *z = static_cast<T *>(is_q ? gx.q : gx.k) + s.m * (is_q ? gx.q_token : gx.k_token) + s.c0;
            const int64_t x_head = is_q ? a.q_head : a.k_head, y_head = is_q ? gy.q_head : gy.k_head,
                          z_head = is_q ? gx.q_head : gx.k_head;
            float w[8];
            load_weight(is_q ? a.weight_q : a.weight_k, s, w);
            constexpr int AHEAD = 2;
            for (int h0 = 0; h0 < heads; h0 += AHEAD * split) {
                Raw8<T> rx[AHEAD], ry[AHEAD];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int h = h0 + j * split + s.part;
                    zero8(rx[j]);
                    zero8(ry[j]);
                    if (h < heads) {
                        load_row<T, VEC>(x + h * x_head, s, rx[j]);
                        load_row<T, VEC>(y + h * y_head, s, ry[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (h0 + j * split >= heads) break;      // (the same for every thread)
                    const int h = h0 + j * split + s.part;
                    float xh[8], du[8], dot = 0.0f;
                    widen8(rx[j], xh);
                    widen8(ry[j], du);
                    const float r = scale_of(c, xh, lanes);
#pragma unroll
                    for (int i = 0; i < 8; ++i) du[i] *= scale;
                    turns.template turn<true>(c, row, s.c0, du);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        xh[i] *= r;
                        dw[which][i] = fmaf(du[i], xh[i], dw[which][i]);
                        du[i] *= w[i];
                        dot = fmaf(xh[i], du[i], dot);
                    }
                    for (int o = lanes / 2; o > 0; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    if (c.norm == LQ_NORM_RMS) dot /= (float)c.d;
#pragma unroll
                    for (int i = 0; i < 8; ++i) du[i] = r * fmaf(-xh[i], dot, du[i]);
                    if (h < heads && s.on) store8<VEC>(z + h * z_head, s.n, du);
                }
            }
        }
    }
    if (partials == nullptr) return;
    // the row groups' parts, channel by channel in a fixed order
    const int dp = lanes * 8, n_rows = kQkThreads / lanes;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[threadIdx.x * 8 + i] = dw[k][i];
        __syncthreads();
        for (int e = threadIdx.x; e < c.d; e += kQkThreads) {
            float t = 0.0f;
            for (int i = 0; i < n_rows; ++i) t += rows[i * dp + e];
            partials[((int64_t)k * gridDim.x + blockIdx.x) * c.d + e] = t;
        }
    }
}

// grad_weight[e] = the sum of the CTAs' parts; one CTA for 32 channels of each
// of q and k, 32 threads a channel.
__global__ void __launch_bounds__(1024) qk_weight_sum_kernel(const float *partials, int n, int d, float *gwq, float *gwk) {
    __shared__ float part[32][33];
    float *dst = blockIdx.y == 0 ? gwq : gwk;
    if (dst == nullptr) return;
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, e = blockIdx.x * 32 + x;
    float s = 0.0f;
    if (e < d)
        for (int i = y; i < n; i += 32) s += partials[((int64_t)blockIdx.y * n + i) * d + e];
    part[x][y] = s;
    __syncthreads();
    const float t = group_sum<32>(part[y][x]);
    if (x == 0 && blockIdx.x * 32 + y < d) dst[blockIdx.x * 32 + y] = t;
}

template <typename T, bool VEC, int ROT>
struct Qk {
    using Type = T;
    static constexpr bool V = VEC;
    static constexpr int R = ROT;
};
template <typename T, bool VEC, typename F>
cudaError_t by_rotation(const lq_qk_norm_config &c, F &&f) {
    if (c.rot_dim == 0) return f(Qk<T, VEC, ROT_NONE>());
    if (c.pairs == LQ_PAIRS_NEIGHBOURS) return f(Qk<T, VEC, ROT_NEIGHBOURS>());
    return c.rot_dim % 16 == 0 ? f(Qk<T, VEC, ROT_SHUFFLE>()) : f(Qk<T, VEC, ROT_SHARED>());
}
template <typename F>
cudaError_t by_kind(const lq_qk_norm_config &c, bool vec, F &&f) {
    if (c.dtype == LQ_DTYPE_BF16)
        return vec ? by_rotation<__nv_bfloat16, true>(c, f) : by_rotation<__nv_bfloat16, false>(c, f);
    return vec ? by_rotation<float, true>(c, f) : by_rotation<float, false>(c, f);
}

// Parts that a token's heads are taken in: one where there are tokens enough to
// fill the device (a thread's angles then serve all heads), and more for few.
int split_of(const lq_qk_norm_config &c, int64_t n_tokens, int lanes) {
    const int64_t want = 1024LL * sm_count();      // threads that keep the memory busy
    const int heads = c.heads_q > c.heads_k ? c.heads_q : c.heads_k;
    int split = 1;
    while (split < heads && n_tokens * split * lanes < want) split *= 2;
    return split;
}

}  // namespace

cudaError_t launch_qk_norm(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &out, bool vec,
                           cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    const int lanes = row_lanes(c.d), split = split_of(c, a.n_tokens, lanes), rows = kQkThreads / lanes;
    return by_kind(c, vec, [&](auto k) {
        using K = decltype(k);
        qk_norm_kernel<typename K::Type, K::V, K::R>
            <<<(unsigned)((a.n_tokens * split + rows - 1) / rows), kQkThreads, 0, s>>>(c, a, out, lanes, split);
        return cudaGetLastError();
    });
}

cudaError_t launch_qk_norm_backward(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &gy,
                                    const lq_qk_pair &gx, float *gwq, float *gwk, float *partials, bool vec,
                                    cudaStream_t s) {
    const int lanes = row_lanes(c.d), split = split_of(c, a.n_tokens, lanes), rows = kQkThreads / lanes;
    const int64_t groups = a.n_tokens * split, want = (groups + rows - 1) / rows;
    const bool sums = gwq != nullptr || gwk != nullptr;
    const unsigned grid = (unsigned)(want < kQkPartials ? want : kQkPartials);
    if (grid > 0) {
        const cudaError_t e = by_kind(c, vec, [&](auto k) {
            using K = decltype(k);
            qk_norm_backward_kernel<typename K::Type, K::V, K::R>
                <<<grid, kQkThreads, 0, s>>>(c, a, gy, gx, sums ? partials : nullptr, lanes, split, groups);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    if (!sums) return cudaSuccess;
    qk_weight_sum_kernel<<<dim3((unsigned)((c.d + 31) / 32), 2), 1024, 0, s>>>(partials, (int)grid, c.d, gwq, gwk);
    return cudaGetLastError();
}

}  // namespace lq

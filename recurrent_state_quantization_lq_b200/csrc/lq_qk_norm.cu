// Norms of queries and keys for each head with the position rotation in the
// same pass, and their gradients.
//
// For a row x of d channels, r = (sum x^2 (or mean x^2) + eps)^(-1/2):
//     xh = x r,  u = xh w,  y = s R(theta) u,
// with R a turn of the first rot_dim channels in pairs.  Backward, from dy:
//     dz = s R(-theta) dy,  dw = sum over rows of dz xh,  du = dz w,
//     dx = r (du - xh c),   c = sum xh du (L2) or its d-th part (RMS).
#include "lq_ops.h"
#include "lq_kernels.h"
#include "lq_vec8.cuh"

namespace lq {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float *p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16 *p) { *p = __float2bfloat16_rn(x); }

// cos and sin of position * inv_freq: the angle is formed in FP64 and reduced
// to half a turn there, so a far position loses nothing; the FP32 functions
// then see at most pi.
__device__ __forceinline__ void angle_of(int position, double inv_freq, float *cosine, float *sine) {
    double turns = (double)position * inv_freq * 0.15915494309189535;   // 1 / (2 pi)
    turns -= rint(turns);
    sincospif((float)(2.0 * turns), sine, cosine);
}

// Channel e of a rotated row: its pair's index, and whether it is the pair's first.
__device__ __forceinline__ int pair_of(const lq_qk_norm_config &c, int e, bool *first, int *partner) {
    const int half = c.rot_dim / 2;
    if (c.pairs == LQ_PAIRS_HALF) {
        *first = e < half;
        *partner = *first ? e + half : e - half;
        return *first ? e : e - half;
    }
    *first = (e & 1) == 0;
    *partner = e ^ 1;
    return e / 2;
}

// One warp per token: lane l holds channels l, l + 32, ... of a row, and a
// rotated channel's partner comes through shared memory.
struct Lane {
    float cs[8], sn[8];        // of the lane's channels (1 and 0 past rot_dim); sn signed for the forward turn
    int partner[8];
};

__device__ __forceinline__ void turn_of(const lq_qk_norm_config &c, const lq_qk_norm_args &a, int64_t m, int lane,
                                        Lane &w) {
    const int pos = c.rot_dim > 0 ? __ldg(a.positions + m) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        w.cs[j] = 1.0f;
        w.sn[j] = 0.0f;
        w.partner[j] = e;
        if (e < c.rot_dim) {
            bool first;
            const int i = pair_of(c, e, &first, &w.partner[j]);
            angle_of(pos, __ldg(a.inv_freq + i), &w.cs[j], &w.sn[j]);
            if (first) w.sn[j] = -w.sn[j];
        }
    }
}

// y_e = u_e cos + u_partner sin (signed); back: the transpose turn.
__device__ __forceinline__ void turn(const Lane &w, float *row, int lane, int d, const float *u, bool back, float *y) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < d) row[lane + 32 * j] = u[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] = lane + 32 * j < d ? fmaf(back ? -w.sn[j] : w.sn[j], row[w.partner[j]], w.cs[j] * u[j]) : 0.0f;
    __syncwarp();
}

__device__ __forceinline__ float scale_of(const lq_qk_norm_config &c, const float *x) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(x[j], x[j], s);
    s = group_sum<32>(s);
    return rsqrtf((c.norm == LQ_NORM_RMS ? s / (float)c.d : s) + c.eps);
}

template <typename T>
__device__ __forceinline__ void load_row(const T *p, int lane, int d, float *x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = lane + 32 * j < d ? to_f32(p[lane + 32 * j]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_row(T *p, int lane, int d, const float *x) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < d) from_f32(x[j], p + lane + 32 * j);
}

template <typename T>
__global__ void __launch_bounds__(kQkThreads) qk_norm_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair out) {
    __shared__ float rows[kQkWarps][256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t m = (int64_t)blockIdx.x * kQkWarps + warp;
    if (m >= a.n_tokens) return;
    Lane w;
    turn_of(c, a, m, lane, w);
    for (int hd = 0; hd < c.heads_q + c.heads_k; ++hd) {
        const bool is_q = hd < c.heads_q;
        const int h = is_q ? hd : hd - c.heads_q;
        const float *weight = is_q ? a.weight_q : a.weight_k;
        float x[8], y[8];
        load_row(static_cast<const T *>(is_q ? a.q : a.k) + m * (is_q ? a.q_token : a.k_token) +
                     h * (is_q ? a.q_head : a.k_head), lane, c.d, x);
        const float r = scale_of(c, x), s = is_q ? c.q_scale : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] *= r;
            if (weight != nullptr && lane + 32 * j < c.d) x[j] *= __ldg(weight + lane + 32 * j);
        }
        turn(w, rows[warp], lane, c.d, x, false, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= s;
        store_row(static_cast<T *>(is_q ? out.q : out.k) + m * (is_q ? out.q_token : out.k_token) +
                      h * (is_q ? out.q_head : out.k_head), lane, c.d, y);
    }
}

template <typename T>
__global__ void __launch_bounds__(kQkThreads)
    qk_norm_backward_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair gy, lq_qk_pair gx, float *partials) {
    __shared__ float rows[kQkWarps][256];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    float dw[2][8] = {};                  // this warp's part of the weight gradients, q and k
    for (int64_t m = (int64_t)blockIdx.x * kQkWarps + warp; m < a.n_tokens; m += (int64_t)gridDim.x * kQkWarps) {
        Lane w;
        turn_of(c, a, m, lane, w);
        for (int hd = 0; hd < c.heads_q + c.heads_k; ++hd) {
            const bool is_q = hd < c.heads_q;
            const int h = is_q ? hd : hd - c.heads_q;
            const float *weight = is_q ? a.weight_q : a.weight_k;
            float x[8], dy[8], dz[8];
            load_row(static_cast<const T *>(is_q ? a.q : a.k) + m * (is_q ? a.q_token : a.k_token) +
                         h * (is_q ? a.q_head : a.k_head), lane, c.d, x);
            load_row(static_cast<const T *>(is_q ? gy.q : gy.k) + m * (is_q ? gy.q_token : gy.k_token) +
                         h * (is_q ? gy.q_head : gy.k_head), lane, c.d, dy);
            const float r = scale_of(c, x), s = is_q ? c.q_scale : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] *= s;
            turn(w, rows[warp], lane, c.d, dy, true, dz);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] *= r;                                      // xh
                if (is_q) dw[0][j] = fmaf(dz[j], x[j], dw[0][j]);
                else dw[1][j] = fmaf(dz[j], x[j], dw[1][j]);
                if (weight != nullptr && lane + 32 * j < c.d) dz[j] *= __ldg(weight + lane + 32 * j);
                dot = fmaf(x[j], dz[j], dot);
            }
            dot = group_sum<32>(dot);
            if (c.norm == LQ_NORM_RMS) dot /= (float)c.d;
#pragma unroll
            for (int j = 0; j < 8; ++j) dz[j] = r * fmaf(-x[j], dot, dz[j]);
            store_row(static_cast<T *>(is_q ? gx.q : gx.k) + m * (is_q ? gx.q_token : gx.k_token) +
                          h * (is_q ? gx.q_head : gx.k_head), lane, c.d, dz);
        }
    }
    if (partials == nullptr) return;
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) rows[warp][lane + 32 * j] = dw[k][j];
        __syncthreads();
        if (threadIdx.x < c.d) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kQkWarps; ++i) s += rows[i][threadIdx.x];
            partials[((int64_t)k * gridDim.x + blockIdx.x) * c.d + threadIdx.x] = s;
        }
    }
}

// grad_weight[c] = the sum of the CTAs' partial sums; one CTA for each of q and k.
__global__ void __launch_bounds__(1024) qk_weight_sum_kernel(const float *partials, int n, int d, float *gwq, float *gwk) {
    __shared__ float part[1024];
    float *dst = blockIdx.x == 0 ? gwq : gwk;
    if (dst == nullptr) return;
    const int lanes = 1024 / d, c = threadIdx.x % d, l = threadIdx.x / d;
    float s = 0.0f;
    if (l < lanes)
        for (int i = l; i < n; i += lanes) s += partials[((int64_t)blockIdx.x * n + i) * d + c];
    part[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < d) {
        float t = 0.0f;
        for (int i = 0; i < lanes; ++i) t += part[i * d + threadIdx.x];
        dst[threadIdx.x] = t;
    }
}

}  // namespace

cudaError_t launch_qk_norm(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &out,
                           cudaStream_t s) {
    const unsigned grid = (unsigned)((a.n_tokens + kQkWarps - 1) / kQkWarps);
    if (grid == 0) return cudaSuccess;
    if (c.dtype == LQ_DTYPE_BF16) qk_norm_kernel<__nv_bfloat16><<<grid, kQkThreads, 0, s>>>(c, a, out);
    else qk_norm_kernel<float><<<grid, kQkThreads, 0, s>>>(c, a, out);
    return cudaGetLastError();
}

cudaError_t launch_qk_norm_backward(const lq_qk_norm_config &c, const lq_qk_norm_args &a, const lq_qk_pair &gy,
                                    const lq_qk_pair &gx, float *gwq, float *gwk, float *partials, cudaStream_t s) {
    const int64_t want = (a.n_tokens + kQkWarps - 1) / kQkWarps;
    const bool sums = gwq != nullptr || gwk != nullptr;
    const unsigned grid = (unsigned)(want < kQkPartials ? want : kQkPartials);
    if (grid > 0) {
        float *p = sums ? partials : nullptr;
        if (c.dtype == LQ_DTYPE_BF16) qk_norm_backward_kernel<__nv_bfloat16><<<grid, kQkThreads, 0, s>>>(c, a, gy, gx, p);
        else qk_norm_backward_kernel<float><<<grid, kQkThreads, 0, s>>>(c, a, gy, gx, p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (sums) {
        qk_weight_sum_kernel<<<2, 1024, 0, s>>>(partials, (int)grid, c.d, gwq, gwk);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

}  // namespace lq

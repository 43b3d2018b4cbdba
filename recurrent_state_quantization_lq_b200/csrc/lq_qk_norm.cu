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

// cos and sin of position * inv_freq.  The angle is formed in turns, in FP64
// with the products' remainders (1 / (2 pi) has a tail, too), and reduced to half
// a turn there, so a far position loses nothing; what rounding the reduced angle
// to FP32 takes from it is turned on in first order.  What is left is the error
// of the FP32 functions and one rounding.  (Device times are the same without.)
__device__ __forceinline__ void angle_of(int position, double inv_freq, float *cosine, float *sine) {
    constexpr double kHead = 0.15915494309189535, kTail = -9.839338337591243e-18;    // 1 / (2 pi)
    const double p = (double)position, f = inv_freq * kHead, t = p * f;
    const double f_low = fma(inv_freq, kTail, fma(inv_freq, kHead, -f)), t_low = fma(p, f_low, fma(p, f, -t));
    const double half_turns = 2.0 * ((t - rint(t)) + t_low);
    const float x = (float)half_turns, rest = (float)(half_turns - (double)x) * 3.14159265f;
    float c, s;
    sincospif(x, &s, &c);
    *cosine = fmaf(-rest, s, c);
    *sine = fmaf(rest, c, s);
}

// How a pair's two channels meet.
enum { ROT_NONE, ROT_NEIGHBOURS, ROT_SHUFFLE, ROT_SHARED };

// A thread's turns at a token: channel i of its eight becomes cs[i] u_i + sn[i] u_partner.
template <int ROT>
struct Turns {
    float cs[ROT == ROT_NONE ? 1 : 8], sn[ROT == ROT_NONE ? 1 : 8];
    int partner;             // ROT_SHUFFLE: the partners' lane

    __device__ __forceinline__ void set(const lq_qk_norm_config &c, const lq_qk_norm_args &a, int64_t m, int c0, int lane) {
        if constexpr (ROT != ROT_NONE) {
            const int pos = __ldg(a.positions + m), half = c.rot_dim / 2;
            if constexpr (ROT == ROT_SHUFFLE) {
                // the partners have the same eight angles: each forms four
                const bool any = c0 < c.rot_dim, second = c0 >= half;
                partner = !any ? lane : second ? lane - half / 8 : lane + half / 8;
                const int k = second ? c0 - half + 4 : c0;
                float ca[4], sa[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ca[i] = 1.0f;
                    sa[i] = 0.0f;
                    if (any) angle_of(pos, __ldg(a.inv_freq + k + i), &ca[i], &sa[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float co = __shfl_sync(0xffffffffu, ca[i], partner), so = __shfl_sync(0xffffffffu, sa[i], partner);
                    cs[i] = second ? co : ca[i];
                    cs[i + 4] = second ? ca[i] : co;
                    sn[i] = second ? so : -sa[i];
                    sn[i + 4] = second ? sa[i] : -so;
                }
                return;
            }
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
    __device__ __forceinline__ static int partner_of(const lq_qk_norm_config &c, int e) {
        const int half = c.rot_dim / 2;
        return e >= c.rot_dim ? e : c.pairs == LQ_PAIRS_HALF ? (e < half ? e + half : e - half) : e ^ 1;
    }
    // The partners of a row's eight channels u, as they lie in `raw`.  row: the
    // row's place in shared memory (ROT_SHARED).
    template <typename T>
    __device__ __forceinline__ void partners(const lq_qk_norm_config &c, const Raw8<T> &raw, const float2 *u, float *row,
                                             int c0, float2 *p) const {
        if constexpr (ROT == ROT_NEIGHBOURS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = make_float2(u[i].y, u[i].x);
        } else if constexpr (ROT == ROT_SHUFFLE && sizeof(T) == 2) {     // half the shuffles: two channels a word
            Raw8<T> r;
            r.w.x = __shfl_sync(0xffffffffu, raw.w.x, partner);
            r.w.y = __shfl_sync(0xffffffffu, raw.w.y, partner);
            r.w.z = __shfl_sync(0xffffffffu, raw.w.z, partner);
            r.w.w = __shfl_sync(0xffffffffu, raw.w.w, partner);
            widen8(r, p);
        } else if constexpr (ROT == ROT_SHUFFLE) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = make_float2(__shfl_sync(0xffffffffu, u[i].x, partner), __shfl_sync(0xffffffffu, u[i].y, partner));
        } else if constexpr (ROT == ROT_SHARED) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<float2 *>(row + c0 + 2 * i) = u[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = make_float2(row[partner_of(c, c0 + 2 * i)], row[partner_of(c, c0 + 2 * i + 1)]);
        }
    }
};

// The linear part of a token's rows: y_i = C_i x_i + S_i x_partner.  Forward the
// weights are in C and S, so that they cost a token's rows nothing; BACK is the
// opposite turn.
template <int ROT>
struct Linear {
    float2 C[4], S[ROT == ROT_NONE ? 1 : 4];
    template <bool BACK>
    __device__ __forceinline__ void set(const Turns<ROT> &t, const float *w, const float *w_partner) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float cs = ROT == ROT_NONE ? 1.0f : t.cs[ROT == ROT_NONE ? 0 : i];
            (i & 1 ? C[i / 2].y : C[i / 2].x) = BACK ? cs : cs * w[i];
            if constexpr (ROT != ROT_NONE) {
                const float sn = t.sn[i];
                (i & 1 ? S[i / 2].y : S[i / 2].x) = BACK ? -sn : sn * w_partner[i];
            }
        }
    }
    __device__ __forceinline__ void apply(const float2 *x, const float2 *p, float2 *y) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i] = mul2(C[i], x[i]);
            if constexpr (ROT != ROT_NONE) y[i] = fma2(S[i], p[i], y[i]);
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

template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const T *p, const Share &s, Raw8<T> &r) {
    zero8(r);
    if (s.on) load8<VEC>(p, s.n, r);
}

// The weights of a thread's channels, and (forward) of their partners.
__device__ __forceinline__ void load_weight(const float *w, const Share &s, float *x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w != nullptr && i < s.n ? __ldg(w + s.c0 + i) : 1.0f;
}
template <int ROT>
__device__ __forceinline__ void load_partners(const lq_qk_norm_config &c, const float *w, const Share &s, float *x) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = ROT != ROT_NONE && w != nullptr && i < s.n ? __ldg(w + Turns<ROT>::partner_of(c, s.c0 + i)) : 1.0f;
}

// The sum over a row of the products of two pairs' lists, and r from it.
__device__ __forceinline__ float row_dot(const float2 *x, const float2 *y, int lanes) {
    float2 t = mul2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) t = fma2(x[i], y[i], t);
    float s = t.x + t.y;
    for (int o = lanes / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ float scale_of(const lq_qk_norm_config &c, float sum, float mean_of) {
    return rsqrtf(fmaf(sum, mean_of, c.eps));
}

// Rows in flight per thread, forward.  Threads count for more than registers
// here: for 32768 tokens of 40 heads x 128 four CTAs an SM with four rows each
// take 129 us, three 141 and two 167.  (Backward, 16384 tokens: three CTAs
// with a row and its gradient ahead 128 us, four 159, two 143.)
constexpr int kAhead = 4;

template <typename T, bool VEC, int ROT, int LANES>
__global__ void __launch_bounds__(kQkThreads, 4)
    qk_norm_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair out, int any_lanes, int split) {
    const int lanes = LANES > 0 ? LANES : any_lanes;
    __shared__ __align__(16) float rows[ROT == ROT_SHARED ? kQkWarps * 32 * 8 : 4];
    const int64_t group = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) / lanes;
    Share s = share_of(c.d, lanes, split, group);
    const bool live = s.m < a.n_tokens;
    if (!live) s.m = a.n_tokens - 1, s.on = false;   // (the warp's shuffles want every lane)
    float *row = rows + (ROT == ROT_SHARED ? (threadIdx.x / lanes) * lanes * 8 : 0);
    const float mean_of = c.norm == LQ_NORM_RMS ? 1.0f / (float)c.d : 1.0f;
    Turns<ROT> turns;
    turns.set(c, a, s.m, s.c0, s.lane);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const bool is_q = which == 0;
        const int heads = is_q ? c.heads_q : c.heads_k;
        const int64_t x_head = is_q ? a.q_head : a.k_head, y_head = is_q ? out.q_head : out.k_head;
        const T *x = static_cast<const T *>(is_q ? a.q : a.k) + s.m * (is_q ? a.q_token : a.k_token) + s.part * x_head + s.c0;
        T *y = static_cast<T *>(is_q ? out.q : out.k) + s.m * (is_q ? out.q_token : out.k_token) + s.part * y_head + s.c0;
        const float *weight = is_q ? a.weight_q : a.weight_k;
        float w[8], wp[8];
        load_weight(weight, s, w);
        load_partners<ROT>(c, weight, s, wp);
        Linear<ROT> linear;
        linear.template set<false>(turns, w, wp);
        const float scale = is_q ? c.q_scale : 1.0f;
        for (int h0 = 0; h0 < heads; h0 += kAhead * split) {
            Raw8<T> raw[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                zero8(raw[j]);
                if (h0 + j * split + s.part < heads) load_row<T, VEC>(x, s, raw[j]);
                x += split * x_head;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (h0 + j * split >= heads) break;      // (the same for every thread)
                float2 u[4], p[4], z[4];
                widen8(raw[j], u);
                const float r = scale * scale_of(c, row_dot(u, u, lanes), mean_of);
                turns.partners(c, raw[j], u, row, s.c0, p);
                linear.apply(u, p, z);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = mul2(make_float2(r, r), z[i]);
                if (h0 + j * split + s.part < heads && s.on) store8<VEC>(y, s.n, z);
                y += split * y_head;
            }
        }
    }
}

// A sum in two FP32 parts: the second has what the additions to the first round
// off (Knuth's two-sum).  The weight gradients' sums of many parts, over a
// thread's rounds, a CTA's rows and the CTAs, are taken so, and their error does
// not grow with the tokens.  Up to kPlainRows rows of a thread (or the heads of
// one token), and as many threads' parts, are added up in plain FP32: a thread's
// registers are full, and what it carries over rounds lies in shared memory.
struct TwoSum {
    float s = 0.0f, e = 0.0f;
    __device__ __forceinline__ void add(float x, float rest = 0.0f) {
        const float t = __fadd_rn(s, x), b = __fsub_rn(t, s);
        e += __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)) + rest;
        s = t;
    }
    __device__ __forceinline__ float value() const { return isfinite(s) ? s + e : s; }
};
constexpr int kPlainRows = 32;
// The rounds of the backward kernel whose rows a thread adds up plainly.
__host__ __device__ inline int rounds_of_plain_sums(int heads, int split) {
    const int per_round = (heads + split - 1) / split;
    return per_round < kPlainRows ? kPlainRows / per_round : 1;
}

template <typename T, bool VEC, int ROT, int LANES>
__global__ void __launch_bounds__(kQkThreads, 3)
    qk_norm_backward_kernel(lq_qk_norm_config c, lq_qk_norm_args a, lq_qk_pair gy, lq_qk_pair gx, float *partials,
                            int any_lanes, int split, int64_t groups) {
    const int lanes = LANES > 0 ? LANES : any_lanes;
    __shared__ __align__(16) float rows[kQkThreads * 8];
    extern __shared__ float2 sums[];             // the threads' parts over the rounds (a TwoSum each), where carried
    float *row = rows + (threadIdx.x / lanes) * lanes * 8;
    const int64_t first = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) / lanes;
    const int64_t all = (int64_t)gridDim.x * (kQkThreads / lanes);
    const int64_t rounds = (groups + all - 1) / all;
    const float mean_of = c.norm == LQ_NORM_RMS ? 1.0f / (float)c.d : 1.0f;
    // the CTAs of blockIdx.y = 0 take the queries and the others the keys: with
    // both, the weight gradients' parts alone took 16 registers
    const bool is_q = blockIdx.y == 0;
    const int heads = is_q ? c.heads_q : c.heads_k;
    const float scale = is_q ? c.q_scale : 1.0f;          // of the results: they are linear in dy
    const int64_t x_head = is_q ? a.q_head : a.k_head, y_head = is_q ? gy.q_head : gy.k_head,
                  z_head = is_q ? gx.q_head : gx.k_head;
    float2 dw[4] = {};                    // this thread's part of the weight gradient: of `every` rounds
    const int every = rounds_of_plain_sums(heads, split);
    const bool carried = partials != nullptr && rounds > every;
    if (carried)
        for (int i = 0; i < 8; ++i) sums[i * kQkThreads + threadIdx.x] = make_float2(0.0f, 0.0f);
    for (int64_t round = 0; round < rounds; ++round) {
        Share s = share_of(c.d, lanes, split, first + round * all);
        const bool live = s.m < a.n_tokens;
        if (!live) s.m = a.n_tokens - 1, s.on = false;
        Linear<ROT> linear;
        Turns<ROT> turns;
        turns.set(c, a, s.m, s.c0, s.lane);
        linear.template set<true>(turns, nullptr, nullptr);
        const T *x = static_cast<const T *>(is_q ? a.q : a.k) + s.m * (is_q ? a.q_token : a.k_token) + s.part * x_head + s.c0;
        const T *y = static_cast<const T *>(is_q ? gy.q : gy.k) + s.m * (is_q ? gy.q_token : gy.k_token) + s.part * y_head + s.c0;
        T *z = static_cast<T *>(is_q ? gx.q : gx.k) + s.m * (is_q ? gx.q_token : gx.k_token) + s.part * z_head + s.c0;
        float w[8];
        load_weight(is_q ? a.weight_q : a.weight_k, s, w);
        Raw8<T> next_x, next_y;                           // a row ahead
        auto fetch = [&](int h0) {
            zero8(next_x);
            zero8(next_y);
            if (h0 + s.part < heads) {
                load_row<T, VEC>(x, s, next_x);
                load_row<T, VEC>(y, s, next_y);
            }
            x += split * x_head;
            y += split * y_head;
        };
        fetch(0);
        for (int h0 = 0; h0 < heads; h0 += split) {
            const bool mine = h0 + s.part < heads;
            const Raw8<T> rx = next_x, ry = next_y;
            fetch(h0 + split);
            float2 xh[4], dy[4], p[4], du[4];
            widen8(rx, xh);
            widen8(ry, dy);
            const float r = scale_of(c, row_dot(xh, xh, lanes), mean_of);
            turns.partners(c, ry, dy, row, s.c0, p);
            linear.apply(dy, p, du);                      // dz
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xh[i] = mul2(make_float2(r, r), xh[i]);
                dw[i] = fma2(du[i], xh[i], dw[i]);
                du[i] = mul2(make_float2(w[2 * i], w[2 * i + 1]), du[i]);
            }
            const float dot = -row_dot(xh, du, lanes) * mean_of, rs = r * scale;
#pragma unroll
            for (int i = 0; i < 4; ++i) du[i] = mul2(make_float2(rs, rs), fma2(make_float2(dot, dot), xh[i], du[i]));
            if (mine && s.on) store8<VEC>(z, s.n, du);
            z += split * z_head;
        }
        if (carried && ((round + 1) % every == 0 || round + 1 == rounds)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 so_far = sums[i * kQkThreads + threadIdx.x];
                TwoSum t{so_far.x, so_far.y};
                float &x = i & 1 ? dw[i / 2].y : dw[i / 2].x;
                t.add(x);
                sums[i * kQkThreads + threadIdx.x] = make_float2(t.s, t.e);
                x = round + 1 < rounds ? 0.0f : t.value();
            }
        }
    }
    if (partials == nullptr) return;
    // the row groups' parts, channel by channel in a fixed order
    const int dp = lanes * 8, n_rows = kQkThreads / lanes;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<float2 *>(rows + threadIdx.x * 8 + 2 * i) = dw[i];
    __syncthreads();
    for (int e = threadIdx.x; e < c.d; e += kQkThreads) {
        TwoSum t;
        for (int i0 = 0; i0 < n_rows; i0 += kPlainRows) {
            float x = 0.0f;
            for (int i = i0; i < min(i0 + kPlainRows, n_rows); ++i) x += rows[i * dp + e];
            t.add(x);
        }
        partials[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * c.d + e] = scale * t.value();
    }
}

// grad_weight[e] = the sum of the CTAs' parts; one CTA for eight channels of each
// of q and k, 32 threads a channel.  (With 32 channels a CTA the two-part sums of
// its 1024 threads took 1 us more than plain ones; so they take none.)
constexpr int kSumChannels = 8;
__global__ void __launch_bounds__(32 * kSumChannels)
    qk_weight_sum_kernel(const float *partials, int n, int d, float *gwq, float *gwk) {
    __shared__ float part[kSumChannels][33], rest[kSumChannels][33];
    float *dst = blockIdx.y == 0 ? gwq : gwk;
    if (dst == nullptr) return;
    const int x = threadIdx.x % kSumChannels, y = threadIdx.x / kSumChannels, e = blockIdx.x * kSumChannels + x;
    TwoSum s;
    constexpr int AHEAD = 8;         // parts in flight; one at a time took 10 us more
    const float *from = partials + (int64_t)blockIdx.y * n * d + min(e, d - 1);
    for (int i0 = y; i0 < n; i0 += 32 * AHEAD) {
        float t[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) t[j] = __ldg(from + (int64_t)min(i0 + 32 * j, n - 1) * d);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) s.add(i0 + 32 * j < n ? t[j] : 0.0f);
    }
    part[x][y] = s.s;
    rest[x][y] = s.e;
    __syncthreads();
    const int channel = threadIdx.x / 32, lane = threadIdx.x % 32, to = blockIdx.x * kSumChannels + channel;
    TwoSum t{part[channel][lane], rest[channel][lane]};
    for (int o = 16; o > 0; o /= 2) t.add(__shfl_down_sync(0xffffffffu, t.s, o), __shfl_down_sync(0xffffffffu, t.e, o));
    if (lane == 0 && to < d) dst[to] = t.value();
}

template <typename T, bool VEC, int ROT, int LANES_>
struct Qk {
    using Type = T;
    static constexpr bool V = VEC;
    static constexpr int R = ROT, LANES = LANES_;    // LANES: of a row, where the kernel is compiled for them (0: any)
};
// Aligned rows are compiled for heads of 33..64, 65..128 and 129..256 channels:
// the sums over a row then have no loop.
template <typename T, bool VEC, int ROT, typename F>
cudaError_t by_lanes(int d, F &&f) {
    if constexpr (VEC) {
        switch (row_lanes(d)) {
            case 8: return f(Qk<T, VEC, ROT, 8>());
            case 16: return f(Qk<T, VEC, ROT, 16>());
            case 32: return f(Qk<T, VEC, ROT, 32>());
            default: break;
        }
    }
    return f(Qk<T, VEC, ROT, 0>());
}
template <typename T, bool VEC, typename F>
cudaError_t by_rotation(const lq_qk_norm_config &c, F &&f) {
    if (c.rot_dim == 0) return by_lanes<T, VEC, ROT_NONE>(c.d, f);
    if (c.pairs == LQ_PAIRS_NEIGHBOURS) return by_lanes<T, VEC, ROT_NEIGHBOURS>(c.d, f);
    return c.rot_dim % 16 == 0 ? by_lanes<T, VEC, ROT_SHUFFLE>(c.d, f) : by_lanes<T, VEC, ROT_SHARED>(c.d, f);
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
        qk_norm_kernel<typename K::Type, K::V, K::R, K::LANES>
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
        const int64_t rounds = (want + grid - 1) / grid;
        const bool carried = sums && (rounds > rounds_of_plain_sums(c.heads_q, split) ||
                                      (c.heads_k > 0 && rounds > rounds_of_plain_sums(c.heads_k, split)));
        const int smem = carried ? 8 * kQkThreads * (int)sizeof(float2) : 0;
        const cudaError_t e = by_kind(c, vec, [&](auto k) {
            using K = decltype(k);
            qk_norm_backward_kernel<typename K::Type, K::V, K::R, K::LANES>
                <<<dim3(grid, c.heads_k > 0 ? 2 : 1), kQkThreads, smem, s>>>(c, a, gy, gx, sums ? partials : nullptr, lanes,
                                                                            split, groups);
            return cudaGetLastError();
        });
        if (e != cudaSuccess) return e;
    }
    if (!sums) return cudaSuccess;
    qk_weight_sum_kernel<<<dim3((unsigned)((c.d + kSumChannels - 1) / kSumChannels), 2), 32 * kSumChannels, 0, s>>>(
        partials, (int)grid, c.d, gwq, gwk);
    return cudaGetLastError();
}

}  // namespace lq

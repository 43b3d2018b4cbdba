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
// Both passes are bound by memory: forward, a token of a head is read once and
// written once; backward, v and grad_out are read and grad_v written once.
//
// Layout of the work.  A thread holds eight channels of a row (lq_vec8.cuh);
// row_lanes(d) adjacent lanes hold a row.  A cluster of CTAs takes one unit:
// `ranks` CTAs x (rows of lanes) x R consecutive tokens a step.
//   Pass one: each row runs its R tokens from zero; the rows' maps are composed
//     over the warp by shuffles and left in shared memory.
//   The composer, a warp of its own, composes the eight warps' maps, exchanges
//     the CTA's map with the cluster through distributed shared memory and
//     leaves the true state before each warp's tokens.
//   Pass two: each row runs its tokens, still in shared memory, from their true
//     start and stores the results.
// The workers take pass two of a step after pass one of the next one, so that
// the composer's chain of latencies (about 1500 cycles in a cluster) costs no
// time; a third kind of warp, the loader, keeps the tokens of up to three steps
// in flight or in use.  Measured without that split, with every warp waiting
// for the maps of its own step, a step of 32 KB took 6400 cycles (8200 in a
// cluster) where the memory needs 5800 for two CTAs.
#include <cooperative_groups.h>

#include <algorithm>

#include "lq_ops.h"
#include "lq_kernels.h"
#include "lq_vec8.cuh"

namespace cg = cooperative_groups;

namespace lq {

constexpr int kWorkers = 256;                    // threads that run tokens: warps 0..7
constexpr int kWorkerWarps = kWorkers / 32;
constexpr int kSplitThreads = kWorkers + 64;     // and the composer (warp 8) and the loader (warp 9)
constexpr int kStages = 3;                       // steps whose tokens are in shared memory
constexpr int kMostRanks = 8;                    // CTAs of a cluster (the portable size)
constexpr int kRowsThreads = 256;                // of the kernel for a few tokens

// Consecutive tokens that a row of lanes takes in a step: as many as let two
// CTAs' stages share an SM.
constexpr int forward_run(bool bf16, bool chan) { return chan ? 2 : bf16 ? 8 : 4; }
constexpr int backward_run(bool bf16, bool chan) { return bf16 && !chan ? 4 : 2; }

int scan_checkpoint_tokens(const lq_scan_config &c) {
    return kWorkers / row_lanes(c.d) * backward_run(c.in_dtype == LQ_DTYPE_BF16, c.gate == LQ_GATE_CHANNEL);
}

namespace {

// alpha = exp(g).  A gate near 1 acts over a thousand tokens, so its last bit
// counts: 1 + (Taylor's g + g^2/2 + ... + g^6/720) is rounded once, at the
// sum, where |g| <= 1/4 (remainder below 1.3e-8), and has no bias there.
__device__ __forceinline__ float2 taylor_exp2(float2 g) {
    auto k = [](float x) { return make_float2(x, x); };
    float2 p = fma2(g, k(1.0f / 720.0f), k(1.0f / 120.0f));
    p = fma2(g, p, k(1.0f / 24.0f));
    p = fma2(g, p, k(1.0f / 6.0f));
    p = fma2(g, p, k(0.5f));
    p = fma2(g, p, k(1.0f));
    return fma2(g, p, k(1.0f));
}
__device__ __forceinline__ float2 gates_of(float2 g) {
    float2 a = taylor_exp2(g);
    if (!(fabsf(g.x) <= 0.25f)) a.x = expf(g.x);
    if (!(fabsf(g.y) <= 0.25f)) a.y = expf(g.y);
    return a;
}
__device__ __forceinline__ float gate_of(float g) { return gates_of(make_float2(g, 0.0f)).x; }

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

// The gates of a thread's eight channels, in pairs (scalar gate: one pair of equal values).
template <bool CHAN>
struct Gates {
    static constexpr int N = CHAN ? 4 : 1;
    float2 a[N];
    __device__ __forceinline__ float2 operator[](int i) const { return a[CHAN ? i : 0]; }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = make_float2(x, x);
    }
    template <bool VEC>
    __device__ __forceinline__ void load(const float *p, int n) {   // log gates, as they lie in memory
        if constexpr (CHAN) {
            Raw8<float> r;
            load8<VEC>(p, n, r);
            widen8(r, a);
        } else {
            fill(__ldg(p));
        }
    }
    __device__ __forceinline__ void exponentiate() {
        if constexpr (CHAN) {
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = gates_of(a[i]);
        } else {
            fill(gate_of(a[0].x));
        }
    }
    __device__ __forceinline__ void times(const Gates &b) {
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = mul2(a[i], b.a[i]);
    }
    // the gates `o` lanes before (after) this one
    __device__ __forceinline__ Gates before(int o) const {
        Gates r;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r.a[i].x = __shfl_up_sync(0xffffffffu, a[i].x, o);
            r.a[i].y = CHAN ? __shfl_up_sync(0xffffffffu, a[i].y, o) : r.a[i].x;
        }
        return r;
    }
    __device__ __forceinline__ Gates after(int o) const {
        Gates r;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r.a[i].x = __shfl_down_sync(0xffffffffu, a[i].x, o);
            r.a[i].y = CHAN ? __shfl_down_sync(0xffffffffu, a[i].y, o) : r.a[i].x;
        }
        return r;
    }
};

__device__ __forceinline__ float2 pair_before(float2 x, int o) {
    return make_float2(__shfl_up_sync(0xffffffffu, x.x, o), __shfl_up_sync(0xffffffffu, x.y, o));
}
__device__ __forceinline__ float2 pair_after(float2 x, int o) {
    return make_float2(__shfl_down_sync(0xffffffffu, x.x, o), __shfl_down_sync(0xffffffffu, x.y, o));
}

// -------------------------------------------------- tokens in shared memory

// One tensor's rows [token][sequence][head][d] as the tensor-map copies see
// them: a box is some consecutive tokens of one (sequence, head).
constexpr int kMostBox = 256;       // tokens a box may have
struct RowMap {
    CUtensorMap map;
};

__device__ __forceinline__ void bring_boxes(unsigned char *base, const RowMap &m, const Unit &w, int t_first, int tokens,
                                            int row_bytes, uint64_t *bar) {
    const int box = min(tokens, kMostBox);
    for (int t = 0; t < tokens; t += box)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
            "%5}], [%6];" ::"r"(smem_u32(base + t * row_bytes)),
            "l"(&m.map), "r"(0), "r"(w.h), "r"(w.b), "r"(t_first + t), "r"(smem_u32(bar))
            : "memory");
}
// Where a tensor's rows are not whole pieces of 16 bytes, each thread copies
// the channels that it will read.
template <typename T>
__device__ __forceinline__ void bring_row(unsigned char *base, int pitch, const T *src, int64_t token_stride, int first,
                                          int live, int c0, int n) {
    T *q = reinterpret_cast<T *>(base) + first * pitch + c0;
    for (int i = 0; i < live; ++i, src += token_stride, q += pitch) {
        Raw8<T> r;
        load8<false>(src, n, r);
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(q) = r.w;
        } else {
            reinterpret_cast<float4 *>(q)[0] = r.lo;
            reinterpret_cast<float4 *>(q)[1] = r.hi;
        }
    }
}
// Eight channels of a token in shared memory, as pairs (where fewer exist, what
// follows them is read too).
template <typename T>
__device__ __forceinline__ void read_shared(const unsigned char *base, int pitch, int token, int c0, float2 *x) {
    const T *q = reinterpret_cast<const T *>(base) + token * pitch + c0;
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
        r.w = *reinterpret_cast<const uint4 *>(q);
    } else {
        r.lo = reinterpret_cast<const float4 *>(q)[0];
        r.hi = reinterpret_cast<const float4 *>(q)[1];
    }
    widen8(r, x);
}
__device__ __forceinline__ void read_shared(const float *q, float2 *x) {
    Raw8<float> r;
    r.lo = reinterpret_cast<const float4 *>(q)[0];
    r.hi = reinterpret_cast<const float4 *>(q)[1];
    widen8(r, x);
}

__device__ __forceinline__ void cp_async4(float *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrive at `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The workers and the composer meet.
__device__ __forceinline__ void maps_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kWorkers + 32) : "memory"); }

// The shared memory of one CTA: the stages (the tensors, then a pair (log gate,
// beta) a token) and, twice by the parity of the step, the warps' maps.
// BYTES: of a channel of a token; DIRS: maps a warp leaves (1 forward, 2 backward).
template <int BYTES, bool CHAN, int DIRS>
struct Space {
    int tokens, dp;
    __host__ __device__ Space(int n_tokens, int d) : tokens(n_tokens), dp((d + 7) / 8 * 8) {}
    // rows that a tensor map fills are packed; the last thread of the last row may read 16 bytes past them
    __host__ __device__ int scalars() const { return (tokens * dp * BYTES + 16 + 127) / 128 * 128; }
    __host__ __device__ int stage() const { return (scalars() + tokens * 8 + 127) / 128 * 128; }
    __host__ __device__ int map() const { return kWorkerWarps * (DIRS * dp + (CHAN ? dp : 4)); }   // floats
    __host__ __device__ int peer() const { return dp + (CHAN ? dp : 4); }                          // floats
    __host__ __device__ int bytes(int ranks) const {
        return kStages * stage() + 2 * map() * 4 + (ranks > 1 ? 2 * ranks * peer() * 4 : 0);
    }
};

// Barriers of a CTA.
struct Bars {
    uint64_t full[kStages];      // the loader's copies of a stage have landed
    uint64_t empty[kStages];     // the eight warps have read a stage
    uint64_t peer[2];            // the cluster's maps of a step are here
};
__device__ __forceinline__ void init_bars(Bars &b) {
    for (int i = 0; i < kStages; ++i) {
        mbar_init(&b.full[i], 1 + 32);
        mbar_init(&b.empty[i], kWorkerWarps);
    }
    mbar_init(&b.peer[0], 1);
    mbar_init(&b.peer[1], 1);
    fence_mbar_init();
}

// The stage of a step and the parity of its use, counted without divisions.
struct Turn {
    int stage = 0, parity = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
        }
    }
};

// ---------------------------------------- one vector from every CTA of a cluster

__device__ __forceinline__ uint32_t peer_address(uint32_t local, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
// Store four values in a peer's shared memory and count their bytes at the peer's barrier.
__device__ __forceinline__ void peer_store(uint32_t dst, float4 x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(x.x)), "r"(__float_as_uint(x.y)), "r"(__float_as_uint(x.z)),
                 "r"(__float_as_uint(x.w)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool peer_wait(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if (clock64() - t0 > kWaitBudgetCycles) return false;
    }
}

// Four channels' maps h -> A h + H, and their use.
struct Map4 {
    float4 A, H;
};
__device__ __forceinline__ float4 apply(const Map4 &m, float4 h) {
    return make_float4(fmaf(m.A.x, h.x, m.H.x), fmaf(m.A.y, h.y, m.H.y), fmaf(m.A.z, h.z, m.H.z), fmaf(m.A.w, h.w, m.H.w));
}
__device__ __forceinline__ float4 times4(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 four(float x) { return make_float4(x, x, x, x); }
// The first n (0..4) of four values.
__device__ __forceinline__ float4 load4(const float *p, int n) {
    float4 x = four(0.0f);
    if (n > 0) x.x = p[0];
    if (n > 1) x.y = p[1];
    if (n > 2) x.z = p[2];
    if (n > 3) x.w = p[3];
    return x;
}
__device__ __forceinline__ void store4(float *p, int n, const float4 &x) {
    if (n > 0) p[0] = x.x;
    if (n > 1) p[1] = x.y;
    if (n > 2) p[2] = x.z;
    if (n > 3) p[3] = x.w;
}

// The composer's work.  A lane owns channels 4 q .. 4 q + 3 for q = lane and
// lane + 32.  A step's maps are [H][kWorkerWarps][dp] (backward: then E), then
// A [kWorkerWarps][dp or 4].  BACK: the cluster's order runs from its last CTA
// to its first.
template <bool CHAN, bool BACK>
struct Composer {
    float *peers;            // [2][ranks][H dp, A (dp, or 4 equal)]
    uint64_t *bars;          // [2]
    int ranks, rank, dp;
    float4 carry[2];         // what enters the step
    bool alive = true;       // a wait that ran out is the last one, and what follows it is NaN

    __device__ __forceinline__ int owned() const { return (dp / 4 - (int)(threadIdx.x % 32) + 31) / 32; }
    __device__ __forceinline__ Map4 map(const float *H, const float *A, int k, int q) const {
        return Map4{*reinterpret_cast<const float4 *>(A + k * (CHAN ? dp : 4) + (CHAN ? 4 * q : 0)),
                    *reinterpret_cast<const float4 *>(H + k * dp + 4 * q)};
    }
    // Replace the warps' maps of `step` by what enters each warp.  Every CTA
    // stores its map in all CTAs and waits at its own barrier for everybody's:
    // unlike a cluster barrier this waits for no store to global memory.  A CTA
    // stores its map of step s + 2 only after it has those of s + 1, whose
    // senders had read step s.
    __device__ __forceinline__ void run(int step, float *H, const float *A) {
        const int lane = threadIdx.x % 32, p = step & 1, size = dp + (CHAN ? dp : 4);
        if (ranks > 1) {
            if (lane == 0) mbar_arrive_expect_tx(bars + p, (uint32_t)(ranks * size * 4));
            for (int j = 0; j < owned(); ++j) {
                const int q = lane + 32 * j;
                Map4 all = map(H, A, BACK ? kWorkerWarps - 1 : 0, q);
#pragma unroll
                for (int k = 1; k < kWorkerWarps; ++k) {
                    const Map4 m = map(H, A, BACK ? kWorkerWarps - 1 - k : k, q);
                    all.H = apply(m, all.H);
                    all.A = times4(all.A, m.A);
                }
                const uint32_t at = smem_u32(peers + (p * ranks + rank) * size), bar = smem_u32(bars + p);
                for (int r = 0; r < ranks; ++r) {
                    const uint32_t dst = peer_address(at, r), b = peer_address(bar, r);
                    peer_store(dst + q * 16, all.H, b);
                    if (CHAN || q == 0) peer_store(dst + (dp + 4 * q) * 4, all.A, b);
                }
            }
            if (alive) alive = peer_wait(bars + p, (step >> 1) & 1);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j >= owned()) break;
            const int q = lane + 32 * j;
            float4 x = carry[j];
            if (ranks > 1) {
                if (!alive) carry[j] = four(nanf(""));
#pragma unroll
                for (int i = 0; i < kMostRanks; ++i) {
                    if (i >= ranks) break;
                    const int r = BACK ? ranks - 1 - i : i;
                    const float *m = peers + (p * ranks + r) * size;
                    if (r == rank) x = carry[j];
                    carry[j] = apply(map(m, m + dp, 0, q), carry[j]);
                }
            }
#pragma unroll
            for (int i = 0; i < kWorkerWarps; ++i) {
                const int k = BACK ? kWorkerWarps - 1 - i : i;
                const Map4 m = map(H, A, k, q);
                *reinterpret_cast<float4 *>(H + k * dp + 4 * q) = x;
                x = apply(m, x);
            }
            if (ranks == 1) carry[j] = x;
        }
    }
};

// ------------------------------------------------------------------- forward

// Token after token, one row of lanes per unit.
template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kRowsThreads) scan_rows_kernel(lq_scan_args a, int heads, int units, int d,
                                                                 int lanes, int every) {
    const int id = blockIdx.x * kRowsThreads + threadIdx.x;
    const int u = id / lanes, c0 = (id % lanes) * 8;
    if (u >= units || c0 >= d) return;
    const Unit w = unit_of(a, heads, u);
    const int n = min(8, d - c0);
    const int64_t state = (int64_t)u * d + c0;
    float2 h[4] = {};
    if (a.h0 != nullptr) {
        Raw8<float> r;
        load8<VEC>(a.h0 + state, n, r);
        widen8(r, h);
    }
    for (int t = 0; t < w.len; ++t) {
        Raw8<InT> raw;
        load8<VEC>(static_cast<const InT *>(a.v) + row_of(a.v_stride, w, t) + c0, n, raw);
        Gates<CHAN> gate;
        gate.template load<VEC>(a.g + row_of(a.g_stride, w, t) + (CHAN ? c0 : 0), n);
        const float beta = a.beta != nullptr ? __ldg(a.beta + row_of(a.beta_stride, w, t)) : 1.0f;
        if (a.checkpoints != nullptr && t % every == 0)
            store8<VEC>(a.checkpoints + (int64_t)(t / every) * units * d + state, n, h);
        gate.exponentiate();
        float2 v[4];
        widen8(raw, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fma2(gate[i], h[i], mul2(make_float2(beta, beta), v[i]));
        if (a.out != nullptr) store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, h);
    }
    if (a.h_last != nullptr) store8<VEC>(a.h_last + state, n, h);
    if (a.zero_past && a.out != nullptr) {
        const float2 zero[4] = {};
        for (int t = w.len; t < a.n_tokens; ++t)
            store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, zero);
    }
}

template <typename InT, bool CHAN>
using ForwardSpace = Space<(int)sizeof(InT) + (CHAN ? 4 : 0), CHAN, 1>;

template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kSplitThreads, 2)
    scan_forward_kernel(lq_scan_args a, const __grid_constant__ RowMap map_v, const __grid_constant__ RowMap map_g,
                        int heads, int units, int d, int lanes, int every) {
    constexpr int R = forward_run(sizeof(InT) == 2, CHAN);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Bars bars;
    const int rows = kWorkers / lanes, chunk = rows * R;
    const ForwardSpace<InT, CHAN> space(chunk, d);
    const int dp = space.dp, pitch = VEC ? d : dp;
    const int gates_at = chunk * pitch * (int)sizeof(InT);          // the log gates of channels in a stage
    float *maps = reinterpret_cast<float *>(smem + kStages * space.stage());
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) init_bars(bars);
    __syncthreads();
    if (ranks > 1) cluster.sync();

    const Unit w = unit_of(a, heads, blockIdx.x / ranks);
    const int stride = ranks * chunk, steps = (w.len + stride - 1) / stride;
    const InT *pv = static_cast<const InT *>(a.v) + row_of(a.v_stride, w, 0);
    const float *pg = a.g + row_of(a.g_stride, w, 0);
    const float *pb = a.beta != nullptr ? a.beta + row_of(a.beta_stride, w, 0) : nullptr;

    if (warp == kWorkerWarps + 1) {                  // the loader
        Turn turn;
        for (int s = 0; s < steps; ++s, turn.next()) {
            const int t_cta = s * stride + rank * chunk, live = min(max(w.len - t_cta, 0), chunk);
            if (s >= kStages && !mbar_wait(&bars.empty[turn.stage], turn.parity ^ 1, kWaitBudgetCycles)) break;
            unsigned char *base = smem + turn.stage * space.stage();
            float2 *sc = reinterpret_cast<float2 *>(base + space.scalars());
            uint64_t *full = &bars.full[turn.stage];
            if (lane == 0) {
                const int row_bytes = d * (int)sizeof(InT);
                mbar_arrive_expect_tx(full, VEC && live > 0 ? (uint32_t)(chunk * (row_bytes + (CHAN ? d * 4 : 0))) : 0u);
                if (VEC && live > 0) {
                    bring_boxes(base, map_v, w, t_cta, chunk, row_bytes, full);
                    if (CHAN) bring_boxes(base + gates_at, map_g, w, t_cta, chunk, d * 4, full);
                }
            }
            for (int i = lane; i < live; i += 32) {
                if (!CHAN) cp_async4(&sc[i].x, pg + (t_cta + i) * a.g_stride.token);
                if (pb != nullptr) cp_async4(&sc[i].y, pb + (t_cta + i) * a.beta_stride.token);
            }
            cp_async_arrive(full);
        }
    } else if (warp == kWorkerWarps) {               // the composer
        Composer<CHAN, false> composer{maps + 2 * space.map(), bars.peer, ranks, rank, dp};
        const int64_t state = (int64_t)w.u * d;
        for (int j = 0; j < 2; ++j) {
            const int c = 4 * (lane + 32 * j);
            composer.carry[j] = a.h0 != nullptr ? load4(a.h0 + state + c, d - c) : four(0.0f);
        }
        for (int s = 0; s < steps; ++s) {
            float *H = maps + (s & 1) * space.map();
            maps_barrier();
            composer.run(s, H, H + kWorkerWarps * dp);
        }
        maps_barrier();
        if (rank == 0 && a.h_last != nullptr)
            for (int j = 0; j < 2; ++j) {
                const int c = 4 * (lane + 32 * j);
                store4(a.h_last + state + c, d - c, composer.carry[j]);
            }
    } else {                                         // the workers
        const int c0 = (lane % lanes) * 8, row = tid / lanes;
        const bool on = c0 < d;
        const int n = on ? min(8, d - c0) : 0;
        auto bring = [&](int s, int stage) {
            const int t_row = s * stride + rank * chunk + row * R, live = min(max(w.len - t_row, 0), R);
            unsigned char *base = smem + stage * space.stage();
            if (!on) return;
            bring_row(base, pitch, pv + c0 + t_row * a.v_stride.token, a.v_stride.token, row * R, live, c0, n);
            if (CHAN) bring_row(base + gates_at, pitch, pg + c0 + t_row * a.g_stride.token, a.g_stride.token, row * R, live, c0, n);
        };
        if (!VEC)
            for (int s = 0; s < kStages; ++s) bring(s, s);
        bool alive = true;           // a wait that ran out is the last one, and what follows it is NaN
        Turn one, two;               // the stages of pass one and pass two
        Gates<CHAN> A_before;        // of the step whose pass two is due: the map of its warp's rows before this one
        float2 H_before[4];
        for (int s = 0; s <= steps; ++s) {
            Gates<CHAN> A;
            float2 H[4] = {};
            A.fill(1.0f);
            if (s < steps) {
                const int live = min(max(w.len - (s * stride + rank * chunk + row * R), 0), R);
                unsigned char *base = smem + one.stage * space.stage();
                float2 *sc = reinterpret_cast<float2 *>(base + space.scalars()) + row * R;
                float *sH = maps + (s & 1) * space.map(), *sA = sH + kWorkerWarps * dp;
                if (alive) alive = mbar_wait(&bars.full[one.stage], one.parity, kWaitBudgetCycles);
                if (!alive) A.fill(nanf(""));
                if (!CHAN) {                         // each gate is raised once, by one lane of its row
                    for (int i = lane % lanes; i < live; i += lanes) sc[i].x = gate_of(sc[i].x);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (i >= live || !on) break;
                    const float2 gb = sc[i];
                    const float b = pb != nullptr ? gb.y : 1.0f;
                    Gates<CHAN> gate;
                    if constexpr (CHAN) {            // raised once: pass two finds alpha in its place
                        float *g = reinterpret_cast<float *>(base + gates_at) + (row * R + i) * pitch + c0;
                        read_shared(g, gate.a);
                        gate.exponentiate();
                        store8<true>(g, n, gate.a);
                    } else {
                        gate.fill(gb.x);
                    }
                    float2 v[4];
                    read_shared<InT>(base, pitch, row * R + i, c0, v);
#pragma unroll
                    for (int c = 0; c < 4; ++c) H[c] = fma2(gate[c], H[c], mul2(make_float2(b, b), v[c]));
                    A.times(gate);
                }
                for (int o = lanes; o < 32; o *= 2) {
                    const Gates<CHAN> before = A.before(o);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 hp = pair_before(H[c], o);
                        if (lane >= o) H[c] = fma2(A[c], hp, H[c]);
                    }
                    if (lane >= o) A.times(before);
                }
                if (on && lane >= 32 - lanes) {
                    store8<true>(sH + warp * dp + c0, 8, H);
                    if constexpr (CHAN) store8<true>(sA + warp * dp + c0, 8, A.a);
                    else if (c0 == 0) *reinterpret_cast<float4 *>(sA + warp * 4) = four(A.a[0].x);
                }
                A = A.before(lanes);
#pragma unroll
                for (int c = 0; c < 4; ++c) H[c] = pair_before(H[c], lanes);
                one.next();
            }
            maps_barrier();          // the maps of step s are there, and the states of step s - 1
            if (s > 0) {
                const int t_row = (s - 1) * stride + rank * chunk + row * R, live = min(max(w.len - t_row, 0), R);
                const unsigned char *base = smem + two.stage * space.stage();
                const float2 *sc = reinterpret_cast<const float2 *>(base + space.scalars()) + row * R;
                if (on && live > 0) {
                    float2 h[4];
                    read_shared(maps + ((s - 1) & 1) * space.map() + warp * dp + c0, h);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (lane >= lanes) h[c] = fma2(A_before[c], h[c], H_before[c]);
                    if (a.checkpoints != nullptr && t_row % every == 0)
                        store8<VEC>(a.checkpoints + ((int64_t)(t_row / every) * units + w.u) * d + c0, n, h);
                    if (a.out != nullptr) {
                        OutT *po = static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t_row) + c0;
#pragma unroll
                        for (int i = 0; i < R; ++i, po += a.out_stride.token) {
                            if (i >= live) break;
                            const float2 gb = sc[i];
                            const float b = pb != nullptr ? gb.y : 1.0f;
                            Gates<CHAN> gate;
                            if constexpr (CHAN) read_shared<float>(base + gates_at, pitch, row * R + i, c0, gate.a);
                            else gate.fill(gb.x);
                            float2 v[4];
                            read_shared<InT>(base, pitch, row * R + i, c0, v);
#pragma unroll
                            for (int c = 0; c < 4; ++c) h[c] = fma2(gate[c], h[c], mul2(make_float2(b, b), v[c]));
                            store8<VEC>(po, n, h);
                        }
                    }
                }
                if (!VEC && s - 1 + kStages < steps) bring(s - 1 + kStages, two.stage);
                if (CHAN) fence_proxy_async_smem();  // alpha was written where the next copy lands
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.empty[two.stage]);
                two.next();
            }
            A_before = A;
#pragma unroll
            for (int c = 0; c < 4; ++c) H_before[c] = H[c];
        }
        if (a.zero_past && a.out != nullptr && on) {
            const float2 zero[4] = {};
            for (int t = w.len + rank * rows + row; t < a.n_tokens; t += ranks * rows)
                store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, zero);
        }
    }
    __syncthreads();
    if (ranks > 1) cluster.sync();                   // no CTA leaves while another may still store to it
}

// ------------------------------------------------------------------ backward

// Sums of N values over the lanes of a row, N a power of two up to the lanes:
// at each of the first levels a lane hands half of its values over, so a value
// costs about one shuffle.  The lane is left with the sum of value *index.
template <int N>
__device__ __forceinline__ float sum_row(float (&x)[N], int lanes, int lane, int *index) {
    int o = lanes / 2, at = 0;
#pragma unroll
    for (int m = N / 2; m >= 1; m /= 2, o /= 2) {
        const bool high = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float keep = high ? x[i + m] : x[i], give = high ? x[i] : x[i + m];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
        at += high ? m : 0;
    }
    float s = x[0];
    for (; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    *index = at;
    return s;
}

template <typename InT, typename OutT, bool CHAN>
using BackwardSpace = Space<(int)sizeof(InT) + (int)sizeof(OutT) + (CHAN ? 4 : 0), CHAN, 2>;

// Steps run from the sequence's end.  Pass one also runs a row's tokens
// backwards from zero (E); the composer starts a step's states from the CTA's
// checkpoint, so only the gradient's maps cross the cluster; pass two runs the
// states up and the gradients down and multiplies them.
template <typename InT, typename OutT, bool CHAN, bool VEC>
__global__ void __launch_bounds__(kSplitThreads, 2)
    scan_backward_kernel(lq_scan_args a, lq_scan_grads g, const __grid_constant__ RowMap map_v,
                         const __grid_constant__ RowMap map_y, const __grid_constant__ RowMap map_g, int heads, int units,
                         int d, int lanes) {
    constexpr int R = backward_run(sizeof(InT) == 2, CHAN);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Bars bars;
    const int rows = kWorkers / lanes, chunk = rows * R;
    const BackwardSpace<InT, OutT, CHAN> space(chunk, d);
    const int dp = space.dp, pitch = VEC ? d : dp;
    const int y_at = chunk * pitch * (int)sizeof(InT), gates_at = y_at + chunk * pitch * (int)sizeof(OutT);
    float *maps = reinterpret_cast<float *>(smem + kStages * space.stage());
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) init_bars(bars);
    __syncthreads();
    if (ranks > 1) cluster.sync();

    const Unit w = unit_of(a, heads, blockIdx.x / ranks);
    const int stride = ranks * chunk, steps = (w.len + stride - 1) / stride;
    auto first_of = [&](int s) { return (steps - 1 - s) * stride + rank * chunk; };     // this CTA's first token of a step
    const InT *pv = static_cast<const InT *>(a.v) + row_of(a.v_stride, w, 0);
    const OutT *py = g.grad_out != nullptr ? static_cast<const OutT *>(g.grad_out) + row_of(g.grad_out_stride, w, 0) : nullptr;
    const float *pg = a.g + row_of(a.g_stride, w, 0);
    const float *pb = a.beta != nullptr ? a.beta + row_of(a.beta_stride, w, 0) : nullptr;

    if (warp == kWorkerWarps + 1) {                  // the loader
        Turn turn;
        const int v_bytes = d * (int)sizeof(InT), y_bytes = py != nullptr ? d * (int)sizeof(OutT) : 0;
        for (int s = 0; s < steps; ++s, turn.next()) {
            const int t_cta = first_of(s), live = min(max(w.len - t_cta, 0), chunk);
            if (s >= kStages && !mbar_wait(&bars.empty[turn.stage], turn.parity ^ 1, kWaitBudgetCycles)) break;
            unsigned char *base = smem + turn.stage * space.stage();
            float2 *sc = reinterpret_cast<float2 *>(base + space.scalars());
            uint64_t *full = &bars.full[turn.stage];
            if (lane == 0) {
                mbar_arrive_expect_tx(full, VEC && live > 0 ? (uint32_t)(chunk * (v_bytes + y_bytes + (CHAN ? d * 4 : 0))) : 0u);
                if (VEC && live > 0) {
                    bring_boxes(base, map_v, w, t_cta, chunk, v_bytes, full);
                    if (py != nullptr) bring_boxes(base + y_at, map_y, w, t_cta, chunk, y_bytes, full);
                    if (CHAN) bring_boxes(base + gates_at, map_g, w, t_cta, chunk, d * 4, full);
                }
            }
            for (int i = lane; i < live; i += 32) {
                if (!CHAN) cp_async4(&sc[i].x, pg + (t_cta + i) * a.g_stride.token);
                if (pb != nullptr) cp_async4(&sc[i].y, pb + (t_cta + i) * a.beta_stride.token);
            }
            cp_async_arrive(full);
        }
    } else if (warp == kWorkerWarps) {               // the composer
        Composer<CHAN, true> composer{maps + 2 * space.map(), bars.peer, ranks, rank, dp};
        const int64_t state = (int64_t)w.u * d;
        float4 mark[2];              // the state before the CTA's tokens of the step
        auto mark_of = [&](int s) {
            for (int j = 0; j < 2; ++j) {
                const int c = 4 * (lane + 32 * j), t_cta = first_of(s);
                const bool live = s < steps && t_cta < w.len;
                mark[j] = live ? load4(a.checkpoints + (int64_t)(t_cta / chunk) * units * d + state + c, d - c) : four(0.0f);
            }
        };
        for (int j = 0; j < 2; ++j) {
            const int c = 4 * (lane + 32 * j);
            composer.carry[j] = g.grad_last != nullptr ? load4(g.grad_last + state + c, d - c) : four(0.0f);
        }
        mark_of(0);
        for (int s = 0; s < steps; ++s) {
            float *H = maps + (s & 1) * space.map(), *E = H + kWorkerWarps * dp, *A = E + kWorkerWarps * dp;
            maps_barrier();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (j >= composer.owned()) break;
                const int q = lane + 32 * j;
#pragma unroll
                for (int k = 0; k < kWorkerWarps; ++k) {
                    const Map4 m = composer.map(H, A, k, q);
                    *reinterpret_cast<float4 *>(H + k * dp + 4 * q) = mark[j];
                    mark[j] = apply(m, mark[j]);
                }
            }
            mark_of(s + 1);
            composer.run(s, E, A);
        }
        maps_barrier();
        if (rank == 0 && g.grad_h0 != nullptr)
            for (int j = 0; j < 2; ++j) {
                const int c = 4 * (lane + 32 * j);
                store4(g.grad_h0 + state + c, d - c, composer.carry[j]);
            }
    } else {                                         // the workers
        const int c0 = (lane % lanes) * 8, row = tid / lanes;
        const bool on = c0 < d;
        const int n = on ? min(8, d - c0) : 0;
        auto bring = [&](int s, int stage) {
            if (!on || s >= steps) return;
            const int t_row = first_of(s) + row * R, live = min(max(w.len - t_row, 0), R);
            unsigned char *base = smem + stage * space.stage();
            bring_row(base, pitch, pv + c0 + t_row * a.v_stride.token, a.v_stride.token, row * R, live, c0, n);
            if (py != nullptr)
                bring_row(base + y_at, pitch, py + c0 + t_row * g.grad_out_stride.token, g.grad_out_stride.token, row * R, live, c0, n);
            if (CHAN) bring_row(base + gates_at, pitch, pg + c0 + t_row * a.g_stride.token, a.g_stride.token, row * R, live, c0, n);
        };
        if (!VEC)
            for (int s = 0; s < kStages; ++s) bring(s, s);
        // eight channels of grad_out; channels past d are no part of any sum
        auto grad_of = [&](const unsigned char *base, int i, float2 *y) {
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = make_float2(0.0f, 0.0f);
            if (py != nullptr) read_shared<OutT>(base + y_at, pitch, row * R + i, c0, y);
        };
        bool alive = true;           // a wait that ran out is the last one, and what follows it is NaN
        Turn one, two;               // the stages of pass one and pass two
        Gates<CHAN> A_before, B_after;           // of the step whose pass two is due: the maps of its warp's rows
        float2 H_before[4], E_after[4];          // before and after this one
        for (int s = 0; s <= steps; ++s) {
            Gates<CHAN> A, B;
            float2 H[4] = {}, E[4] = {};
            A.fill(1.0f);
            if (s < steps) {
                const int live = min(max(w.len - (first_of(s) + row * R), 0), R);
                unsigned char *base = smem + one.stage * space.stage();
                float2 *sc = reinterpret_cast<float2 *>(base + space.scalars()) + row * R;
                float *sH = maps + (s & 1) * space.map(), *sE = sH + kWorkerWarps * dp, *sA = sE + kWorkerWarps * dp;
                if (alive) alive = mbar_wait(&bars.full[one.stage], one.parity, kWaitBudgetCycles);
                if (!alive) A.fill(nanf(""));
                if (!CHAN) {                         // each gate is raised once, by one lane of its row
                    for (int i = lane % lanes; i < live; i += lanes) sc[i].x = gate_of(sc[i].x);
                    __syncwarp();
                }
                Gates<CHAN> gate[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    gate[i].fill(1.0f);
                    if (i < live && on) {
                        const float2 gb = sc[i];
                        const float b = pb != nullptr ? gb.y : 1.0f;
                        if constexpr (CHAN) {        // raised once: pass two finds alpha in its place
                            float *q = reinterpret_cast<float *>(base + gates_at) + (row * R + i) * pitch + c0;
                            read_shared(q, gate[i].a);
                            gate[i].exponentiate();
                            store8<true>(q, n, gate[i].a);
                        } else {
                            gate[i].fill(gb.x);
                        }
                        float2 v[4];
                        read_shared<InT>(base, pitch, row * R + i, c0, v);
#pragma unroll
                        for (int c = 0; c < 4; ++c) H[c] = fma2(gate[i][c], H[c], mul2(make_float2(b, b), v[c]));
                        A.times(gate[i]);
                    }
                }
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    if (i < live && on) {
                        float2 y[4];
                        grad_of(base, i, y);
#pragma unroll
                        for (int c = 0; c < 4; ++c) E[c] = mul2(gate[i][c], add2(y[c], E[c]));
                    }
                }
                B = A;
                for (int o = lanes; o < 32; o *= 2) {
                    const Gates<CHAN> ap = A.before(o), bp = B.after(o);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 hp = pair_before(H[c], o), ep = pair_after(E[c], o);
                        if (lane >= o) H[c] = fma2(A[c], hp, H[c]);
                        if (lane + o < 32) E[c] = fma2(B[c], ep, E[c]);
                    }
                    if (lane >= o) A.times(ap);
                    if (lane + o < 32) B.times(bp);
                }
                if (on && lane >= 32 - lanes) {
                    store8<true>(sH + warp * dp + c0, 8, H);
                    if constexpr (CHAN) store8<true>(sA + warp * dp + c0, 8, A.a);
                    else if (c0 == 0) *reinterpret_cast<float4 *>(sA + warp * 4) = four(A.a[0].x);
                }
                if (on && lane < lanes) store8<true>(sE + warp * dp + c0, 8, E);
                A = A.before(lanes);
                B = B.after(lanes);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    H[c] = pair_before(H[c], lanes);
                    E[c] = pair_after(E[c], lanes);
                }
                one.next();
            }
            maps_barrier();          // the maps of step s are there, and what enters the warps of step s - 1
            if (s > 0) {
                const int t_row = first_of(s - 1) + row * R, live = min(max(w.len - t_row, 0), R);
                const unsigned char *base = smem + two.stage * space.stage();
                const float2 *sc = reinterpret_cast<const float2 *>(base + space.scalars()) + row * R;
                const float *sH = maps + ((s - 1) & 1) * space.map(), *sE = sH + kWorkerWarps * dp;
                float2 h[4] = {}, x[4] = {}, ah[R][4];           // ah = alpha_t h_{t-1}
                if (on) {
                    read_shared(sH + warp * dp + c0, h);
                    read_shared(sE + warp * dp + c0, x);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (lane >= lanes) h[c] = fma2(A_before[c], h[c], H_before[c]);
                    if (lane + lanes < 32) x[c] = fma2(B_after[c], x[c], E_after[c]);
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (i < live && on) {
                        const float2 gb = sc[i];
                        const float b = pb != nullptr ? gb.y : 1.0f;
                        Gates<CHAN> gate;
                        if constexpr (CHAN) read_shared<float>(base + gates_at, pitch, row * R + i, c0, gate.a);
                        else gate.fill(gb.x);
                        float2 v[4];
                        read_shared<InT>(base, pitch, row * R + i, c0, v);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            ah[i][c] = mul2(gate[c], h[c]);
                            h[c] = fma2(make_float2(b, b), v[c], ah[i][c]);
                        }
                    }
                }
                constexpr int N = CHAN ? R : 2 * R;              // sums over a token's channels: grad_beta, then grad_g
                float sums[N] = {};
                InT *gv = static_cast<InT *>(g.grad_v) + row_of(g.grad_v_stride, w, t_row) + c0;
                float *gg = g.grad_g + row_of(g.grad_g_stride, w, t_row) + (CHAN ? c0 : 0);
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    if (i < live && on) {
                        const float2 gb = sc[i];
                        const float b = pb != nullptr ? gb.y : 1.0f;
                        Gates<CHAN> gate;
                        if constexpr (CHAN) read_shared<float>(base + gates_at, pitch, row * R + i, c0, gate.a);
                        else gate.fill(gb.x);
                        float2 y[4], v[4], dv[4], sb = {}, sg = {};
                        grad_of(base, i, y);
                        read_shared<InT>(base, pitch, row * R + i, c0, v);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float2 D = add2(y[c], x[c]);
                            x[c] = mul2(gate[c], D);
                            dv[c] = mul2(make_float2(b, b), D);
                            y[c] = mul2(ah[i][c], D);            // grad_g of the channel
                            if (2 * c < n) {                     // (beyond an odd d the pair's second half is zero)
                                sb = fma2(v[c], D, sb);
                                sg = add2(sg, y[c]);
                            }
                        }
                        sums[i] = sb.x + sb.y;
                        if (!CHAN) sums[N - R + i] = sg.x + sg.y;
                        if (g.grad_v != nullptr) store8<VEC>(gv + i * g.grad_v_stride.token, n, dv);
                        if (CHAN && g.grad_g != nullptr) store8<VEC>(gg + i * g.grad_g_stride.token, n, y);
                    }
                }
                float *gb_row = g.grad_beta != nullptr ? g.grad_beta + row_of(g.grad_beta_stride, w, t_row) : nullptr;
                if (!CHAN || gb_row != nullptr) {
                    auto put = [&](int j, float x) {
                        const int i = j % R;
                        if (i >= live) return;
                        if (j < R) {
                            if (gb_row != nullptr) gb_row[i * g.grad_beta_stride.token] = x;
                        } else if (g.grad_g != nullptr) {
                            gg[i * g.grad_g_stride.token] = x;
                        }
                    };
                    if (lanes >= N) {
                        int j;
                        const float x = sum_row(sums, lanes, lane, &j);
                        if (lane % (lanes / N) == 0) put(j, x);
                    } else {
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            for (int o = lanes / 2; o >= 1; o /= 2) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
                            if (c0 == 0) put(j, sums[j]);
                        }
                    }
                }
                if (!VEC) bring(s - 1 + kStages, two.stage);
                if (CHAN) fence_proxy_async_smem();  // alpha was written where the next copy lands
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.empty[two.stage]);
                two.next();
            }
            A_before = A;
            B_after = B;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                H_before[c] = H[c];
                E_after[c] = E[c];
            }
        }
        if (a.zero_past && on) {
            const float2 zero[4] = {};
            for (int t = w.len + rank * rows + row; t < a.n_tokens; t += ranks * rows) {
                if (g.grad_v != nullptr) store8<VEC>(static_cast<InT *>(g.grad_v) + row_of(g.grad_v_stride, w, t) + c0, n, zero);
                if (CHAN && g.grad_g != nullptr) store8<VEC>(g.grad_g + row_of(g.grad_g_stride, w, t) + c0, n, zero);
                if (!CHAN && c0 == 0 && g.grad_g != nullptr) g.grad_g[row_of(g.grad_g_stride, w, t)] = 0.0f;
                if (c0 == 0 && g.grad_beta != nullptr) g.grad_beta[row_of(g.grad_beta_stride, w, t)] = 0.0f;
            }
        }
    }
    __syncthreads();
    if (ranks > 1) cluster.sync();                   // no CTA leaves while another may still store to it
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


// A launch of `ranks` CTAs a unit as clusters.  `most`: the dynamic shared
// memory that the kernel may ask for at all.
template <auto kernel, typename... V>
cudaError_t launch_clusters(int units, int ranks, int smem, int most, cudaStream_t s, const V &...args) {
    const cudaError_t e = opt_in_smem<kernel>(most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units * (unsigned)ranks);
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The tensor map of one tensor's rows.  A dimension of one entry gets a stride
// of one row; the others are positive (the callers see to that).
cudaError_t row_map(RowMap *m, const void *p, const lq_strides &s, const lq_scan_config &c, int tokens, int dtype,
                    int chunk) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t size = dtype == LQ_DTYPE_BF16 ? 2 : 4, row = (cuuint64_t)c.d * size;
    const cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.heads, (cuuint64_t)c.batch, (cuuint64_t)tokens};
    const cuuint64_t strides[3] = {c.heads > 1 ? (cuuint64_t)s.head * size : row,
                                   c.batch > 1 ? (cuuint64_t)s.seq * size : row,
                                   tokens > 1 ? (cuuint64_t)s.token * size : row};
    const cuuint32_t box[4] = {(cuuint32_t)c.d, 1, 1, (cuuint32_t)std::min(chunk, kMostBox)};
    const cuuint32_t each[4] = {1, 1, 1, 1};
    const CUresult r = encode(&m->map, dtype == LQ_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                              4, const_cast<void *>(p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// CTAs that share a unit: the number that takes the fewest steps one after
// another, counting two steps' time for the start and end of each round of CTAs
// on the device.
int ranks_of(int units, long long tokens, int chunk, int ctas_per_sm) {
    const long long slots = (long long)ctas_per_sm * sm_count();
    int best = 1;
    long long least = -1;
    for (int r = 1; r <= kMostRanks; ++r) {
        const long long rounds = ((long long)units * r + slots - 1) / slots, stride = (long long)r * chunk;
        const long long cost = rounds * ((tokens + stride - 1) / stride + 2);
        if (least < 0 || cost < least) {
            least = cost;
            best = r;
        }
    }
    return best;
}

// Shared memory of a kernel whose stages are S: what a call needs, the most
// that any d wants, and the CTAs that then fit an SM (registers leave two).
struct Room {
    int smem, most, ctas;
};
template <typename S>
Room room_of(int d, int run) {
    auto bytes = [run](int dd) { return S(kWorkers / row_lanes(dd) * run, dd).bytes(kMostRanks); };
    Room r{bytes(d), 0, 1};
    for (int dd = 8; dd <= 256; dd *= 2) r.most = std::max(r.most, bytes(dd));
    if (2 * (r.smem + 2048) <= 228 * 1024) r.ctas = 2;
    return r;
}

}  // namespace

cudaError_t launch_scan_forward(const lq_scan_config &c, const lq_scan_args &a, bool vec, cudaStream_t s) {
    const int units = c.batch * c.heads, lanes = row_lanes(c.d), every = scan_checkpoint_tokens(c);
    return by_variant(c, vec, [&](auto k) {
        using K = decltype(k);
        using In = typename K::In;
        if (a.n_tokens <= 4) {
            const long long threads = (long long)units * lanes;
            scan_rows_kernel<In, typename K::Out, K::CHAN, K::VEC>
                <<<(unsigned)((threads + kRowsThreads - 1) / kRowsThreads), kRowsThreads, 0, s>>>(a, c.heads, units, c.d,
                                                                                                 lanes, every);
            return cudaGetLastError();
        }
        constexpr int run = forward_run(sizeof(In) == 2, K::CHAN);
        const Room room = room_of<ForwardSpace<In, K::CHAN>>(c.d, run);
        const int chunk = kWorkers / lanes * run, ranks = ranks_of(units, a.n_tokens, chunk, room.ctas);
        RowMap v = {}, g = {};
        if (K::VEC) {
            cudaError_t e = row_map(&v, a.v, a.v_stride, c, a.n_tokens, c.in_dtype, chunk);
            if (e == cudaSuccess && K::CHAN) e = row_map(&g, a.g, a.g_stride, c, a.n_tokens, LQ_DTYPE_F32, chunk);
            if (e != cudaSuccess) return e;
        }
        return launch_clusters<scan_forward_kernel<In, typename K::Out, K::CHAN, K::VEC>>(
            units, ranks, room.smem, room.most, s, a, v, g, c.heads, units, c.d, lanes, every);
    });
}

cudaError_t launch_scan_backward(const lq_scan_config &c, const lq_scan_args &a, const lq_scan_grads &g, bool vec,
                                 cudaStream_t s) {
    const int units = c.batch * c.heads, lanes = row_lanes(c.d);
    return by_variant(c, vec && a.n_tokens > 0, [&](auto k) {
        using K = decltype(k);
        using In = typename K::In;
        using Out = typename K::Out;
        constexpr int run = backward_run(sizeof(In) == 2, K::CHAN);
        const Room room = room_of<BackwardSpace<In, Out, K::CHAN>>(c.d, run);
        const int chunk = kWorkers / lanes * run, ranks = ranks_of(units, a.n_tokens, chunk, room.ctas);
        RowMap v = {}, y = {}, gate = {};
        if (K::VEC) {
            cudaError_t e = row_map(&v, a.v, a.v_stride, c, a.n_tokens, c.in_dtype, chunk);
            if (e == cudaSuccess && g.grad_out != nullptr)
                e = row_map(&y, g.grad_out, g.grad_out_stride, c, a.n_tokens, c.out_dtype, chunk);
            if (e == cudaSuccess && K::CHAN) e = row_map(&gate, a.g, a.g_stride, c, a.n_tokens, LQ_DTYPE_F32, chunk);
            if (e != cudaSuccess) return e;
        }
        return launch_clusters<scan_backward_kernel<In, Out, K::CHAN, K::VEC>>(
            units, ranks, room.smem, room.most, s, a, g, v, y, gate, c.heads, units, c.d, lanes);
    });
}

}  // namespace lq

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
//   Pass one: each row runs its R tokens from zero.
//   The rows' maps are composed over the CTA and, through distributed shared
//     memory, over the cluster, so that each row gets the true state before its
//     tokens.
//   Pass two: the results from there.
// One warp, the loader, keeps the tokens of up to three steps in shared memory.
//   Forward, rows compose their maps over a warp by shuffles and a composer warp
// does the rest.  Pass two runs the row's tokens, still in shared memory, again,
// and comes after pass one of the next step, so that the composer's chain of
// latencies (about 1500 cycles in a cluster) costs no time.  Without that, every
// warp waiting for the maps of its own step, a step of 64 KB of an SM took 6400
// cycles (8200 in a cluster) where the memory needs 5800.  Measured, BF16, one
// gate a head: 64 x 32 heads x 128 x 2048 tokens 365 us (0.93 of the rate of a
// plain copy), one sequence of 65536 tokens 220 us (0.77; 256 CTAs).
//   Backward there are twice the results a token and the instructions count:
// pass one keeps its local results in registers, a worker thread composes a
// channel, and pass two corrects the local results by what enters the row; the
// two CTAs of an SM cover each other's waits.  Measured: 8 x 32 heads x 128 x
// 8192 tokens 346 us (0.72 of the copy rate), from 630 with the tokens run again.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "lq_ops.h"
#include "lq_kernels.h"
#include "lq_vec8.cuh"

namespace cg = cooperative_groups;

namespace lq {

// Warps that run tokens, beside the composer and the loader.  Forward, three
// stages of tokens and two steps' maps of two CTAs just fit an SM's shared
// memory; backward, two CTAs of eight warps leave a thread 128 registers.
constexpr int forward_warps(bool chan) { return chan ? 6 : 7; }
constexpr int kBackwardWarps = 6;
constexpr int kStages = 3;                       // steps whose tokens are in shared memory
constexpr int kMostRanks = 8;                    // CTAs of a cluster (the portable size)
constexpr int kRowsThreads = 256;                // of the kernel for a few tokens

// Consecutive tokens that a row of lanes takes in a step: as many as the two
// CTAs' stages have room for.
constexpr int forward_run(bool bf16, bool chan) { return chan ? (bf16 ? 3 : 2) : bf16 ? 8 : 4; }
constexpr int backward_run(bool bf16, bool chan) { return bf16 && !chan ? 4 : 2; }

// (a multiple of every forward_run of the same types, so that a checkpoint
// falls on the start of a row's tokens there)
int scan_checkpoint_tokens(const lq_scan_config &c) {
    return 32 * kBackwardWarps / row_lanes(c.d) * backward_run(c.in_dtype == LQ_DTYPE_BF16, c.gate == LQ_GATE_CHANNEL);
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

// The gates of a thread's eight channels: four pairs, or one value for all.
template <bool CHAN>
struct Gates {
    float2 a[4];
    __device__ __forceinline__ float2 operator[](int i) const { return a[i]; }
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = make_float2(x, x);
    }
    template <bool VEC>
    __device__ __forceinline__ void load(const float *p, int n) {   // log gates, as they lie in memory
        Raw8<float> r;
        load8<VEC>(p, n, r);
        widen8(r, a);
    }
    __device__ __forceinline__ void exponentiate() {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = gates_of(a[i]);
    }
    __device__ __forceinline__ void times(const Gates &b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = mul2(a[i], b.a[i]);
    }
    // the gates `o` lanes before (after) this one
    __device__ __forceinline__ Gates before(int o) const {
        Gates r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.a[i] = make_float2(__shfl_up_sync(0xffffffffu, a[i].x, o), __shfl_up_sync(0xffffffffu, a[i].y, o));
        return r;
    }
    __device__ __forceinline__ Gates after(int o) const {
        Gates r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.a[i] = make_float2(__shfl_down_sync(0xffffffffu, a[i].x, o), __shfl_down_sync(0xffffffffu, a[i].y, o));
        return r;
    }
};
template <>
struct Gates<false> {
    float a;
    __device__ __forceinline__ float2 operator[](int) const { return make_float2(a, a); }
    __device__ __forceinline__ void fill(float x) { a = x; }
    template <bool VEC>
    __device__ __forceinline__ void load(const float *p, int) {
        a = __ldg(p);
    }
    __device__ __forceinline__ void exponentiate() { a = gate_of(a); }
    __device__ __forceinline__ void times(const Gates &b) { a *= b.a; }
    __device__ __forceinline__ Gates before(int o) const { return Gates{__shfl_up_sync(0xffffffffu, a, o)}; }
    __device__ __forceinline__ Gates after(int o) const { return Gates{__shfl_down_sync(0xffffffffu, a, o)}; }
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
struct RowMap {
    CUtensorMap map;
};
// Tokens of a box: the step's tokens of a CTA (three or seven times a power of
// two), halved until a box may have them (256).
__host__ __device__ inline int box_of(int tokens) {
    while (tokens > 256) tokens /= 2;
    return tokens;
}

__device__ __forceinline__ void bring_boxes(unsigned char *base, const RowMap &m, const Unit &w, int t_first, int tokens,
                                            int row_bytes, uint64_t *bar) {
    const int box = box_of(tokens);
#pragma unroll 1
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
#pragma unroll 1
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
// Eight channels of a token in shared memory (where fewer exist, what follows
// them is read too), as they lie there or as pairs.
template <typename T>
__device__ __forceinline__ void read_shared(const unsigned char *base, int pitch, int token, int c0, Raw8<T> &r) {
    const T *q = reinterpret_cast<const T *>(base) + token * pitch + c0;
    if constexpr (sizeof(T) == 2) {
        r.w = *reinterpret_cast<const uint4 *>(q);
    } else {
        r.lo = reinterpret_cast<const float4 *>(q)[0];
        r.hi = reinterpret_cast<const float4 *>(q)[1];
    }
}
template <typename T>
__device__ __forceinline__ void read_shared(const unsigned char *base, int pitch, int token, int c0, float2 *x) {
    Raw8<T> r;
    read_shared(base, pitch, token, c0, r);
    widen8(r, x);
}
// Its first n channels (rounded up to 16 bytes) set to zero.
template <typename T>
__device__ __forceinline__ void clear_shared(unsigned char *base, int pitch, int token, int c0, int n) {
    const float2 zero[4] = {};
    store8<true>(reinterpret_cast<T *>(base) + token * pitch + c0, n, zero);
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
// A named barrier of some of a CTA's warps.
template <int ID, int THREADS>
__device__ __forceinline__ void meet() {
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// The stages of one CTA in shared memory: up to three tensors, then a pair (log
// gate or alpha, beta) a token, then (backward) the state before the tokens.
// NW: workers' warps; B0, B1, B2: bytes of a channel of the tensors.
template <int NW_, int B0, int B1, int B2, bool CHAN, bool BACK>
struct Space {
    static constexpr int NW = NW_;
    int tokens, dp, rows;
    __host__ __device__ Space(int d, int lanes, int run)
        : tokens(32 * NW / lanes * run), dp((d + 7) / 8 * 8), rows(32 * NW / lanes) {}
    __host__ __device__ static int up(int bytes) { return (bytes + 127) / 128 * 128; }
    // where a tensor starts (a tensor map's copies want 128 bytes), and what follows them
    __host__ __device__ int second() const { return up(tokens * dp * B0); }
    __host__ __device__ int third() const { return second() + up(tokens * dp * B1); }
    __host__ __device__ int scalars() const { return third() + up(tokens * dp * B2); }
    __host__ __device__ int mark() const { return up(scalars() + tokens * 8); }
    __host__ __device__ int stage() const { return mark() + (BACK ? up(dp * 4) : 0); }
    // In floats, the maps of a step.  Forward, of the warps: H [NW][dp], A [NW][dp
    // or 4].  Backward, of the rows: H, E [rows][dp], A, B [rows][dp or 1] (A:
    // the gates' product from the group's first row on, B: from its last).
    __host__ __device__ int gate_row() const { return CHAN ? dp : BACK ? 1 : 4; }
    __host__ __device__ int E() const { return rows * dp; }
    __host__ __device__ int A() const { return BACK ? 2 * rows * dp : NW * dp; }
    __host__ __device__ int B() const { return A() + rows * gate_row(); }
    __host__ __device__ int map() const { return BACK ? (B() + rows * gate_row() + 3) / 4 * 4 : A() + NW * gate_row(); }
    __host__ __device__ int maps() const { return (BACK ? 1 : 2) * map(); }
    // a CTA's map as its peers see it: H or E [dp], then A [dp, or 4 equal]
    __host__ __device__ int peer() const { return dp + (CHAN ? dp : 4); }
    __host__ __device__ int bytes(int ranks) const {
        return kStages * stage() + maps() * 4 + (ranks > 1 ? 2 * ranks * peer() * 4 : 0);
    }
};

// Barriers of a CTA.
struct Bars {
    uint64_t full[kStages];      // a stage's tokens are there
    uint64_t empty[kStages];     // the workers' warps have read a stage
    uint64_t peer[2];            // the cluster's maps of a step are here
};
__device__ __forceinline__ void init_bars(Bars &b, int workers) {
    for (int i = 0; i < kStages; ++i) {
        mbar_init(&b.full[i], 1 + 32);
        mbar_init(&b.empty[i], workers);
    }
    mbar_init(&b.peer[0], 1);
    mbar_init(&b.peer[1], 1);
    fence_mbar_init();
}

// Every wait is bounded.  After one that ran out (tokens or a peer's map never
// came) the later ones are short, and what came too late or depends on it is
// NaN: forward the tokens from the late ones on, backward the late tokens, what
// their gradient reaches before them and grad_g behind them in the same step.
constexpr long long kLateCycles = 200000;
__device__ __forceinline__ long long budget_of(bool alive) { return alive ? kWaitBudgetCycles : kLateCycles; }
// Before the CTA's end: late copies, which still write to its stages, get time to land.
__device__ __forceinline__ void linger() {
    const long long t0 = clock64();
    while (clock64() - t0 < kLateCycles) {}
}

__device__ __forceinline__ void fill_nan(float2 (&x)[4], float2 (&y)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = y[c] = make_float2(nanf(""), nanf(""));
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
// Store values in a peer's shared memory and count their bytes at the peer's barrier.
__device__ __forceinline__ void peer_store(uint32_t dst, float x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
                 "r"(__float_as_uint(x)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t dst, float4 x, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "r"(__float_as_uint(x.x)), "r"(__float_as_uint(x.y)), "r"(__float_as_uint(x.z)),
                 "r"(__float_as_uint(x.w)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool peer_wait(uint64_t *bar, uint32_t parity, long long budget_cycles) {
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
        if (clock64() - t0 > budget_cycles) return false;
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

// The forward composer's work.  A lane owns channels 4 q .. 4 q + 3 for q = lane
// and lane + 32.
template <int NW, bool CHAN>
struct Composer {
    float *peers;            // [2][ranks][H dp, A (dp, or 4 equal)]
    uint64_t *bars;          // [2]
    int ranks, rank, dp;
    float4 carry[2];         // the state before the step
    bool alive = true;       // until a wait runs out

    __device__ __forceinline__ int owned() const { return (dp / 4 - (int)(threadIdx.x % 32) + 31) / 32; }
    __device__ __forceinline__ Map4 map(const float *H, const float *A, int k, int q) const {
        return Map4{*reinterpret_cast<const float4 *>(A + k * (CHAN ? dp : 4) + (CHAN ? 4 * q : 0)),
                    *reinterpret_cast<const float4 *>(H + k * dp + 4 * q)};
    }
    // Replace the warps' maps of `step` by the states before their tokens.  Every
    // CTA stores its map in all CTAs and waits at its own barrier for everybody's:
    // unlike a cluster barrier this waits for no store to global memory.  A CTA
    // stores its map of step s + 2 only after it has those of s + 1, whose
    // senders had read step s.
    __device__ __forceinline__ void run(int step, float *H, const float *A) {
        const int lane = threadIdx.x % 32, p = step & 1, size = dp + (CHAN ? dp : 4);
        if (ranks > 1) {
            if (lane == 0) mbar_arrive_expect_tx(bars + p, (uint32_t)(ranks * size * 4));
            for (int j = 0; j < owned(); ++j) {
                const int q = lane + 32 * j;
                Map4 all = map(H, A, 0, q);
#pragma unroll
                for (int k = 1; k < NW; ++k) {
                    const Map4 m = map(H, A, k, q);
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
            alive = peer_wait(bars + p, (step >> 1) & 1, budget_of(alive)) && alive;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j >= owned()) break;
            const int q = lane + 32 * j;
            float4 x = carry[j];
            if (ranks > 1) {
                if (!alive) carry[j] = four(nanf(""));
#pragma unroll
                for (int r = 0; r < kMostRanks; ++r) {
                    if (r >= ranks) break;
                    const float *m = peers + (p * ranks + r) * size;
                    if (r == rank) x = carry[j];
                    carry[j] = apply(map(m, m + dp, 0, q), carry[j]);
                }
            }
            // four maps are read before the first is replaced: one after another
            // their latencies would add up
#pragma unroll
            for (int k = 0; k < NW; k += 4) {
                Map4 m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (k + i < NW) m[i] = map(H, A, k + i, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (k + i >= NW) break;
                    *reinterpret_cast<float4 *>(H + (k + i) * dp + 4 * q) = x;
                    x = apply(m[i], x);
                }
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
    constexpr int AHEAD = 4;         // tokens in flight
    for (int t0 = 0; t0 < w.len; t0 += AHEAD) {
        Raw8<InT> raw[AHEAD];
        Gates<CHAN> gate[AHEAD];
        float beta[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int t = t0 + i;
            if (t >= w.len) break;
            load8<VEC>(static_cast<const InT *>(a.v) + row_of(a.v_stride, w, t) + c0, n, raw[i]);
            gate[i].template load<VEC>(a.g + row_of(a.g_stride, w, t) + (CHAN ? c0 : 0), n);
            beta[i] = a.beta != nullptr ? __ldg(a.beta + row_of(a.beta_stride, w, t)) : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int t = t0 + i;
            if (t >= w.len) break;
            if (a.checkpoints != nullptr && t % every == 0)
                store8<VEC>(a.checkpoints + (int64_t)(t / every) * units * d + state, n, h);
            gate[i].exponentiate();
            float2 v[4];
            widen8(raw[i], v);
#pragma unroll
            for (int c = 0; c < 4; ++c) h[c] = fma2(gate[i][c], h[c], mul2(make_float2(beta[i], beta[i]), v[c]));
            if (a.out != nullptr) store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, h);
        }
    }
    if (a.h_last != nullptr) store8<VEC>(a.h_last + state, n, h);
    if (a.zero_past && a.out != nullptr) {
        const float2 zero[4] = {};
        for (int t = w.len; t < a.n_tokens; ++t)
            store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, zero);
    }
}

template <typename InT, bool CHAN>
using ForwardSpace = Space<forward_warps(CHAN), (int)sizeof(InT), CHAN ? 4 : 0, 0, CHAN, false>;

template <typename InT, typename OutT, bool CHAN, bool VEC, int D_>
__global__ void __launch_bounds__(32 * forward_warps(CHAN) + 64, 2)
    scan_forward_kernel(lq_scan_args a, const __grid_constant__ RowMap map_v, const __grid_constant__ RowMap map_g,
                        int heads, int units, int any_d, int every) {
    const int d = D_ > 0 ? D_ : any_d, lanes = row_lanes(d);
    constexpr int R = forward_run(sizeof(InT) == 2, CHAN);
    constexpr int NW = forward_warps(CHAN);
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Bars bars;
    const int rows = 32 * NW / lanes, chunk = rows * R;
    const ForwardSpace<InT, CHAN> space(d, lanes, R);
    const int dp = space.dp, pitch = VEC ? d : dp;
    const int gates_at = space.second();                            // the log gates of channels in a stage
    float *maps = reinterpret_cast<float *>(smem + kStages * space.stage());
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) init_bars(bars, NW);
    __syncthreads();
    if (ranks > 1) cluster.sync();

    const Unit w = unit_of(a, heads, blockIdx.x / ranks);
    const int stride = ranks * chunk, steps = (w.len + stride - 1) / stride;
    const InT *pv = static_cast<const InT *>(a.v) + row_of(a.v_stride, w, 0);
    const float *pg = a.g + row_of(a.g_stride, w, 0);
    const float *pb = a.beta != nullptr ? a.beta + row_of(a.beta_stride, w, 0) : nullptr;

    float4 last[2];                        // the composer's: the last state
    if (warp == NW + 1) {                  // the loader
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
#pragma unroll 1
            for (int i = lane; i < live; i += 32) {
                if (!CHAN) cp_async4(&sc[i].x, pg + (t_cta + i) * a.g_stride.token);
                if (pb != nullptr) cp_async4(&sc[i].y, pb + (t_cta + i) * a.beta_stride.token);
            }
            cp_async_arrive(full);
        }
    } else if (warp == NW) {               // the composer
        Composer<NW, CHAN> composer{maps + space.maps(), bars.peer, ranks, rank, dp};
        const int64_t state = (int64_t)w.u * d;
        for (int j = 0; j < 2; ++j) {
            const int c = 4 * (lane + 32 * j);
            composer.carry[j] = a.h0 != nullptr ? load4(a.h0 + state + c, d - c) : four(0.0f);
        }
        for (int s = 0; s < steps; ++s) {
            float *H = maps + (s & 1) * space.map();
            meet<1, 32 * NW + 32>();
            composer.run(s, H, H + NW * dp);
        }
        meet<1, 32 * NW + 32>();
        last[0] = composer.carry[0];
        last[1] = composer.carry[1];
    } else {                                         // the workers
        const int in_row = lane & (lanes - 1), c0 = in_row * 8, row = tid / lanes;
        const bool on = c0 < d;
        const int n = on ? min(8, d - c0) : 0, cr = on ? c0 : 0;     // (lanes past d run with others' channels)
        auto bring = [&](int s, int stage) {
            const int t_row = s * stride + rank * chunk + row * R, live = min(max(w.len - t_row, 0), R);
            unsigned char *base = smem + stage * space.stage();
            if (!on) return;
            bring_row(base, pitch, pv + c0 + t_row * a.v_stride.token, a.v_stride.token, row * R, live, c0, n);
            if (CHAN) bring_row(base + gates_at, pitch, pg + c0 + t_row * a.g_stride.token, a.g_stride.token, row * R, live, c0, n);
        };
        if (!VEC)
            for (int s = 0; s < kStages; ++s) bring(s, s);
        bool alive = true;           // until a wait runs out
        Turn one, two;               // the stages of pass one and pass two
        // the row's first token is past_mark tokens past checkpoint `mark`, step after step
        const int stride_marks = stride / every, stride_past = stride - stride_marks * every;
        int mark = (rank * chunk + row * R) / every, past_mark = rank * chunk + row * R - mark * every;
        Gates<CHAN> A_before;        // of the step whose pass two is due: the map of its warp's rows before this one
        float2 H_before[4];
        bool alive_before = true;    // (as the maps: of that step)
        for (int s = 0; s <= steps; ++s) {
            Gates<CHAN> A;
            float2 H[4] = {};
            A.fill(1.0f);
            if (s < steps) {
                const int live = min(max(w.len - (s * stride + rank * chunk + row * R), 0), R);
                unsigned char *base = smem + one.stage * space.stage();
                float2 *sc = reinterpret_cast<float2 *>(base + space.scalars()) + row * R;
                float *sH = maps + (s & 1) * space.map(), *sA = sH + NW * dp;
                alive = mbar_wait(&bars.full[one.stage], one.parity, budget_of(alive)) && alive;
                // each gate is raised once, by one lane of its row; past the end it is 1, and beta 0
                for (int i = in_row; i < R; i += lanes) {
                    if (!CHAN) sc[i].x = i < live ? gate_of(sc[i].x) : 1.0f;
                    if (i >= live) sc[i].y = 0.0f;
                    else if (pb == nullptr) sc[i].y = 1.0f;
                }
                __syncwarp();
                if (live < R && on) {                // what lies past the sequence's end is nothing
#pragma unroll 1
                    for (int i = live; i < R; ++i) {
                        clear_shared<InT>(base, pitch, row * R + i, c0, n);
                        if (CHAN) clear_shared<float>(base + gates_at, pitch, row * R + i, c0, n);
                    }
                    fence_proxy_async_smem();
                }
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float2 gb = sc[i];
                    Gates<CHAN> gate;
                    if constexpr (CHAN) {            // raised once: pass two finds alpha in its place
                        float *g = reinterpret_cast<float *>(base + gates_at) + (row * R + i) * pitch + cr;
                        read_shared(g, gate.a);
                        gate.exponentiate();
                        if (on) store8<true>(g, n, gate.a);
                    } else {
                        gate.fill(gb.x);
                    }
                    float2 v[4];
                    read_shared<InT>(base, pitch, row * R + i, cr, v);
#pragma unroll
                    for (int c = 0; c < 4; ++c) H[c] = fma2(gate[c], H[c], mul2(make_float2(gb.y, gb.y), v[c]));
                    A.times(gate);
                }
                if (!alive) fill_nan(H, H);          // the row's map, and with it every later state
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
                    else if (c0 == 0) *reinterpret_cast<float4 *>(sA + warp * 4) = four(A.a);
                }
                A = A.before(lanes);
#pragma unroll
                for (int c = 0; c < 4; ++c) H[c] = pair_before(H[c], lanes);
                one.next();
            }
            meet<1, 32 * NW + 32>();          // the maps of step s are there, and the states of step s - 1
            if (s > 0) {
                const int t_row = (s - 1) * stride + rank * chunk + row * R, live = min(max(w.len - t_row, 0), R);
                const unsigned char *base = smem + two.stage * space.stage();
                const float2 *sc = reinterpret_cast<const float2 *>(base + space.scalars()) + row * R;
                float2 h[4];
                read_shared(maps + ((s - 1) & 1) * space.map() + warp * dp + cr, h);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (lane >= lanes) h[c] = fma2(A_before[c], h[c], H_before[c]);
                if (!alive_before) fill_nan(h, h);
                if (a.checkpoints != nullptr) {
                    if (on && live > 0 && past_mark == 0)
                        store8<VEC>(a.checkpoints + ((int64_t)mark * units + w.u) * d + c0, n, h);
                    mark += stride_marks;
                    past_mark += stride_past;
                    if (past_mark >= every) {
                        past_mark -= every;
                        ++mark;
                    }
                }
                if (a.out != nullptr) {
                    OutT *po = static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t_row) + c0;
#pragma unroll
                    for (int i = 0; i < R; ++i, po += a.out_stride.token) {
                        const float2 gb = sc[i];
                        Gates<CHAN> gate;
                        if constexpr (CHAN) read_shared<float>(base + gates_at, pitch, row * R + i, cr, gate.a);
                        else gate.fill(gb.x);
                        float2 v[4];
                        read_shared<InT>(base, pitch, row * R + i, cr, v);
#pragma unroll
                        for (int c = 0; c < 4; ++c) h[c] = fma2(gate[c], h[c], mul2(make_float2(gb.y, gb.y), v[c]));
                        if (i < live && on) store8<VEC>(po, n, h);
                    }
                }
                if (!VEC && s - 1 + kStages < steps) bring(s - 1 + kStages, two.stage);
                if (CHAN) fence_proxy_async_smem();  // alpha was written where the next copy lands
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.empty[two.stage]);
                two.next();
            }
            A_before = A;
            alive_before = alive;
#pragma unroll
            for (int c = 0; c < 4; ++c) H_before[c] = H[c];
        }
        if (!alive) linger();
        if (a.zero_past && a.out != nullptr && on) {
            const float2 zero[4] = {};
#pragma unroll 1
            for (int t = w.len + rank * rows + row; t < a.n_tokens; t += ranks * rows)
                store8<VEC>(static_cast<OutT *>(a.out) + row_of(a.out_stride, w, t) + c0, n, zero);
        }
    }
    __syncthreads();
    if (ranks > 1) cluster.sync();                   // no CTA leaves while another may still store to it
    // only now: h_last may be h0, which every CTA of the cluster reads
    if (warp == NW && rank == 0 && a.h_last != nullptr)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = 4 * (lane + 32 * j);
            store4(a.h_last + (int64_t)w.u * d + c, d - c, last[j]);
        }
}

// ------------------------------------------------------------------ backward

// Sums of N values over the lanes of a row, N a power of two up to the lanes:
// at each of the first levels a lane hands half of its values over, so a value
// costs about one shuffle; a lane is left with the sum of one value.
template <int N>
__device__ __forceinline__ float sum_row(float (&x)[N], int lanes, int lane) {
    int o = lanes / 2;
#pragma unroll
    for (int m = N / 2; m >= 1; m /= 2, o /= 2) {
        const bool high = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float keep = high ? x[i + m] : x[i], give = high ? x[i] : x[i + m];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float s = x[0];
    for (; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
// The value whose sum sum_row leaves with a lane.
template <int N>
__device__ __forceinline__ int sum_of(int lanes, int lane) {
    int o = lanes / 2, at = 0;
#pragma unroll
    for (int m = N / 2; m >= 1; m /= 2, o /= 2) at += (lane & o) != 0 ? m : 0;
    return at;
}

template <typename InT, typename OutT, bool CHAN>
using BackwardSpace = Space<kBackwardWarps, (int)sizeof(InT), (int)sizeof(OutT), CHAN ? 4 : 0, CHAN, true>;

// Steps run from the sequence's end.  Pass one runs a row's tokens forwards from
// zero (alpha h, H) and backwards from zero (D, E); the composer starts a step's
// states from the CTA's checkpoint, so only the gradient's maps cross the
// cluster.  With h what enters the row from before and X from behind, P_t the
// product of its gates up to t and Q_t of those after t, pass two has
//     alpha_t h_{t-1} = P_t h + its local value,   D_t = Q_t X + its local value.
template <typename InT, typename OutT, bool CHAN, bool VEC, int D_>
__global__ void __launch_bounds__(32 * kBackwardWarps + 32, D_ > 0 ? 2 : 1)
    scan_backward_kernel(lq_scan_args a, lq_scan_grads g, const __grid_constant__ RowMap map_v,
                         const __grid_constant__ RowMap map_y, const __grid_constant__ RowMap map_g, int heads, int units,
                         int any_d) {
    const int d = D_ > 0 ? D_ : any_d, lanes = row_lanes(d);
    constexpr int R = backward_run(sizeof(InT) == 2, CHAN);
    constexpr int NW = kBackwardWarps;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Bars bars;
    const int rows = 32 * NW / lanes, chunk = rows * R;
    const BackwardSpace<InT, OutT, CHAN> space(d, lanes, R);
    const int dp = space.dp, pitch = VEC ? d : dp;
    const int y_at = space.second(), gates_at = space.third();      // grad_out, and the log gates of channels, in a stage
    float *maps = reinterpret_cast<float *>(smem + kStages * space.stage());
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    if (tid == 0) init_bars(bars, NW);
    __syncthreads();
    if (ranks > 1) cluster.sync();

    const Unit w = unit_of(a, heads, blockIdx.x / ranks);
    const int stride = ranks * chunk, steps = (w.len + stride - 1) / stride;
    auto first_of = [&](int s) { return (steps - 1 - s) * stride + rank * chunk; };     // this CTA's first token of a step
    const InT *pv = static_cast<const InT *>(a.v) + row_of(a.v_stride, w, 0);
    const OutT *py = g.grad_out != nullptr ? static_cast<const OutT *>(g.grad_out) + row_of(g.grad_out_stride, w, 0) : nullptr;
    const float *pg = a.g + row_of(a.g_stride, w, 0);
    const float *pb = a.beta != nullptr ? a.beta + row_of(a.beta_stride, w, 0) : nullptr;

    // A worker composes channel tid (and tid + 32 NW where there are as many);
    // where half of the threads are enough for the states, the other half
    // composes the gradients.
    constexpr int NC = D_ > 0 && D_ <= 32 * NW ? 1 : 2;
    const int e_from = dp <= 16 * NW ? 16 * NW : 0;
    float carry[NC];                 // what enters a step from behind
    if (warp == NW) {                                // the loader
        const int v_bytes = d * (int)sizeof(InT), y_bytes = py != nullptr ? d * (int)sizeof(OutT) : 0;
        auto live_of = [&](int s) { return min(max(w.len - first_of(s), 0), chunk); };
        auto issue = [&](int s, int stage) {         // the copies of a step, one group of them
            const int t_cta = first_of(s), live = live_of(s);
            unsigned char *base = smem + stage * space.stage();
            uint64_t *full = &bars.full[stage];
            if (lane == 0) {
                const bool any = VEC && live > 0;
                mbar_arrive_expect_tx(full, any ? (uint32_t)(chunk * (v_bytes + y_bytes + (CHAN ? d * 4 : 0))) : 0u);
                if (any) {
                    bring_boxes(base, map_v, w, t_cta, chunk, v_bytes, full);
                    if (py != nullptr) bring_boxes(base + y_at, map_y, w, t_cta, chunk, y_bytes, full);
                    if (CHAN) bring_boxes(base + gates_at, map_g, w, t_cta, chunk, d * 4, full);
                }
            }
            float2 *sc = reinterpret_cast<float2 *>(base + space.scalars());
#pragma unroll 1
            for (int j = lane; j < live; j += 32) {
                if (!CHAN) cp_async4(&sc[j].x, pg + (t_cta + j) * a.g_stride.token);
                if (pb != nullptr) cp_async4(&sc[j].y, pb + (t_cta + j) * a.beta_stride.token);
            }
            float *mark = reinterpret_cast<float *>(base + space.mark());
            const float *from = a.checkpoints + ((int64_t)(t_cta / chunk) * units + w.u) * d;
            if (live > 0)
#pragma unroll 1
                for (int c = lane; c < d; c += 32) cp_async4(mark + c, from + c);
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Once a step's copies have landed its gates are raised and it is
        // announced, before the loader waits for the workers to leave a stage.
        Turn now, next, left;
        if (steps > 0) issue(0, 0);
        if (steps > 1) issue(1, 1);
        next.next();
        for (int s = 0; s < steps; ++s, now.next()) {
            if (s + 1 < steps) asm volatile("cp.async.wait_group 1;" ::: "memory");      // step s + 1 may be on its way
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            float2 *sc = reinterpret_cast<float2 *>(smem + now.stage * space.stage() + space.scalars());
#pragma unroll 1
            for (int j = lane, live = live_of(s); j < chunk; j += 32) {      // (the lane's own copies)
                if (!CHAN) sc[j].x = j < live ? gate_of(sc[j].x) : 1.0f;     // past the end: 1, and beta 0
                if (j >= live) sc[j].y = 0.0f;
                else if (pb == nullptr) sc[j].y = 1.0f;
            }
            mbar_arrive(&bars.full[now.stage]);
            next.next();
            if (s + 2 < steps) {
                if (s + 2 >= kStages) {
                    if (!mbar_wait(&bars.empty[left.stage], left.parity, kWaitBudgetCycles)) break;
                    left.next();
                }
                issue(s + 2, next.stage);
            }
        }
    } else {                                         // the workers
        const int in_row = lane & (lanes - 1), c0 = in_row * 8, row = tid / lanes;
        const bool on = c0 < d;
        const int n = on ? min(8, d - c0) : 0, cr = on ? c0 : 0;     // (lanes past d run with others' channels)
        const int group = max(lanes, 8), in_group = lane & (group - 1), per_group = group / lanes;
        const int first = row & ~(per_group - 1), last = first + per_group - 1;      // rows of the group
        const int groups = 32 * NW / group, gate_row = space.gate_row(), peer = space.peer();
        float *peers = maps + space.maps();
        float *sH = maps, *sE = maps + space.E(), *sA = maps + space.A(), *sB = maps + space.B();
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

        // where the row's results go, step after step
        constexpr int N = CHAN ? R : 2 * R;          // sums over a token's channels: grad_beta, then grad_g
        const int t_start = first_of(0) + row * R;
        InT *gv = static_cast<InT *>(g.grad_v) + row_of(g.grad_v_stride, w, t_start) + c0;
        float *gg = g.grad_g + row_of(g.grad_g_stride, w, t_start) + c0;
        const int sum_index = sum_of<N>(lanes, lane), sum_token = sum_index % R;     // the sum that this lane is left with
        const bool is_beta = sum_index < R, writer = lanes >= N && (lane & (lanes / N - 1)) == 0;
        const lq_strides &sum_stride = is_beta ? g.grad_beta_stride : g.grad_g_stride;
        float *sum_at = is_beta ? g.grad_beta : g.grad_g;
        const bool puts = writer && sum_at != nullptr;
        sum_at += row_of(sum_stride, w, t_start + sum_token);
        const int64_t gv_step = stride * g.grad_v_stride.token, gg_step = stride * g.grad_g_stride.token,
                      sum_step = stride * sum_stride.token;

#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = tid - e_from + 32 * NW * j;
            carry[j] = c >= 0 && c < d && g.grad_last != nullptr ? g.grad_last[(int64_t)w.u * d + c] : 0.0f;
        }
        bool alive = true;           // until a wait runs out
        Turn turn;
        for (int s = 0; s < steps; ++s) {
            const int t_row = first_of(s) + row * R, live = min(max(w.len - t_row, 0), R);
            unsigned char *base = smem + turn.stage * space.stage();
            const float2 *sc = reinterpret_cast<const float2 *>(base + space.scalars()) + row * R;
            Gates<CHAN> P[R], Q[R], A, B;
            float2 ah[R][4], D[R][4], H[4] = {}, E[4] = {};
            A.fill(1.0f);
            B.fill(1.0f);
            alive = mbar_wait(&bars.full[turn.stage], turn.parity, budget_of(alive)) && alive;
            if (!alive) fill_nan(H, E);              // the row's results and its maps
            if (live < R && on) {                    // what lies past the sequence's end is nothing
#pragma unroll 1
                for (int i = live; i < R; ++i) {
                    clear_shared<InT>(base, pitch, row * R + i, c0, n);
                    clear_shared<OutT>(base + y_at, pitch, row * R + i, c0, n);     // (without grad_out too: whole pieces)
                    if (CHAN) clear_shared<float>(base + gates_at, pitch, row * R + i, c0, n);
                }
                fence_proxy_async_smem();
            }
            {
                Gates<CHAN> gate[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float2 gb = sc[i];
                    if constexpr (CHAN) {
                        read_shared<float>(base + gates_at, pitch, row * R + i, cr, gate[i].a);
                        gate[i].exponentiate();
                    } else {
                        gate[i].fill(gb.x);
                    }
                    float2 v[4];
                    read_shared<InT>(base, pitch, row * R + i, cr, v);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        ah[i][c] = mul2(gate[i][c], H[c]);
                        H[c] = fma2(make_float2(gb.y, gb.y), v[c], ah[i][c]);
                    }
                    A.times(gate[i]);
                    P[i] = A;
                }
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    float2 y[4] = {};
                    if (py != nullptr) read_shared<OutT>(base + y_at, pitch, row * R + i, cr, y);
                    Q[i] = B;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        D[i][c] = add2(y[c], E[c]);
                        E[c] = mul2(gate[i][c], D[i][c]);
                    }
                    B.times(gate[i]);
                }
            }
            for (int o = lanes; o < group; o *= 2) {
                const Gates<CHAN> ap = A.before(o), bp = B.after(o);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 hp = pair_before(H[c], o), ep = pair_after(E[c], o);
                    if (in_group >= o) H[c] = fma2(A[c], hp, H[c]);
                    if (in_group + o < group) E[c] = fma2(B[c], ep, E[c]);
                }
                if (in_group >= o) A.times(ap);
                if (in_group + o < group) B.times(bp);
            }
            if (on) {
                store8<true>(sH + row * dp + c0, 8, H);
                store8<true>(sE + row * dp + c0, 8, E);
                if constexpr (CHAN) {
                    store8<true>(sA + row * dp + c0, 8, A.a);
                    if (per_group > 1) store8<true>(sB + row * dp + c0, 8, B.a);
                } else if (c0 == 0) {
                    sA[row] = A.a;
                    sB[row] = B.a;
                }
            }
            meet<1, 32 * NW>();
            // The groups' H and E are replaced by what enters them.  A group's H and
            // A are its last row's, its E its first row's.  The cluster's maps cross
            // as Composer's do.
            const int step_h = per_group * dp, step_a = per_group * gate_row, p = s & 1;
            const float *A_last = sA + (per_group - 1) * gate_row;
            static_assert(NW % 3 == 0, "groups of rows in threes");
            if (ranks > 1) {         // this CTA's map to the cluster
                if (tid == e_from) mbar_arrive_expect_tx(bars.peer + p, (uint32_t)(ranks * (CHAN ? 2 * dp : dp + 1) * 4));
                const uint32_t at = smem_u32(peers + (p * ranks + rank) * peer), bar = smem_u32(bars.peer + p);
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const int c = tid - e_from + 32 * NW * j;
                    if (c < 0 || c >= dp) break;
                    const float *Ec = sE + c, *Ac = A_last + (CHAN ? c : 0);
                    float all_a = 1.0f, all_e = 0.0f;
#pragma unroll 1
                    for (int k = groups - 1; k >= 0; k -= 3) {
                        const float e0 = Ec[k * step_h], e1 = Ec[(k - 1) * step_h], e2 = Ec[(k - 2) * step_h];
                        const float a0 = Ac[k * step_a], a1 = Ac[(k - 1) * step_a], a2 = Ac[(k - 2) * step_a];
                        all_e = fmaf(a2, fmaf(a1, fmaf(a0, all_e, e0), e1), e2);
                        all_a *= a0 * a1 * a2;
                    }
#pragma unroll
                    for (int r = 0; r < kMostRanks; ++r) {
                        if (r >= ranks) break;
                        const uint32_t dst = peer_address(at, r), b = peer_address(bar, r);
                        peer_store(dst + c * 4, all_e, b);
                        if (CHAN || c == 0) peer_store(dst + (dp + c) * 4, all_a, b);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NC; ++j) {           // the states, from the CTA's checkpoint on
                const int c = tid + 32 * NW * j;
                if (c >= dp) break;
                float *Hc = sH + (per_group - 1) * dp + c;
                const float *Ac = A_last + (CHAN ? c : 0);
                float h = c < d ? reinterpret_cast<const float *>(base + space.mark())[c] : 0.0f;
#pragma unroll 1
                for (int k = 0; k < groups; k += 3) {            // (three are read before one is replaced)
                    const float h0 = Hc[k * step_h], h1 = Hc[(k + 1) * step_h], h2 = Hc[(k + 2) * step_h];
                    const float a0 = Ac[k * step_a], a1 = Ac[(k + 1) * step_a], a2 = Ac[(k + 2) * step_a];
                    Hc[k * step_h] = h;
                    h = fmaf(a0, h, h0);
                    Hc[(k + 1) * step_h] = h;
                    h = fmaf(a1, h, h1);
                    Hc[(k + 2) * step_h] = h;
                    h = fmaf(a2, h, h2);
                }
            }
#pragma unroll
            for (int j = 0; j < NC; ++j) {           // the gradients
                const int c = tid - e_from + 32 * NW * j;
                if (c < 0 || c >= dp) break;
                float *Ec = sE + c;
                const float *Ac = A_last + (CHAN ? c : 0);
                float x = carry[j];
                if (ranks > 1) {
                    alive = peer_wait(bars.peer + p, (s >> 1) & 1, budget_of(alive)) && alive;
                    if (!alive) carry[j] = nanf("");
#pragma unroll 1
                    for (int r = ranks - 1; r >= 0; --r) {
                        const float *m = peers + (p * ranks + r) * peer;
                        if (r == rank) x = carry[j];
                        carry[j] = fmaf(m[dp + (CHAN ? c : 0)], carry[j], m[c]);
                    }
                }
#pragma unroll 1
                for (int k = groups - 1; k >= 0; k -= 3) {
                    const float e0 = Ec[k * step_h], e1 = Ec[(k - 1) * step_h], e2 = Ec[(k - 2) * step_h];
                    const float a0 = Ac[k * step_a], a1 = Ac[(k - 1) * step_a], a2 = Ac[(k - 2) * step_a];
                    Ec[k * step_h] = x;
                    x = fmaf(a0, x, e0);
                    Ec[(k - 1) * step_h] = x;
                    x = fmaf(a1, x, e1);
                    Ec[(k - 2) * step_h] = x;
                    x = fmaf(a2, x, e2);
                }
                if (ranks == 1) carry[j] = x;
            }
            meet<1, 32 * NW>();      // what enters the groups of rows is there
            float2 h[4], x[4];
            read_shared(sH + last * dp + cr, h);
            read_shared(sE + first * dp + cr, x);
            if (per_group > 1) {     // the maps of the group's rows before and after this one
                if (row != first) {
                    Gates<CHAN> m;
                    float2 y[4];
                    if constexpr (CHAN) read_shared(sA + (row - 1) * dp + cr, m.a);
                    else m.fill(sA[row - 1]);
                    read_shared(sH + (row - 1) * dp + cr, y);
#pragma unroll
                    for (int c = 0; c < 4; ++c) h[c] = fma2(m[c], h[c], y[c]);
                }
                if (row != last) {
                    Gates<CHAN> m;
                    float2 y[4];
                    if constexpr (CHAN) read_shared(sB + (row + 1) * dp + cr, m.a);
                    else m.fill(sB[row + 1]);
                    read_shared(sE + (row + 1) * dp + cr, y);
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[c] = fma2(m[c], x[c], y[c]);
                }
                __syncwarp();        // the group's rows have read each other's maps
            }
            float sums[N];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float2 v[4], dv[4], dg[4], sb = {}, sg = {};
                read_shared<InT>(base, pitch, row * R + i, cr, v);
                const float beta = sc[i].y;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 Dt = fma2(Q[i][c], x[c], D[i][c]), aht = fma2(P[i][c], h[c], ah[i][c]);
                    dv[c] = mul2(make_float2(beta, beta), Dt);
                    if (CHAN) dg[c] = mul2(aht, Dt);
                    if (2 * c < n) {                 // (beyond an odd d the pair's second half is zero)
                        sb = fma2(v[c], Dt, sb);
                        if (!CHAN) sg = fma2(aht, Dt, sg);
                    }
                }
                sums[i] = sb.x + sb.y;
                if (!CHAN) sums[N - R + i] = sg.x + sg.y;
                if (on && i < live) {
                    if (g.grad_v != nullptr) store8<VEC>(gv + i * g.grad_v_stride.token, n, dv);
                    if (CHAN && g.grad_g != nullptr) store8<VEC>(gg + i * g.grad_g_stride.token, n, dg);
                }
            }
            if (!CHAN || g.grad_beta != nullptr) {
                if (lanes >= N) {
                    const float sum = sum_row(sums, lanes, lane);
                    if (puts && sum_token < live) *sum_at = sum;
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        for (int o = lanes / 2; o >= 1; o /= 2) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
                        const int t = t_row + j % R;
                        if (c0 == 0 && j % R < live) {
                            if (j < R && g.grad_beta != nullptr) g.grad_beta[row_of(g.grad_beta_stride, w, t)] = sums[j];
                            if (j >= R && g.grad_g != nullptr) g.grad_g[row_of(g.grad_g_stride, w, t)] = sums[j];
                        }
                    }
                }
            }
            gv -= gv_step;
            gg -= gg_step;
            sum_at -= sum_step;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.empty[turn.stage]);     // the stage is read
            if (!VEC) bring(s + kStages, turn.stage);
            turn.next();
        }
        if (!alive) linger();
        if (a.zero_past && on) {
            const float2 zero[4] = {};
#pragma unroll 1
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
    // only now: grad_h0 may be grad_last, which every CTA of the cluster reads
    if (warp < NW && rank == 0 && g.grad_h0 != nullptr)
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = tid - e_from + 32 * NW * j;
            if (c >= 0 && c < d) g.grad_h0[(int64_t)w.u * d + c] = carry[j];
        }
}

// ------------------------------------------------------------------ dispatch

// A kernel's types and variants, as one value.
template <typename In_, typename Out_, bool CHAN_, bool VEC_, int D_>
struct Variant {
    using In = In_;
    using Out = Out_;
    static constexpr bool CHAN = CHAN_, VEC = VEC_;
    static constexpr int D = D_;             // channels, where the kernel is compiled for them (0: any)
};

// Aligned heads of 64, 128 and 256 channels, one type in and out, have kernels
// of their own.  With the channels known, so is every place in shared memory:
// registers were full before, and the places were worked out again at each use
// (backward, composing took 3100 of 5850 cycles a step; one spilled register
// cost thousands, the two CTAs of an SM leaving the L1 no room).
template <typename In, typename Out, bool CHAN, typename F>
cudaError_t by_rows(const lq_scan_config &c, bool vec, F &&f) {
    if constexpr (std::is_same<In, Out>::value) {
        if (vec) {
            switch (c.d) {
                case 64: return f(Variant<In, Out, CHAN, true, 64>());
                case 128: return f(Variant<In, Out, CHAN, true, 128>());
                case 256: return f(Variant<In, Out, CHAN, true, 256>());
                default: break;
            }
        }
    }
    return vec ? f(Variant<In, Out, CHAN, true, 0>()) : f(Variant<In, Out, CHAN, false, 0>());
}

template <typename In, typename Out, typename F>
cudaError_t by_gate(const lq_scan_config &c, bool vec, F &&f) {
    return c.gate == LQ_GATE_CHANNEL ? by_rows<In, Out, true>(c, vec, f) : by_rows<In, Out, false>(c, vec, f);
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
cudaError_t launch_clusters(int threads, int units, int ranks, int smem, int most, cudaStream_t s, const V &...args) {
    const cudaError_t e = opt_in_smem<kernel>(most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units * (unsigned)ranks);
    cfg.blockDim = dim3((unsigned)threads);
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
    const cuuint32_t box[4] = {(cuuint32_t)c.d, 1, 1, (cuuint32_t)box_of(chunk)};
    const cuuint32_t each[4] = {1, 1, 1, 1};
    const CUresult r = encode(&m->map, dtype == LQ_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                              4, const_cast<void *>(p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// How a call is split: the CTAs that share a unit, a CTA's shared memory, and
// the most that any d wants (for the kernel's limit).
struct Plan {
    int ranks, smem, most, chunk;
    long long rounds;        // of CTAs on the device
};

// As many CTAs as take the least time: rounds of CTAs on the device, each its
// steps and two more for its start and end, a step in a cluster costing
// `shared` times one without (in hundredths: measured 115 forward, where the
// exchange is hidden, and 160 backward).  Registers leave most_ctas CTAs to an
// SM, and shared memory one or two.
template <typename S>
Plan plan_of(int units, long long tokens, int d, int run, int most_ctas, int shared) {
    auto space = [run](int dd) { return S(dd, row_lanes(dd), run); };
    Plan p{1, 0, 0, space(d).tokens, 1};
    long long least = -1;
    for (int r = 1; r <= kMostRanks; ++r) {
        const int smem = space(d).bytes(r);
        const long long slots = (2 * (smem + 2048) <= 228 * 1024 ? most_ctas : 1) * (long long)sm_count();
        const long long rounds = ((long long)units * r + slots - 1) / slots, stride = (long long)r * p.chunk;
        const long long cost = rounds * ((tokens + stride - 1) / stride + 2) * (r > 1 ? shared : 100);
        if (least < 0 || cost < least) {
            least = cost;
            p.ranks = r;
            p.smem = smem;
            p.rounds = rounds;
        }
    }
    for (int dd = 8; dd <= 256; dd *= 2) p.most = std::max(p.most, space(dd).bytes(kMostRanks));
    return p;
}

}  // namespace

cudaError_t launch_scan_forward(const lq_scan_config &c, const lq_scan_args &a, bool vec, cudaStream_t s) {
    const int units = c.batch * c.heads, lanes = row_lanes(c.d), every = scan_checkpoint_tokens(c);
    return by_variant(c, vec, [&](auto k) {
        using K = decltype(k);
        using In = typename K::In;
        constexpr int run = forward_run(sizeof(In) == 2, K::CHAN);
        const Plan p = plan_of<ForwardSpace<In, K::CHAN>>(units, a.n_tokens, c.d, run, 2, 115);
        // Token after token takes 6 us and 0.35 us a token while the threads fit the
        // device; the split kernel 4 us and 4.4 us a round of CTAs while a CTA has
        // one step.  (2048 units of 128 channels, 16 tokens: 12 against 31 us; 32
        // units: 10 against 8.)
        if (a.n_tokens <= std::min(12 * p.rounds - 6, 64LL)) {
            const long long threads = (long long)units * lanes;
            scan_rows_kernel<In, typename K::Out, K::CHAN, K::VEC>
                <<<(unsigned)((threads + kRowsThreads - 1) / kRowsThreads), kRowsThreads, 0, s>>>(a, c.heads, units, c.d,
                                                                                                 lanes, every);
            return cudaGetLastError();
        }
        RowMap v = {}, g = {};
        if (K::VEC) {
            cudaError_t e = row_map(&v, a.v, a.v_stride, c, a.n_tokens, c.in_dtype, p.chunk);
            if (e == cudaSuccess && K::CHAN) e = row_map(&g, a.g, a.g_stride, c, a.n_tokens, LQ_DTYPE_F32, p.chunk);
            if (e != cudaSuccess) return e;
        }
        return launch_clusters<scan_forward_kernel<In, typename K::Out, K::CHAN, K::VEC, K::D>>(
            32 * forward_warps(K::CHAN) + 64, units, p.ranks, p.smem, p.most, s, a, v, g, c.heads, units, c.d, every);
    });
}

cudaError_t launch_scan_backward(const lq_scan_config &c, const lq_scan_args &a, const lq_scan_grads &g, bool vec,
                                 cudaStream_t s) {
    const int units = c.batch * c.heads;
    return by_variant(c, vec && a.n_tokens > 0, [&](auto k) {
        using K = decltype(k);
        using In = typename K::In;
        using Out = typename K::Out;
        constexpr int run = backward_run(sizeof(In) == 2, K::CHAN);
        const Plan p = plan_of<BackwardSpace<In, Out, K::CHAN>>(units, a.n_tokens, c.d, run, K::D > 0 ? 2 : 1, 160);
        RowMap v = {}, y = {}, gate = {};
        if (K::VEC) {
            cudaError_t e = row_map(&v, a.v, a.v_stride, c, a.n_tokens, c.in_dtype, p.chunk);
            if (e == cudaSuccess && g.grad_out != nullptr)
                e = row_map(&y, g.grad_out, g.grad_out_stride, c, a.n_tokens, c.out_dtype, p.chunk);
            if (e == cudaSuccess && K::CHAN) e = row_map(&gate, a.g, a.g_stride, c, a.n_tokens, LQ_DTYPE_F32, p.chunk);
            if (e != cudaSuccess) return e;
        }
        return launch_clusters<scan_backward_kernel<In, Out, K::CHAN, K::VEC, K::D>>(
            32 * kBackwardWarps + 32, units, p.ranks, p.smem, p.most, s, a, g, v, y, gate, c.heads, units, c.d);
    });
}

}  // namespace lq

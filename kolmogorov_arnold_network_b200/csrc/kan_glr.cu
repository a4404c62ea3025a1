// kan_glr.cu -- gated linear recurrence over time, forward, backward and the
// single step.
//
// Per channel c, sequence b and step t, with s = sigmoid(r_t), lambda =
// softplus(decay_c):
//   log a_t = -lambda s,  m_t = sqrt(1 - a_t^2),  u_t = sigmoid(g_t) x_t
//   h_t = a_t h_{t-1} + m_t u_t,   y_t = h_t
// and at a step with reset set, h_{t-1} counts as 0 whatever it holds.
// Backward, gamma_t the gradient that flows into h_{t-1}:
//   d_t = dy_t + gamma_{t+1},  gamma_t = a_t d_t (0 at a reset)
//   dx = d m sigmoid(g),  dg = dx x (1 - sigmoid(g))
//   dL = d (a h_{t-1} - a^2 u / m)          (with respect to L = log a)
//   dr = dL L (1 - s),  ddecay = sum dL L sigmoid(decay) / lambda
//
// Both directions are scans of affine maps h -> A h + B.  Within a thread's
// steps a step is one fused multiply-add.  Between threads factors multiply as
// sums of y = -log a, and A goes as A - 1 above about one half (a long memory
// has A next to 1, where fp32 holds A - 1 but not A to 24 bits) and as A below
// (next to 0 it is the other way round): see Factor.
//
// Split (one pass over HBM): a warp's lanes hold neighbouring channels, a
// thread S steps of its channels in registers; the W warps of a block and the
// CTAs of a cluster hold the blocks of S steps side by side in time.  Each
// thread composes its S steps, the maps meet in shared memory (warps of a
// block) and in distributed shared memory (blocks of the cluster), each
// thread composes what lies before it in a fixed order and walks its S steps
// again from the state that enters them.  The cluster walks along the
// sequence this way, the next inputs being loaded before this step's
// exchange.  No block waits for another one outside its cluster, and the
// order of every sum is fixed.
//
// The forward can keep the state that enters each block of S = 8 steps
// (fp32): the backward recomputes the states within a block from it, so it
// reads 1/2 byte an element instead of y, and unrounded states.
#include <algorithm>
#include <atomic>

#include "kan_device.cuh"
#include "kan_vec.cuh"

namespace kan {
namespace {

constexpr int kSteps = 8;         // steps per thread, and the spacing of the kept states

constexpr int kMaxCluster = 8;    // blocks of a cluster (the portable bound)
constexpr int64_t kMaxStride = 1 << 20;   // elements from a step to the next: a span of 512 steps stays within 32 bits of bytes

struct GlrArgs {
    const void *x, *r, *g;
    int64_t xb, xt, rb, rt, gb, gt;     // strides (elements) of sequence and step
    const float* decay;
    const unsigned char* reset;         // [B, T] or null
    const float* h0;                    // [B, C] or null
    void* y;                            // [B, T, C]
    float* h_last;                      // [B, C] or null
    float* kept;                        // [B, ceil(T / 8), C] or null (forward: written, backward: read)
    // backward
    const void* dy;                     // [B, T, C]
    const float* dh_last;               // [B, C] or null
    void *dx, *dr, *dg;                 // [B, T, C] or null
    float* dh0;                         // [B, C] or null
    double* part;                       // [B * cluster][C] partial sums for ddecay, or null
    int64_t B, T, C;
    int strips;                         // of 128 bytes
    unsigned int* status;
};

constexpr float kTiny = 1e-37f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsq(float x)
{
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the smaller of both; a NaN passes
__device__ __forceinline__ float min_nan(float x, float y)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// E neighbouring channels of a thread.
template <int E> struct F {
    float v[E];
    __device__ __forceinline__ static F all(float x)
    {
        F r;
#pragma unroll
        for (int e = 0; e < E; ++e) r.v[e] = x;
        return r;
    }
    __device__ __forceinline__ static F of(const float (&x)[E])
    {
        F r;
#pragma unroll
        for (int e = 0; e < E; ++e) r.v[e] = x[e];
        return r;
    }
    __device__ __forceinline__ void get(float (&x)[E]) const
    {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = v[e];
    }
};
template <int E> __device__ __forceinline__ F<E> fma(F<E> x, F<E> y, F<E> z)
{
    F<E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = fmaf(x.v[e], y.v[e], z.v[e]);
    return r;
}
template <int E> __device__ __forceinline__ F<E> operator*(F<E> x, F<E> y)
{
    F<E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = x.v[e] * y.v[e];
    return r;
}
template <int E> __device__ __forceinline__ F<E> operator+(F<E> x, F<E> y)
{
    F<E> r;
#pragma unroll
    for (int e = 0; e < E; ++e) r.v[e] = x.v[e] + y.v[e];
    return r;
}
// f of each channel
template <int E, typename Fn> __device__ __forceinline__ F<E> each(F<E> x, Fn f)
{
    float v[E];
    x.get(v);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = f(v[e]);
    return F<E>::of(v);
}
template <int E, typename Fn> __device__ __forceinline__ F<E> each(F<E> x, F<E> y, Fn f)
{
    float v[E], w[E];
    x.get(v);
    y.get(w);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = f(v[e], w[e]);
    return F<E>::of(v);
}

// e^-x; with TOP, held at 2^TOP from above, so that what is made of it stays finite (a NaN passes).
template <int TOP, int E> __device__ __forceinline__ F<E> exp_minus(F<E> x)
{
    return each(x * F<E>::all(-kLog2e), [](float t) { return ex2(min_nan(t, (float)TOP)); });
}
template <int E> __device__ __forceinline__ F<E> exp_minus(F<E> x)
{
    return each(x * F<E>::all(-kLog2e), [](float t) { return ex2(t); });
}
template <int E> __device__ __forceinline__ F<E> rsq_of(F<E> x)
{
    return each(x, [](float t) { return rsq(t); });
}
template <int E> __device__ __forceinline__ F<E> rcp_of(F<E> x)
{
    return each(x, [](float t) { return rcp(t); });
}

// 1 - e^-y for 0 <= y <= 1/4: y sum_{k=0..6} (-y)^k / (k+1)!; the next term is below 2^-29 of it
template <int E> __device__ __forceinline__ F<E> rest_series(F<E> y)
{
    F<E> s = fma(y, F<E>::all(1.0f / 5040.0f), F<E>::all(-1.0f / 720.0f));
    s = fma(s, y, F<E>::all(1.0f / 120.0f));
    s = fma(s, y, F<E>::all(-1.0f / 24.0f));
    s = fma(s, y, F<E>::all(1.0f / 6.0f));
    s = fma(s, y, F<E>::all(-0.5f));
    return fma(s, y, F<E>::all(1.0f)) * y;
}
template <int E> __device__ __forceinline__ F<E> exp_neg(F<E> y)
{
    return each(y * F<E>::all(-kLog2e), [](float t) { return ex2(t); });
}
template <int E> __device__ __forceinline__ F<E> pick_small(F<E> y, F<E> small, F<E> large)
{
    float t[E], p[E], q[E];
    y.get(t);
    small.get(p);
    large.get(q);
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = t[e] < 0.25f ? p[e] : q[e];
    return F<E>::of(p);
}
// 1 - a of a step with a = e^-y (a NaN passes), and a itself to its own last bit where it is small.
template <int E> __device__ __forceinline__ F<E> rest_of(F<E> y)
{
    return pick_small(y, rest_series(y), fma(exp_neg(y), F<E>::all(-1.0f), F<E>::all(1.0f)));
}
template <int E> __device__ __forceinline__ void decay_of(F<E> y, F<E>& av, F<E>& rest)
{
    const F<E> r = rest_series(y), big = exp_neg(y), one = F<E>::all(1.0f), neg = F<E>::all(-1.0f);
    rest = pick_small(y, r, fma(big, neg, one));
    av = pick_small(y, fma(r, neg, one), big);
}
// 1 - a^2
template <int E> __device__ __forceinline__ F<E> square_rest(F<E> rest)
{
    return rest * fma(rest, F<E>::all(-1.0f), F<E>::all(2.0f));
}

// The map h -> A h + B of many steps as h -> (k h + (p h + B)): k = 1, p = A - 1 for A above 3/4, else k = 0, p = A.
// A reset among the steps (y is inf) gives k = 0, p = -0: B alone for every finite h, and CUTS looks at p for the others.
template <int E> struct Map {
    F<E> p, k, b;
};
template <int E> __device__ __forceinline__ Map<E> map_of(F<E> y, F<E> B)
{
    Map<E> m;
    m.p = pick_small(y, fma(rest_series(y), F<E>::all(-1.0f), F<E>::all(0.0f)), exp_neg(y));      // never -0
    m.p = each(m.p, y, [](float p, float t) { return t == INFINITY ? -0.0f : p; });
    m.k = each(y, [](float t) { return t < 0.25f ? 1.0f : 0.0f; });
    m.b = B;
    return m;
}
template <bool CUTS, int E> __device__ __forceinline__ F<E> apply(const Map<E>& m, F<E> h)
{
    if (CUTS) h = each(m.p, h, [](float p, float x) { return __float_as_uint(p) == 0x80000000u ? 0.0f : x; });
    return fma(m.k, h, fma(m.p, h, m.b));
}

__device__ __forceinline__ float softplus_of(float d) { return fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d))); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank)
{
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(local), "r"(rank));
    return d;
}
// 16, 8 or 4 bytes to another block's shared memory; its mbarrier counts them as they arrive.
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float4 v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(to),
                 "r"(bar), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float2 v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];" ::"r"(to),
                 "r"(bar), "f"(v.x), "f"(v.y)
                 : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %2, [%1];" ::"r"(to), "r"(bar), "f"(v)
                 : "memory");
}

template <int E> struct Vecs;
template <> struct Vecs<1> {
    using One = float;
    using Two = float2;
};
template <> struct Vecs<2> {
    using One = float2;
    using Two = float4;
};
__device__ __forceinline__ float one_of(F<1> x) { return x.v[0]; }
__device__ __forceinline__ float2 one_of(F<2> x) { return make_float2(x.v[0], x.v[1]); }
__device__ __forceinline__ F<1> of_one(float x) { return {{x}}; }
__device__ __forceinline__ F<2> of_one(float2 x) { return {{x.x, x.y}}; }
__device__ __forceinline__ float2 two_of(F<1> x, F<1> y) { return make_float2(x.v[0], y.v[0]); }
__device__ __forceinline__ float4 two_of(F<2> x, F<2> y) { return make_float4(x.v[0], x.v[1], y.v[0], y.v[1]); }
__device__ __forceinline__ Map<1> of_two(float2 t, float b) { return {{{t.x}}, {{t.y}}, {{b}}}; }
__device__ __forceinline__ Map<2> of_two(float4 t, float2 b) { return {{{t.x, t.y}}, {{t.z, t.w}}, {{b.x, b.y}}}; }

// Shared memory of the exchange, two sets used by turns: maps of the block's warps and their sums of y, maps of the
// cluster's blocks with the mbarrier that counts them.
template <int E, int W, int CL> struct Meet {
    typename Vecs<E>::Two pk[2][W][32], tot_pk[2][CL][32];
    typename Vecs<E>::One b[2][W][32], len[2][W][32], tot_b[2][CL][32];
    uint64_t full[2];
    static constexpr uint32_t kMapBytes = 32 * 12 * E;
};

template <int E, int W, int CL> __device__ __forceinline__ void meet_init(Meet<E, W, CL>& s)
{
    if constexpr (CL > 1) {
        if (threadIdx.x == 0) {
            mbar_init(smem_addr(&s.full[0]), 1);
            mbar_init(smem_addr(&s.full[1]), 1);
            fence_barrier_init();
        }
        cluster_sync_all();                              // every block of the cluster runs, its barriers are set up
    }
}

// Exchange of span n of the cluster: every thread gives its map (y, B); it gets the state that enters its steps, and
// `run` moves past the whole span.  Position 0 comes first in the direction of the scan.  One block barrier a span: a
// set is written again only two spans later, when all warps have passed the barrier in between, and a block's maps
// for that span are sent only after it has the whole cluster's of the span in between.  A wait that gives up is
// recorded; the walk goes on (its results are void) and ends.
template <int E, int W, int CL> struct Walk {
    Meet<E, W, CL>& s;
    int set, lane;
    // the block's warps `from` <= w < `to`
    template <bool CUTS> __device__ __forceinline__ F<E> warps(int from, int to, F<E> h) const
    {
#pragma unroll(CUTS ? 1 : 4)
        for (int w = from; w < to; ++w) h = apply<CUTS>(of_two(s.pk[set][w][lane], s.b[set][w][lane]), h);
        return h;
    }
    // the cluster's blocks
    template <bool CUTS> __device__ __forceinline__ F<E> blocks(int from, int to, F<E> h) const
    {
#pragma unroll(CUTS ? 1 : 4)
        for (int c = from; c < to; ++c) h = apply<CUTS>(of_two(s.tot_pk[set][c][lane], s.tot_b[set][c][lane]), h);
        return h;
    }
    template <bool CUTS> __device__ __forceinline__ void states(int wpos, int cpos, F<E>& run, F<E>& in) const
    {
        if constexpr (CL > 1) {
            in = blocks<CUTS>(0, cpos, run);
            run = blocks<CUTS>(cpos, CL, in);
            in = warps<CUTS>(0, wpos, in);
        } else {
            in = warps<CUTS>(0, wpos, run);
            run = warps<CUTS>(wpos, W, in);
        }
    }
};

// at_barrier runs right before the block's barrier, past_barrier right after it.
template <int E, int W, int CL, typename At, typename Past>
__device__ __forceinline__ F<E> exchange(Meet<E, W, CL>& s, int n, int wpos, int cpos, F<E> y, F<E> B, F<E>& run, bool cuts,
                                         unsigned int* status, bool& waits, At at_barrier, Past past_barrier)
{
    const int lane = threadIdx.x & 31, set = n & 1;
    const Map<E> m = map_of(y, B);
    F<E> in = run;
    if constexpr (W * CL == 1) {
        run = apply<true>(m, run);
    } else {
        const Walk<E, W, CL> walk{s, set, lane};
        s.pk[set][wpos][lane] = two_of(m.p, m.k);
        s.b[set][wpos][lane] = one_of(B);
        if constexpr (CL > 1) s.len[set][wpos][lane] = one_of(y);
        at_barrier();
        __syncthreads();
        if constexpr (CL > 1) {
            if (wpos == 0) {
                F<E> yt = F<E>::all(0.0f);
                const F<E> bt = cuts ? walk.template warps<true>(0, W, yt) : walk.template warps<false>(0, W, yt);
#pragma unroll
                for (int w = 0; w < W; ++w)              // a reset cuts off a NaN before it
                    yt = each(yt, of_one(s.len[set][w][lane]), [](float t, float l) { return l == INFINITY ? l : t + l; });
                const Map<E> t = map_of(yt, bt);
                const uint32_t bar = smem_addr(&s.full[set]), pk = smem_addr(&s.tot_pk[set][cpos][lane]),
                               bb = smem_addr(&s.tot_b[set][cpos][lane]);
                if (lane == 0) mbar_arrive_expect_tx(bar, CL * s.kMapBytes);
#pragma unroll
                for (int c = 0; c < CL; ++c) {
                    const uint32_t pb = peer_addr(bar, c);
                    st_async(peer_addr(pk, c), pb, two_of(t.p, t.k));
                    st_async(peer_addr(bb, c), pb, one_of(t.b));
                }
            }
        }
        past_barrier();
        if constexpr (CL > 1) {
            if (waits) waits = mbar_wait(smem_addr(&s.full[set]), (n >> 1) & 1, status);
        }
        const F<E> first = run;
        walk.template states<false>(wpos, cpos, run, in);
        if (cuts) {
            // A cut map is B + 0 h: right unless h is not finite.  Then (what comes out is a NaN) once more with care.
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) t += run.v[e] + in.v[e];
            if (__any_sync(0xffffffffu, t != t)) {
                run = first;
                walk.template states<true>(wpos, cpos, run, in);
            }
        }
    }
    return in;
}

// Where a thread stands: its block's unit is (sequence b, strip of channels).
template <int E> struct Place {
    int warp, rank, chans;           // chans: channels of this thread that exist (0..E)
    int second;                      // where the second one is read from (a channel that exists)
    int64_t b, c, c0, read;          // c0: the strip's first channel; read: the channel that is read (c, or 0 beyond the last)
    __device__ __forceinline__ Place(const GlrArgs& a, int cl)
    {
        warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
        rank = cl > 1 ? (int)cluster_rank() : 0;
        const int unit = blockIdx.x / cl;
        b = unit / a.strips;
        c0 = (unit - b * a.strips) * (32 * E);
        c = c0 + (threadIdx.x & 31) * E;
        chans = (int)max((int64_t)0, min((int64_t)E, a.C - c));
        read = chans > 0 ? c : 0;
        second = chans > 1 ? 1 : 0;
    }
    // bytes from a span's first step to this thread's first step and channel
    __device__ __forceinline__ uint32_t off(int64_t stride, int64_t first, int size) const
    {
        return (uint32_t)(((uint32_t)first * (uint32_t)stride + (uint32_t)read) * (uint32_t)size);
    }
};

// Inputs straight to registers: a thread's S steps, element by element (rows need not be whole vectors).  A thread beyond
// the last channel reads another one's (and stores nothing).
template <typename T, int E, int S> struct Direct {
    Pack<T, 1> q[S][E];
    // p: the block's address (the same for all its threads) of the span's first step; off: this thread's bytes from it
    template <bool FULL> __device__ __forceinline__ void load(const T* p, uint32_t off, int64_t stride, int live, int second)
    {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const T* at = reinterpret_cast<const T*>(reinterpret_cast<const char*>(p + i * stride) + off);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (!FULL) q[i][e] = Pack<T, 1>::zero();
                if (FULL || i < live) q[i][e] = Pack<T, 1>::load(at + (e ? second : 0));
            }
        }
    }
    __device__ __forceinline__ F<E> get(int i) const
    {
        F<E> r;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float w[1];
            q[i][e].unpack(w);
            r.v[e] = w[0];
        }
        return r;
    }
};

// Inputs through shared memory, two spans ahead, in 16-byte copies: the rows of a block's 64 steps of a strip are 128
// bytes.  Thread k copies the chunk k % 8 of the rows k / 8 and k / 8 + 32 of each array.
constexpr int kRowBytes = 128, kTileBytes = 8 * kSteps * kRowBytes;
struct Copier {
    const char* from;                // this thread's chunk of the next span's tile
    int64_t half, span;              // bytes to the row 32 further, to the next tile in the walk's direction
    // p: the array at the sequence's first step; step: the tile's first step; spans: steps to the next tile (may be negative)
    template <typename T> __device__ __forceinline__ Copier(const T* p, int64_t stride, int64_t c0, int64_t step, int64_t spans)
    {
        from = reinterpret_cast<const char*>(p + (step + (threadIdx.x >> 3)) * stride + c0) + (threadIdx.x & 7) * 16;
        half = 32 * stride * (int64_t)sizeof(T);
        span = spans * stride * (int64_t)sizeof(T);
    }
    // rows and row 32 further: exist
    __device__ __forceinline__ void copy(uint32_t to, bool row, bool further)
    {
        if (row) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        if (further) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 32 * kRowBytes), "l"(from + half) : "memory");
        from += span;
    }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int E> __device__ __forceinline__ F<E> staged(const char* tile, int row)
{
    const Pack<T, E> q = Pack<T, E>::load(reinterpret_cast<const T*>(tile + row * kRowBytes) + (threadIdx.x & 31) * E);
    float v[E];
    q.unpack(v);
    return F<E>::of(v);
}

template <typename T, int LV, int E> __device__ __forceinline__ void store_step(T* p, F<E> x, int chans)
{
    float v[E];
    x.get(v);
#pragma unroll
    for (int j = 0; j < E / LV; ++j) {
        if (j * LV < chans) {
            float w[LV];
#pragma unroll
            for (int e = 0; e < LV; ++e) w[e] = v[j * LV + e];
            Pack<T, LV>::pack(w).store(p + j * LV);
        }
    }
}
template <int E> __device__ __forceinline__ F<E> load_f32(const float* p, int chans)
{
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = e < chans ? p[e] : 0.0f;
    return F<E>::of(v);
}
template <int E> __device__ __forceinline__ void store_f32(float* p, F<E> x, int chans)
{
    float v[E];
    x.get(v);
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < chans) p[e] = v[e];
}
// Forward: S steps a thread, W warps a block, CL blocks a cluster; STAGED: inputs through shared memory (W = 8), else
// into registers.
template <typename T, bool STAGED, int S, int W, int CL>
__global__ void __launch_bounds__(32 * W, W == 8 ? (STAGED ? (sizeof(T) == 2 ? 3 : 4) : 2) : 1) glr_forward_kernel(const GlrArgs a)
{
    constexpr int E = 4 / (int)sizeof(T);
    constexpr int LV = STAGED ? E : 1;
    extern __shared__ __align__(128) char tiles[];       // STAGED: [2][r, g, x] tiles
    __shared__ Meet<E, W, CL> meet;
    const Place<E> at(a, CL);
    constexpr int64_t SPAN = (int64_t)S * W * CL;
    const int64_t mine = (int64_t)at.rank * W * S, first = mine + at.warp * S;   // the block's and the thread's first step
    const int chans = at.chans;
    const int64_t state = at.b * a.C + at.c;
    const T* X = reinterpret_cast<const T*>(a.x) + at.b * a.xb;
    const T* R = reinterpret_cast<const T*>(a.r) + at.b * a.rb;
    const T* G = reinterpret_cast<const T*>(a.g) + at.b * a.gb;
    T* Y = reinterpret_cast<T*>(a.y) + (at.b * a.T + first) * a.C + at.c;      // this thread's first output of the span
    const unsigned char* Z = a.reset ? a.reset + at.b * a.T : nullptr;
    float* K = a.kept ? a.kept + (at.b * ((a.T + kSteps - 1) / kSteps) + first / kSteps) * a.C + at.c : nullptr;

    const F<E> lambda = each(load_f32<E>(a.decay + at.c, chans), [](float d) { return softplus_of(d); });
    const F<E> one = F<E>::all(1.0f), zero = F<E>::all(0.0f), neg = F<E>::all(-1.0f);
    F<E> run = a.h0 ? load_f32<E>(a.h0 + state, chans) : zero;
    Direct<T, E, STAGED ? 1 : S> qx, qr, qg;
    Copier cr(R, a.rt, at.c0, mine, SPAN), cg(G, a.gt, at.c0, mine, SPAN), cx(X, a.xt, at.c0, mine, SPAN);
    const bool chunk = at.c0 + (threadIdx.x & 7) * (16 / (int)sizeof(T)) < a.C;      // a chunk that this thread copies exists
    const uint32_t place = smem_addr(tiles) + threadIdx.x * 16;
    const int lane = threadIdx.x & 31;
    unsigned char zb = 0;                                // the reset byte of this lane's step of the next span
    auto fetch = [&](int64_t base, int set) {
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - base - first));
        if (Z) zb = lane < live ? Z[base + first + lane] : 0;
        if constexpr (STAGED) {
            const int64_t left = a.T - base - mine - (threadIdx.x >> 3);
            const bool r0 = chunk && left > 0, r1 = chunk && left > 32;
            const uint32_t tile = place + set * 3 * kTileBytes;
            cr.copy(tile, r0, r1);
            cg.copy(tile + kTileBytes, r0, r1);
            cx.copy(tile + 2 * kTileBytes, r0, r1);
            copies_commit();
        } else if (live == S) {
            qr.template load<true>(R + base * a.rt, at.off(a.rt, first, sizeof(T)), a.rt, S, at.second);
            qg.template load<true>(G + base * a.gt, at.off(a.gt, first, sizeof(T)), a.gt, S, at.second);
            qx.template load<true>(X + base * a.xt, at.off(a.xt, first, sizeof(T)), a.xt, S, at.second);
        } else {
            qr.template load<false>(R + base * a.rt, at.off(a.rt, first, sizeof(T)), a.rt, live, at.second);
            qg.template load<false>(G + base * a.gt, at.off(a.gt, first, sizeof(T)), a.gt, live, at.second);
            qx.template load<false>(X + base * a.xt, at.off(a.xt, first, sizeof(T)), a.xt, live, at.second);
        }
    };
    meet_init(meet);
    bool waits = true;
    unsigned char zb_now;
    fetch(0, 0);
    zb_now = zb;
    if constexpr (STAGED) {
        fetch(SPAN, 1);                                  // (nothing beyond the end)
        copies_wait<1>();
        __syncthreads();
    }

    int n = 0;
    for (int64_t base = 0; base < a.T; base += SPAN, ++n) {
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - base - first));
        const uint32_t cuts = Z ? __ballot_sync(0xffffffffu, zb_now != 0) : 0;
        const char* tile = tiles + (n & 1) * 3 * kTileBytes;
        auto in_r = [&](int i) { return STAGED ? staged<T, E>(tile, at.warp * S + i) : qr.get(STAGED ? 0 : i); };
        auto in_g = [&](int i) { return STAGED ? staged<T, E>(tile + kTileBytes, at.warp * S + i) : qg.get(STAGED ? 0 : i); };
        auto in_x = [&](int i) { return STAGED ? staged<T, E>(tile + 2 * kTileBytes, at.warp * S + i) : qx.get(STAGED ? 0 : i); };
        F<E> fa[S], bb[S], len = zero, B = zero;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const F<E> y = rcp_of(one + exp_minus(in_r(i))) * lambda;
            const F<E> rest = rest_of(y), m2 = square_rest(rest);
            // m sigmoid(g) = m^2 / sqrt(m^2 (1 + e)^2) with e = exp(-g): one rsqrt, held where m is 0
            const F<E> q = one + exp_minus<60>(in_g(i));
            bb[i] = m2 * rsq_of(fma(m2 * q, q, F<E>::all(kTiny))) * in_x(i);
            fa[i] = one + rest * neg;
            len = len + y;
            B = fma(fa[i], B, bb[i]);
        }
        if (live < S) {                                  // past the end: a = 1, nothing comes in
            len = B = zero;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < live) {
                    len = len + rcp_of(one + exp_minus(in_r(i))) * lambda;
                    B = fma(fa[i], B, bb[i]);
                }
            }
        }
        if (!STAGED && base + SPAN < a.T) fetch(base + SPAN, 0);
        zb_now = zb;
        if (cuts) {                                      // resets among the steps: they cut off what comes before them
            B = zero;
            len = F<E>::all(INFINITY);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (cuts >> i & 1) B = zero;
                if (i < live) B = fma(fa[i], B, bb[i]);
            }
        }
        F<E> h = exchange<E, W, CL>(
            meet, n, at.warp, at.rank, len, B, run, Z != nullptr, a.status, waits,
            [&] {
                if constexpr (STAGED) copies_wait<0>();  // the next span's inputs, before the barrier
            },
            [&] {
                if constexpr (STAGED)                    // all warps have read this span's tiles
                    if (base + 2 * SPAN < a.T) fetch(base + 2 * SPAN, n & 1);
            });
        if (K) {
            if (live > 0) store_f32<E>(K, h, chans);
            K += SPAN / kSteps * a.C;
        }
        if (live == S && !cuts) {
            if (chans > 0) {
                T* y = Y;
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    h = fma(fa[i], h, bb[i]);
                    store_step<T, LV, E>(y, h, STAGED ? E : chans);
                    y += a.C;
                }
            }
        } else {
            T* y = Y;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (cuts >> i & 1) h = zero;
                h = fma(fa[i], h, bb[i]);
                if (i < live) store_step<T, LV, E>(y, h, chans);
                y += a.C;
            }
        }
        Y += SPAN * a.C;
    }
    if (a.h_last && at.rank == 0 && at.warp == 0) store_f32<E>(a.h_last + state, run, chans);
}

// Backward: the same split, walked from the end of the sequence.
template <typename T, bool STAGED, int W, int CL>
__global__ void __launch_bounds__(32 * W, W == 8 ? 2 : 1) glr_backward_kernel(const GlrArgs a)
{
    constexpr int S = kSteps;                            // a thread's steps begin at a kept state
    constexpr int E = 4 / (int)sizeof(T);
    constexpr int LV = STAGED ? E : 1;
    extern __shared__ __align__(128) char tiles[];       // STAGED: [2][r, g, x, dy] tiles
    __shared__ Meet<E, W, CL> meet;
    const Place<E> at(a, CL);
    constexpr int64_t SPAN = (int64_t)S * W * CL;
    const int64_t mine = (int64_t)at.rank * W * S, first = mine + at.warp * S;
    const int chans = at.chans;
    const int64_t state = at.b * a.C + at.c, end = (a.T - 1) / SPAN * SPAN;       // end: the last span's first step
    const T* X = reinterpret_cast<const T*>(a.x) + at.b * a.xb;
    const T* R = reinterpret_cast<const T*>(a.r) + at.b * a.rb;
    const T* G = reinterpret_cast<const T*>(a.g) + at.b * a.gb;
    const T* D = reinterpret_cast<const T*>(a.dy) + at.b * a.T * a.C;
    const unsigned char* Z = a.reset ? a.reset + at.b * a.T : nullptr;
    const float* K = a.kept + (at.b * ((a.T + kSteps - 1) / kSteps) + (end + first) / kSteps) * a.C + at.c;
    int64_t out = (at.b * a.T + end + first) * a.C + at.c;                        // this thread's first output of the span

    const F<E> lambda = each(load_f32<E>(a.decay + at.c, chans), [](float d) { return softplus_of(d); });
    const F<E> one = F<E>::all(1.0f), zero = F<E>::all(0.0f), neg = F<E>::all(-1.0f);
    F<E> run = a.dh_last ? load_f32<E>(a.dh_last + state, chans) : zero;
    double acc[E];                                       // sum of dL L
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0;
    Copier cr(R, a.rt, at.c0, end + mine, -SPAN), cg(G, a.gt, at.c0, end + mine, -SPAN), cx(X, a.xt, at.c0, end + mine, -SPAN),
        cd(D, a.C, at.c0, end + mine, -SPAN);
    const bool chunk = at.c0 + (threadIdx.x & 7) * (16 / (int)sizeof(T)) < a.C;
    const uint32_t place = smem_addr(tiles) + threadIdx.x * 16;
    const int lane = threadIdx.x & 31;
    unsigned char zb = 0;                                // reset byte of this lane's step, and the kept state, of the next span
    F<E> hb = F<E>::all(0.0f);
    auto copy = [&](int64_t base, int set) {
        const int64_t left = a.T - base - mine - (threadIdx.x >> 3);
        const bool r0 = chunk && left > 0, r1 = chunk && left > 32;
        const uint32_t tile = place + set * 4 * kTileBytes;
        cr.copy(tile, r0, r1);
        cg.copy(tile + kTileBytes, r0, r1);
        cx.copy(tile + 2 * kTileBytes, r0, r1);
        cd.copy(tile + 3 * kTileBytes, r0, r1);
        copies_commit();
    };
    auto ahead = [&](int64_t base) {                     // called once for each span, in the walk's order
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - base - first));
        if (Z) zb = lane < live ? Z[base + first + lane] : 0;
        if (live > 0) hb = load_f32<E>(K, chans);
        K -= SPAN / kSteps * a.C;
    };
    meet_init(meet);
    bool waits = true;
    ahead(end);
    if constexpr (STAGED) {
        copy(end, 0);
        if (end >= SPAN) copy(end - SPAN, 1);
        else copies_commit();
        copies_wait<1>();
        __syncthreads();
    }

    int n = 0;
    for (int64_t base = end; base >= 0; base -= SPAN, ++n) {
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - base - first));
        Direct<T, E, STAGED ? 1 : S> qx, qr, qg, qd;
        if constexpr (!STAGED) {
            if (live == S) {
                qr.template load<true>(R + base * a.rt, at.off(a.rt, first, sizeof(T)), a.rt, S, at.second);
                qg.template load<true>(G + base * a.gt, at.off(a.gt, first, sizeof(T)), a.gt, S, at.second);
                qx.template load<true>(X + base * a.xt, at.off(a.xt, first, sizeof(T)), a.xt, S, at.second);
                qd.template load<true>(D + base * a.C, at.off(a.C, first, sizeof(T)), a.C, S, at.second);
            } else {
                qr.template load<false>(R + base * a.rt, at.off(a.rt, first, sizeof(T)), a.rt, live, at.second);
                qg.template load<false>(G + base * a.gt, at.off(a.gt, first, sizeof(T)), a.gt, live, at.second);
                qx.template load<false>(X + base * a.xt, at.off(a.xt, first, sizeof(T)), a.xt, live, at.second);
                qd.template load<false>(D + base * a.C, at.off(a.C, first, sizeof(T)), a.C, live, at.second);
            }
        }
        const char* tile = tiles + (n & 1) * 4 * kTileBytes;
        auto in_r = [&](int i) { return STAGED ? staged<T, E>(tile, at.warp * S + i) : qr.get(STAGED ? 0 : i); };
        auto in_g = [&](int i) { return STAGED ? staged<T, E>(tile + kTileBytes, at.warp * S + i) : qg.get(STAGED ? 0 : i); };
        auto in_x = [&](int i) { return STAGED ? staged<T, E>(tile + 2 * kTileBytes, at.warp * S + i) : qx.get(STAGED ? 0 : i); };
        Pack<T, E> dy[S];                                // (kept packed: the tile is free after the exchange's barrier)
#pragma unroll
        for (int i = 0; i < S; ++i) {
            if constexpr (STAGED) {
                dy[i] = i < live ? Pack<T, E>::load(reinterpret_cast<const T*>(tile + 3 * kTileBytes + (at.warp * S + i) * kRowBytes) + (threadIdx.x & 31) * E)
                                 : Pack<T, E>::zero();
            } else {
                float v[E];
                qd.get(STAGED ? 0 : i).get(v);
                dy[i] = Pack<T, E>::pack(v);
            }
        }
        auto in_d = [&](int i) {
            float v[E];
            dy[i].unpack(v);
            return F<E>::of(v);
        };
        const uint32_t cut = Z ? __ballot_sync(0xffffffffu, zb != 0) : 0;
        F<E> h = hb;
        if (base > 0) ahead(base - SPAN);
        // per step: the factor, and what d multiplies in each gradient:
        //   dx = d cx_,  dg = dx cg_,  dL L = d cl,  dr = dL L cr_
        F<E> fa[S], cx_[S], cg_[S], cl[S], cr_[S], len = zero, B = zero;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const F<E> er = exp_minus<115>(in_r(i)), eg = exp_minus<115>(in_g(i));
            const F<E> s = rcp_of(one + er), sg = rcp_of(one + eg), x = in_x(i);
            const F<E> y = s * lambda;
            F<E> rest;
            decay_of(y, fa[i], rest);
            // 1 / m, held where m is 0 (there y is 0 too, and y / m goes to 0 with it)
            const F<E> m2 = square_rest(rest), rm = rsq_of(m2 + F<E>::all(kTiny));
            cx_[i] = m2 * rm * sg;
            cg_[i] = x * (eg * sg);
            cr_[i] = er * s;
            if (cut && cut >> i & 1) h = zero;
            // a L (h - a u / m), L = -y
            cl[i] = fa[i] * y * fma(fa[i] * rm, sg * x, h * neg);
            h = fma(fa[i], h, cx_[i] * x);
            len = len + y;
        }
        if (live < S) {                                  // past the end: gamma passes (dy is 0 there)
            len = zero;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (i < live) len = len + rcp_of(one + exp_minus<115>(in_r(i))) * lambda;
                else fa[i] = one;
            }
        }
        // the map of these steps, from the last to the first: gamma -> a (gamma + dy)
#pragma unroll
        for (int i = S - 1; i >= 0; --i) B = fa[i] * (B + in_d(i));
        if (cut) {
            B = zero;
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                B = fa[i] * (B + in_d(i));
                if (cut >> i & 1) B = zero;
            }
            len = F<E>::all(INFINITY);
        }
        F<E> flow = exchange<E, W, CL>(
            meet, n, W - 1 - at.warp, CL - 1 - at.rank, len, B, run, Z != nullptr, a.status, waits,
            [&] {
                if constexpr (STAGED) copies_wait<0>();
            },
            [&] {
                if constexpr (STAGED)
                    if (base >= 2 * SPAN) copy(base - 2 * SPAN, n & 1);
            });
        F<E> part = zero;
        T *ox = reinterpret_cast<T*>(a.dx) + out + S * a.C, *orr = reinterpret_cast<T*>(a.dr) + out + S * a.C,
          *og = reinterpret_cast<T*>(a.dg) + out + S * a.C;
        if (live == S && !cut) {
            if (chans > 0) {
#pragma unroll
                for (int i = S - 1; i >= 0; --i) {
                    const F<E> d = flow + in_d(i), gx = d * cx_[i], gl = d * cl[i];
                    flow = fa[i] * d;
                    part = part + gl;
                    ox -= a.C, orr -= a.C, og -= a.C;
                    if (a.dx) store_step<T, LV, E>(ox, gx, STAGED ? E : chans);
                    if (a.dr) store_step<T, LV, E>(orr, gl * cr_[i], STAGED ? E : chans);
                    if (a.dg) store_step<T, LV, E>(og, gx * cg_[i], STAGED ? E : chans);
                }
            }
        } else {
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                const F<E> d = flow + in_d(i), gx = d * cx_[i], gl = d * cl[i];
                flow = fa[i] * d;
                if (cut >> i & 1) flow = zero;
                ox -= a.C, orr -= a.C, og -= a.C;
                if (i < live) {
                    part = part + gl;
                    if (a.dx) store_step<T, LV, E>(ox, gx, chans);
                    if (a.dr) store_step<T, LV, E>(orr, gl * cr_[i], chans);
                    if (a.dg) store_step<T, LV, E>(og, gx * cg_[i], chans);
                }
            }
        }
        out -= SPAN * a.C;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += (double)part.v[e];
    }
    if (a.dh0 && at.rank == 0 && at.warp == 0) store_f32<E>(a.dh0 + state, run, chans);
    if (a.part) {
        __shared__ double red[W][E][32];
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < E; ++e) red[at.warp][e][lane] = acc[e];
        __syncthreads();
        if (at.warp == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                double v = 0.0;
                for (int w = 0; w < W; ++w) v += red[w][e][lane];
                if (e < chans) a.part[(at.b * CL + at.rank) * a.C + at.c + e] = v;
            }
        }
    }
}

// ddecay from the partial sums of dL L, in their order.
__global__ void glr_decay_kernel(const double* __restrict__ part, int64_t n, int64_t C, const float* __restrict__ decay,
                                 float* __restrict__ ddecay)
{
    const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (c >= C) return;
    double v = 0.0;
    for (int64_t i = 0; i < n; ++i) v += part[i * C + c];
    const float d = decay[c];
    // sigmoid(d) / softplus(d), which goes to 1 as d falls
    const float ratio = d > -15.0f ? 1.0f / ((1.0f + expf(-d)) * softplus_of(d)) : 1.0f;
    ddecay[c] = (float)(v * (double)ratio);
}

kan_status gl_fail(kan_status st, const char* msg) { return set_last_error(st, msg); }

kan_status validate(const kan_glr_shape* s)
{
    if (!s) return gl_fail(KAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->batch < 0 || s->time < 0 || s->channels < 1) return gl_fail(KAN_ERR_INVALID_ARG, "batch >= 0, time >= 0, channels >= 1");
    if (s->dtype != KAN_F32 && s->dtype != KAN_BF16) return gl_fail(KAN_ERR_INVALID_ARG, "unknown dtype");
    const int64_t st[] = {s->x_stride_b, s->x_stride_t, s->r_stride_b, s->r_stride_t, s->g_stride_b, s->g_stride_t};
    for (int64_t v : st)
        if (v < 0) return gl_fail(KAN_ERR_INVALID_ARG, "negative stride");
    for (int i = 1; i < 6; i += 2)
        if (st[i] > kMaxStride) return gl_fail(KAN_ERR_UNSUPPORTED, "a stride of steps above 2^20 elements");
    if (s->channels > kMaxStride || s->time > ((int64_t)1 << 40) || s->batch > ((int64_t)1 << 31) ||
        s->batch * ((s->channels + 31) / 32) > ((int64_t)1 << 27))
        return gl_fail(KAN_ERR_UNSUPPORTED, "sizes too large");
    return KAN_OK;
}

// Clusters of a kernel that run at once on the current device, looked up once per device (a table per kernel).
template <typename K> int resident(K kernel, int warps, int cluster, size_t smem, std::atomic<int> (&known)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg{};
    if (smem && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = 1;
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <typename K> cudaError_t launch(K kernel, int warps, int cluster, size_t smem, const GlrArgs& a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * a.strips * cluster));
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) count_launch();
    return e;
}

// The kernels of one direction and operand type: blocks of 8 warps in clusters of 1 to 8, and a block of one warp for
// sequences of at most 8 steps (and, forward, for a single one).
template <typename T, bool STAGED, bool BWD> struct Kernels {
    static constexpr size_t kSmem = STAGED ? 2 * (BWD ? 4 : 3) * kTileBytes : 0;
    static void (*of(int cluster))(const GlrArgs)
    {
        if constexpr (BWD)
            return cluster == 1 ? glr_backward_kernel<T, STAGED, 8, 1> : cluster == 2 ? glr_backward_kernel<T, STAGED, 8, 2>
                 : cluster == 4 ? glr_backward_kernel<T, STAGED, 8, 4> : glr_backward_kernel<T, STAGED, 8, 8>;
        else
            return cluster == 1 ? glr_forward_kernel<T, STAGED, kSteps, 8, 1> : cluster == 2 ? glr_forward_kernel<T, STAGED, kSteps, 8, 2>
                 : cluster == 4 ? glr_forward_kernel<T, STAGED, kSteps, 8, 4> : glr_forward_kernel<T, STAGED, kSteps, 8, 8>;
    }
    // Blocks of a cluster lie side by side in time: the size that needs the fewest rounds of spans on a full device,
    // a span costing a little more with each block whose maps are walked.
    static int cluster_for(const GlrArgs& a)
    {
        static std::atomic<int> known[4][64];
        const int64_t units = a.B * a.strips;
        int best = 0;
        int64_t cost = -1;
        for (int i = 0; i < 4; ++i) {
            const int cl = 1 << i;
            const int64_t at_once = resident(of(cl), 8, cl, kSmem, known[i]);
            if (at_once < 1) return 0;
            const int64_t c = (units + at_once - 1) / at_once * ((a.T + 8 * kSteps * cl - 1) / (8 * kSteps * cl)) * (16 + cl);
            if (cost < 0 || c < cost) {
                cost = c;
                best = cl;
            }
        }
        return best;
    }
    static cudaError_t run(GlrArgs& a, int& cluster, cudaStream_t st)
    {
        cluster = cluster_for(a);
        return cluster ? launch(of(cluster), 8, cluster, kSmem, a, st) : cudaErrorInvalidValue;
    }
};
template <typename T, bool BWD> cudaError_t run_short(const GlrArgs& a, cudaStream_t st)
{
    if constexpr (BWD) return launch(glr_backward_kernel<T, false, 1, 1>, 1, 1, 0, a, st);
    else if (a.T == 1) return launch(glr_forward_kernel<T, false, 1, 1, 1>, 1, 1, 0, a, st);
    else return launch(glr_forward_kernel<T, false, kSteps, 1, 1>, 1, 1, 0, a, st);
}

// Inputs go through shared memory where their rows begin on 16 bytes and outputs on what a thread stores.
bool staged_ok(const kan_glr_shape& s, const GlrArgs& a)
{
    const int esz = s.dtype == KAN_F32 ? 4 : 2;
    const uint64_t strides = (uint64_t)(s.channels | s.x_stride_b | s.x_stride_t | s.r_stride_b | s.r_stride_t | s.g_stride_b |
                                        s.g_stride_t) * esz;
    const uint64_t in = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) |
                         reinterpret_cast<uintptr_t>(a.g) | reinterpret_cast<uintptr_t>(a.dy));
    const uint64_t out = (reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.dx) |
                          reinterpret_cast<uintptr_t>(a.dr) | reinterpret_cast<uintptr_t>(a.dg));
    return strides % 16 == 0 && in % 16 == 0 && out % 4 == 0;
}

template <typename T, bool BWD> cudaError_t run_type(const kan_glr_shape& s, GlrArgs& a, int& cluster, cudaStream_t st)
{
    a.strips = (int)((s.channels + 32 * (4 / sizeof(T)) - 1) / (32 * (4 / sizeof(T))));
    cluster = 1;
    if (a.T <= kSteps) return run_short<T, BWD>(a, st);
    return staged_ok(s, a) ? Kernels<T, true, BWD>::run(a, cluster, st) : Kernels<T, false, BWD>::run(a, cluster, st);
}
template <bool BWD> cudaError_t run(const kan_glr_shape& s, GlrArgs& a, int& cluster, cudaStream_t st)
{
    return s.dtype == KAN_F32 ? run_type<float, BWD>(s, a, cluster, st) : run_type<__nv_bfloat16, BWD>(s, a, cluster, st);
}

void common_args(const kan_glr_shape& s, GlrArgs& a)
{
    a.xb = s.x_stride_b, a.xt = s.x_stride_t;
    a.rb = s.r_stride_b, a.rt = s.r_stride_t;
    a.gb = s.g_stride_b, a.gt = s.g_stride_t;
    a.B = s.batch, a.T = s.time, a.C = s.channels;
    a.status = device_status_ptr();
}

bool misaligned(const kan_glr_shape& s, std::initializer_list<const void*> ops, std::initializer_list<const void*> f32)
{
    const uintptr_t esz = s.dtype == KAN_F32 ? 4 : 2;
    for (const void* p : ops)
        if (reinterpret_cast<uintptr_t>(p) % esz) return true;
    for (const void* p : f32)
        if (reinterpret_cast<uintptr_t>(p) % 4) return true;
    return false;
}

}  // namespace
}  // namespace kan

using namespace kan;

extern "C" {

kan_status kan_glr_workspace_size(const kan_glr_shape* s, size_t* bytes)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (!bytes) return gl_fail(KAN_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = (size_t)s->batch * kMaxCluster * s->channels * sizeof(double);
    return KAN_OK;
}

kan_status kan_glr_forward(const kan_glr_shape* s, const void* x, const void* r, const void* g, const float* decay,
                           const unsigned char* reset, const float* h0, void* y, float* h_last, float* kept, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    const bool none = s->batch == 0 || s->time == 0;
    if (!none && (!x || !r || !g || !decay || !y)) return gl_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {x, r, g, y}, {decay, h0, h_last, kept}))
        return gl_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (none) {                                          // the state stays what it was
        const size_t n = (size_t)s->batch * s->channels * sizeof(float);
        if (h_last && n && h_last != h0)
            e = h0 ? cudaMemcpyAsync(h_last, h0, n, cudaMemcpyDeviceToDevice, cs) : cudaMemsetAsync(h_last, 0, n, cs);
        return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
    }
    GlrArgs a{};
    common_args(*s, a);
    a.x = x, a.r = r, a.g = g, a.decay = decay, a.reset = reset, a.h0 = h0;
    a.y = y, a.h_last = h_last, a.kept = kept;
    int cluster;
    e = run<false>(*s, a, cluster, cs);
    return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

kan_status kan_glr_backward(const kan_glr_shape* s, const void* x, const void* r, const void* g, const float* decay,
                            const unsigned char* reset, const float* kept, const void* dy, const float* dh_last, void* dx,
                            void* dr, void* dg, float* ddecay, float* dh0, void* workspace, size_t ws_bytes, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    const bool none = s->batch == 0 || s->time == 0;
    if (!none && (!x || !r || !g || !decay || !kept || !dy)) return gl_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {x, r, g, dy, dx, dr, dg}, {decay, kept, dh_last, ddecay, dh0}) || !aligned16(workspace))
        return gl_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements, the workspace to 16 bytes");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (none) {
        const size_t n = (size_t)s->batch * s->channels * sizeof(float);
        if (ddecay) e = cudaMemsetAsync(ddecay, 0, (size_t)s->channels * sizeof(float), cs);
        if (e == cudaSuccess && dh0 && n && dh0 != dh_last)
            e = dh_last ? cudaMemcpyAsync(dh0, dh_last, n, cudaMemcpyDeviceToDevice, cs) : cudaMemsetAsync(dh0, 0, n, cs);
        return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
    }
    GlrArgs a{};
    common_args(*s, a);
    a.x = x, a.r = r, a.g = g, a.decay = decay, a.reset = reset, a.kept = const_cast<float*>(kept);
    a.dy = dy, a.dh_last = dh_last, a.dx = dx, a.dr = dr, a.dg = dg, a.dh0 = dh0;
    if (ddecay) {
        if (!workspace || ws_bytes < (size_t)s->batch * kMaxCluster * s->channels * sizeof(double))
            return gl_fail(KAN_ERR_WORKSPACE, "workspace too small");
        a.part = reinterpret_cast<double*>(workspace);
    }
    int cluster;
    e = run<true>(*s, a, cluster, cs);
    if (e == cudaSuccess && ddecay) {
        glr_decay_kernel<<<(unsigned)((s->channels + 127) / 128), 128, 0, cs>>>(a.part, s->batch * cluster, s->channels, decay, ddecay);
        count_launch();
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

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
// Both directions are scans of affine maps h -> A h + B.  A long memory has A
// next to 1, where fp32 holds A - 1 but not A to 24 bits, a short one has A
// next to 0, where it is the other way round: a factor is kept as A - 1 (not
// positive) above about one half and as A (positive) below, see Factor.
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

#include "kan_device.cuh"
#include "kan_vec.cuh"

namespace kan {
namespace {

constexpr int kSteps = 8;         // steps per thread, and the spacing of the kept states

constexpr int kMaxCluster = 8;    // blocks of a cluster (the portable bound)

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
    int strips;                         // ceil(C / (32 VEC))
};

// Factor: a number v that stands for A in [0, 1].  v in (-1, 0]: A = 1 + v;  v > 0: A = v;  v = kHard: A = 0, and what
// it multiplies is cut off even if it is not finite (L = -inf, which stands for a reset).
constexpr float kHard = -2.0f;
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

// E neighbouring channels of a thread; two of them go through the packed f32x2 instructions.
template <int E> struct F;
template <> struct F<1> {
    float a;
    __device__ __forceinline__ static F all(float x) { return {x}; }
    __device__ __forceinline__ static F of(const float (&v)[1]) { return {v[0]}; }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = a; }
};
template <> struct F<2> {
    uint64_t q;
    __device__ __forceinline__ static F two(float x, float y)
    {
        F r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.q) : "f"(x), "f"(y));
        return r;
    }
    __device__ __forceinline__ static F all(float x) { return two(x, x); }
    __device__ __forceinline__ static F of(const float (&v)[2]) { return two(v[0], v[1]); }
    __device__ __forceinline__ void get(float (&v)[2]) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(q)); }
};
__device__ __forceinline__ F<1> fma(F<1> x, F<1> y, F<1> z) { return {fmaf(x.a, y.a, z.a)}; }
__device__ __forceinline__ F<1> operator*(F<1> x, F<1> y) { return {x.a * y.a}; }
__device__ __forceinline__ F<1> operator+(F<1> x, F<1> y) { return {x.a + y.a}; }
__device__ __forceinline__ F<2> fma(F<2> x, F<2> y, F<2> z)
{
    F<2> r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.q) : "l"(x.q), "l"(y.q), "l"(z.q));
    return r;
}
__device__ __forceinline__ F<2> operator*(F<2> x, F<2> y)
{
    F<2> r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(x.q), "l"(y.q));
    return r;
}
__device__ __forceinline__ F<2> operator+(F<2> x, F<2> y)
{
    F<2> r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(x.q), "l"(y.q));
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

// e^-x, held at 2^TOP from above, so that what is made of it stays finite (a NaN passes).
template <int TOP, int E> __device__ __forceinline__ F<E> exp_minus(F<E> x)
{
    return each(x * F<E>::all(-kLog2e), [](float t) { return ex2(min_nan(t, (float)TOP)); });
}
template <int E> __device__ __forceinline__ F<E> rcp_of(F<E> x)
{
    return each(x, [](float t) { return rcp(t); });
}

// The factor exp(L), L <= 0 (a NaN passes).
template <int E> __device__ __forceinline__ F<E> factor_of(F<E> L)
{
    // exp(L) - 1 = sum_{k=1..8} L^k / k!; the next term is below 2^-26 of the sum at L = -0.5
    F<E> s = fma(L, F<E>::all(1.0f / 40320.0f), F<E>::all(1.0f / 5040.0f));
    s = fma(s, L, F<E>::all(1.0f / 720.0f));
    s = fma(s, L, F<E>::all(1.0f / 120.0f));
    s = fma(s, L, F<E>::all(1.0f / 24.0f));
    s = fma(s, L, F<E>::all(1.0f / 6.0f));
    s = fma(s, L, F<E>::all(0.5f));
    s = fma(s, L, F<E>::all(1.0f)) * L;
    const F<E> big = each(L * F<E>::all(kLog2e), [](float t) {
        const float x = ex2(t);
        return x < kTiny ? kTiny : x;
    });
    float l[E], p[E], b[E];
    L.get(l);
    s.get(p);
    big.get(b);
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = l[e] > -0.5f ? p[e] : b[e];
    return F<E>::of(p);
}
__device__ __forceinline__ float value_of(float v) { return v > 0.0f ? v : 1.0f + v; }      // not for kHard
// 1 - A^2
template <int E> __device__ __forceinline__ F<E> one_minus_sq(F<E> v)
{
    // -v v + c with c = 1 (v = A) or -2 v (v = A - 1)
    const F<E> c = each(v, [](float t) { return t > 0.0f ? 1.0f : -2.0f * t; });
    return fma(v * F<E>::all(-1.0f), v, c);
}
// A h + B, v not kHard
template <int E> __device__ __forceinline__ F<E> walk(F<E> v, F<E> B, F<E> h)
{
    return fma(v, h, B) + each(v, h, [](float t, float x) { return t > 0.0f ? 0.0f : x; });
}
template <int E> __device__ __forceinline__ F<E> apply(F<E> v, F<E> B, F<E> h)
{
    float t[E], b[E], r[E];
    walk(v, B, h).get(r);
    v.get(t);
    B.get(b);
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = t[e] == kHard ? b[e] : r[e];
    return F<E>::of(r);
}
// the factor of steps whose L sum up to this; -inf: a reset was among them
template <int E> __device__ __forceinline__ F<E> factor_or_cut(F<E> L)
{
    const F<E> v = factor_of(L);
    return each(L, v, [](float l, float t) { return l == -INFINITY ? kHard : t; });
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
__device__ __forceinline__ void st_cluster(const void* local, uint32_t rank, float2 v)
{
    uint32_t a = (uint32_t)__cvta_generic_to_shared(local), d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(d), "f"(v.x), "f"(v.y) : "memory");
}

// Shared memory of the exchange: maps (factor, offset) and sums of L of the block's warps, maps of the cluster's blocks
// (two sets, written by turns).
template <int E, int W, int CL> struct Meet {
    float2 agg[W][E][32];
    float len[W][E][32];
    float2 tot[2][CL][E][32];
};

// Exchange of one span of the cluster: every thread gives its map (L, B); it gets the state that enters its steps, and
// `run` moves past the whole span.  Position 0 comes first in the direction of the scan.  Factors multiply as sums of L.
template <int E, int W, int CL>
__device__ __forceinline__ F<E> exchange(Meet<E, W, CL>& s, int parity, int wpos, int cpos, F<E> L, F<E> B, F<E>& run)
{
    const int lane = threadIdx.x & 31;
    const F<E> v = factor_or_cut(L);
    F<E> in = run;
    if constexpr (W * CL == 1) {
        run = apply(v, B, run);
        return in;
    }
    auto put = [&](float2 (*to)[32], F<E> x, F<E> y) {
        float p[E], q[E];
        x.get(p);
        y.get(q);
#pragma unroll
        for (int e = 0; e < E; ++e) to[e][lane] = make_float2(p[e], q[e]);
    };
    auto step = [&](const float2 (*from)[32], F<E> h) {
        float p[E], q[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 t = from[e][lane];
            p[e] = t.x;
            q[e] = t.y;
        }
        return apply(F<E>::of(p), F<E>::of(q), h);
    };
    put(s.agg[wpos], v, B);
    if constexpr (CL > 1) {
        float l[E];
        L.get(l);
#pragma unroll
        for (int e = 0; e < E; ++e) s.len[wpos][e][lane] = l[e];
    }
    __syncthreads();
    if constexpr (CL > 1) {
        if (wpos == 0) {
            F<E> bt = F<E>::all(0.0f);
            float lt[E] = {};
#pragma unroll
            for (int w = 0; w < W; ++w) {
                bt = step(s.agg[w], bt);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float l = s.len[w][e][lane];
                    lt[e] = l == -INFINITY ? l : lt[e] + l;          // a reset cuts off a NaN before it
                }
            }
            float p[E], q[E];
            factor_or_cut(F<E>::of(lt)).get(p);
            bt.get(q);
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int c = 0; c < CL; ++c) st_cluster(&s.tot[parity][cpos][e][lane], c, make_float2(p[e], q[e]));
        }
        cluster_sync_all();
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            if (c == cpos) in = run;
            run = step(s.tot[parity][c], run);
        }
        for (int w = 0; w < wpos; ++w) in = step(s.agg[w], in);
        // the next span's maps are written after the next pass of the barrier above at the earliest by this block's
        // warps that have read these: one more block barrier
        __syncthreads();
    } else {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wpos) in = run;
            run = step(s.agg[w], run);
        }
        __syncthreads();
    }
    return in;
}

// Forward: S steps a thread, W warps a block, CL blocks a cluster.
template <typename T, int E, int S, int W, int CL>
__global__ void __launch_bounds__(32 * W, W == 8 ? 4 : 1) glr_forward_kernel(const GlrArgs a)
{
    __shared__ Meet<E, W, CL> meet;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = CL > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / CL;                // (sequence, strip of channels)
    const int64_t b = unit / a.strips;
    const int64_t c = (unit - b * a.strips) * (32 * E) + lane * E;
    const bool on = c < a.C;                             // E divides C
    constexpr int64_t SPAN = (int64_t)S * W * CL;
    using V = Pack<T, E>;
    const int64_t first = ((int64_t)rank * W + warp) * S;    // this thread's first step within a span
    const T* X = reinterpret_cast<const T*>(a.x) + b * a.xb + c;
    const T* R = reinterpret_cast<const T*>(a.r) + b * a.rb + c;
    const T* G = reinterpret_cast<const T*>(a.g) + b * a.gb + c;
    T* Y = reinterpret_cast<T*>(a.y) + b * a.T * a.C + c;
    const unsigned char* Z = a.reset ? a.reset + b * a.T : nullptr;
    float* K = a.kept ? a.kept + b * ((a.T + kSteps - 1) / kSteps) * a.C + c : nullptr;

    float t0[E], t1[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        t0[e] = on ? -softplus_of(a.decay[c + e]) : 0.0f;
        t1[e] = on && a.h0 ? a.h0[b * a.C + c + e] : 0.0f;
    }
    const F<E> neg_lambda = F<E>::of(t0), one = F<E>::all(1.0f), zero = F<E>::all(0.0f);
    F<E> run = F<E>::of(t1);
    if constexpr (CL > 1) cluster_sync_all();            // every block of the cluster runs before its memory is written

    int parity = 0;
    for (int64_t base = 0; base < a.T; base += SPAN, parity ^= 1) {
        const int64_t t = base + first;
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - t));
        V qx[S], qr[S], qg[S];
        uint32_t cut = 0;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            qx[i] = qr[i] = qg[i] = V::zero();
            if (i < live && on) {
                qr[i] = V::load(R + (t + i) * a.rt);
                qg[i] = V::load(G + (t + i) * a.gt);
                qx[i] = V::load(X + (t + i) * a.xt);
            }
        }
        if (Z) {
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (i < live && Z[t + i]) cut |= 1u << i;
        }
        F<E> fa[S], bb[S], L = zero, B = zero;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            float vx[E], vr[E], vg[E];
            qx[i].unpack(vx);
            qr[i].unpack(vr);
            qg[i].unpack(vg);
            const F<E> s = rcp_of(one + exp_minus<115>(F<E>::of(vr)));
            const F<E> l = s * (i < live ? neg_lambda : zero);       // past the end: a = 1
            fa[i] = factor_of(l);
            // m sigmoid(g) = sqrt(m^2) / (1 + e) = m^2 / sqrt(m^2 (1 + e)^2), one rsqrt
            const F<E> m2 = one_minus_sq(fa[i]), q = one + exp_minus<60>(F<E>::of(vg));
            const F<E> w = m2 * each(m2 * q * q, [](float u) { return rsq(u < kTiny ? kTiny : u); });
            bb[i] = w * F<E>::of(vx);
            const bool z = cut >> i & 1;
            L = z ? F<E>::all(-INFINITY) : L + l;
            B = walk(fa[i], bb[i], z ? zero : B);
        }
        F<E> h = exchange<E, W, CL>(meet, parity, warp, rank, L, B, run);
        if (K && live > 0 && on) {
            float f[E];
            h.get(f);
#pragma unroll
            for (int e = 0; e < E; ++e) K[(t / kSteps) * a.C + e] = f[e];
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            h = walk(fa[i], bb[i], cut >> i & 1 ? zero : h);
            if (i < live && on) {
                float f[E];
                h.get(f);
                V::pack(f).store(Y + (t + i) * a.C);
            }
        }
    }
    if (a.h_last && on && rank == 0 && warp == 0) {
        float f[E];
        run.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) a.h_last[b * a.C + c + e] = f[e];
    }
}

// Backward: the same split, walked from the end of the sequence.
template <typename T, int E, int S, int W, int CL>
__global__ void __launch_bounds__(32 * W, W == 8 ? 2 : 1) glr_backward_kernel(const GlrArgs a)
{
    static_assert(S == kSteps, "a thread's steps begin at a kept state");
    __shared__ Meet<E, W, CL> meet;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = CL > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / CL;
    const int64_t b = unit / a.strips;
    const int64_t c = (unit - b * a.strips) * (32 * E) + lane * E;
    const bool on = c < a.C;
    constexpr int64_t SPAN = (int64_t)S * W * CL;
    using V = Pack<T, E>;
    const int64_t first = ((int64_t)rank * W + warp) * S;
    const T* X = reinterpret_cast<const T*>(a.x) + b * a.xb + c;
    const T* R = reinterpret_cast<const T*>(a.r) + b * a.rb + c;
    const T* G = reinterpret_cast<const T*>(a.g) + b * a.gb + c;
    const int64_t dense = b * a.T * a.C + c;
    const T* D = reinterpret_cast<const T*>(a.dy) + dense;
    const unsigned char* Z = a.reset ? a.reset + b * a.T : nullptr;
    const float* K = a.kept + b * ((a.T + kSteps - 1) / kSteps) * a.C + c;

    float t0[E], t1[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        t0[e] = on ? -softplus_of(a.decay[c + e]) : 0.0f;
        t1[e] = on && a.dh_last ? a.dh_last[b * a.C + c + e] : 0.0f;
    }
    const F<E> neg_lambda = F<E>::of(t0), one = F<E>::all(1.0f), zero = F<E>::all(0.0f);
    F<E> run = F<E>::of(t1);
    double acc[E];                                       // sum of dL L
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0;
    if constexpr (CL > 1) cluster_sync_all();

    int parity = 0;
    for (int64_t base = (a.T - 1) / SPAN * SPAN; base >= 0; base -= SPAN, parity ^= 1) {
        const int64_t t = base + first;
        const int live = (int)min((int64_t)S, max((int64_t)0, a.T - t));
        V qx[S], qr[S], qg[S], qd[S];
        uint32_t cut = 0;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            qx[i] = qr[i] = qg[i] = qd[i] = V::zero();
            if (i < live && on) {
                qr[i] = V::load(R + (t + i) * a.rt);
                qg[i] = V::load(G + (t + i) * a.gt);
                qx[i] = V::load(X + (t + i) * a.xt);
                qd[i] = V::load(D + (t + i) * a.C);
            }
        }
        if (Z) {
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (i < live && Z[t + i]) cut |= 1u << i;
        }
        F<E> h = zero;
        if (live > 0 && on) {
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = K[(t / kSteps) * a.C + e];
            h = F<E>::of(f);
        }
        // per step: the factor, and what d multiplies in each gradient:
        //   dx = d cx,  dg = dx cg,  dL L = d cl,  dr = dL L cr
        F<E> fa[S], cx[S], cg[S], cl[S], cr[S], L = zero;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            float vx[E], vr[E], vg[E];
            qx[i].unpack(vx);
            qr[i].unpack(vr);
            qg[i].unpack(vg);
            const F<E> er = exp_minus<115>(F<E>::of(vr)), eg = exp_minus<115>(F<E>::of(vg));
            const F<E> s = rcp_of(one + er), sg = rcp_of(one + eg), x = F<E>::of(vx);
            const F<E> l = s * (i < live ? neg_lambda : zero);
            fa[i] = factor_of(l);
            const F<E> m2 = one_minus_sq(fa[i]);
            const F<E> rm = each(m2, [](float u) { return u < kTiny ? 0.0f : rsq(u); });   // 1 / m; L / m goes to 0 with L
            const F<E> av = each(fa[i], [](float v) { return value_of(v); });
            const F<E> u = sg * x, hp = cut >> i & 1 ? zero : h;
            cx[i] = m2 * rm * sg;
            cg[i] = x * (eg * sg);
            cr[i] = er * s;
            cl[i] = av * l * fma(av * F<E>::all(-1.0f), u * rm, hp);
            h = walk(fa[i], cx[i] * x, hp);
            L = cut >> i & 1 ? F<E>::all(-INFINITY) : L + l;
        }
        // the map of these steps, from the last to the first: gamma -> a (gamma + dy)
        F<E> B = zero;
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
            float vd[E];
            qd[i].unpack(vd);
            const F<E> d = B + F<E>::of(vd);
            B = cut >> i & 1 ? zero : walk(fa[i], zero, d);
        }
        // (a reset cuts off what comes from later steps, a NaN of which would pass the sum of L)
        if (cut) L = F<E>::all(-INFINITY);
        F<E> flow = exchange<E, W, CL>(meet, parity, W - 1 - warp, CL - 1 - rank, L, B, run);
        F<E> part = zero;
#pragma unroll
        for (int i = S - 1; i >= 0; --i) {
            if (i < live) {
                float vd[E], f[E];
                qd[i].unpack(vd);
                const F<E> d = flow + F<E>::of(vd);
                const F<E> ox = d * cx[i], ol = d * cl[i];
                part = part + ol;
                flow = cut >> i & 1 ? zero : walk(fa[i], zero, d);
                if (on) {
                    const int64_t at = dense + (t + i) * a.C;
                    if (a.dx) {
                        ox.get(f);
                        V::pack(f).store(reinterpret_cast<T*>(a.dx) + at);
                    }
                    if (a.dr) {
                        (ol * cr[i]).get(f);
                        V::pack(f).store(reinterpret_cast<T*>(a.dr) + at);
                    }
                    if (a.dg) {
                        (ox * cg[i]).get(f);
                        V::pack(f).store(reinterpret_cast<T*>(a.dg) + at);
                    }
                }
            }
        }
        float f[E];
        part.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += (double)f[e];
    }
    if (a.dh0 && on && rank == 0 && warp == 0) {
        float f[E];
        run.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) a.dh0[b * a.C + c + e] = f[e];
    }
    if (a.part) {
        __shared__ double red[W][E][32];
#pragma unroll
        for (int e = 0; e < E; ++e) red[warp][e][lane] = acc[e];
        __syncthreads();
        if (warp == 0 && on) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                double v = 0.0;
                for (int w = 0; w < W; ++w) v += red[w][e][lane];
                a.part[(b * CL + rank) * a.C + c + e] = v;
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
    if (s->channels > ((int64_t)1 << 24) || s->time > ((int64_t)1 << 40) || s->batch > ((int64_t)1 << 31) ||
        s->batch * ((s->channels + 31) / 32) > ((int64_t)1 << 27))
        return gl_fail(KAN_ERR_UNSUPPORTED, "sizes too large");
    return KAN_OK;
}

struct GlrPlan {
    int vec, cluster, warps, steps, strips;
};

// Blocks of 8 warps; as many blocks of a cluster side by side in time as fill the SMs once (kResident blocks fit), at
// most 8, no more than the sequence has steps for.  A block of one warp where 8 steps (or one) are all there is.
GlrPlan plan_of(const kan_glr_shape& s, int vec, bool backward)
{
    GlrPlan P{};
    P.vec = vec;
    P.strips = (int)((s.channels + 32 * vec - 1) / (32 * vec));
    P.steps = s.time == 1 && !backward ? 1 : kSteps;
    P.warps = s.time <= kSteps ? 1 : 8;
    P.cluster = 1;
    const int64_t resident = 148 * (backward ? 2 : 4), units = s.batch * P.strips;
    if (P.warps == 8)
        while (P.cluster < kMaxCluster && units * P.cluster * 2 <= resident && s.time > (int64_t)P.cluster * 8 * kSteps)
            P.cluster *= 2;
    return P;
}

template <typename K> cudaError_t launch(K kernel, int warps, int cluster, const GlrArgs& a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * a.strips * cluster));
    cfg.blockDim = dim3(32 * warps);
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

template <typename T, int E> cudaError_t forward_of(const GlrPlan& P, const GlrArgs& a, cudaStream_t st)
{
    if (P.steps == 1) return launch(glr_forward_kernel<T, E, 1, 1, 1>, 1, 1, a, st);
    if (P.warps == 1) return launch(glr_forward_kernel<T, E, kSteps, 1, 1>, 1, 1, a, st);
    switch (P.cluster) {
    case 1: return launch(glr_forward_kernel<T, E, kSteps, 8, 1>, 8, 1, a, st);
    case 2: return launch(glr_forward_kernel<T, E, kSteps, 8, 2>, 8, 2, a, st);
    case 4: return launch(glr_forward_kernel<T, E, kSteps, 8, 4>, 8, 4, a, st);
    default: return launch(glr_forward_kernel<T, E, kSteps, 8, 8>, 8, 8, a, st);
    }
}

template <typename T, int E> cudaError_t backward_of(const GlrPlan& P, const GlrArgs& a, cudaStream_t st)
{
    if (P.warps == 1) return launch(glr_backward_kernel<T, E, kSteps, 1, 1>, 1, 1, a, st);
    switch (P.cluster) {
    case 1: return launch(glr_backward_kernel<T, E, kSteps, 8, 1>, 8, 1, a, st);
    case 2: return launch(glr_backward_kernel<T, E, kSteps, 8, 2>, 8, 2, a, st);
    case 4: return launch(glr_backward_kernel<T, E, kSteps, 8, 4>, 8, 4, a, st);
    default: return launch(glr_backward_kernel<T, E, kSteps, 8, 8>, 8, 8, a, st);
    }
}

// Two bf16 channels per thread where every row of every operand begins on 4 bytes.
int vec_of(const kan_glr_shape& s, const GlrArgs& a)
{
    if (s.dtype == KAN_F32) return 1;
    const uint64_t odd = (uint64_t)(s.channels | s.x_stride_b | s.x_stride_t | s.r_stride_b | s.r_stride_t | s.g_stride_b |
                                    s.g_stride_t) & 1;
    const uint64_t addr = (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.r) |
                           reinterpret_cast<uintptr_t>(a.g) | reinterpret_cast<uintptr_t>(a.y) |
                           reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.dx) |
                           reinterpret_cast<uintptr_t>(a.dr) | reinterpret_cast<uintptr_t>(a.dg)) & 3;
    return odd || addr ? 1 : 2;
}

void common_args(const kan_glr_shape& s, GlrArgs& a)
{
    a.xb = s.x_stride_b, a.xt = s.x_stride_t;
    a.rb = s.r_stride_b, a.rt = s.r_stride_t;
    a.gb = s.g_stride_b, a.gt = s.g_stride_t;
    a.B = s.batch, a.T = s.time, a.C = s.channels;
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
    const GlrPlan P = plan_of(*s, vec_of(*s, a), false);
    a.strips = P.strips;
    if (s->dtype == KAN_F32) e = forward_of<float, 1>(P, a, cs);
    else e = P.vec == 2 ? forward_of<__nv_bfloat16, 2>(P, a, cs) : forward_of<__nv_bfloat16, 1>(P, a, cs);
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
    const GlrPlan P = plan_of(*s, vec_of(*s, a), true);
    a.strips = P.strips;
    const int64_t parts = s->batch * P.cluster;
    if (ddecay) {
        if (!workspace || ws_bytes < (size_t)parts * s->channels * sizeof(double))
            return gl_fail(KAN_ERR_WORKSPACE, "workspace too small");
        a.part = reinterpret_cast<double*>(workspace);
    }
    if (s->dtype == KAN_F32) e = backward_of<float, 1>(P, a, cs);
    else e = P.vec == 2 ? backward_of<__nv_bfloat16, 2>(P, a, cs) : backward_of<__nv_bfloat16, 1>(P, a, cs);
    if (e == cudaSuccess && ddecay) {
        glr_decay_kernel<<<(unsigned)((s->channels + 127) / 128), 128, 0, cs>>>(a.part, parts, s->channels, decay, ddecay);
        count_launch();
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

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
constexpr float kHard = -2.0f;    // the factor of a map that a reset cuts

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

// What the CUDA functions give: the accurate ones for fp32 operands, the fast ones (about two units in the last place
// of fp32 for these arguments) for bf16 operands.
template <typename T> __device__ __forceinline__ float exp_of(float v) { return sizeof(T) == 4 ? expf(v) : __expf(v); }
template <typename T> __device__ __forceinline__ float recip(float v) { return sizeof(T) == 4 ? __frcp_rn(v) : __fdividef(1.0f, v); }
// sigmoid(v), and 1 - sigmoid(v) without cancellation.  Below -80 the sigmoid is held at e^-80, so that e stays finite;
// a NaN passes.
template <typename T> __device__ __forceinline__ float sigmoid_of(float v, float& rest)
{
    const float e = exp_of<T>(-v > 80.0f ? 80.0f : -v);
    const float s = recip<T>(1.0f + e);
    rest = e * s;
    return s;
}
template <typename T> __device__ __forceinline__ float sigmoid_of(float v)
{
    float rest;
    return sigmoid_of<T>(v, rest);
}

// Factor: a number v that stands for A in [0, 1].  v in (-1, 0]: A = 1 + v;  v > 0: A = v;  v = kHard: A = 0, and what
// it multiplies is cut off even if it is not finite (a reset, or a product below fp32's range).
constexpr float kTiny = 1e-37f;

// The factor exp(L), L <= 0 (a NaN passes).
template <typename T> __device__ __forceinline__ float factor_of(float L)
{
    const float big = exp_of<T>(L);
    // exp(L) - 1 = sum_{k=1..8} L^k / k!; the next term is below 2^-26 of the sum at L = -0.5
    float s = fmaf(L, 1.0f / 40320.0f, 1.0f / 5040.0f);
    s = fmaf(s, L, 1.0f / 720.0f);
    s = fmaf(s, L, 1.0f / 120.0f);
    s = fmaf(s, L, 1.0f / 24.0f);
    s = fmaf(s, L, 1.0f / 6.0f);
    s = fmaf(s, L, 0.5f);
    s = fmaf(s, L, 1.0f);
    return L > -0.5f ? s * L : (big < kTiny ? kTiny : big);
}
__device__ __forceinline__ float value_of(float v) { return v > 0.0f ? v : 1.0f + v; }      // not for kHard
__device__ __forceinline__ float one_minus_sq(float v) { return v > 0.0f ? fmaf(-v, v, 1.0f) : -v * (2.0f + v); }
// A h + B, v not kHard
__device__ __forceinline__ float walk(float v, float B, float h)
{
    return fmaf(v, h, B) + (v > 0.0f ? 0.0f : h);
}

template <typename T> __device__ __forceinline__ float sqrt_of(float v) { return sizeof(T) == 4 ? __fsqrt_rn(v) : v * rsqrtf(fmaxf(v, 1e-37f)); }

__device__ __forceinline__ float softplus_of(float d) { return fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d))); }

__device__ __forceinline__ float apply(float v, float B, float h) { return v == kHard ? B : walk(v, B, h); }
// (V, B) first, then (v, b)
__device__ __forceinline__ void compose(float& V, float& B, float v, float b)
{
    B = apply(v, b, B);
    const float sum = fmaf(V, v, V + v), prod = value_of(V) * value_of(v);
    const bool small = V > 0.0f || v > 0.0f || sum < -0.5f;   // the product is kept as A
    V = V == kHard || v == kHard || (small && prod < kTiny) ? kHard : (small ? prod : sum);
}

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

// Exchange of one step of the cluster: every thread gives its map (P, B); on
// return each thread holds the state that enters its steps in `in`, and `run`
// has moved past the whole cluster's steps.  Position 0 comes first in the
// direction of the scan.
template <int VEC, int W, int CL>
__device__ __forceinline__ void exchange(float2 (*agg)[VEC][32], float2 (*tot)[CL][VEC][32], int parity, int wpos,
                                         int cpos, const float (&P)[VEC], const float (&B)[VEC], float (&run)[VEC],
                                         float (&in)[VEC])
{
    const int lane = threadIdx.x & 31;
    if constexpr (W * CL == 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            in[e] = run[e];
            run[e] = apply(P[e], B[e], run[e]);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) agg[wpos][e][lane] = make_float2(P[e], B[e]);
    __syncthreads();
    float Pp[VEC], Bp[VEC], Pt[VEC], Bt[VEC];            // what lies before this warp in the block; the whole block
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        Pt[e] = 0.0f;
        Bt[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wpos) {
                Pp[e] = Pt[e];
                Bp[e] = Bt[e];
            }
            const float2 q = agg[w][e][lane];
            compose(Pt[e], Bt[e], q.x, q.y);
        }
    }
    if constexpr (CL > 1) {
        if (wpos == 0) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
#pragma unroll
                for (int q = 0; q < CL; ++q) st_cluster(&tot[parity][cpos][e][lane], q, make_float2(Pt[e], Bt[e]));
        }
        cluster_sync_all();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float h = run[e];
#pragma unroll
            for (int q = 0; q < CL; ++q) {
                if (q == cpos) in[e] = h;
                const float2 v = tot[parity][q][e][lane];
                h = apply(v.x, v.y, h);
            }
            run[e] = h;
            in[e] = apply(Pp[e], Bp[e], in[e]);
        }
    } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            in[e] = apply(Pp[e], Bp[e], run[e]);
            run[e] = apply(Pt[e], Bt[e], run[e]);
        }
    }
}

template <typename T, int VEC, int S, int W, int CL, bool BWD>
__global__ void __launch_bounds__(32 * W) glr_kernel(const GlrArgs a)
{
    __shared__ float2 agg[W][VEC][32];
    __shared__ float2 tot[2][CL][VEC][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = CL > 1 ? (int)cluster_rank() : 0;
    const int64_t unit = blockIdx.x / CL;                // (sequence, strip of channels)
    const int64_t b = unit / a.strips;
    const int64_t c = (unit - b * a.strips) * (32 * VEC) + lane * VEC;
    const bool on = c < a.C;                             // VEC divides C
    const int wpos = BWD ? W - 1 - warp : warp, cpos = BWD ? CL - 1 - rank : rank;
    constexpr int64_t SPAN = (int64_t)S * W * CL;
    const int64_t spans = (a.T + SPAN - 1) / SPAN;
    const int64_t off = ((int64_t)rank * W + warp) * S;  // this thread's first step within a span
    using V = Pack<T, VEC>;
    const T* X = reinterpret_cast<const T*>(a.x) + b * a.xb + c;
    const T* R = reinterpret_cast<const T*>(a.r) + b * a.rb + c;
    const T* G = reinterpret_cast<const T*>(a.g) + b * a.gb + c;
    const int64_t bt = b * a.T;
    const int64_t blocks = (a.T + kSteps - 1) / kSteps;

    float lambda[VEC], run[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        lambda[e] = on ? softplus_of(a.decay[c + e]) : 0.0f;
        const float* first = BWD ? a.dh_last : a.h0;
        run[e] = on && first ? first[b * a.C + c + e] : 0.0f;
    }
    double acc[VEC];                                     // sum of dL L
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.0;

    V qx[S], qr[S], qg[S], qd[BWD ? S : 1];
    float kept[VEC];
    uint32_t cut = 0, live = 0;                          // steps of this thread: reset set; within the sequence
    auto fetch = [&](int64_t span) {
        const int64_t t0 = span * SPAN + off;
        cut = live = 0;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int64_t t = t0 + i;
            if (t < a.T) {
                live |= 1u << i;
                if (a.reset && a.reset[bt + t]) cut |= 1u << i;
                if (on) {
                    qx[i] = V::load(X + t * a.xt);
                    qr[i] = V::load(R + t * a.rt);
                    qg[i] = V::load(G + t * a.gt);
                    if constexpr (BWD) qd[i] = V::load(reinterpret_cast<const T*>(a.dy) + (bt + t) * a.C + c);
                }
            }
        }
        if constexpr (BWD) {
            if (on && t0 < a.T) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) kept[e] = a.kept[(b * blocks + t0 / kSteps) * a.C + c + e];
            }
        }
    };
    fetch(BWD ? spans - 1 : 0);
    if constexpr (CL > 1) cluster_sync_all();            // every block of the cluster runs before its memory is written
    for (int64_t n = 0; n < spans; ++n) {
        const int64_t span = BWD ? spans - 1 - n : n;
        const int64_t t0 = span * SPAN + off;
        const uint32_t live_n = on ? live : 0, cut_n = cut;
        float fa[S][VEC], in[VEC];
        if constexpr (!BWD) {
            float bb[S][VEC], P[VEC], B[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) P[e] = B[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                float fx[VEC], fr[VEC], fg[VEC];
                qx[i].unpack(fx);
                qr[i].unpack(fr);
                qg[i].unpack(fg);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    fa[i][e] = factor_of<T>(-lambda[e] * sigmoid_of<T>(fr[e]));
                    bb[i][e] = sqrt_of<T>(one_minus_sq(fa[i][e])) * (sigmoid_of<T>(fg[e]) * fx[e]);
                    if (!(live_n >> i & 1)) fa[i][e] = bb[i][e] = 0.0f;
                    compose(P[e], B[e], cut_n >> i & 1 ? kHard : fa[i][e], bb[i][e]);
                }
            }
            if (n + 1 < spans) fetch(span + 1);
            exchange<VEC, W, CL>(agg, tot, (int)(n & 1), wpos, cpos, P, B, run, in);
            if (a.kept && live_n) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) a.kept[(b * blocks + t0 / kSteps) * a.C + c + e] = in[e];
            }
            T* Y = reinterpret_cast<T*>(a.y) + (bt + t0) * a.C + c;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                if (live_n >> i & 1) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) in[e] = apply(cut_n >> i & 1 ? kHard : fa[i][e], bb[i][e], in[e]);
                    V::pack(in).store(Y + (int64_t)i * a.C);
                }
            }
        } else {
            float hp[S][VEC], P[VEC], B[VEC];
            // the states before each step, from the kept one
#pragma unroll
            for (int e = 0; e < VEC; ++e) in[e] = live_n ? kept[e] : 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                float fx[VEC], fr[VEC], fg[VEC];
                qx[i].unpack(fx);
                qr[i].unpack(fr);
                qg[i].unpack(fg);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    fa[i][e] = factor_of<T>(-lambda[e] * sigmoid_of<T>(fr[e]));
                    const float bb = sqrt_of<T>(one_minus_sq(fa[i][e])) * (sigmoid_of<T>(fg[e]) * fx[e]);
                    hp[i][e] = cut_n >> i & 1 ? 0.0f : in[e];
                    in[e] = walk(fa[i][e], bb, hp[i][e]);
                    if (!(live_n >> i & 1)) fa[i][e] = 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) P[e] = B[e] = 0.0f;
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                float fd[VEC];
                qd[i].unpack(fd);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    // gamma -> a (gamma + dy): offset a dy
                    const float d = live_n >> i & 1 ? fd[e] : 0.0f;
                    if (cut_n >> i & 1) {
                        P[e] = kHard;
                        B[e] = 0.0f;
                    } else {
                        compose(P[e], B[e], fa[i][e], walk(fa[i][e], 0.0f, d));
                    }
                }
            }
            exchange<VEC, W, CL>(agg, tot, (int)(n & 1), wpos, cpos, P, B, run, in);
            const int64_t o = (bt + t0) * a.C + c;
            float part[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) part[e] = 0.0f;
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                if (!(live_n >> i & 1)) continue;
                float fx[VEC], fr[VEC], fg[VEC], fd[VEC], ox[VEC], orr[VEC], og[VEC];
                qx[i].unpack(fx);
                qr[i].unpack(fr);
                qg[i].unpack(fg);
                qd[i].unpack(fd);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float rest_r, rest_g;
                    const float s = sigmoid_of<T>(fr[e], rest_r), L = -lambda[e] * s, av = value_of(fa[i][e]);
                    const float sg = sigmoid_of<T>(fg[e], rest_g), m = sqrt_of<T>(one_minus_sq(fa[i][e]));
                    // as L -> 0, L / m -> 0: no division by zero
                    const float rm = m > 1e-18f ? recip<T>(m) : 0.0f;
                    const float d = fd[e] + in[e];
                    const float u = sg * fx[e];
                    const float dl = d * av * (hp[i][e] - av * u * rm) * L;
                    ox[e] = d * m * sg;
                    og[e] = ox[e] * fx[e] * rest_g;
                    orr[e] = dl * rest_r;
                    part[e] += dl;
                    in[e] = cut_n >> i & 1 ? 0.0f : walk(fa[i][e], 0.0f, d);
                }
                const int64_t at = o + (int64_t)i * a.C;
                if (a.dx) V::pack(ox).store(reinterpret_cast<T*>(a.dx) + at);
                if (a.dr) V::pack(orr).store(reinterpret_cast<T*>(a.dr) + at);
                if (a.dg) V::pack(og).store(reinterpret_cast<T*>(a.dg) + at);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += (double)part[e];
            if (n + 1 < spans) fetch(span - 1);
        }
    }
    float* last = BWD ? a.dh0 : a.h_last;
    if (last && on && rank == 0 && warp == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) last[b * a.C + c + e] = run[e];
    }
    if constexpr (BWD) {
        if (a.part) {
            __shared__ double red[W][VEC][32];
#pragma unroll
            for (int e = 0; e < VEC; ++e) red[warp][e][lane] = acc[e];
            __syncthreads();
            if (warp == 0 && on) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    double v = 0.0;
                    for (int w = 0; w < W; ++w) v += red[w][e][lane];
                    a.part[(b * CL + rank) * a.C + c + e] = v;
                }
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

GlrPlan plan_of(const kan_glr_shape& s, int vec)
{
    GlrPlan P{};
    P.vec = vec;
    P.strips = (int)((s.channels + 32 * vec - 1) / (32 * vec));
    P.warps = 8;
    P.steps = kSteps;
    P.cluster = 8;
    return P;
}

template <typename T, int VEC, int S, int W, int CL, bool BWD>
cudaError_t launch(const GlrArgs& a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.B * a.strips * CL));
    cfg.blockDim = dim3(32 * W);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CL > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, glr_kernel<T, VEC, S, W, CL, BWD>, a);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T, int VEC, bool BWD>
cudaError_t run(const GlrPlan&, const GlrArgs& a, cudaStream_t st)
{
    return launch<T, VEC, kSteps, 8, 8, BWD>(a, st);
}

template <bool BWD> cudaError_t run_any(const kan_glr_shape& s, const GlrPlan& P, const GlrArgs& a, cudaStream_t st)
{
    if (s.dtype == KAN_F32) return run<float, 1, BWD>(P, a, st);
    return P.vec == 2 ? run<__nv_bfloat16, 2, BWD>(P, a, st) : run<__nv_bfloat16, 1, BWD>(P, a, st);
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

constexpr int kMaxCluster = 8;

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
    const GlrPlan P = plan_of(*s, vec_of(*s, a));
    a.strips = P.strips;
    e = run_any<false>(*s, P, a, cs);
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
    const GlrPlan P = plan_of(*s, vec_of(*s, a));
    a.strips = P.strips;
    const int64_t parts = s->batch * P.cluster;
    if (ddecay) {
        if (!workspace || ws_bytes < (size_t)parts * s->channels * sizeof(double))
            return gl_fail(KAN_ERR_WORKSPACE, "workspace too small");
        a.part = reinterpret_cast<double*>(workspace);
    }
    e = run_any<true>(*s, P, a, cs);
    if (e == cudaSuccess && ddecay) {
        glr_decay_kernel<<<(unsigned)((s->channels + 127) / 128), 128, 0, cs>>>(a.part, parts, s->channels, decay, ddecay);
        count_launch();
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? KAN_OK : gl_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

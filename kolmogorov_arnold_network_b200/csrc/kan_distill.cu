// kan_distill.cu -- distillation from a teacher's top logits: the loss of each
// row and its gradient.
//
// Row n has student logits z over the vocabulary and K teacher entries
// (id_k, t_k); with temperature T, over the entries that count:
//   p = softmax(t / T),  q = softmax(z / T)
//   loss_n = w_n T^2 sum_k p_k (log p_k - log q_{id_k})
//   dz_v   = dloss_n w_n T (q_v - sum_{k: id_k = v} p_k)
//
// exp((z - max) / T) is taken as 2^((z - m) k) with m the row's maximum and
// k = log2(e) / T.  The difference comes first: it is exact for the logits
// next to the maximum, and a row that a mask fills with its type's lowest value
// stays finite.
#include <algorithm>
#include <atomic>

#include "kan_device.cuh"
#include "kan_vec.cuh"

namespace kan {
namespace {

constexpr int kMaxK = 1024;       // teacher entries per row
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct DistArgs {
    const void* z;
    const void* ids;
    const float* teacher;
    const float* weight;          // [N] or null (1)
    const float* dloss;           // [N] or null (1)
    float* loss;                  // [N] or null
    float2* stats;                // [N] (m, sum of 2^((z - m) k))
    void* dz;
    int64_t n, vocab, ld, ld_grad;
    int k, id_bytes;
    float temp, inv_temp, scale2;   // scale2 = log2(e) / T
    unsigned int* status;
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float block_max(float v, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, red[w]);
    __syncthreads();
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kWarps; ++w) v += red[w];
    __syncthreads();
    return v;
}

// The teacher's entries of a row, in shared memory.
struct Teacher {
    int32_t id[kMaxK];            // -1: the entry does not count
    float p[kMaxK];               // its probability
};

// Loads row n's entries and makes their probabilities; logp[i] is log p of entry threadIdx.x + i kThreads.  Returns
// whether any entry counts.
__device__ bool load_teacher(const DistArgs& a, int64_t n, Teacher& t, float* red, float (&logp)[kMaxK / kThreads])
{
    float mx = neg_inf();
    bool any = false;
    float v[kMaxK / kThreads];
#pragma unroll
    for (int i = 0; i < kMaxK / kThreads; ++i) {
        const int j = threadIdx.x + i * kThreads;
        v[i] = neg_inf();
        if (j < a.k) {
            const int64_t at = n * a.k + j;
            int64_t id = a.id_bytes == 8 ? reinterpret_cast<const int64_t*>(a.ids)[at]
                                         : (int64_t)reinterpret_cast<const int32_t*>(a.ids)[at];
            if (id >= a.vocab) {
                record_status(a.status, KAN_ERR_DEVICE_CHECK);
                id = -1;
            }
            const float x = id < 0 ? neg_inf() : a.teacher[at];
            if (x == neg_inf()) id = -1;
            t.id[j] = id < 0 ? -1 : (int32_t)id;
            v[i] = x;
            any |= id >= 0;
            mx = fmaxf(mx, x);
        }
    }
    any = __syncthreads_or(any);
    if (!any) return false;
    mx = block_max(mx, red);
    float e[kMaxK / kThreads], s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxK / kThreads; ++i) {
        e[i] = v[i] == neg_inf() ? 0.0f : expf((v[i] - mx) * a.inv_temp);
        s += e[i];
    }
    s = block_sum(s, red);
    const float ls = logf(s);
#pragma unroll
    for (int i = 0; i < kMaxK / kThreads; ++i) {
        const int j = threadIdx.x + i * kThreads;
        logp[i] = (v[i] - mx) * a.inv_temp - ls;
        if (j < a.k) t.p[j] = e[i] / s;
    }
    __syncthreads();
    return true;
}

template <typename T> __device__ __forceinline__ float elem(const T* p)
{
    float f[1];
    Pack<T, 1>::load(p).unpack(f);
    return f[0];
}

// A row in 16-byte vectors: elements before the first aligned address, vectors, elements after the last one.
template <typename T> struct RowSplit {
    static constexpr int N = 16 / (int)sizeof(T);
    int64_t head, vecs, tail0;
    __device__ RowSplit(const T* row, int64_t vocab)
    {
        const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
        head = min(vocab, (int64_t)((N - off) % N));
        vecs = (vocab - head) / N;
        tail0 = head + vecs * N;
    }
};

// 2^((z - m) k)
__device__ __forceinline__ float term(float z, float m, float k) { return ex2((z - m) * k); }

// (m, sum) of a row in one reading: each thread keeps a running maximum and the sum relative to it.
template <typename T> __device__ float2 row_stats(const DistArgs& a, const T* row, float* red)
{
    constexpr int N = RowSplit<T>::N;
    const RowSplit<T> sp(row, a.vocab);
    float m = neg_inf(), s = 0.0f;
    auto add = [&](const auto& f) {
        constexpr int CNT = sizeof(f) / sizeof(float);
        float vm = f[0];
#pragma unroll
        for (int e = 1; e < CNT; ++e) vm = fmaxf(vm, f[e]);
        if (vm > m) {
            s *= term(m, vm, a.scale2);                  // 0 for the first one
            m = vm;
        }
        const float ref = m == neg_inf() ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < CNT; ++e) s += term(f[e], ref, a.scale2);
    };
    for (int64_t i = threadIdx.x; i < sp.vecs; i += kThreads) {
        float f[N];
        Pack<T, N>::load(row + sp.head + i * N).unpack(f);
        add(f);
    }
    if (threadIdx.x < sp.head) {
        const float f[1] = {elem(row + threadIdx.x)};
        add(f);
    }
    if (sp.tail0 + threadIdx.x < a.vocab) {
        const float f[1] = {elem(row + sp.tail0 + threadIdx.x)};
        add(f);
    }
    const float M = block_max(m, red);
    s = block_sum(m == neg_inf() ? s : s * term(m, M, a.scale2), red);
    // a row of -inf alone has no distribution
    if (M == neg_inf()) s = __int_as_float(0x7fc00000);
    return make_float2(M, s);
}

template <typename T> __global__ void __launch_bounds__(kThreads) distill_forward_kernel(const DistArgs a)
{
    __shared__ Teacher t;
    __shared__ float red[kWarps];
    const int64_t n = blockIdx.x;
    const float w = a.weight ? a.weight[n] : 1.0f;
    float logp[kMaxK / kThreads];
    if (w == 0.0f || !load_teacher(a, n, t, red, logp)) {
        if (threadIdx.x == 0) {
            a.loss[n] = 0.0f;
            a.stats[n] = make_float2(0.0f, 1.0f);
        }
        return;
    }
    const T* row = reinterpret_cast<const T*>(a.z) + n * a.ld;
    const float2 st = row_stats<T>(a, row, red);
    const float lsum = logf(st.y);
    float l = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxK / kThreads; ++i) {
        const int j = threadIdx.x + i * kThreads;
        if (j < a.k && t.id[j] >= 0 && !(t.p[j] == 0.0f))
            l += t.p[j] * (logp[i] - ((elem(row + t.id[j]) - st.x) * a.inv_temp - lsum));
    }
    l = block_sum(l, red);
    if (threadIdx.x == 0) {
        a.loss[n] = w * a.temp * a.temp * l;
        a.stats[n] = st;
    }
}

// The teacher's part of the gradient, after the row is written: one thread for each entry that is the first with its id.
// zk: the student's logits at this thread's entries (read before the row, which may lie in the same place, was written).
template <typename T>
__device__ void subtract_teacher(const DistArgs& a, const Teacher& t, const float (&zk)[kMaxK / kThreads], T* out,
                                 float2 st, float c)
{
    const float inv = 1.0f / st.y;
#pragma unroll
    for (int q = 0; q < kMaxK / kThreads; ++q) {
        const int j = threadIdx.x + q * kThreads;
        if (j >= a.k) break;
        const int32_t id = t.id[j];
        if (id < 0) continue;
        float p = 0.0f;
        bool first = true;
        for (int i = 0; i < a.k; ++i) {
            if (t.id[i] == id) {
                first &= i >= j;
                p += t.p[i];
            }
        }
        if (!first) continue;
        const float f[1] = {c * (term(zk[q], st.x, a.scale2) * inv - p)};
        Pack<T, 1>::pack(f).store(out + id);
    }
}

template <typename T> __global__ void __launch_bounds__(kThreads) distill_backward_kernel(const DistArgs a)
{
    constexpr int N = RowSplit<T>::N;
    __shared__ Teacher t;
    __shared__ float red[kWarps];
    const int64_t n = blockIdx.x;
    const float w = (a.weight ? a.weight[n] : 1.0f) * (a.dloss ? a.dloss[n] : 1.0f);
    T* out = reinterpret_cast<T*>(a.dz) + n * a.ld_grad;
    const RowSplit<T> so(out, a.vocab);
    float logp[kMaxK / kThreads];
    if (w == 0.0f || !load_teacher(a, n, t, red, logp)) {
        for (int64_t i = threadIdx.x; i < so.vecs; i += kThreads) Pack<T, N>::zero().store(out + so.head + i * N);
        if (threadIdx.x < so.head) Pack<T, 1>::zero().store(out + threadIdx.x);
        if (so.tail0 + threadIdx.x < a.vocab) Pack<T, 1>::zero().store(out + so.tail0 + threadIdx.x);
        return;
    }
    const T* row = reinterpret_cast<const T*>(a.z) + n * a.ld;
    const RowSplit<T> sp(row, a.vocab);
    const float2 st = a.stats[n];
    const float c = w * a.temp, cq = c / st.y;
    float zk[kMaxK / kThreads];
#pragma unroll
    for (int q = 0; q < kMaxK / kThreads; ++q) {
        const int j = threadIdx.x + q * kThreads;
        zk[q] = j < a.k && t.id[j] >= 0 ? elem(row + t.id[j]) : 0.0f;
    }
    __syncthreads();
    auto one = [&](int64_t v) {
        const float f[1] = {cq * term(elem(row + v), st.x, a.scale2)};
        Pack<T, 1>::pack(f).store(out + v);
    };
    if (sp.head == so.head) {
        for (int64_t i = threadIdx.x; i < sp.vecs; i += kThreads) {
            float f[N];
            Pack<T, N>::load(row + sp.head + i * N).unpack(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = cq * term(f[e], st.x, a.scale2);
            Pack<T, N>::pack(f).store(out + sp.head + i * N);
        }
        if (threadIdx.x < sp.head) one(threadIdx.x);
        if (sp.tail0 + threadIdx.x < a.vocab) one(sp.tail0 + threadIdx.x);
    } else {
        for (int64_t v = threadIdx.x; v < a.vocab; v += kThreads) one(v);
    }
    __syncthreads();
    subtract_teacher<T>(a, t, zk, out, st, c);
}

// ---- both in one pass ----
// A cluster of CL blocks takes a row at a time, a block a slice of it, which lies in its shared memory from the load to the
// store: the logits are read once and the gradient is written in their place there.  Two buffers: while a row is worked
// on, the next one is loaded and the last one stored, in bulk copies of whole 16-byte chunks (the elements of a row's or
// slice's broken chunks go by plain loads and stores).  The blocks of a cluster exchange the slices' (maximum, sum) and
// the logits at the teacher's tokens (for the loss, which block 0 writes) through st.async and an mbarrier.
struct FusedArgs {
    DistArgs d;
    int per;                      // elements of a slice (the last one may be shorter): whole chunks
    int buf;                      // bytes of a buffer
    int kp;                       // teacher entries, rounded up to 4
    int kpow;                     // and to a power of two, at most the block's threads
};

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
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float2 v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];" ::"r"(to), "r"(bar),
                 "f"(v.x), "f"(v.y)
                 : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %2, [%1];" ::"r"(to), "r"(bar), "f"(v)
                 : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes) : "memory");
}

// A sum kept relative to its own maximum m, relative to M instead (nothing to scale where there is no element).
__device__ __forceinline__ float rescale(float2 st, float M, float k) { return st.x == neg_inf() ? st.y : st.y * term(st.x, M, k); }
// (m, s) of the lanes together, in every lane
template <int LANES> __device__ __forceinline__ float2 join_lanes(float2 st, float k)
{
    float M = st.x;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float s = rescale(st, M, k);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return make_float2(M, s);
}

// Two fp32 values in the packed f32x2 instructions.
__device__ __forceinline__ uint64_t two(float x, float y)
{
    uint64_t q;
    asm("mov.b64 %0, {%1, %2};" : "=l"(q) : "f"(x), "f"(y));
    return q;
}
__device__ __forceinline__ void halves(uint64_t q, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(q)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ uint64_t ex2_2(uint64_t q)
{
    float x, y;
    halves(q, x, y);
    return two(ex2(x), ex2(y));
}
// Element pair i of a chunk.
__device__ __forceinline__ uint64_t pair(const Pack<float, 4>& c, int i) { return two(__uint_as_float(c.word(2 * i)), __uint_as_float(c.word(2 * i + 1))); }
__device__ __forceinline__ uint64_t pair(const Pack<__nv_bfloat16, 8>& c, int i)
{
    return two(__uint_as_float(c.word(i) << 16), __uint_as_float(c.word(i) & 0xFFFF0000u));
}
// The largest element (a NaN is passed over; the sums see it).
__device__ __forceinline__ float chunk_max(const Pack<float, 4>& c)
{
    return fmaxf(fmaxf(__uint_as_float(c.q.x), __uint_as_float(c.q.y)), fmaxf(__uint_as_float(c.q.z), __uint_as_float(c.q.w)));
}
__device__ __forceinline__ float chunk_max(const Pack<__nv_bfloat16, 8>& c)
{
    auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(h(c.q.x), h(c.q.y)), __hmax2(h(c.q.z), h(c.q.w)));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Beyond this magnitude m k may overflow: exponents are then taken from the difference z - m alone.
constexpr float kLarge = 1e30f;

// A thread's running (m, sum of 2^((z - m) k)) over chunks.  With bf16 logits the exponent is one multiply-add (z k - m k:
// m k's rounding, 2^-24 of it, is far below what the logits' own type resolves), with fp32 logits the difference first.
template <typename T> struct Running {
    static constexpr int N = 16 / (int)sizeof(T);
    float m = neg_inf(), mk = 0.0f;
    uint64_t acc = 0;                                    // two partial sums
    float k;
    __device__ __forceinline__ void add(const Pack<T, N>& c)
    {
        const float vm = chunk_max(c);
        if (vm > m) {
            const float f = term(m, vm, k);              // 0 for the first one
            acc = mul2(acc, two(f, f));
            m = vm;
            mk = m * k;
        }
        if (fabsf(m) < kLarge) {
            const uint64_t kk = two(k, k), off = sizeof(T) == 2 ? two(-mk, -mk) : two(-m, -m);
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                acc = add2(acc, ex2_2(sizeof(T) == 2 ? fma2(pair(c, i), kk, off) : mul2(add2(pair(c, i), off), kk)));
        } else {
            const float ref = m == neg_inf() ? 0.0f : m;
            float x[N], s = 0.0f;
            c.unpack(x);
#pragma unroll
            for (int e = 0; e < N; ++e) s += term(x[e], ref, k);
            acc = add2(acc, two(s, 0.0f));
        }
    }
    __device__ __forceinline__ float2 get() const
    {
        float x, y;
        halves(acc, x, y);
        return make_float2(m, x + y);
    }
};

template <typename T, int CL, int NT>
__global__ void __launch_bounds__(NT, NT == 512 ? 2 : 6) distill_fused_kernel(const FusedArgs f)
{
    constexpr int N = 16 / (int)sizeof(T), WARPS = NT / 32, J = 2;       // at most J entries a thread
    extern __shared__ __align__(128) unsigned char smem[];
    const DistArgs& a = f.d;
    int32_t* const tid_ = reinterpret_cast<int32_t*>(smem + 2 * (size_t)f.buf);      // [kp] ids of the entries, -1: none
    float* const te = reinterpret_cast<float*>(tid_ + f.kp);                         // [kp] exp((t - max) / T)
    float* const zk = te + f.kp;                                                     // [2][kp] block 0: logits at the entries
    __shared__ float2 wstat[WARPS], cstat[2][CL];
    __shared__ float wmax[WARPS], wsum[WARPS], wloss[WARPS];
    __shared__ int wvalid[WARPS];
    __shared__ uint64_t full[2], met[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CL > 1 ? (int)cluster_rank() : 0;
    const int64_t clusters = gridDim.x / CL;
    const int64_t v0 = (int64_t)rank * f.per;
    const int len = (int)min((int64_t)f.per, a.vocab - v0);
    const int warps_k = min(WARPS, (a.k + 31) / 32);                     // warps that hold entries
    if (tid == 0) {
        mbar_init(smem_addr(&full[0]), 1);
        mbar_init(smem_addr(&full[1]), 1);
        mbar_init(smem_addr(&met[0]), 1);
        mbar_init(smem_addr(&met[1]), 1);
        fence_barrier_init();
    }
    if constexpr (CL > 1) cluster_sync_all();
    else __syncthreads();

    const T* const Z = reinterpret_cast<const T*>(a.z) + v0;
    T* const G = reinterpret_cast<T*>(a.dz) + v0;
    // element e of the slice lies at buffer[off + e]
    auto off_of = [&](int64_t n) { return (int)((reinterpret_cast<uintptr_t>(Z + n * a.ld) & 15u) / sizeof(T)); };
    // chunks of the buffer that a bulk copy may load: not those that reach beyond the row
    auto load_chunks = [&](int off, int& ca, int& cb) {
        ca = rank == 0 && off > 0 ? 1 : 0;
        const int64_t in_row = ((int64_t)off + (a.vocab - v0)) / N;
        cb = (int)min((int64_t)((off + len + N - 1) / N), in_row);
        if (cb < ca) cb = ca;
    };
    // the broken chunks' elements of row n: thread < 2 N; index in the slice, or -1
    auto edge_of = [&](int off, int ca, int cb) {
        const int head = min(len, max(0, ca * N - off)), tail = max(head, cb * N - off);
        if (tid < N) return tid < head ? tid : -1;
        if (tid < 2 * N) return tail + tid - N < len ? tail + tid - N : -1;
        return -1;
    };
    auto load = [&](int64_t n, int b) {                                  // thread 0: row n into buffer b
        const int off = off_of(n);
        int ca, cb;
        load_chunks(off, ca, cb);
        const uint32_t bar = smem_addr(&full[b]);
        const uint32_t bytes = (uint32_t)(cb - ca) * 16;
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes) bulk_load(smem_addr(smem + (size_t)b * f.buf) + ca * 16, Z + n * a.ld - off + ca * N, bytes, bar);
    };
    auto edge_load = [&](int64_t n, int& at) {                           // thread < 2 N: its broken chunk's element
        const int off = off_of(n);
        int ca, cb;
        load_chunks(off, ca, cb);
        at = edge_of(off, ca, cb);
        const float v = at >= 0 ? elem(Z + n * a.ld + at) : 0.0f;
        at += off;
        return v;
    };
    auto edge_put = [&](int b, int64_t n, int at, float v) {
        if (at >= off_of(n)) {
            const float x[1] = {v};
            Pack<T, 1>::pack(x).store(reinterpret_cast<T*>(smem + (size_t)b * f.buf) + at);
        }
    };
    // a row's teacher entries of this thread
    int id_next[J];
    float t_next[J];
    float w_next = 0.0f;
    auto teacher = [&](int64_t n) {
        w_next = a.weight ? a.weight[n] : 1.0f;
#pragma unroll
        for (int q = 0; q < J; ++q) {
            const int j = tid + q * NT;
            id_next[q] = -1;
            t_next[q] = neg_inf();
            if (j < a.k) {
                const int64_t at = n * a.k + j;
                const int64_t id = a.id_bytes == 8 ? reinterpret_cast<const int64_t*>(a.ids)[at]
                                                   : (int64_t)reinterpret_cast<const int32_t*>(a.ids)[at];
                const float t = a.teacher[at];
                if (id >= a.vocab && w_next != 0.0f) record_status(a.status, KAN_ERR_DEVICE_CHECK);
                if (id >= 0 && id < a.vocab && t != neg_inf()) {
                    id_next[q] = (int)id;
                    t_next[q] = t;
                }
            }
        }
    };

    const int64_t n0 = blockIdx.x / CL;
    if (n0 < a.n) {
        int at;
        float v;
        if (tid < 2 * N) {
            v = edge_load(n0, at);
            edge_put(0, n0, at, v);
            if (n0 + clusters < a.n) {
                v = edge_load(n0 + clusters, at);
                edge_put(1, n0 + clusters, at, v);
            }
        }
        if (tid == 0) {
            load(n0, 0);
            if (n0 + clusters < a.n) load(n0 + clusters, 1);
        }
        teacher(n0);
    }
    __syncthreads();
    bool waits = true;
    int it = 0, ex = 0;                                                  // rows so far; exchanges so far
    for (int64_t n = n0; n < a.n; n += clusters, ++it) {
        const int b = it & 1;
        const int64_t after = n + clusters;
        T* const buf = reinterpret_cast<T*>(smem + (size_t)b * f.buf);
        const int off = off_of(n), chunks = (off + len + N - 1) / N;
        int id[J];
        float t[J], z[J];
        const float w = w_next;
        bool any = false;
#pragma unroll
        for (int q = 0; q < J; ++q) {
            id[q] = id_next[q];
            t[q] = t_next[q];
            any |= id[q] >= 0;
        }
        if (after < a.n) teacher(after);
        // the row after next goes where the last one was; its broken chunks' elements, ahead
        const bool refill = it > 0 && after < a.n;
        int edge_at = -1;
        float edge_v = 0.0f;
        if (refill && tid < 2 * N) edge_v = edge_load(after, edge_at);
        if (waits) waits = mbar_wait(smem_addr(&full[b]), (it >> 1) & 1, a.status);

        // maximum and sum of the slice, each thread's own at first
        Running<T> mine;
        mine.k = a.scale2;
        if (w != 0.0f) {
            const int first = off > 0 ? 1 : 0, last = (off + len) / N;    // whole chunks
#pragma unroll 2
            for (int c = first + tid; c < last; c += NT) mine.add(Pack<T, N>::load(buf + c * N));
            if (tid < 2 && (tid == 0 ? first > 0 : last < chunks && last >= first)) {     // the broken ones
                const int c = tid == 0 ? 0 : last;
                Pack<T, N> q = Pack<T, N>::load(buf + c * N);
                float x[N];
                q.unpack(x);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int i = c * N - off + e;
                    if (i < 0 || i >= len) x[e] = neg_inf();
                }
                mine.add(Pack<T, N>::pack(x));
            }
        }
        float2 st = join_lanes<32>(mine.get(), a.scale2);
        float mt = neg_inf();
#pragma unroll
        for (int q = 0; q < J; ++q) {
            const int64_t i = (int64_t)id[q] - v0;
            z[q] = id[q] >= 0 && i >= 0 && i < len ? elem(buf + off + i) : 0.0f;
            mt = fmaxf(mt, t[q]);
        }
        if (warp < warps_k) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        }
        if (lane == 0) {
            wstat[warp] = st;
            wmax[warp] = mt;
        }
        // (the row before is stored by now or soon: its buffer takes the row after)
        if (refill && warp == 0) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            if (tid < 2 * N) edge_put(b ^ 1, after, edge_at, edge_v);
            if (lane == 0) load(after, b ^ 1);
        }
        any = __syncthreads_or(any);                                     // 1: partial results are there
        const bool counts = any && w != 0.0f;
        float cq = 0.0f, M = 0.0f, S = 1.0f, c = 0.0f, E = 1.0f;
        if (counts) {
            const int set = ex & 1;
            mt = wmax[0];
            for (int i = 1; i < warps_k; ++i) mt = fmaxf(mt, wmax[i]);
            if (warp == 0) {                                             // the slice's (m, s) to every block
                st = join_lanes<WARPS>(lane < WARPS ? wstat[lane] : make_float2(neg_inf(), 0.0f), a.scale2);
                if constexpr (CL > 1) {
                    if (lane < CL) st_async(peer_addr(smem_addr(&cstat[set][rank]), lane), peer_addr(smem_addr(&met[set]), lane), st);
                } else {
                    if (lane == 0) cstat[0][0] = st;
                }
            }
            // the teacher's weights, and the logits at its tokens to block 0
            float e[J], es = 0.0f;
            int valid = 0;
#pragma unroll
            for (int q = 0; q < J; ++q) {
                const int j = tid + q * NT;
                e[q] = id[q] < 0 ? 0.0f : expf((t[q] - mt) * a.inv_temp);
                es += e[q];
                valid += id[q] >= 0;
                if (j < a.k) {
                    tid_[j] = id[q];
                    te[j] = e[q];
                    if constexpr (CL > 1) {
                        const int64_t i = (int64_t)id[q] - v0;
                        if (id[q] >= 0 && i >= 0 && i < len)
                            st_async(peer_addr(smem_addr(zk + set * f.kp + j), 0), peer_addr(smem_addr(&met[set]), 0), z[q]);
                    }
                }
            }
            if (warp < warps_k) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
                valid = __reduce_add_sync(0xffffffffu, valid);
                if (lane == 0) {
                    wsum[warp] = es;
                    wvalid[warp] = valid;
                }
            }
            __syncthreads();                                             // 2: the teacher's entries (and, alone, the sums)
            if constexpr (CL > 1) {
                if (tid == 0) {
                    int all = 0;
                    if (rank == 0)
                        for (int i = 0; i < warps_k; ++i) all += wvalid[i];
                    mbar_arrive_expect_tx(smem_addr(&met[set]), CL * (int)sizeof(float2) + all * 4);
                }
                if (waits) waits = mbar_wait(smem_addr(&met[set]), (ex >> 1) & 1, a.status);
            }
            M = cstat[CL > 1 ? set : 0][0].x;
#pragma unroll
            for (int i = 1; i < CL; ++i) M = fmaxf(M, cstat[set][i].x);
            S = rescale(cstat[CL > 1 ? set : 0][0], M, a.scale2);
#pragma unroll
            for (int i = 1; i < CL; ++i) S += rescale(cstat[set][i], M, a.scale2);
            if (M == neg_inf()) S = __int_as_float(0x7fc00000);          // a row of -inf alone has no distribution
            E = wsum[0];
            for (int i = 1; i < warps_k; ++i) E += wsum[i];
            c = w * a.temp;
            cq = c / S;
            if (rank == 0) {
                float l = 0.0f;
                const float le = logf(E), ls = logf(S);
#pragma unroll
                for (int q = 0; q < J; ++q) {
                    const int j = tid + q * NT;
                    const float p = e[q] / E;
                    if (id[q] >= 0 && !(p == 0.0f)) {
                        const float zj = CL > 1 ? zk[set * f.kp + j] : z[q];
                        l += p * ((t[q] - mt) * a.inv_temp - le - ((zj - M) * a.inv_temp - ls));
                    }
                }
                if (warp < warps_k) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (lane == 0) wloss[warp] = l;
                }
            }
            ++ex;
        }
        // the gradient in the logits' place (broken chunks too: their elements outside the slice are not stored)
        if (!counts) {
            for (int i = tid; i < chunks; i += NT) Pack<T, N>::zero().store(buf + i * N);
        } else if (sizeof(T) == 2 && fabsf(M) < kLarge && fabsf(cq) > 1.0f / kLarge && fabsf(cq) < kLarge) {
            // c q = +-2^(z k + (log2 |c / S| - m k)): one multiply-add and one ex2 an element
            const float shift = log2f(fabsf(cq)) - M * a.scale2;
            const uint64_t kk = two(a.scale2, a.scale2), add = two(shift, shift);
            const uint32_t sign = cq < 0.0f ? 0x80008000u : 0u;
#pragma unroll 2
            for (int i = tid; i < chunks; i += NT) {
                const Pack<T, N> q = Pack<T, N>::load(buf + i * N);
                float x[N];
#pragma unroll
                for (int e = 0; e < N / 2; ++e) halves(ex2_2(fma2(pair(q, e), kk, add)), x[2 * e], x[2 * e + 1]);
                Pack<T, N> r = Pack<T, N>::pack(x);
                r.q = make_uint4(r.q.x ^ sign, r.q.y ^ sign, r.q.z ^ sign, r.q.w ^ sign);
                r.store(buf + i * N);
            }
        } else {
            const uint64_t kk = two(a.scale2, a.scale2), mm = two(-M, -M), cc = two(cq, cq);
#pragma unroll 2
            for (int i = tid; i < chunks; i += NT) {
                const Pack<T, N> q = Pack<T, N>::load(buf + i * N);
                float x[N];
#pragma unroll
                for (int e = 0; e < N / 2; ++e) halves(mul2(ex2_2(mul2(add2(pair(q, e), mm), kk)), cc), x[2 * e], x[2 * e + 1]);
                Pack<T, N>::pack(x).store(buf + i * N);
            }
        }
        // does an id occur twice?  The block's threads share the comparisons: 2^k of them, each with all others' part
        bool twice = false;
        if (counts) {
            const int parts = NT / f.kpow, part = tid / f.kpow;          // (entries beyond kpow: the thread's second one)
#pragma unroll
            for (int q = 0; q < J; ++q) {
                const int j = (tid & (f.kpow - 1)) + q * f.kpow;
                if (j < a.k && tid_[j] >= 0) {
                    const int me = tid_[j];
                    for (int o = part * 4; o < a.k; o += parts * 4) {
                        const int4 v = *reinterpret_cast<const int4*>(tid_ + o);
                        twice |= (v.x == me && o != j) | (v.y == me && o + 1 != j && o + 1 < a.k) |
                                 (v.z == me && o + 2 != j && o + 2 < a.k) | (v.w == me && o + 3 != j && o + 3 < a.k);
                    }
                }
                if (a.k <= f.kpow) break;
            }
        }
        twice = __syncthreads_or(twice);                                 // 3: the slice is written
        // the teacher's part: an entry of this slice that is the first with its id takes all of them
#pragma unroll
        for (int q = 0; q < J; ++q) {
            const int j = tid + q * NT;
            const int64_t i = (int64_t)id[q] - v0;
            if (counts && id[q] >= 0 && i >= 0 && i < len) {
                float sum = te[j];
                bool first = true;
                if (twice) {
                    sum = 0.0f;
                    for (int o = 0; o < a.k; ++o) {
                        if (tid_[o] == id[q]) {
                            first &= o >= j;
                            sum += te[o];
                        }
                    }
                }
                if (first) {
                    const float x[1] = {c * (term(z[q], M, a.scale2) / S - sum / E)};
                    Pack<T, 1>::pack(x).store(buf + off + i);
                }
            }
        }
        if (tid == 0 && rank == 0) {
            float l = 0.0f;
            if (counts)
                for (int i = 0; i < warps_k; ++i) l += wloss[i];
            a.loss[n] = counts ? w * a.temp * a.temp * l : 0.0f;
            a.stats[n] = make_float2(counts ? M : 0.0f, counts ? S : 1.0f);
        }
        fence_async_smem();
        __syncthreads();                                                 // 4: the teacher's part too
        T* const out = G + n * a.ld_grad;
        const int sa = off > 0 ? 1 : 0, sb = max(sa, (off + len) / N);   // whole chunks of the slice
        if (tid == 0) {
            if (sb > sa) bulk_store(out - off + sa * N, smem_addr(buf) + sa * 16, (uint32_t)(sb - sa) * 16);
            bulk_commit();
        }
        const int i = edge_of(off, sa, sb);
        if (i >= 0) Pack<T, 1>::load(buf + off + i).store(out + i);
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if constexpr (CL > 1) cluster_sync_all();                            // no block leaves while another's logits may arrive
}

kan_status di_fail(kan_status st, const char* msg) { return set_last_error(st, msg); }

kan_status validate(const kan_distill_shape* s)
{
    if (!s) return di_fail(KAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->rows < 0 || s->vocab < 1 || s->entries < 1) return di_fail(KAN_ERR_INVALID_ARG, "rows >= 0, vocab >= 1, entries >= 1");
    if (s->ld < s->vocab || s->ld_grad < s->vocab) return di_fail(KAN_ERR_INVALID_ARG, "a row stride below vocab");
    if (s->dtype != KAN_F32 && s->dtype != KAN_BF16) return di_fail(KAN_ERR_INVALID_ARG, "unknown dtype");
    if (s->id_bytes != 4 && s->id_bytes != 8) return di_fail(KAN_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
    if (!(s->temperature > 0.0f) || !(s->temperature - s->temperature == 0.0f))
        return di_fail(KAN_ERR_INVALID_ARG, "temperature must be positive and finite");
    if (s->entries > kMaxK) return di_fail(KAN_ERR_UNSUPPORTED, "more than 1024 teacher entries per row");
    if (s->rows > ((int64_t)1 << 31) - 1 || s->vocab > ((int64_t)1 << 30)) return di_fail(KAN_ERR_UNSUPPORTED, "sizes too large");
    return KAN_OK;
}

DistArgs args_of(const kan_distill_shape& s, const void* z, const void* ids, const float* teacher, const float* weight)
{
    DistArgs a{};
    a.z = z;
    a.ids = ids;
    a.teacher = teacher;
    a.weight = weight;
    a.n = s.rows;
    a.vocab = s.vocab;
    a.ld = s.ld;
    a.ld_grad = s.ld_grad;
    a.k = s.entries;
    a.id_bytes = s.id_bytes;
    a.temp = s.temperature;
    a.inv_temp = 1.0f / s.temperature;
    a.scale2 = (float)(1.4426950408889634 / (double)s.temperature);
    a.status = device_status_ptr();
    return a;
}

bool misaligned(const kan_distill_shape& s, std::initializer_list<const void*> ops, const void* ids,
                std::initializer_list<const void*> f32)
{
    const uintptr_t esz = s.dtype == KAN_F32 ? 4 : 2;
    for (const void* p : ops)
        if (reinterpret_cast<uintptr_t>(p) % esz) return true;
    for (const void* p : f32)
        if (reinterpret_cast<uintptr_t>(p) % 4) return true;
    return reinterpret_cast<uintptr_t>(ids) % s.id_bytes != 0;
}

template <typename F32, typename B16> cudaError_t by_type(const kan_distill_shape& s, F32 f32, B16 b16, const DistArgs& a, cudaStream_t st)
{
    if (s.dtype == KAN_F32) f32<<<(unsigned)s.rows, kThreads, 0, st>>>(a);
    else b16<<<(unsigned)s.rows, kThreads, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

// The fused kernel's shape: the fewest blocks a row whose two buffers let two blocks share an SM, else one block an SM;
// none (0) if not even 8 slices fit, or if the gradient's rows do not begin where the logits' do within 16 bytes.
struct FusedPlan {
    int cluster, per, buf, kp;
    size_t smem;
};
FusedPlan plan_of(const kan_distill_shape& s, const void* z, const void* dz)
{
    FusedPlan P{};
    const int64_t esz = s.dtype == KAN_F32 ? 4 : 2, n = 16 / esz;
    if ((reinterpret_cast<uintptr_t>(z) - reinterpret_cast<uintptr_t>(dz)) % 16 || (s.ld - s.ld_grad) * esz % 16) return P;
    P.kp = (s.entries + 3) / 4 * 4;
    for (size_t limit : {(size_t)112 << 10, (size_t)224 << 10}) {
        for (int cl = 1; cl <= 8; cl *= 2) {
            const int64_t per = ((s.vocab + cl - 1) / cl + n - 1) / n * n;
            const int64_t buf = per * esz + 16;
            const size_t smem = 2 * (size_t)buf + 16 * (size_t)P.kp;
            if (smem <= limit && per * (cl - 1) < s.vocab) {
                P.cluster = cl;
                P.per = (int)per;
                P.buf = (int)buf;
                P.smem = smem;
                return P;
            }
        }
    }
    return P;
}

template <typename T, int CL, int NT> cudaError_t launch_fused(FusedArgs f, const FusedPlan& P, cudaStream_t st)
{
    f.kpow = 4;
    while (f.kpow < f.d.k && f.kpow < NT) f.kpow *= 2;
    // clusters that run at once, looked up again when the shared memory or the device differs from the last call's
    static std::atomic<uint64_t> known{0};
    auto kernel = distill_fused_kernel<T, CL, NT>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = P.smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const uint64_t key = (uint64_t)P.smem << 8 | (uint64_t)(dev & 0xff);
    uint64_t got = known.load(std::memory_order_relaxed);
    int n = (int)(got >> 48);
    if (!n || (got & 0xffffffffffffull) != key) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 << 10);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(CL);
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        n = std::min(std::max(n, 1), 0x7fff);
        known.store((uint64_t)n << 48 | key, std::memory_order_relaxed);
    }
    cfg.gridDim = dim3((unsigned)(std::min<int64_t>(n, f.d.n) * CL));
    cfg.numAttrs = CL > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kernel, f);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename T> cudaError_t fused_of(const FusedArgs& f, const FusedPlan& P, cudaStream_t st)
{
    // short rows: more and smaller blocks on an SM, so that other rows' phases fill the barriers of one
    if (P.cluster == 1 && P.buf <= 16 << 10 && f.d.k <= 256) return launch_fused<T, 1, 128>(f, P, st);
    switch (P.cluster) {
    case 1: return launch_fused<T, 1, 512>(f, P, st);
    case 2: return launch_fused<T, 2, 512>(f, P, st);
    case 4: return launch_fused<T, 4, 512>(f, P, st);
    default: return launch_fused<T, 8, 512>(f, P, st);
    }
}

}  // namespace
}  // namespace kan

using namespace kan;

extern "C" {

kan_status kan_distill_forward(const kan_distill_shape* s, const void* z, const void* ids, const float* teacher,
                               const float* weight, float* loss, float* stats, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (s->rows == 0) return KAN_OK;
    if (!z || !ids || !teacher || !loss || !stats) return di_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {z}, ids, {teacher, weight, loss}) || reinterpret_cast<uintptr_t>(stats) % 8)
        return di_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements, stats to 8 bytes");
    DistArgs a = args_of(*s, z, ids, teacher, weight);
    a.loss = loss;
    a.stats = reinterpret_cast<float2*>(stats);
    const cudaError_t e = by_type(*s, distill_forward_kernel<float>, distill_forward_kernel<__nv_bfloat16>, a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KAN_OK : di_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

kan_status kan_distill_backward(const kan_distill_shape* s, const void* z, const void* ids, const float* teacher,
                                const float* weight, const float* stats, const float* dloss, void* dz, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (s->rows == 0) return KAN_OK;
    if (!z || !ids || !teacher || !stats || !dz) return di_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {z, dz}, ids, {teacher, weight, dloss}) || reinterpret_cast<uintptr_t>(stats) % 8)
        return di_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements, stats to 8 bytes");
    DistArgs a = args_of(*s, z, ids, teacher, weight);
    a.stats = reinterpret_cast<float2*>(const_cast<float*>(stats));
    a.dloss = dloss;
    a.dz = dz;
    const cudaError_t e = by_type(*s, distill_backward_kernel<float>, distill_backward_kernel<__nv_bfloat16>, a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? KAN_OK : di_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

kan_status kan_distill_loss_grad(const kan_distill_shape* s, const void* z, const void* ids, const float* teacher,
                                 const float* weight, float* loss, float* stats, void* dz, void* stream)
{
    kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (s->rows == 0) return KAN_OK;
    if (!z || !ids || !teacher || !loss || !stats || !dz) return di_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {z, dz}, ids, {teacher, weight, loss}) || reinterpret_cast<uintptr_t>(stats) % 8)
        return di_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements, stats to 8 bytes");
    const FusedPlan P = plan_of(*s, z, dz);
    if (!P.cluster) {
        st = kan_distill_forward(s, z, ids, teacher, weight, loss, stats, stream);
        return st == KAN_OK ? kan_distill_backward(s, z, ids, teacher, weight, stats, nullptr, dz, stream) : st;
    }
    FusedArgs f{};
    f.d = args_of(*s, z, ids, teacher, weight);
    f.d.loss = loss;
    f.d.stats = reinterpret_cast<float2*>(stats);
    f.d.dz = dz;
    f.per = P.per;
    f.buf = P.buf;
    f.kp = P.kp;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = s->dtype == KAN_F32 ? fused_of<float>(f, P, cs) : fused_of<__nv_bfloat16>(f, P, cs);
    return e == cudaSuccess ? KAN_OK : di_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

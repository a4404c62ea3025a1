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
    if (s->rows > 0 && !dz) return di_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (misaligned(*s, {dz}, nullptr, {})) return di_fail(KAN_ERR_UNSUPPORTED, "operands must be aligned to their elements, stats to 8 bytes");
    st = kan_distill_forward(s, z, ids, teacher, weight, loss, stats, stream);
    if (st != KAN_OK) return st;
    return kan_distill_backward(s, z, ids, teacher, weight, stats, nullptr, dz, stream);
}

}  // extern "C"

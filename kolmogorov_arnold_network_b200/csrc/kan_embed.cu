// kan_embed.cu -- embedding lookup with scaling, and its gradient by sorted
// tokens.
//
//   y[t, :]  = scale W[id_t, :]
//   dW[v, :] = scale sum_{t : id_t = v} dY[t, :]        (t ascending)
//
// Forward: one warp per (token, 128-vector segment of its row), the widest
// vectors that the rows allow; bound by HBM (each token's row written, each
// distinct row read).
//
// Backward, without atomic adds and with one fixed order of summation:
//   1. embed_sort_kernel orders the tokens by id, stably.  Block p owns the
//      ids with id % P == p (P a power of two): neighbouring ids, whose
//      frequencies are alike in a vocabulary, fall to different blocks.
//      Every block reads all ids twice (they stay in L2); the first reading
//      counts, per warp, the tokens of each owned id and all tokens of the
//      blocks before it, which gives the block's place in the order without
//      any exchange between blocks; the second one places its tokens.  The
//      block also writes the zero rows of its ids that no token has.
//   2. embed_sum_kernel cuts the ordered list into chunks of kChunk tokens;
//      a thread keeps one vector of columns and adds the chunk's rows in
//      order.  Runs that lie within a chunk are written at once, the pieces
//      of runs that cross a border go to the workspace as fp32 partials:
//      the work is even however often a token occurs.
//   3. embed_join_kernel adds the partials of each such run in chunk order.
// Sums are fp32 and rounded once, when the row of dW is written.
#include <algorithm>

#include "kan_device.cuh"
#include "kan_vec.cuh"

namespace kan {
namespace {

constexpr int kSegVecs = 128;     // forward: vectors of a row that one warp copies
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 1536;    // ids per sort block (their per-warp counts lie in shared memory)
constexpr int kChunk = 64;        // tokens per chunk of the ordered list
constexpr int kJoinRows = 4;      // partials that a block of the join adds side by side

template <typename I> __device__ __forceinline__ int64_t id_at(const void* ids, int64_t t)
{
    return (int64_t)reinterpret_cast<const I*>(ids)[t];
}

// ---- forward ----
template <typename T, int N, typename I>
__global__ void __launch_bounds__(128) embed_forward_kernel(const void* __restrict__ ids, const T* __restrict__ W,
                                                            T* __restrict__ y, int64_t tokens, int64_t rows, int64_t dim,
                                                            int segs, float scale, unsigned int* status)
{
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t t = w / segs;
    if (t >= tokens) return;
    const int64_t vecs = dim / N;
    const int64_t v0 = (w - t * segs) * kSegVecs + lane;
    const int64_t id = id_at<I>(ids, t);
    const bool ok = id >= 0 && id < rows;
    if (!ok && lane == 0) record_status(status, KAN_ERR_DEVICE_CHECK);
    const T* src = W + (ok ? id : 0) * dim;
    T* dst = y + t * dim;
    Pack<T, N> q[kSegVecs / 32];
#pragma unroll
    for (int i = 0; i < kSegVecs / 32; ++i)
        q[i] = ok && v0 + 32 * i < vecs ? Pack<T, N>::load(src + (v0 + 32 * i) * N) : Pack<T, N>::zero();
#pragma unroll
    for (int i = 0; i < kSegVecs / 32; ++i) {
        if (v0 + 32 * i < vecs) {
            float f[N];
            q[i].unpack(f);
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = ok ? f[e] * scale : 0.0f;
            Pack<T, N>::pack(f).store(dst + (v0 + 32 * i) * N);
        }
    }
}

// ---- backward: the order ----
struct SortArgs {
    const void* ids;
    int32_t* perm;       // [tokens] token numbers, ordered by (block, id), ascending within an id
    int32_t* key;        // [tokens] their ids
    int32_t* count;      // [1] tokens that take part
    void* dW;
    int64_t tokens, rows, pad;
    int64_t row_bytes;
    int shift;           // log2 P
    int bins;            // ids per block
    int wide;            // dW's rows are whole 16-byte vectors
    unsigned int* status;
};

template <typename I>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SortArgs a)
{
    extern __shared__ int32_t cnt[];                // [kSortWarps][bins] counts, then next places
    int32_t* total = cnt + (size_t)kSortWarps * a.bins;   // [bins] tokens of each id
    __shared__ int32_t wsum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int p = blockIdx.x;
    const int64_t mask = ((int64_t)1 << a.shift) - 1;
    for (int i = tid; i < kSortWarps * a.bins; i += kSortThreads) cnt[i] = 0;
    __syncthreads();

    // tokens of this warp: a contiguous piece, whole 32-token steps
    const int64_t piece = ((a.tokens + kSortThreads - 1) / kSortThreads) * 32;
    const int64_t t0 = min(a.tokens, piece * warp), t1 = min(a.tokens, t0 + piece);
    int32_t* mine = cnt + (size_t)warp * a.bins;
    int below = 0;
    bool bad = false;
#pragma unroll 4
    for (int64_t t = t0 + lane; t < t1; t += 32) {
        const int64_t id = id_at<I>(a.ids, t);
        const bool in = id >= 0 && id < a.rows;
        bad |= !in;
        if (in && id != a.pad) {
            const int o = (int)(id & mask);
            below += o < p;
            if (o == p) atomicAdd(&mine[id >> a.shift], 1);   // an integer count: no order
        }
    }
    if (p == 0 && bad) record_status(a.status, KAN_ERR_DEVICE_CHECK);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
    if (lane == 0) wsum[warp] = below;
    __syncthreads();
    int base = 0;
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) base += wsum[w];
    __syncthreads();

    // places: ids ascending, and within an id the warps' pieces in order
    int carry = base;
    for (int b0 = 0; b0 < a.bins; b0 += kSortThreads) {
        const int b = b0 + tid;
        int n = 0;
        if (b < a.bins)
            for (int w = 0; w < kSortWarps; ++w) n += cnt[(size_t)w * a.bins + b];
        int s = n;                                   // inclusive sum over the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (b < a.bins) {
            total[b] = n;
            int at = carry + before + s - n;
            for (int w = 0; w < kSortWarps; ++w) {
                int32_t& c = cnt[(size_t)w * a.bins + b];
                const int k = c;
                c = at;
                at += k;
            }
        }
        carry += all;
        __syncthreads();
    }
    if (p == (int)mask && tid == 0) *a.count = carry;

    // second reading: every token to its place
    for (int64_t t = t0; t < t1; t += 32) {
        const int64_t tl = t + lane;
        const int64_t id = tl < t1 ? id_at<I>(a.ids, tl) : -1;
        const bool own = id >= 0 && id < a.rows && id != a.pad && (int)(id & mask) == p;
        const unsigned act = __ballot_sync(0xffffffffu, own);
        if (act == 0) continue;
        if (own) {
            const int b = (int)(id >> a.shift);
            const unsigned same = __match_any_sync(act, b);
            const int rank = __popc(same & ((1u << lane) - 1));
            const int at = mine[b];
            __syncwarp(act);
            if (rank == 0) mine[b] = at + __popc(same);
            a.perm[at + rank] = (int32_t)tl;
            a.key[at + rank] = (int32_t)id;
        }
        __syncwarp();
    }

    // rows that no token has
    for (int b = warp; b < a.bins; b += kSortWarps) {
        const int64_t id = ((int64_t)b << a.shift) + p;
        if (id >= a.rows || total[b] != 0) continue;
        char* row = reinterpret_cast<char*>(a.dW) + id * a.row_bytes;
        if (a.wide) {
            for (int64_t i = (int64_t)lane * 16; i < a.row_bytes; i += 512) *reinterpret_cast<uint4*>(row + i) = uint4{};
        } else {
            for (int64_t i = (int64_t)lane * 2; i < a.row_bytes; i += 64) *reinterpret_cast<uint16_t*>(row + i) = 0;
        }
    }
}

// ---- backward: the sums ----
struct SumArgs {
    const void* dY;
    void* dW;
    const int32_t* perm;
    const int32_t* key;
    const int32_t* count;
    float* part;         // [chunks][2][dim]: a chunk's first piece (of a run that began before it), its last piece
    int64_t dim;
    float scale;
};

template <typename T, typename O, int N>
__device__ __forceinline__ void store_row(O* p, const float (&acc)[N], float scale)
{
    // N vectors of T; the output type may need two stores (fp32 from bf16 vectors)
    constexpr int NO = N * (int)sizeof(O) > 16 ? 16 / (int)sizeof(O) : N;
#pragma unroll
    for (int i = 0; i < N; i += NO) {
        float f[NO];
#pragma unroll
        for (int e = 0; e < NO; ++e) f[e] = acc[i + e] * scale;
        Pack<O, NO>::pack(f).store(p + i);
    }
}

template <typename T, typename O, int N>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a)
{
    __shared__ int32_t sp[kChunk], sk[kChunk + 2];       // token numbers; ids with the neighbours' on both sides
    const int m = *a.count;
    const int64_t c0 = (int64_t)blockIdx.x * kChunk;
    if (c0 >= m) return;
    const int len = (int)min((int64_t)kChunk, m - c0);
    for (int i = threadIdx.x; i < len; i += blockDim.x) sp[i] = a.perm[c0 + i];
    for (int i = threadIdx.x; i < len + 2; i += blockDim.x) {
        const int64_t j = c0 + i - 1;
        sk[i] = j >= 0 && j < m ? a.key[j] : -1;
    }
    __syncthreads();
    const int64_t v = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
    if (v * N >= a.dim) return;
    const T* src = reinterpret_cast<const T*>(a.dY) + v * N;
    O* dst = reinterpret_cast<O*>(a.dW) + v * N;
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.dim + v * N;
    bool from_before = sk[1] == sk[0];
    float acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    constexpr int U = 8;
    for (int i0 = 0; i0 < len; i0 += U) {
        Pack<T, N> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < len) q[u] = Pack<T, N>::load(src + (int64_t)sp[i0 + u] * a.dim);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u;
            if (i < len) {
                float f[N];
                q[u].unpack(f);
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] += f[e];
                const int id = sk[i + 1];
                const bool last = i + 1 == len;
                if (last || sk[i + 2] != id) {           // the run's end, or the chunk's
                    const bool goes_on = sk[i + 2] == id;
                    if (!from_before && !goes_on) store_row<T, O, N>(dst + (int64_t)id * a.dim, acc, a.scale);
                    else store_row<T, float, N>(part + (from_before ? 0 : a.dim), acc, 1.0f);
                    from_before = false;
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
                }
            }
        }
    }
}

// A run that crosses chunk borders is joined by the block of the chunk where
// it begins: that chunk's last piece and the first pieces of the chunks after
// it, kJoinRows sums side by side, added in a fixed order at the end.
template <typename O>
__global__ void __launch_bounds__(64 * kJoinRows) embed_join_kernel(const SumArgs a)
{
    const int m = *a.count;
    const int64_t c = blockIdx.x, end = (c + 1) * kChunk;
    if (end >= m) return;
    const int id = a.key[end - 1];
    if (a.key[end] != id) return;
    // it begins here if the chunk's first token is another id's, or the run's very first one
    const int64_t c0 = c * kChunk;
    if (a.key[c0] == id && c0 > 0 && a.key[c0 - 1] == id) return;
    // the chunks after it whose first token is still of the run (equal ids lie side by side)
    int64_t last_chunk = c;
    for (;;) {
        const int64_t at = (last_chunk + 1 + threadIdx.x) * kChunk;
        const int n = __syncthreads_count(at < m && a.key[at] == id);
        last_chunk += n;
        if (n < (int)blockDim.x) break;
    }
    __shared__ float red[kJoinRows][64];
    const int col = threadIdx.x & 63, row = threadIdx.x >> 6;
    const int64_t d = (int64_t)blockIdx.y * 64 + col;
    float acc = 0.0f;
    if (d < a.dim) {
        if (row == 0) acc = a.part[(c * 2 + 1) * a.dim + d];
        for (int64_t k = c + 1 + row; k <= last_chunk; k += kJoinRows) acc += a.part[k * 2 * a.dim + d];
    }
    red[row][col] = acc;
    __syncthreads();
    if (row == 0 && d < a.dim) {
        float s = red[0][col];
#pragma unroll
        for (int r = 1; r < kJoinRows; ++r) s += red[r][col];
        const float f[1] = {s * a.scale};
        Pack<O, 1>::pack(f).store(reinterpret_cast<O*>(a.dW) + (int64_t)id * a.dim + d);
    }
}

kan_status em_fail(kan_status st, const char* msg) { return set_last_error(st, msg); }

kan_status validate(const kan_embed_shape* s)
{
    if (!s) return em_fail(KAN_ERR_INVALID_ARG, "shape is NULL");
    if (s->tokens < 0 || s->rows < 1 || s->dim < 1) return em_fail(KAN_ERR_INVALID_ARG, "tokens >= 0, rows >= 1, dim >= 1");
    if (s->dtype != KAN_F32 && s->dtype != KAN_BF16) return em_fail(KAN_ERR_INVALID_ARG, "unknown dtype");
    if (s->grad_dtype != KAN_F32 && s->grad_dtype != KAN_BF16) return em_fail(KAN_ERR_INVALID_ARG, "unknown grad_dtype");
    if (s->id_bytes != 4 && s->id_bytes != 8) return em_fail(KAN_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
    if (!(s->scale - s->scale == 0.0f)) return em_fail(KAN_ERR_INVALID_ARG, "scale must be finite");
    if (s->padding_idx < -1 || s->padding_idx >= s->rows)
        return em_fail(KAN_ERR_INVALID_ARG, "padding_idx must be -1 (none) or a row");
    if (s->tokens > ((int64_t)1 << 31) - 1024 || s->rows > ((int64_t)1 << 30) || s->dim > ((int64_t)1 << 21))
        return em_fail(KAN_ERR_UNSUPPORTED, "sizes too large");
    if (s->tokens * ((s->dim + kSegVecs - 1) / kSegVecs) > ((int64_t)1 << 32))
        return em_fail(KAN_ERR_UNSUPPORTED, "tokens times dim too large");
    return KAN_OK;
}

// Sort blocks: 256 (all resident at once on 148 SMs), more for tables of more than 256 * kMaxBins rows.
int sort_shift(const kan_embed_shape& s)
{
    int sh = 8;
    while (((s.rows - 1) >> sh) + 1 > kMaxBins) ++sh;
    return sh;
}

struct Layout {
    size_t perm, key, count, part, bytes;
    int64_t chunks;
};

Layout layout_of(const kan_embed_shape& s)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout L{};
    L.chunks = (s.tokens + kChunk - 1) / kChunk;
    L.perm = 0;
    L.key = L.perm + up((size_t)s.tokens * 4);
    L.count = L.key + up((size_t)s.tokens * 4);
    L.part = L.count + 256;
    L.bytes = L.part + up((size_t)L.chunks * 2 * s.dim * 4);
    return L;
}

template <typename T, int N>
cudaError_t launch_forward(const kan_embed_shape& s, const void* ids, const void* W, void* y, cudaStream_t st)
{
    const int64_t segs = (s.dim / N + kSegVecs - 1) / kSegVecs;
    const int64_t blocks = (s.tokens * segs + 3) / 4;
    unsigned int* status = device_status_ptr();
    if (s.id_bytes == 8)
        embed_forward_kernel<T, N, int64_t><<<(unsigned)blocks, 128, 0, st>>>(ids, (const T*)W, (T*)y, s.tokens, s.rows, s.dim, (int)segs, s.scale, status);
    else
        embed_forward_kernel<T, N, int32_t><<<(unsigned)blocks, 128, 0, st>>>(ids, (const T*)W, (T*)y, s.tokens, s.rows, s.dim, (int)segs, s.scale, status);
    count_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t forward_of(const kan_embed_shape& s, const void* ids, const void* W, void* y, cudaStream_t st)
{
    switch (common_vector_bytes((uint64_t)s.dim * sizeof(T)) / (int)sizeof(T)) {
    case 8: if constexpr (sizeof(T) == 2) return launch_forward<T, 8>(s, ids, W, y, st);
    case 4: return launch_forward<T, 4>(s, ids, W, y, st);
    case 2: return launch_forward<T, 2>(s, ids, W, y, st);
    default: return launch_forward<T, 1>(s, ids, W, y, st);
    }
}

template <typename T, typename O, int N>
cudaError_t launch_sum(const kan_embed_shape& s, const SumArgs& a, int64_t chunks, cudaStream_t st)
{
    const int64_t vecs = s.dim / N;
    const int64_t slices = (vecs + 255) / 256;
    const int threads = (int)(((vecs + slices - 1) / slices + 31) / 32 * 32);
    embed_sum_kernel<T, O, N><<<dim3((unsigned)chunks, (unsigned)slices), threads, 0, st>>>(a);
    count_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    embed_join_kernel<O><<<dim3((unsigned)chunks, (unsigned)((s.dim + 63) / 64)), 64 * kJoinRows, 0, st>>>(a);
    count_launch();
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t sum_of(const kan_embed_shape& s, const SumArgs& a, int64_t chunks, cudaStream_t st)
{
    switch (common_vector_bytes((uint64_t)s.dim * sizeof(T)) / (int)sizeof(T)) {
    case 8: if constexpr (sizeof(T) == 2) return launch_sum<T, O, 8>(s, a, chunks, st);
    case 4: return launch_sum<T, O, 4>(s, a, chunks, st);
    case 2: return launch_sum<T, O, 2>(s, a, chunks, st);
    default: return launch_sum<T, O, 1>(s, a, chunks, st);
    }
}

}  // namespace
}  // namespace kan

using namespace kan;

extern "C" {

kan_status kan_embed_workspace_size(const kan_embed_shape* s, size_t* bytes)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (!bytes) return em_fail(KAN_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = s->tokens ? layout_of(*s).bytes : 0;
    return KAN_OK;
}

kan_status kan_embed_forward(const kan_embed_shape* s, const void* ids, const void* W, void* y, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (s->tokens == 0) return KAN_OK;
    if (!ids || !W || !y) return em_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if (reinterpret_cast<uintptr_t>(ids) % s->id_bytes || !aligned16(W) || !aligned16(y))
        return em_fail(KAN_ERR_UNSUPPORTED, "W and y must be 16-byte aligned, ids to their size");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = s->dtype == KAN_F32 ? forward_of<float>(*s, ids, W, y, cs)
                                              : forward_of<__nv_bfloat16>(*s, ids, W, y, cs);
    return e == cudaSuccess ? KAN_OK : em_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

kan_status kan_embed_backward(const kan_embed_shape* s, const void* ids, const void* dY, void* dW, void* workspace,
                              size_t ws_bytes, void* stream)
{
    const kan_status st = validate(s);
    if (st != KAN_OK) return st;
    if (!dW || (s->tokens > 0 && (!ids || !dY))) return em_fail(KAN_ERR_INVALID_ARG, "a null pointer");
    if ((ids && reinterpret_cast<uintptr_t>(ids) % s->id_bytes) || !aligned16(dY) || !aligned16(dW) || !aligned16(workspace))
        return em_fail(KAN_ERR_UNSUPPORTED, "dY, dW and the workspace must be 16-byte aligned, ids to their size");
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int64_t row_bytes = s->dim * (s->grad_dtype == KAN_F32 ? 4 : 2);
    if (s->tokens == 0) {
        const cudaError_t e = cudaMemsetAsync(dW, 0, (size_t)(s->rows * row_bytes), cs);
        return e == cudaSuccess ? KAN_OK : em_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
    }
    const Layout L = layout_of(*s);
    if (!workspace || ws_bytes < L.bytes) return em_fail(KAN_ERR_WORKSPACE, "workspace too small");
    char* ws = reinterpret_cast<char*>(workspace);
    SortArgs o{};
    o.ids = ids;
    o.perm = reinterpret_cast<int32_t*>(ws + L.perm);
    o.key = reinterpret_cast<int32_t*>(ws + L.key);
    o.count = reinterpret_cast<int32_t*>(ws + L.count);
    o.dW = dW;
    o.tokens = s->tokens;
    o.rows = s->rows;
    o.pad = s->padding_idx;
    o.row_bytes = row_bytes;
    o.shift = sort_shift(*s);
    o.bins = (int)(((s->rows - 1) >> o.shift) + 1);
    o.wide = row_bytes % 16 == 0;
    o.status = device_status_ptr();
    const size_t smem = (size_t)(kSortWarps + 1) * o.bins * 4;
    const void* fn = s->id_bytes == 8 ? reinterpret_cast<const void*>(&embed_sort_kernel<int64_t>)
                                      : reinterpret_cast<const void*>(&embed_sort_kernel<int32_t>);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) {
        const unsigned P = 1u << o.shift;
        if (s->id_bytes == 8) embed_sort_kernel<int64_t><<<P, kSortThreads, smem, cs>>>(o);
        else embed_sort_kernel<int32_t><<<P, kSortThreads, smem, cs>>>(o);
        count_launch();
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        SumArgs a{};
        a.dY = dY;
        a.dW = dW;
        a.perm = o.perm;
        a.key = o.key;
        a.count = o.count;
        a.part = reinterpret_cast<float*>(ws + L.part);
        a.dim = s->dim;
        a.scale = s->scale;
        const bool g32 = s->grad_dtype == KAN_F32;
        if (s->dtype == KAN_F32)
            e = g32 ? sum_of<float, float>(*s, a, L.chunks, cs) : sum_of<float, __nv_bfloat16>(*s, a, L.chunks, cs);
        else
            e = g32 ? sum_of<__nv_bfloat16, float>(*s, a, L.chunks, cs)
                    : sum_of<__nv_bfloat16, __nv_bfloat16>(*s, a, L.chunks, cs);
    }
    return e == cudaSuccess ? KAN_OK : em_fail(KAN_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"

// kan_vec.cuh -- vectors of 2 to 16 bytes of fp32 or bf16 elements, for the
// streaming kernels whose rows need not be whole 16-byte vectors: the widest
// vector that divides a row (and every row's first address) is chosen at
// launch, down to single elements.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "kan_internal.h"

namespace kan {

template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };

// N elements of T as they lie in memory (kept packed while in flight).
template <typename T, int N> struct Pack {
    static constexpr int BYTES = N * (int)sizeof(T);
    using Raw = typename RawOf<BYTES>::type;
    Raw q;

    __device__ __forceinline__ static Pack load(const T* p)
    {
        Pack r;
        r.q = *reinterpret_cast<const Raw*>(p);
        return r;
    }
    __device__ __forceinline__ static Pack zero()
    {
        Pack r;
        r.q = Raw{};
        return r;
    }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = q; }
    __device__ __forceinline__ uint32_t word(int i) const
    {
        if constexpr (BYTES == 16) return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
        else if constexpr (BYTES == 8) return i == 0 ? q.x : q.y;
        else return (uint32_t)q;
    }
    __device__ __forceinline__ void unpack(float (&v)[N]) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __uint_as_float(word(i));
        } else if constexpr (N == 1) {
            v[0] = __uint_as_float((uint32_t)q << 16);
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                v[2 * i] = __uint_as_float(word(i) << 16);
                v[2 * i + 1] = __uint_as_float(word(i) & 0xFFFF0000u);
            }
        }
    }
    // round to nearest even, once, to T
    __device__ __forceinline__ static Pack pack(const float (&v)[N])
    {
        Pack r;
        if constexpr (sizeof(T) == 4) {
            if constexpr (N == 1) r.q = __float_as_uint(v[0]);
            else if constexpr (N == 2) r.q = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
            else r.q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        } else if constexpr (N == 1) {
            r.q = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
            uint32_t w[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if constexpr (N == 2) r.q = w[0];
            else if constexpr (N == 4) r.q = make_uint2(w[0], w[1]);
            else r.q = make_uint4(w[0], w[1], w[2], w[3]);
        }
        return r;
    }
};

// The largest power of two, at most 16, that divides every one of the given
// byte counts (row lengths, addresses).
inline int common_vector_bytes(uint64_t a, uint64_t b = 0, uint64_t c = 0, uint64_t d = 0)
{
    const uint64_t all = a | b | c | d | 16u;
    return (int)(all & (~all + 1));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace kan

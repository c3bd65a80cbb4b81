// The 4-bit key/value cache as its kernels see it: where a token's codes and
// parameters are, which sequence a row of the batch belongs to, and what a
// stored value stands for.
//
// A pool is [pages][kv_heads] blocks.  The block of one page and head holds
// page_size tokens:  key codes [page_size][D/2 bytes] (two per byte, low
// nibble first), key parameters [page_size][D/G] (half step, half minimum),
// then value codes and value parameters in the same form.  So a tile of
// consecutive tokens of one head is four contiguous pieces, each a multiple
// of 16 bytes for 16 tokens or more: what a bulk copy wants.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bq_common.cuh"
#include "bq_internal.h"

namespace bq {

// Sequence of row t of the batch: the number of ends cu[1..batch] at or below
// t, for every row with t < cu[batch].  Called by a whole block; a block-wide
// count, so the table is read in parallel and not by dependent steps.
__device__ __forceinline__ int kv4_find_seq(const Kv4Seqs &s, int64_t t) {
    if (s.cu == nullptr) return static_cast<int>(t / s.uniform_n);
    int found = 0;
    for (int base = 0; base < s.batch; base += static_cast<int>(blockDim.x)) {
        const int i = base + static_cast<int>(threadIdx.x);
        found += __syncthreads_count(i < s.batch && __ldg(s.cu + i + 1) <= t);
    }
    return found;
}

// First row and number of rows of sequence b.
__device__ __forceinline__ void kv4_rows(const Kv4Seqs &s, int b, int64_t &first, int &n) {
    if (s.cu == nullptr) {
        first = static_cast<int64_t>(b) * s.uniform_n;
        n = s.uniform_n;
    } else {
        first = __ldg(s.cu + b);
        n = static_cast<int>(__ldg(s.cu + b + 1) - first);
    }
}

// Position of the first of n rows of sequence b.  A length below 0 holds as
// few tokens as 0 does: with no less than -n, the distance from any row to any
// token has 32 bits.
__device__ __forceinline__ int kv4_first_position(const Kv4Seqs &s, int b, int n) {
    return max(__ldg(s.lens + b), 0) - max(n, 0);
}

// Positions that attention reaches: those of the table, and no more than leave
// room above them, so that the first token of a tile, of a copy, or of a page
// looked up ahead is a 32-bit number for every tile that begins below.
constexpr int kKv4MaxTokens = 0x7fff0000;
__device__ __forceinline__ int kv4_capacity(const Kv4Pool &p) {
    return static_cast<int>(min(static_cast<int64_t>(p.table_width) << p.page_log2, static_cast<int64_t>(kKv4MaxTokens)));
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Eight consecutive elements of one type as fp32.
template <typename T>
struct Kv4In;
template <>
struct Kv4In<float> {
    static constexpr int kVec = 2;
    static __device__ __forceinline__ void unpack(const uint4 (&v)[2], float (&f)[8]) {
        f[0] = __uint_as_float(v[0].x), f[1] = __uint_as_float(v[0].y);
        f[2] = __uint_as_float(v[0].z), f[3] = __uint_as_float(v[0].w);
        f[4] = __uint_as_float(v[1].x), f[5] = __uint_as_float(v[1].y);
        f[6] = __uint_as_float(v[1].z), f[7] = __uint_as_float(v[1].w);
    }
    static __device__ __forceinline__ void pack(const float (&f)[8], uint4 (&v)[2]) {
        v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
};
template <>
struct Kv4In<__nv_bfloat16> {
    static constexpr int kVec = 1;
    static __device__ __forceinline__ void unpack(const uint4 (&v)[1], float (&f)[8]) {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void pack(const float (&f)[8], uint4 (&v)[1]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Kv4In<__half> {
    static constexpr int kVec = 1;
    static __device__ __forceinline__ void unpack(const uint4 (&v)[1], float (&f)[8]) {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
    static __device__ __forceinline__ void pack(const float (&f)[8], uint4 (&v)[1]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// What the eight codes of a word stand for: step * code + minimum.  A code
// masked in place is an fp16 subnormal, code * 2^-24 or (the upper half of a
// byte) code * 2^-20; times the step with that power of two in it (4 x 11 bits)
// it is exact in fp32, so the sum is the only rounding.
__device__ __forceinline__ void kv4_values(uint32_t word, float2 step_minimum, float (&f)[8]) {
    const float s0 = step_minimum.x * 16777216.0f, s1 = step_minimum.x * 1048576.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t w = word >> (8 * j), lo = w & 0x000f000fu, hi = w & 0x00f000f0u;
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));  // elements 2 j, 2 j + 4
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));  // 2 j + 1, 2 j + 5
        f[2 * j] = fmaf(a.x, s0, step_minimum.y);
        f[2 * j + 4] = fmaf(a.y, s0, step_minimum.y);
        f[2 * j + 1] = fmaf(b.x, s1, step_minimum.y);
        f[2 * j + 5] = fmaf(b.y, s1, step_minimum.y);
    }
}

}  // namespace bq

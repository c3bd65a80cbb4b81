// What the attention kernels over the 4-bit cache share: small arithmetic, the
// partial results of work that spans several CTAs, and the kernel that joins
// them.
#pragma once

#include "kv4_common.cuh"

namespace bq {
namespace {

constexpr int kKv4MaxSms = 160;
constexpr float kNoMax = -3.0e38f;  // running maximum (in powers of two) before any token
constexpr float kLift = 7.0f;       // weights are 2^(z - maximum + kLift)

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// {lo, hi} as a pair of fp16
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) { return pack_f16(lo, hi); }

// A part of the work whose results are joined: `count` CTAs from this one on
// hold partial results of columns [col0, col0 + cols) of one key head.  Column
// c is query row first + c / share, head c % share of the group.
struct Kv4Partial {
    int64_t first;
    int col0, cols, head, count;
};

// A CTA leaves at most two partial results, in slot 2 cta + 1 for work that
// begins in it and goes on, in slot 2 cta for work that began earlier.  A slot
// holds D + 4 floats for each column: D weighted sums, the maximum (kNoMax
// before any token), the sum of the weights (0: nothing was seen, and the
// other sums mean nothing), and the divisor of each group.
struct Kv4Ws {
    Kv4Partial *desc;
    float *slots;
};
inline Kv4Ws kv4_workspace(void *ws) {
    return {static_cast<Kv4Partial *>(ws),
            reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + 2 * kKv4MaxSms * sizeof(Kv4Partial))};
}

constexpr int kJoinThreads = 256;

template <int D, int G, int COLS, typename T>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnArgs a, const Kv4Ws ws) {
    constexpr int64_t SLOT = static_cast<int64_t>(COLS) * (D + 4);
    pdl_wait();
    const int64_t cta = blockIdx.x;
    const Kv4Partial it = ws.desc[cta];
    if (it.count <= 1) return;
    const int share = a.q_heads / a.pool.kv_heads;
    for (int e = blockIdx.y * kJoinThreads + threadIdx.x; e < it.cols * (D / 4); e += gridDim.y * kJoinThreads) {
        const int c = e / (D / 4), d = e % (D / 4) * 4;
        const float *s0 = ws.slots + (2 * cta + 1) * SLOT + c * (D + 4);
        const float *s1 = ws.slots + 2 * (cta + 1) * SLOT + c * (D + 4);  // then 2 slots on
        float top = s0[D];
#pragma unroll 8
        for (int i = 1; i < it.count; ++i) top = fmaxf(top, s1[(i - 1) * 2 * SLOT + D]);
        float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float den = 0.0f, sum = 0.0f;
#pragma unroll 4
        for (int i = 0; i < it.count; ++i) {
            const float *s = i == 0 ? s0 : s1 + (i - 1) * 2 * SLOT;
            const float m = s[D];
            if (s[D + 1] == 0.0f) continue;
            const float k = ex2(m - top);
            const float4 v = *reinterpret_cast<const float4 *>(s + d);
            num.x = fmaf(v.x, k, num.x);
            num.y = fmaf(v.y, k, num.y);
            num.z = fmaf(v.z, k, num.z);
            num.w = fmaf(v.w, k, num.w);
            den = fmaf(s[D + 2 + d / G], k, den);
            sum = fmaf(s[D + 1], k, sum);
        }
        const int col = it.col0 + c, row = col / share, hh = col - row * share;
        const int64_t to = (it.first + row) * a.q_heads + static_cast<int64_t>(it.head) * share + hh;
        const float inv = den == 0.0f ? 0.0f : __fdividef(1.0f, den);
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + to * D + d) =
            make_uint2(pack2(num.x * inv, num.y * inv, T()), pack2(num.z * inv, num.w * inv, T()));
        if (a.lse != nullptr && d == 0)
            a.lse[to] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
    }
}

// Joins what `grid` CTAs left, as a programmatic dependent of their kernel.
template <int D, int G, int COLS, typename T>
cudaError_t kv4_launch_join(const Kv4AttnArgs &a, const Kv4Ws &ws, unsigned grid, cudaStream_t s) {
    if (grid < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid - 1, COLS > 24 ? 32 : (COLS * D / 4 + kJoinThreads - 1) / kJoinThreads);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, G, COLS, T>, a, ws);
}

}  // namespace
}  // namespace bq

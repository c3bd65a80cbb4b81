// What the attention kernels over the 4-bit cache share: small arithmetic, the
// partial results of work that spans several CTAs, and the kernel that joins
// them.
#pragma once

#include <algorithm>

#include "kv4_common.cuh"

namespace bq {
namespace {

constexpr int kKv4MaxSms = 160;
constexpr int kKv4MaxCtas = 3 * kKv4MaxSms;
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
// Capped scores, cap tanh(x / cap), from v = 2 log2(e) x / cap.  cap (1 - 2 /
// (2^v + 1)) is off by cap 2^-22 (exponential, reciprocal): 2^-16 at kFarCap, a
// 30th of a weight's own rounding.  Beyond it that would grow with the cap, so
// where |x / cap| < 1/4 the first terms of tanh's power series take its place:
// off by 2^-21 of the score; the other form is by 2^-20 there.
// (A variant of its own: in one with small caps and biases its registers cost
// prompts with a bias 4% of their time, one token with a cap of 30 3%; itself
// it takes 858 us for 2048 rows after 8192, where a cap of 30 takes 767.)
constexpr float kFarCap = 64.0f;
enum Mods { kPlain, kNearMods, kFarMods };  // nothing beside the products; a cap up to kFarCap, a bias, or both; a cap beyond
inline Mods mods_of(const Kv4AttnArgs &a) {
    return a.softcap > kFarCap ? kFarMods : a.softcap > 0.0f || a.slopes != nullptr ? kNearMods : kPlain;
}
constexpr float kSeries = 0.72134752044448170f;  // v at x / cap = 1/4
__device__ __forceinline__ float cap_series(float v, float scale) {  // scale v (1 - u^2 / 3 + 2 u^4 / 15 - 17 u^6 / 315)
    constexpr float k = 1.0f / (2.8853900817779268f * 2.8853900817779268f);  // u^2 = k v^2
    const float s = v * v;
    const float p = fmaf(s, fmaf(s, -17.0f / 315.0f * k * k * k, 2.0f / 15.0f * k * k), -1.0f / 3.0f * k);
    return fmaf(scale * v, s * p, scale * v);
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
            reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kKv4MaxCtas * sizeof(Kv4Partial))};
}

constexpr int kJoinThreads = 256;
// Threads that share the partial results of four dims: few rows are split over many CTAs, many rows over two or three.
constexpr int join_ways(int cols) { return cols > 24 ? 1 : 8; }

// Every load of a partial result is independent of the others (no branch
// between them), and join_ways threads take every so many-th one: what bounds
// this kernel is the latency of a few dependent steps.
template <int D, int G, int COLS, typename T>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4AttnArgs a, const Kv4Ws ws) {
    constexpr int64_t SLOT = static_cast<int64_t>(COLS) * (D + 4);
    constexpr int kJoinWays = join_ways(COLS);
    constexpr int PER = kJoinThreads / kJoinWays;  // groups of four dims of a block, one way each
    __shared__ float4 s_num[kJoinWays][PER];
    __shared__ float s_top[kJoinWays][PER], s_den[kJoinWays][PER], s_sum[kJoinWays][PER];
    pdl_wait();
    const int64_t cta = blockIdx.x;
    const Kv4Partial it = ws.desc[cta];
    if (it.count <= 1) return;
    const int share = a.q_heads / a.pool.kv_heads;
    const int way = threadIdx.x / PER, mine = threadIdx.x % PER;
    for (int e0 = blockIdx.y * PER; e0 < it.cols * (D / 4); e0 += gridDim.y * PER) {
        const int e = e0 + mine;  // (D / 4 is a multiple of 16, but a block may reach past the last column)
        const bool on = e < it.cols * (D / 4);
        const int c = on ? e / (D / 4) : 0, d = e % (D / 4) * 4;
        // slot 2 cta + 1 first, then every second one
        const float *s0 = ws.slots + 2 * cta * SLOT + c * (D + 4);
        auto part = [&](int i) { return s0 + (i == 0 ? SLOT : 2 * i * SLOT); };
        float top = kNoMax;
#pragma unroll 8
        for (int i = way; i < it.count; i += kJoinWays) top = fmaxf(top, part(i)[D]);
        float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float den = 0.0f, sum = 0.0f;
#pragma unroll 4
        for (int i = way; i < it.count; i += kJoinWays) {
            const float *s = part(i);
            float4 v = *reinterpret_cast<const float4 *>(s + d);
            const float4 st = *reinterpret_cast<const float4 *>(s + D);  // maximum, sum, divisors
            float ds = d < G ? st.z : st.w;
            const bool none = st.y == 0.0f;  // (the rest of the slot may never have been written)
            const float k = none ? 0.0f : ex2(st.x - top);
            if (none) {
                v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                ds = 0.0f;
            }
            num.x = fmaf(v.x, k, num.x);
            num.y = fmaf(v.y, k, num.y);
            num.z = fmaf(v.z, k, num.z);
            num.w = fmaf(v.w, k, num.w);
            den = fmaf(ds, k, den);
            sum = fmaf(st.y, k, sum);
        }
        s_num[way][mine] = num;
        s_top[way][mine] = top;
        s_den[way][mine] = den;
        s_sum[way][mine] = sum;
        __syncthreads();
        if (way == 0 && on) {
            top = s_top[0][mine];
#pragma unroll
            for (int w = 1; w < kJoinWays; ++w) top = fmaxf(top, s_top[w][mine]);
            num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            den = sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWays; ++w) {
                const float k = ex2(s_top[w][mine] - top);
                const float4 v = s_num[w][mine];
                num.x = fmaf(v.x, k, num.x);
                num.y = fmaf(v.y, k, num.y);
                num.z = fmaf(v.z, k, num.z);
                num.w = fmaf(v.w, k, num.w);
                den = fmaf(s_den[w][mine], k, den);
                sum = fmaf(s_sum[w][mine], k, sum);
            }
            const int col = it.col0 + c, row = col / share, hh = col - row * share;
            const int64_t to = (it.first + row) * a.q_heads + static_cast<int64_t>(it.head) * share + hh;
            const float inv = den == 0.0f ? 0.0f : __fdividef(1.0f, den);
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + to * D + d) =
                make_uint2(pack2(num.x * inv, num.y * inv, T()), pack2(num.z * inv, num.w * inv, T()));
            if (a.lse != nullptr && d == 0)
                a.lse[to] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// Joins what `grid` CTAs left, as a programmatic dependent of their kernel.
template <int D, int G, int COLS, typename T>
cudaError_t kv4_launch_join(const Kv4AttnArgs &a, const Kv4Ws &ws, unsigned grid, cudaStream_t s) {
    if (grid < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid - 1, std::min(COLS * D / 4 * join_ways(COLS) / kJoinThreads, 32));
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

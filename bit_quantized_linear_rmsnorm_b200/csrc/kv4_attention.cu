// Attention of query rows over the 4-bit key/value cache.
//
// One warp per (row, query head): tokens one at a time, each lane holding
// D / 32 dims, with a running maximum and sum in fp32.
#include <algorithm>

#include "kv4_common.cuh"

namespace bq {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half *p, float v) { *p = __float2half_rn(v); }

template <typename T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) kv4_attention_kernel(const Kv4AttnArgs a, uint32_t *status) {
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int b = kv4_find_seq(a.seqs, t);
    if (b >= a.seqs.batch) return;  // a row behind the last sequence
    int64_t first;
    int n;
    kv4_rows(a.seqs, b, first, n);
    const int64_t pos = static_cast<int64_t>(__ldg(a.seqs.lens + b)) - n + (t - first);
    const int share = a.q_heads / a.pool.kv_heads;
    const int page = 1 << a.pool.page_log2;
    for (int h = blockIdx.y * kWarps + warp; h < a.q_heads; h += gridDim.y * kWarps) {
        const T *q = static_cast<const T *>(a.q) + t * a.q_tok + h * a.q_head + lane * E;
        float qf[E], acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            qf[e] = to_f32(q[e]);
            acc[e] = 0.0f;
        }
        float top = -INFINITY, sum = 0.0f;
        const float slope = a.slopes != nullptr ? a.slopes[h] : 0.0f;
        for (int64_t key = a.window > 0 ? max(pos - a.window + 1, int64_t(0)) : 0; key <= pos; ++key) {
            const uint8_t *blk = kv4_block(a.pool, b, static_cast<int>(key), h / share, status, SITE_KV4_ATTENTION);
            float x = NAN, ks = NAN, km = NAN, vs = NAN, vm = NAN;
            uint32_t kc = 0, vc = 0;
            if (blk != nullptr) {
                const int slot = static_cast<int>(key) & (page - 1);
                const int half = static_cast<int>(a.pool.block_bytes >> 1);
                const int par = page * (D / 2) + (slot * (D / G) + lane * E / G) * 4;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    kc |= static_cast<uint32_t>(blk[slot * (D / 2) + lane * E / 2 + i]) << (8 * i);
                    vc |= static_cast<uint32_t>(blk[half + slot * (D / 2) + lane * E / 2 + i]) << (8 * i);
                }
                const float2 kp = __half22float2(*reinterpret_cast<const __half2 *>(blk + par));
                const float2 vp = __half22float2(*reinterpret_cast<const __half2 *>(blk + half + par));
                ks = kp.x, km = kp.y, vs = vp.x, vm = vp.y;
            }
            x = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(qf[e], kv4_value(kc, e, ks, km), x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            x *= a.scale;
            if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
            x = fmaf(slope, static_cast<float>(key - pos), x);
            const float now = max_nan(top, x);
            const float keep = top == -INFINITY ? 0.0f : expf(top - now), p = x == -INFINITY ? 0.0f : expf(x - now);
            sum = sum * keep + p;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(p, kv4_value(vc, e, vs, vm), acc[e] * keep);
            top = now;
        }
        T *o = static_cast<T *>(a.out) + (t * a.q_heads + h) * D + lane * E;
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int e = 0; e < E; ++e) from_f32(o + e, acc[e] * inv);
        if (a.lse != nullptr && lane == 0) a.lse[t * a.q_heads + h] = sum == 0.0f ? -INFINITY : top + logf(sum);
    }
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t s, const DevInfo &dev) {
    const dim3 grid(static_cast<unsigned>(a.total), static_cast<unsigned>((a.q_heads + kWarps - 1) / kWarps));
    auto by_shape = [&](auto tag) {
        using T = decltype(tag);
        auto kern = a.pool.head_dim == 64 ? kv4_attention_kernel<T, 64, 64>
                    : a.pool.group_size == 64 ? kv4_attention_kernel<T, 128, 64> : kv4_attention_kernel<T, 128, 128>;
        kern<<<grid, kWarps * 32, 0, s>>>(a, dev.status);
        return cudaGetLastError();
    };
    return a.dtype == BQ_F16 ? by_shape(__half()) : by_shape(__nv_bfloat16());
}

}  // namespace bq

// The 4-bit key/value cache: quantizing rows into their pages (write) and
// reading pages back as fp32, bf16 or fp16 rows.
//
// Write, for each group of G values x of one token, head and K or V:
//   m = half(clamp(min x, +-65504)),  s = half(min(fl32((max x - m) / 15), 65504))
//   c = clamp(rne((x - m) / s), 0, 15)            (s = 0: c = 0)
// with (max - m) in fp32 and the quotient (x - m) / s that of the real
// numbers: the fp32 quotient is used except within 2e-5 of a half, where its
// error (below 5e-6) could put a code on the wrong side; there fp64 decides.
// A group whose range is not finite (an infinity or a NaN in it) gets NaN
// parameters, so that reading it, and attention on it, give NaN.
//
// One thread holds eight values = one word of codes; D / 8 neighbouring
// threads a row, and a group's extrema meet by shuffles inside G / 8 threads.
// Both kernels read each byte once and write each byte once.
#include "kv4_common.cuh"

namespace bq {
namespace {

constexpr int kThreads = 256;

template <typename T, int D, int G, int U>
__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const T *__restrict__ k, const T *__restrict__ v, int64_t k_tok, int64_t k_head, int64_t v_tok,
                     int64_t v_head, int64_t total, int tokens_per_block, const Kv4Seqs seqs, const Kv4Pool pool,
                     uint32_t *status) {
    constexpr int LPR = D / 8;               // threads per row
    constexpr int RPB = kThreads / LPR;      // rows of a block at a time
    constexpr int NV = Kv4In<T>::kVec;
    __shared__ int s_seq[kKv4BlockTokens], s_pos[kKv4BlockTokens];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), total - t0));
    const int b0 = kv4_find_seq(seqs, t0);
    if (static_cast<int>(threadIdx.x) < nt) {
        const int64_t t = t0 + threadIdx.x;
        int b = seqs.cu == nullptr ? static_cast<int>(t / seqs.uniform_n) : b0;
        if (seqs.cu != nullptr)
            while (b < seqs.batch && __ldg(seqs.cu + b + 1) <= t) ++b;
        int pos = -1;
        if (b < seqs.batch) {
            int64_t first;
            int n;
            kv4_rows(seqs, b, first, n);
            const int len = __ldg(seqs.lens + b);
            const int64_t at = static_cast<int64_t>(len) - n + (t - first);
            if (at >= 0 && at < len) pos = static_cast<int>(at);
        }
        s_seq[threadIdx.x] = b;
        s_pos[threadIdx.x] = pos;
    }
    __syncthreads();

    const int lr = threadIdx.x % LPR;
    const int rows = nt * 2 * pool.kv_heads;  // (token, K or V, head), heads fastest
    // (a warp runs as long as its first row is in range: the shuffles need all of it)
    for (int w0 = (threadIdx.x & ~31) / LPR; w0 < rows; w0 += RPB * U) {
        const int r0 = w0 + (threadIdx.x & 31) / LPR;
        uint4 raw[U][NV];
        uint8_t *dst[U];
        bool isv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RPB;
            dst[u] = nullptr;
            isv[u] = false;
            if (r >= rows) continue;
            const int q = r / pool.kv_heads, head = r - q * pool.kv_heads;
            const int ti = q >> 1;
            isv[u] = q & 1;
            const T *src = isv[u] ? v + (t0 + ti) * v_tok + head * v_head : k + (t0 + ti) * k_tok + head * k_head;
            const int pos = s_pos[ti];
            if (pos < 0) continue;
            uint8_t *blk = kv4_block(pool, s_seq[ti], pos, head, status, SITE_KV4_WRITE);
            if (blk == nullptr) continue;
            const int slot = pos & ((1 << pool.page_log2) - 1);
            const int half = static_cast<int>(pool.block_bytes >> 1);
            // the word of this thread; the row's parameters follow the codes of the page
            dst[u] = blk + (isv[u] ? half : 0) + slot * (D / 2);
#pragma unroll
            for (int i = 0; i < NV; ++i) raw[u][i] = __ldg(reinterpret_cast<const uint4 *>(src) + lr * NV + i);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8];
            if (dst[u] == nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = 0.0f;
            } else {
                Kv4In<T>::unpack(raw[u], f);
            }
            float mn = f[0], mx = f[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                mn = min_nan(mn, f[j]);
                mx = max_nan(mx, f[j]);
            }
#pragma unroll
            for (int o = G / 16; o > 0; o >>= 1) {
                mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const bool finite = fabsf(mx - mn) <= 3.402823466e38f;
            const __half hm = __float2half_rn(fminf(fmaxf(mn, -65504.0f), 65504.0f));
            const float m = __half2float(hm);
            const __half hs = __float2half_rn(fminf(__fdiv_rn(fmaxf(mx - m, 0.0f), 15.0f), 65504.0f));
            const float s = __half2float(hs);
            const float inv15 = finite && s > 0.0f ? __fdividef(1.0f, 15.0f * s) : 0.0f;
            uint32_t word = 0;
            float worst = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c15 = __saturatef((f[j] - m) * inv15);  // clamps to 0..15 (times 1/15); NaN to 0
                const float r = fmaf(c15, 15.0f, 12582912.0f);      // rounds to an integer, ties to even
                worst = fmaxf(worst, fabsf(fmaf(c15, 15.0f, -(r - 12582912.0f))));
                word |= (__float_as_uint(r) & 15u) << (4 * j);
            }
            if (worst > 0.49998f) {
                word = 0;
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    // (indexing f by a loop variable would put it in local memory)
                    float x = f[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) x = j == i ? f[i] : x;
                    const double q = (static_cast<double>(x) - static_cast<double>(m)) / static_cast<double>(s);
                    word |= static_cast<uint32_t>(fmin(fmax(rint(q), 0.0), 15.0)) << (4 * j);
                }
            }
            if (dst[u] != nullptr) {
                const int slot_bytes = (1 << pool.page_log2) * (D / 2);
                *reinterpret_cast<uint32_t *>(dst[u] + lr * 4) = word;
                if (lr % (G / 8) == 0) {
                    // parameters of group lr / (G / 8): the row's place in the page from its codes' address
                    const __half2 par = finite ? __halves2half2(hs, hm)
                                               : __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
                    const int ti = (r0 + u * RPB) / pool.kv_heads >> 1;
                    const int slot = s_pos[ti] & ((1 << pool.page_log2) - 1);
                    uint8_t *pp = dst[u] - slot * (D / 2) + slot_bytes + (slot * (D / G) + lr / (G / 8)) * 4;
                    *reinterpret_cast<__half2 *>(pp) = par;
                }
            }
        }
    }
}

template <typename T, int D, int G, int U>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4Seqs seqs, const int32_t *__restrict__ starts, const Kv4Pool pool, int64_t total,
                    int tokens_per_block, T *__restrict__ k, T *__restrict__ v, uint32_t *status) {
    constexpr int LPR = D / 8;
    constexpr int RPB = kThreads / LPR;
    constexpr int NV = Kv4In<T>::kVec;
    __shared__ int s_seq[kKv4BlockTokens], s_pos[kKv4BlockTokens];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), total - t0));
    const int b0 = kv4_find_seq(seqs, t0);
    if (static_cast<int>(threadIdx.x) < nt) {
        const int64_t t = t0 + threadIdx.x;
        int b = b0;
        while (b < seqs.batch && __ldg(seqs.cu + b + 1) <= t) ++b;
        int pos = -1;
        if (b < seqs.batch) {
            const int64_t at = (t - __ldg(seqs.cu + b)) + (starts != nullptr ? __ldg(starts + b) : 0);
            if (at >= 0 && at <= 0x7fffffff)
                pos = static_cast<int>(at);
            else
                report(status, BQ_ERR_INVALID_ARG, SITE_KV4_READ);
        }
        s_seq[threadIdx.x] = b;
        s_pos[threadIdx.x] = pos;
    }
    __syncthreads();

    const int lr = threadIdx.x % LPR;
    const int rows = nt * 2 * pool.kv_heads;
    for (int r0 = threadIdx.x / LPR; r0 < rows; r0 += RPB * U) {
        uint32_t word[U];
        __half2 par[U];
        T *dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + u * RPB;
            dst[u] = nullptr;
            if (r >= rows) continue;
            const int q = r / pool.kv_heads, head = r - q * pool.kv_heads;
            const int ti = q >> 1;
            if (s_seq[ti] >= seqs.batch) continue;  // a row behind the last sequence stays as it was
            dst[u] = ((q & 1) ? v : k) + ((t0 + ti) * pool.kv_heads + head) * D;
            word[u] = 0;
            par[u] = __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
            const int pos = s_pos[ti];
            if (pos < 0) continue;
            const uint8_t *blk = kv4_block(pool, s_seq[ti], pos, head, status, SITE_KV4_READ);
            if (blk == nullptr) continue;  // (no page there: NaN)
            const int slot = pos & ((1 << pool.page_log2) - 1);
            blk += (q & 1) ? static_cast<int>(pool.block_bytes >> 1) : 0;
            word[u] = *reinterpret_cast<const uint32_t *>(blk + slot * (D / 2) + lr * 4);
            par[u] = *reinterpret_cast<const __half2 *>(blk + (1 << pool.page_log2) * (D / 2) +
                                                        (slot * (D / G) + lr / (G / 8)) * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (dst[u] == nullptr) continue;
            const float2 sm = __half22float2(par[u]);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = kv4_value(word[u], j, sm.x, sm.y);
            uint4 o[NV];
            Kv4In<T>::pack(f, o);
#pragma unroll
            for (int i = 0; i < NV; ++i) __stcs(reinterpret_cast<uint4 *>(dst[u]) + lr * NV + i, o[i]);
        }
    }
}

// Tokens of one block: enough rows for U in flight per thread where the call
// is large, one token where it is small (a decode step), so that the blocks
// spread over the SMs.
int tokens_per_block(int64_t total, int kv_heads, int rows_at_a_time, int U, int num_sms) {
    const int64_t want = (static_cast<int64_t>(rows_at_a_time) * U + 2 * kv_heads - 1) / (2 * kv_heads);
    const int64_t spread = (total + 4 * num_sms - 1) / (4 * num_sms);
    int64_t n = want < spread ? want : spread;
    if (n < 1) n = 1;
    return static_cast<int>(n > kKv4BlockTokens ? kKv4BlockTokens : n);
}

template <typename T, int D, int G>
cudaError_t write_t(const Kv4WriteArgs &a, cudaStream_t s, const DevInfo &dev) {
    constexpr int U = sizeof(T) == 4 ? 2 : 4;
    const int tpb = tokens_per_block(a.total, a.pool.kv_heads, kThreads / (D / 8), U, dev.num_sms);
    const unsigned grid = static_cast<unsigned>((a.total + tpb - 1) / tpb);
    kv4_write_kernel<T, D, G, U><<<grid, kThreads, 0, s>>>(
        static_cast<const T *>(a.k), static_cast<const T *>(a.v), a.k_tok, a.k_head, a.v_tok, a.v_head, a.total, tpb,
        a.seqs, a.pool, dev.status);
    return cudaGetLastError();
}

template <typename T, int D, int G>
cudaError_t read_t(const Kv4ReadArgs &a, cudaStream_t s, const DevInfo &dev) {
    constexpr int U = 4;
    const int tpb = tokens_per_block(a.total, a.pool.kv_heads, kThreads / (D / 8), U, dev.num_sms);
    const unsigned grid = static_cast<unsigned>((a.total + tpb - 1) / tpb);
    kv4_read_kernel<T, D, G, U><<<grid, kThreads, 0, s>>>(a.seqs, a.starts, a.pool, a.total, tpb, static_cast<T *>(a.k),
                                                           static_cast<T *>(a.v), dev.status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto by_shape = [&](auto tag) {
        using T = decltype(tag);
        if (a.pool.head_dim == 64) return write_t<T, 64, 64>(a, s, dev);
        return a.pool.group_size == 64 ? write_t<T, 128, 64>(a, s, dev) : write_t<T, 128, 128>(a, s, dev);
    };
    if (a.dtype == BQ_F32) return by_shape(float());
    return a.dtype == BQ_F16 ? by_shape(__half()) : by_shape(__nv_bfloat16());
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto by_shape = [&](auto tag) {
        using T = decltype(tag);
        if (a.pool.head_dim == 64) return read_t<T, 64, 64>(a, s, dev);
        return a.pool.group_size == 64 ? read_t<T, 128, 64>(a, s, dev) : read_t<T, 128, 128>(a, s, dev);
    };
    if (a.dtype == BQ_F32) return by_shape(float());
    return a.dtype == BQ_F16 ? by_shape(__half()) : by_shape(__nv_bfloat16());
}

}  // namespace bq

// The 4-bit key/value cache: quantizing rows into their pages (write) and
// reading pages back as fp32, bf16 or fp16 rows.
//
// Write, for each group of G values x of one token, head and K or V:
//   m = half(clamp(min x, +-65504)),  s = half(min(fl32((max x - m) / 15), 65504))
//   c = clamp(rne((x - m) / s), 0, 15)            (s = 0: c = 0)
// with (max - m) in fp32 and the quotient (x - m) / s that of the real
// numbers: the fp32 quotient is used except within 2e-5 of a half, where its
// error (below 5e-6) could put a code on the wrong side; there x is
// compared with m + (k + 1/2) s in fp64, where that is exact.
// A group whose range is not finite (an infinity or a NaN in it) gets NaN
// parameters, so that reading it, and attention on it, give NaN.
//
// One thread holds eight values = one word of codes; D / 8 neighbouring
// threads a row, and a group's extrema meet by shuffles inside G / 8 threads.
// Both kernels read each byte once and write each byte once.  A block first
// works out where its tokens lie, once for all heads; a warp then walks the
// tokens of one head and side (keys or values), so that a row costs two
// additions of addresses.  (With a row of any head and side at a time, and its
// page looked up for each, the same work was bound by its own instructions:
// 104 us instead of 67 us, with 52 us for its bytes, to read 65537 tokens of 8
// heads of 128 as bf16.)
#include <algorithm>

#include "kv4_common.cuh"

namespace bq {
namespace {

constexpr int kThreads = 256;

// Where the tokens of a block lie in the pool, without the head and the side.
struct Places {
    int64_t code[kKv4BlockTokens];  // byte offset of the row's codes, or -1: no place (-2: NaN is read there)
    int64_t par[kKv4BlockTokens];   // of its parameters
};
template <int D, int G>
__device__ __forceinline__ void set_place(Places &p, int i, const Kv4Pool &pool, int b, int64_t at, uint32_t *status,
                                          uint32_t site) {
    int page = -1;
    const int64_t entry = at >> pool.page_log2;
    if (at >= 0 && entry < pool.table_width) page = __ldg(pool.table + static_cast<int64_t>(b) * pool.table_ld + entry);
    if (page < 0 || page >= pool.pages) {
        report(status, BQ_ERR_INVALID_ARG, site);
        p.code[i] = -2;
        return;
    }
    const int slot = static_cast<int>(at) & ((1 << pool.page_log2) - 1);
    const int64_t base = static_cast<int64_t>(page) * pool.page_stride;
    p.code[i] = base + slot * (D / 2);
    p.par[i] = base + (D / 2 << pool.page_log2) + slot * (4 * (D / G));
}

template <typename T, int D, int G, int U>
__global__ void __launch_bounds__(kThreads)
    kv4_write_kernel(const T *__restrict__ k, const T *__restrict__ v, int64_t k_tok, int64_t k_head, int64_t v_tok,
                     int64_t v_head, int64_t total, int tokens_per_block, const Kv4Seqs seqs, const Kv4Pool pool,
                     uint32_t *status) {
    constexpr int LPR = D / 8;           // threads per row
    constexpr int TPW = 32 / LPR;        // tokens of a warp at a time
    constexpr int NV = Kv4In<T>::kVec;
    __shared__ Places places;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), total - t0));
    const int b0 = kv4_find_seq(seqs, t0);
    if (static_cast<int>(threadIdx.x) < nt) {
        const int64_t t = t0 + threadIdx.x;
        int b = seqs.cu == nullptr ? static_cast<int>(t / seqs.uniform_n) : b0;
        if (seqs.cu != nullptr)
            while (b < seqs.batch && __ldg(seqs.cu + b + 1) <= t) ++b;
        places.code[threadIdx.x] = -1;
        if (b < seqs.batch) {
            int64_t first;
            int n;
            kv4_rows(seqs, b, first, n);
            const int len = __ldg(seqs.lens + b);
            const int64_t at = static_cast<int64_t>(len) - n + (t - first);
            if (at >= 0 && at < len) set_place<D, G>(places, threadIdx.x, pool, b, at, status, SITE_KV4_WRITE);
        }
    }
    __syncthreads();

    const int lane = threadIdx.x & 31, lr = lane % LPR, lt = lane / LPR;
    const int warps = kThreads / 32, pairs = 2 * pool.kv_heads;
    // a warp takes (head, side) pairs, or, where there are few, some of the tokens of one
    const int split = max(1, min(warps / pairs, (nt + TPW * U - 1) / (TPW * U)));
    for (int w = threadIdx.x >> 5; w < pairs * split; w += warps) {
        const int pair = w / split, from = (w - pair * split) * TPW * U;
        const bool isv = pair & 1;
        const int head = pair >> 1;
        const T *src = (isv ? v + head * v_head : k + head * k_head) + lr * 8;
        const int64_t tok = isv ? v_tok : k_tok;
        uint8_t *dst = pool.pool + head * pool.block_bytes + (isv ? pool.block_bytes >> 1 : 0);
        for (int ti0 = from; ti0 < nt; ti0 += TPW * U * split) {
            uint4 raw[U][NV];
            int64_t code[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ti = ti0 + u * TPW + lt;
                code[u] = ti < nt ? places.code[ti] : -1;
                if (code[u] >= 0) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) raw[u][i] = __ldg(reinterpret_cast<const uint4 *>(src + (t0 + ti) * tok) + i);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (ti0 + u * TPW >= nt) break;  // (no lane has a row: the shuffles need all of them)
                float f[8];
                if (code[u] < 0) {
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
                uint32_t word = 0, near = 0;  // near: elements whose quotient may be on the wrong side of a half
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c15 = __saturatef((f[j] - m) * inv15);  // clamps to 0..15 (times 1/15); NaN to 0
                    const float r = fmaf(c15, 15.0f, 12582912.0f);      // rounds to an integer, ties to even
                    near |= fabsf(fmaf(c15, 15.0f, -(r - 12582912.0f))) > 0.49998f ? 1u << j : 0u;
                    word |= (__float_as_uint(r) & 15u) << (4 * j);
                }
                while (near != 0) {  // one element in about 25000: the exact comparison with the half between two codes
                    const int j = __ffs(near) - 1;
                    near &= near - 1;
                    // (indexing f by a variable would put it in local memory)
                    float x = f[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) x = j == i ? f[i] : x;
                    const int k = static_cast<int>(__saturatef((x - m) * inv15) * 15.0f);  // the code below the half
                    const double half = static_cast<double>(m) + (k + 0.5) * static_cast<double>(s);  // (exact)
                    const int c = x > half || (x == half && (k & 1)) ? k + 1 : k;
                    word = (word & ~(15u << (4 * j))) | static_cast<uint32_t>(c) << (4 * j);
                }
                if (code[u] >= 0) {
                    *reinterpret_cast<uint32_t *>(dst + code[u] + lr * 4) = word;
                    if (lr % (G / 8) == 0)
                        *reinterpret_cast<__half2 *>(dst + places.par[ti0 + u * TPW + lt] + lr / (G / 8) * 4) =
                            finite ? __halves2half2(hs, hm) : __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));
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
    constexpr int TPW = 32 / LPR;
    constexpr int NV = Kv4In<T>::kVec;
    __shared__ Places places;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), total - t0));
    const int b0 = kv4_find_seq(seqs, t0);
    if (static_cast<int>(threadIdx.x) < nt) {
        const int64_t t = t0 + threadIdx.x;
        int b = b0;
        while (b < seqs.batch && __ldg(seqs.cu + b + 1) <= t) ++b;
        places.code[threadIdx.x] = -1;  // a row behind the last sequence stays as it was
        if (b < seqs.batch) {
            const int64_t at = (t - __ldg(seqs.cu + b)) + (starts != nullptr ? __ldg(starts + b) : 0);
            set_place<D, G>(places, threadIdx.x, pool, b, at <= 0x7fffffff ? at : -1, status, SITE_KV4_READ);
        }
    }
    __syncthreads();

    const int lane = threadIdx.x & 31, lr = lane % LPR, lt = lane / LPR;
    const int warps = kThreads / 32, pairs = 2 * pool.kv_heads;
    const int split = max(1, min(warps / pairs, (nt + TPW * U - 1) / (TPW * U)));
    const int64_t row = static_cast<int64_t>(pool.kv_heads) * D;
    for (int w = threadIdx.x >> 5; w < pairs * split; w += warps) {
        const int pair = w / split, from = (w - pair * split) * TPW * U;
        const bool isv = pair & 1;
        const int head = pair >> 1;
        const uint8_t *src = pool.pool + head * pool.block_bytes + (isv ? pool.block_bytes >> 1 : 0);
        T *dst = (isv ? v : k) + t0 * row + head * D + lr * 8;
        for (int ti0 = from; ti0 < nt; ti0 += TPW * U * split) {
            uint32_t word[U];
            __half2 par[U];
            bool on[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ti = ti0 + u * TPW + lt;
                const int64_t code = ti < nt ? places.code[ti] : -1;
                on[u] = code != -1;
                word[u] = 0;
                par[u] = __halves2half2(__ushort_as_half(0x7fff), __ushort_as_half(0x7fff));  // (no page there: NaN)
                if (code >= 0) {
                    word[u] = *reinterpret_cast<const uint32_t *>(src + code + lr * 4);
                    par[u] = *reinterpret_cast<const __half2 *>(src + places.par[ti] + lr / (G / 8) * 4);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!on[u]) continue;
                float f[8];
                kv4_values(word[u], __half22float2(par[u]), f);
                uint4 o[NV];
                Kv4In<T>::pack(f, o);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    __stcs(reinterpret_cast<uint4 *>(dst + (ti0 + u * TPW + lt) * row) + i, o[i]);
            }
        }
    }
}

// Tokens of one block: the most where the call is large, fewer where it is
// small (a decode step), so that the blocks spread over the SMs; a warp takes
// `step` at a time.
int tokens_per_block(int64_t total, int step, int blocks) {
    int64_t n = (total + blocks - 1) / blocks;
    if (n > step / 2) n = (n + step - 1) / step * step;
    return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 1), kKv4BlockTokens));
}

template <typename T, int D, int G>
cudaError_t write_t(const Kv4WriteArgs &a, cudaStream_t s, const DevInfo &dev) {
    constexpr int U = 2;
    const int tpb = tokens_per_block(a.total, 256 / D * U, 12 * dev.num_sms);
    const unsigned grid = static_cast<unsigned>((a.total + tpb - 1) / tpb);
    kv4_write_kernel<T, D, G, U><<<grid, kThreads, 0, s>>>(
        static_cast<const T *>(a.k), static_cast<const T *>(a.v), a.k_tok, a.k_head, a.v_tok, a.v_head, a.total, tpb,
        a.seqs, a.pool, dev.status);
    return cudaGetLastError();
}

template <typename T, int D, int G>
cudaError_t read_t(const Kv4ReadArgs &a, cudaStream_t s, const DevInfo &dev) {
    constexpr int U = 8;
    const int tpb = tokens_per_block(a.total, 256 / D * U, 6 * dev.num_sms);
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

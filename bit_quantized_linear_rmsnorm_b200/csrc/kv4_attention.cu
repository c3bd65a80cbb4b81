// Attention of a few query rows over the 4-bit key/value cache (decoding, and
// verifying a few drafted tokens): bound by reading the cache.
//
// Arithmetic.  A stored element is s * c + m with one step s and minimum m per
// group of G elements of a token, so both leave the products:
//
//   q . K[t]   = sum_g s_k[t,g] (q_g . c[t,g]) + m_k[t,g] sum(q_g)
//   sum p V[t] = sum_t (p_t s_v[t]) (c[t] - 8) + sum_t p_t (m_v[t] + 8 s_v[t])
//
// and the matrix instructions (mma.sync m16n8k16, fp16 x fp16 -> fp32) see
// the codes themselves.  A code masked in place out of its word, (w &
// 0x000f000f) or (w & 0x00f000f0), is a pair of fp16 subnormals c * 2^-24 or
// c * 2^-20, exact: two elements cost one AND and half a shift, and the powers
// of two go into the query (odd codes' 2^4) and the final scale.  Values' codes
// are taken from the middle (one subtraction for two, exact): the instruction's
// additions round toward zero, and sums of 0..15 drift with every step while the
// result is what the minima's term leaves of them (one row over 131072 tokens:
// relative error 0.0018 against 0.0016 of a 32-bit computation rounded to bf16;
// now the same).  Keys are the A
// operand of K q^T (rows: 16 tokens), values that of V^T p (rows: 16 dims),
// so 8 columns carry the query rows and heads that share a key head, and p
// moves from one product to the next by two 8 x 8 register transposes.
//
// Roundings.  q is scaled by a power of two into fp16, odd elements 2^4 lower:
// exact for bf16 values within 2^-27 of the row's largest, fp16 values within
// 2^-24; what is smaller is off by 2^-35 of it at most.  p * s_v is rounded
// once to fp16, the type of the instruction (a second half of it would double
// the products with the values, and a bf16 result's error, 0.0017 of the
// largest, is that of a 32-bit computation as it is; fp16 results have 0.0003
// where that has 0.0002); the sums that go with it (the divisor, and the
// minima's term, and with them lse) are taken of the same rounded weights, so
// the rounding acts as a relative error of a weight, 2^-11 at most (weights
// below 2^-21 of the largest: 2^-32 of that one), and cancels for a
// single token.  (A step far below the others' can leave fp16's normal range
// with its weight: such a weight counts in the sums as it is.)
// Running maximum, sums and products are fp32.  The maximum is
// that of z + log2 s_v, which keeps p * s_v within fp16 whatever the steps
// are; it is raised only when a score passes it by 2^8 (the weights then stay
// below 2^15), so most tiles need no shuffles and no rescaling.
//
// Work.  Up to 72 columns (bq_internal.h has the measurements), in blocks of
// 8, 16 or 24.  The tiles (32 tokens of one key head and column block) of the whole
// batch, and kStart tiles' worth for beginning an item, are one list, cut into
// equal shares for the CTAs, whatever the lengths are: three CTAs per SM (two
// where more columns take the registers), 4 warps each, every warp with a ring
// of tiles of its own that bulk copies fill.  The warps of a share meet in
// shared memory; a (sequence, head, columns) item that spans several CTAs
// leaves partial results in the workspace, and a second kernel, launched as a
// programmatic dependent, joins them.
//
// What bounds it: DRAM traffic is the cache read once (321 MB for 64 ragged
// sequences of up to 8192 tokens, 8 heads of 128), but at 96 to 98 us (50% of the
// measured copy bandwidth) it is the issue of instructions: about 720 for a
// tile, of which 192 bring codes into registers, at 57% of the issue slots,
// the rest being fixed latencies of 12 warps.  Measured against this split:
// two CTAs of 8 warps (128 registers, addresses worked out again for each
// tile) 119 us; copies by cp.async of all lanes 122 us; without kStart 129 us.
//
// Every wait on a copy is bounded; if one runs out, the kernel records
// BQ_ERR_TIMEOUT, lets its copies land (bounded again) and finishes.
#include <algorithm>

#include "kv4_attention.cuh"

namespace bq {
namespace {

constexpr int kTile = 32;
constexpr int kW = 4;  // warps
constexpr int kThreads = kW * 32;
constexpr int kStart = 12;  // cost of starting an item, in tiles (64 ragged sequences: 115, 109, 105, 102 us at 3, 6, 10, 14)
constexpr float kSlack = 8.0f;  // a maximum is raised when passed by more
constexpr float kFarStep = 0.001953125f;  // a step below 2^-9 of the largest is far from it

// (D, G) shape of the cache and the geometry that follows from it.
template <int D_, int G_, int NB_>
struct Shape {
    static constexpr int D = D_, G = G_, NB = NB_;
    static constexpr int HV = D / 64;            // 64-element halves of a row
    static constexpr int GR = D / G;             // groups of a row
    static constexpr int ROW = D / 2;            // bytes of codes of a token
    static constexpr int PAR = 4 * GR;           // bytes of parameters of a token
    static constexpr int CODES = kTile * ROW, PARS = kTile * PAR;
    static constexpr int STAGE = 2 * (CODES + PARS);
    static constexpr int CTAS = NB == 1 ? 3 : 2;  // per SM
    static constexpr int S = NB == 1 ? 3 : 5;  // stages of a warp (a fourth gains nothing)
    static constexpr int COLS = 8 * NB;
    static constexpr int CSTR = D + 8;  // floats between columns of a warp's results
    static constexpr int RES = (COLS * CSTR + COLS * (2 + GR)) * 4;  // bytes of a warp's results
    static constexpr int QSM = NB == 1 ? 0 : HV * 4 * NB * 32 * 8;   // query fragments in shared memory
    static constexpr int RING = kW * S * STAGE;
    static_assert(kW * RES <= RING, "the results of the warps share the ring");
    static constexpr int OFF_Q = RING;
    static constexpr int OFF_BAR = OFF_Q + QSM;
    static constexpr int SMEM = OFF_BAR + kW * S * 8;
    static constexpr size_t SLOT = static_cast<size_t>(COLS) * (D + 4);  // floats of a partial result
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes less 8, both as pairs of fp16 subnormals: exact.
__device__ __forceinline__ uint32_t from_middle(uint32_t codes, uint32_t eight) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(codes), "r"(eight));
    return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// What the rows of sequence b need of the cache.
struct SeqPlan {
    int64_t first;  // first row
    int rows;       // rows computed (at most max_q)
    int pos0;       // position of the first row
    int lo, hi;     // first and last position that a row sees (hi -1: none)
    int t0, tiles;  // first tile and number of tiles (1 for rows that see nothing)
    int blocks;     // column blocks
};
__device__ __forceinline__ SeqPlan plan_seq(const Kv4AttnArgs &a, int b, int share, int cols) {
    SeqPlan p;
    int n;
    kv4_rows(a.seqs, b, p.first, n);
    // (a row past the tensor is never touched, whatever the offsets say)
    p.rows = static_cast<int>(min(static_cast<int64_t>(min(n, a.max_q)), a.total - p.first));
    if (n <= 0 || p.rows < 0 || p.first < 0) p.rows = 0;
    p.pos0 = kv4_first_position(a.seqs, b, n);
    const int cap = kv4_capacity(a.pool);
    p.hi = static_cast<int>(min(static_cast<int64_t>(p.pos0) + p.rows, static_cast<int64_t>(cap))) - 1;
    p.lo = a.window > 0 ? static_cast<int>(max(static_cast<int64_t>(p.pos0) - a.window + 1, int64_t(0))) : 0;
    if (p.hi < p.lo) p.hi = -1;
    p.t0 = p.lo / kTile;
    p.tiles = p.hi < 0 ? 1 : p.hi / kTile - p.t0 + 1;
    p.blocks = static_cast<int>((static_cast<int64_t>(p.rows) * share + cols - 1) / cols);
    return p;
}

template <typename C, Mods MODS, typename T>
__global__ void __launch_bounds__(kThreads, C::CTAS) kv4_decode_kernel(const Kv4AttnArgs a, const Kv4Ws ws, uint32_t *status) {
    constexpr int D = C::D, NB = C::NB, HV = C::HV, GR = C::GR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_sum[kW];
    __shared__ int s_b;
    __shared__ int64_t s_before;
    __shared__ uint32_t s_nan;  // columns whose query is not finite
    pdl_launch_dependents();    // the joining kernel waits for this grid before it reads
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    // token of score row g (of 8): tokens 4, 5 and 6, 7 change places, so that the value words of lanes t = 0, 1 and
    // t = 2, 3, which are then of tokens of different parity, lie in different banks
    const int gt = g ^ (g >> 2);
    const int share = a.q_heads / a.pool.kv_heads;
    const int page_log2 = a.pool.page_log2;
    const uint32_t ring = smem_u32(smem) + warp * C::S * C::STAGE;
    const uint32_t bars = smem_u32(smem) + C::OFF_BAR + warp * C::S * 8;
    if (lane < C::S) mbar_init(bars + 8 * lane, 1);
    fence_mbarrier_init();

    // ---- the share of this CTA: units [u, u_end) of the batch's list, whose
    // items (a head's column block of a sequence) count their tiles and
    // kStart, column blocks fastest, then heads, then sequences
    const int64_t per = (a.seqs.batch + kThreads - 1) / kThreads;
    const int64_t b_lo = min(per * threadIdx.x, static_cast<int64_t>(a.seqs.batch));
    const int64_t b_hi = min(b_lo + per, static_cast<int64_t>(a.seqs.batch));
    int64_t mine = 0;
    for (int64_t b = b_lo; b < b_hi; ++b) {
        const SeqPlan p = plan_seq(a, static_cast<int>(b), share, C::COLS);
        mine += static_cast<int64_t>(p.tiles + kStart) * p.blocks * a.pool.kv_heads;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    // a share is at least about one tile per warp
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + kW - 1) / kW);
    const int64_t cta = blockIdx.x;
    if (threadIdx.x == 0 && ws.desc != nullptr) ws.desc[cta].count = 0;
    if (cta >= ctas) return;
    const int64_t u_begin = total * cta / ctas, u_end = total * (cta + 1) / ctas;
    if (u_begin >= before && u_begin < before + mine) {
        int64_t at = before;
        for (int64_t b = b_lo; b < b_hi; ++b) {
            const SeqPlan p = plan_seq(a, static_cast<int>(b), share, C::COLS);
            const int64_t n = static_cast<int64_t>(p.tiles + kStart) * p.blocks * a.pool.kv_heads;
            if (u_begin < at + n) {
                s_b = static_cast<int>(b);
                s_before = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int b = s_b;
    int64_t seq_begin = s_before;  // first unit of sequence b

    int issued = 0, taken = 0;  // tiles of this warp's ring, over all segments
    bool dead = false;          // a wait ran out
    for (int64_t u = u_begin; u < u_end;) {
        // ---- next segment: the part of one item that falls into the share
        SeqPlan p = plan_seq(a, b, share, C::COLS);
        const auto cost = [&] { return static_cast<int64_t>(p.tiles + kStart) * p.blocks * a.pool.kv_heads; };
        while (u >= seq_begin + cost()) {
            seq_begin += cost();
            p = plan_seq(a, ++b, share, C::COLS);
        }
        const int item_cost = p.tiles + kStart;
        const int64_t item = (u - seq_begin) / item_cost;
        const int64_t item_begin = seq_begin + item * item_cost, item_end = item_begin + item_cost;
        const int head = static_cast<int>(item / p.blocks), cb = static_cast<int>(item % p.blocks);
        const int64_t seg_end = min(item_end, u_end);
        // (a part's tiles are in proportion to its cost; there may be none)
        const int64_t first_tile = (u - item_begin) * p.tiles / item_cost;
        const int tile0 = p.t0 + static_cast<int>(first_tile);
        const int ntiles = static_cast<int>((seg_end - item_begin) * p.tiles / item_cost - first_tile);
        const int col0 = cb * C::COLS;  // columns: row of the sequence * share + head of the group
        const int ncols = min(C::COLS, p.rows * share - col0);
        const int cap = kv4_capacity(a.pool);

        // ---- the warp's own tiles: tile0 + warp, + kW, ...; their pages are
        // looked up 32 tiles ahead, a lane each
        const int mytiles = ntiles > warp ? (ntiles - warp + kW - 1) / kW : 0;
        int64_t src0 = 0, src1 = 0;  // block of the page (both halves of a tile where pages are 16 tokens), -1: none
        auto look_up = [&](int i0) {
            src0 = src1 = -1;
            const int tok = (tile0 + warp + (i0 + lane) * kW) * kTile;
            if (i0 + lane < mytiles) {
                auto page_at = [&](int pos) -> int64_t {
                    const int i = pos >> page_log2;  // (pos <= hi < capacity of the table)
                    const int pg = __ldg(a.pool.table + static_cast<int64_t>(b) * a.pool.table_ld + i);
                    if (pg < 0 || pg >= a.pool.pages) {
                        report(status, BQ_ERR_INVALID_ARG, SITE_KV4_ATTENTION);
                        return -2;
                    }
                    return static_cast<int64_t>(pg) * a.pool.page_stride +
                           static_cast<int64_t>(head) * a.pool.block_bytes;
                };
                // (a page that ends before the window may be gone, and its entry name none)
                if (tok <= p.hi && (page_log2 != 4 || tok + 16 > p.lo)) src0 = page_at(tok);
                if (page_log2 == 4 && tok + 16 <= p.hi) src1 = page_at(tok + 16);
            }
        };
        uint32_t bad_bits = 0;  // per stage, 2 bits: a half of the tile has no page
        auto issue = [&](int i) {
            const int stage = issued % C::S;
            const int64_t s0 = __shfl_sync(0xffffffffu, src0, i & 31);
            const int64_t s1 = page_log2 == 4 ? __shfl_sync(0xffffffffu, src1, i & 31) : -1;
            const uint32_t dst = ring + stage * C::STAGE, bar = bars + 8 * stage;
            const int parts = page_log2 == 4 ? 2 : 1;
            const int toks = kTile / parts;
            const uint32_t bytes = static_cast<uint32_t>(toks * (C::ROW + C::PAR) * 2);
            if (lane == 0) mbar_arrive_expect_tx(bar, (s0 >= 0 ? bytes : 0) + (s1 >= 0 ? bytes : 0));
            __syncwarp();
            const int part = lane >> 2, what = lane & 3;  // K codes, K parameters, V codes, V parameters
            const int64_t s = part == 0 ? s0 : s1;
            if (part < parts && s >= 0) {
                const int slot = ((tile0 + warp + i * kW) * kTile) & ((1 << page_log2) - 1);
                const int off = (what >> 1) * static_cast<int>(a.pool.block_bytes >> 1) +
                                ((what & 1) ? (C::ROW << page_log2) + (part ? 0 : slot) * C::PAR
                                            : (part ? 0 : slot) * C::ROW);
                const uint32_t to = (what >> 1) * (C::CODES + C::PARS) + ((what & 1) ? C::CODES + part * toks * C::PAR
                                                                                    : part * toks * C::ROW);
                bulk_load(dst + to, a.pool.pool + s + off, static_cast<uint32_t>(toks * ((what & 1) ? C::PAR : C::ROW)),
                          bar);
            }
            const uint32_t bad = (s0 == -2 ? (parts == 1 ? 3u : 1u) : 0u) | (s1 == -2 ? 2u : 0u);
            bad_bits = (bad_bits & ~(3u << (2 * stage))) | (bad << (2 * stage));
            ++issued;
        };
        look_up(0);
        int next = 0;
        for (; next < min(C::S, mytiles) && !dead; ++next) issue(next);

        // ---- the query: this lane's fragments are of column g (of 8), dims
        // 64 h + 16 t .. + 15
        uint32_t qf[NB == 1 ? HV * 8 : 1];
        float f[NB][2], sq[NB][2][GR];
        int pos[NB][2];
        float slope[NB][2];
        if (threadIdx.x == 0) s_nan = 0;
        __syncthreads();
        {
            float fc[NB], sc[NB][GR];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int c = col0 + nb * 8 + g;
                const bool on = nb * 8 + g < ncols;
                const int row = c / share, hh = c - row * share;
                const T *q = static_cast<const T *>(a.q) + (p.first + row) * a.q_tok +
                             (static_cast<int64_t>(head) * share + hh) * a.q_head;
                float v[HV][16];
                float top = 0.0f;
                bool finite = true;
#pragma unroll
                for (int h = 0; h < HV; ++h) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint4 raw[1] = {make_uint4(0, 0, 0, 0)};
                        if (on) raw[0] = __ldg(reinterpret_cast<const uint4 *>(q + 64 * h + 16 * t) + i);
                        float x[8];
                        Kv4In<T>::unpack(raw, x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            v[h][8 * i + j] = x[j];
                            top = fmaxf(top, fabsf(x[j]));
                            finite &= fabsf(x[j]) <= 3.402823466e38f;
                        }
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    finite &= __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, o) != 0;
                }
                if (!finite && warp == 0 && t == 0) atomicOr(&s_nan, 1u << (nb * 8 + g));
                // 2^k brings the largest into [2^14, 2^15)
                int k = top > 0.0f && finite ? 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127) : 0;
                k = min(k, 120);
                const float up = finite ? __uint_as_float(static_cast<uint32_t>(127 + k) << 23) : 0.0f;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                const float zs = a.scale * (MODS != kPlain ? 1.0f : 1.4426950408889634f) * down;
                fc[nb] = zs * 16777216.0f;
#pragma unroll
                for (int r = 0; r < GR; ++r) sc[nb][r] = 0.0f;
#pragma unroll
                for (int h = 0; h < HV; ++h) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[h][j] = finite ? v[h][j] * up : 0.0f;
                        sc[nb][h % GR] += v[h][j];
                    }
                }
#pragma unroll
                for (int r = 0; r < GR; ++r) {
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) sc[nb][r] += __shfl_xor_sync(0xffffffffu, sc[nb][r], o);
                    sc[nb][r] *= zs;
                }
                // step (h, word w, half j) of the product: elements (n, n + 4) and, 2^4 up, (n + 1, n + 5), n = 2 j
#pragma unroll
                for (int h = 0; h < HV; ++h) {
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        const int n = (st >> 1) * 8 + (st & 1) * 2;
                        const uint32_t q0 = pack_f16(v[h][n], v[h][n + 4]);
                        const uint32_t q1 = pack_f16(v[h][n + 1] * 0.0625f, v[h][n + 5] * 0.0625f);
                        if constexpr (NB == 1) {
                            qf[(h * 4 + st) * 2] = q0;
                            qf[(h * 4 + st) * 2 + 1] = q1;
                        } else if (warp == nb) {
                            *reinterpret_cast<uint2 *>(smem + C::OFF_Q + (((h * 4 + st) * NB + nb) * 32 + lane) * 8) =
                                make_uint2(q0, q1);
                        }
                    }
                }
            }
            // factors of the columns that this lane holds scores of: 2 t and 2 t + 1
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int from = (2 * t + cc) * 4;
                    f[nb][cc] = __shfl_sync(0xffffffffu, fc[nb], from);
#pragma unroll
                    for (int r = 0; r < GR; ++r) sq[nb][cc][r] = __shfl_sync(0xffffffffu, sc[nb][r], from);
                    const int c = nb * 8 + 2 * t + cc;
                    pos[nb][cc] = c < ncols ? p.pos0 + (col0 + c) / share : -1;
                    slope[nb][cc] = 0.0f;
                    if (MODS != kPlain && a.slopes != nullptr && c < ncols)
                        slope[nb][cc] = __ldg(a.slopes + head * share + (col0 + c) % share);
                }
            }
        }
        if (NB > 1) __syncthreads();
        // positions that every column sees
        const int row_lo = col0 / share, row_hi = (col0 + ncols - 1) / share;
        const int all_hi = p.pos0 + row_lo;  // up to the first row's position
        const int all_lo = a.window > 0 ? p.pos0 + row_hi - a.window + 1 : 0;

        float step_ref = 0.0f;  // about the largest value step so far
        float o[NB][HV][4][4], m[NB][2], l[NB][2][GR], mo[NB][2][GR];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int h = 0; h < HV; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[nb][h][i][j] = 0.0f;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                m[nb][cc] = kNoMax;
#pragma unroll
                for (int r = 0; r < GR; ++r) l[nb][cc][r] = mo[nb][cc][r] = 0.0f;
            }
        }

#pragma unroll 1
        for (int i = 0; i < mytiles && !dead; ++i) {
            const int stage = taken % C::S;
            bool ok = mbar_wait_timed(bars + 8 * stage, (taken / C::S) & 1, status, SITE_KV4_ATTENTION);
            if (!__all_sync(0xffffffffu, ok)) {
                dead = true;
                break;
            }
            const uint32_t kc = ring + stage * C::STAGE, kp = kc + C::CODES, vc = kp + C::PARS, vp = vc + C::CODES;
            const int tok0 = (tile0 + warp + i * kW) * kTile;
            const uint32_t bad = (bad_bits >> (2 * stage)) & 3u;
            const bool edge = tok0 + kTile - 1 > all_hi || tok0 < all_lo || bad != 0;

            // ---- scores: z[block][nb][row half * 2 + column], in powers of two
            float z[2][NB][4];
            float sv[2][2][GR], mv[2][2][GR], ri[2][2][GR];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float s[GR][NB][4];
#pragma unroll
                for (int r = 0; r < GR; ++r)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[r][nb][j] = 0.0f;
#pragma unroll
                for (int h = 0; h < HV; ++h) {
                    const uint2 w0 = lds64(kc + (16 * k + gt) * C::ROW + 32 * h + 8 * t);
                    const uint2 w1 = lds64(kc + (16 * k + gt + 8) * C::ROW + 32 * h + 8 * t);
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        const uint32_t x0 = (st < 2 ? w0.x : w0.y) >> (8 * (st & 1));
                        const uint32_t x1 = (st < 2 ? w1.x : w1.y) >> (8 * (st & 1));
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            uint32_t b0, b1;
                            if constexpr (NB == 1) {
                                b0 = qf[(h * 4 + st) * 2];
                                b1 = qf[(h * 4 + st) * 2 + 1];
                            } else {
                                const uint2 v = lds64(smem_u32(smem) + C::OFF_Q + (((h * 4 + st) * NB + nb) * 32 + lane) * 8);
                                b0 = v.x;
                                b1 = v.y;
                            }
                            mma_f16(s[h % GR][nb], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u,
                                    x1 & 0x00f000f0u, b0, b1);
                        }
                    }
                }
#pragma unroll
                for (int rh = 0; rh < 2; ++rh) {
                    const int tok = 16 * k + gt + 8 * rh;
                    float ks[GR], km[GR];
#pragma unroll
                    for (int r = 0; r < GR; ++r) {
                        const float2 x = unpack_f16(lds32(kp + tok * C::PAR + 4 * r));
                        ks[r] = x.x;
                        km[r] = x.y;
                        const float2 y = unpack_f16(lds32(vp + tok * C::PAR + 4 * r));
                        sv[k][rh][r] = y.x;
                        mv[k][rh][r] = fmaf(8.0f, y.x, y.y);  // (codes are taken from 8)
                        ri[k][rh][r] = rcp(y.x);
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            float x, y = 0.0f;
                            if constexpr (GR == 1) {
                                x = s[0][nb][2 * rh + cc] * ks[0];
                                y = km[0] * sq[nb][cc][0];
                            } else {
                                x = fmaf(s[1][nb][2 * rh + cc], ks[1], s[0][nb][2 * rh + cc] * ks[0]);
                                y = fmaf(km[1], sq[nb][cc][1], km[0] * sq[nb][cc][0]);
                            }
                            x = fmaf(x, f[nb][cc], y);
                            if constexpr (MODS != kPlain) {
                                if (a.softcap > 0.0f) {
                                    const float v = x * a.cap_rate;
                                    x = fmaf(-2.0f * a.softcap, rcp(ex2(v) + 1.0f), a.softcap);
                                    if (MODS == kFarMods && fabsf(v) < kSeries)
                                        x = cap_series(v, a.softcap * (0.5f / 1.4426950408889634f));
                                }
                                x = fmaf(slope[nb][cc], static_cast<float>(tok0 + tok - pos[nb][cc]), x);
                                x *= 1.4426950408889634f;
                            }
                            z[k][nb][2 * rh + cc] = x;
                        }
                    }
                }
            }
            if (edge) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const bool gone = (bad >> k) & 1u;
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh) {
                        const int tok = 16 * k + gt + 8 * rh;
                        if (gone || tok0 + tok > p.hi || tok0 + tok < p.lo) {  // a place that holds nothing for these rows
#pragma unroll
                            for (int r = 0; r < GR; ++r) {
                                sv[k][rh][r] = fmaxf(step_ref, 5.9604644775390625e-08f);
                                mv[k][rh][r] = 0.0f;
                                ri[k][rh][r] = rcp(sv[k][rh][r]);
                            }
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                            for (int cc = 0; cc < 2; ++cc) {
                                const int d = tok0 + tok - pos[nb][cc];
                                if (gone) z[k][nb][2 * rh + cc] = __int_as_float(0x7fffffff);
                                if (d > 0 || (a.window > 0 && d <= -a.window)) z[k][nb][2 * rh + cc] = -INFINITY;
                            }
                        }
                    }
                }
            }

            // ---- tokens that need care: values that are not finite count only for the rows that see them, and a step
            // far below the others' may lose p * s_v to fp16's underflow, so such a token's weight goes into the
            // sums apart (bits 2 (2 k + rh) + group)
            uint32_t direct = 0, spoilt = 0;
            float lv[2][2];  // log2 of the step, for the maximum
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int rh = 0; rh < 2; ++rh) {
                    float x = sv[k][rh][0];
                    if constexpr (GR == 2) x = fmaxf(x, sv[k][rh][1]);
                    lv[k][rh] = lg2(x);
                }
            float lo = INFINITY, hi = 0.0f, odd = 0.0f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int rh = 0; rh < 2; ++rh)
#pragma unroll
                    for (int r = 0; r < GR; ++r) {
                        lo = fminf(lo, sv[k][rh][r]);
                        hi = fmaxf(hi, sv[k][rh][r]);
                        odd = fmaf(0.0f, sv[k][rh][r], fmaf(0.0f, mv[k][rh][r], odd));
                    }
            const bool care =
                __any_sync(0xffffffffu, !(lo > step_ref * kFarStep && hi <= 2.0f * step_ref && odd == 0.0f));
            if (care) {
                hi = step_ref;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh)
#pragma unroll
                        for (int r = 0; r < GR; ++r) {
                            // (mv is m + 8 s: up to 9 x 65504 of what is stored as finite)
                            if (!(fabsf(sv[k][rh][r]) <= 65504.0f && fabsf(mv[k][rh][r]) <= 9.0f * 65504.0f)) {
                                sv[k][rh][r] = mv[k][rh][r] = 0.0f;
                                spoilt |= 1u << (4 * k + 2 * rh + r);
                            }
                            hi = fmaxf(hi, sv[k][rh][r]);
                        }
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                step_ref = hi;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh) {
                        float x = 5.9604644775390625e-08f;
#pragma unroll
                        for (int r = 0; r < GR; ++r) {
                            x = fmaxf(x, sv[k][rh][r]);
                            if (sv[k][rh][r] <= step_ref * kFarStep) {
                                direct |= 1u << (4 * k + 2 * rh + r);
                                ri[k][rh][r] = 0.0f;  // (its share of the sums is added below)
                            }
                        }
                        lv[k][rh] = lg2(x);
                    }
            }

            // ---- running maximum of z + log2(step)
            bool rise = false;
            float top[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    top[nb][cc] = fmaxf(fmaxf(z[0][nb][cc] + lv[0][0], z[0][nb][2 + cc] + lv[0][1]),
                                        fmaxf(z[1][nb][cc] + lv[1][0], z[1][nb][2 + cc] + lv[1][1]));
                    rise |= top[nb][cc] > m[nb][cc] + kSlack;
                }
            }
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        float x = top[nb][cc];
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
                        const float now = fmaxf(m[nb][cc], x);
                        const float keep = ex2(m[nb][cc] - now);
                        m[nb][cc] = now;
#pragma unroll
                        for (int r = 0; r < GR; ++r) {
                            l[nb][cc][r] *= keep;
                            mo[nb][cc][r] *= keep;
                        }
#pragma unroll
                        for (int h = 0; h < HV; ++h)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                o[nb][h][j][cc] *= keep;
                                o[nb][h][j][2 + cc] *= keep;
                            }
                    }
                }
            }

            // ---- weights, and the products with the values
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t pb[NB][GR][2];  // weight * step, column g, tokens 2 t, 2 t + 1 (+ 8)
#pragma unroll
                for (int rh = 0; rh < 2; ++rh) {
                    float zr[GR];
#pragma unroll
                    for (int r = 0; r < GR; ++r) zr[r] = mv[k][rh][r] * ri[k][rh][r];
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const float e0 = ex2(z[k][nb][2 * rh] - (m[nb][0] - kLift));
                        const float e1 = ex2(z[k][nb][2 * rh + 1] - (m[nb][1] - kLift));
#pragma unroll
                        for (int r = 0; r < GR; ++r) {
                            const uint32_t ph = pack_f16(e0 * sv[k][rh][r], e1 * sv[k][rh][r]);
                            const float2 w = unpack_f16(ph);
                            l[nb][0][r] = fmaf(w.x, ri[k][rh][r], l[nb][0][r]);
                            l[nb][1][r] = fmaf(w.y, ri[k][rh][r], l[nb][1][r]);
                            mo[nb][0][r] = fmaf(w.x, zr[r], mo[nb][0][r]);
                            mo[nb][1][r] = fmaf(w.y, zr[r], mo[nb][1][r]);
                            pb[nb][r][rh] = transpose8x8(ph);
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < HV; ++h) {
                    const uint32_t at = vc + (16 * k + 2 * t) * C::ROW + 32 * h + 4 * g;
                    const uint32_t first = at + (t >> 1) * C::ROW, second = at + (1 - (t >> 1)) * C::ROW;  // as gt has them
                    const uint32_t a0 = lds32(first), a1 = lds32(second);
                    const uint32_t b0 = lds32(first + 8 * C::ROW), b1 = lds32(second + 8 * C::ROW);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {  // dims 8 g + 2 w (rows g) and + 1 (rows g + 8)
                        const uint32_t x = __byte_perm(a0, a1, 0x0400 + 0x0101 * w);
                        const uint32_t y = __byte_perm(b0, b1, 0x0400 + 0x0101 * w);
                        const uint32_t x0 = from_middle(x & 0x000f000fu, 0x00080008u), x1 = from_middle(x & 0x00f000f0u, 0x00800080u);
                        const uint32_t y0 = from_middle(y & 0x000f000fu, 0x00080008u), y1 = from_middle(y & 0x00f000f0u, 0x00800080u);
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            mma_f16(o[nb][h][w], x0, x1, y0, y1, pb[nb][h % GR][0], pb[nb][h % GR][1]);
                    }
                }
            }
            if (care) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh)
#pragma unroll
                        for (int r = 0; r < GR; ++r) {
                            if (!((direct >> (4 * k + 2 * rh + r)) & 1u)) continue;
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int cc = 0; cc < 2; ++cc) {
                                    const float x = z[k][nb][2 * rh + cc], e = ex2(x - (m[nb][cc] - kLift));
                                    // (rounded as in the products, for a row to which the step is not small at all;
                                    // as it is below fp16's normal numbers)
                                    const float ps = unpack_f16(pack_f16(e * sv[k][rh][r], 0.0f)).x;
                                    const float w = ps >= 6.103515625e-05f ? ps * rcp(sv[k][rh][r]) : e;
                                    l[nb][cc][r] += w;
                                    mo[nb][cc][r] = fmaf(w, mv[k][rh][r], mo[nb][cc][r]);
                                    // NaN for the rows that see it
                                    if (((spoilt >> (4 * k + 2 * rh + r)) & 1u) && x > -INFINITY)
                                        mo[nb][cc][r] = __int_as_float(0x7fffffff);
                                }
                        }
            }
            ++taken;
            __syncwarp();
            if (next < mytiles) {
                if ((next & 31) == 0) look_up(next);
                issue(next);
                ++next;
            }
        }

        // ---- the warps' results meet in the ring (every copy has landed)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) {
#pragma unroll
                    for (int r = 0; r < GR; ++r) {
                        l[nb][cc][r] += __shfl_xor_sync(0xffffffffu, l[nb][cc][r], s);
                        mo[nb][cc][r] += __shfl_xor_sync(0xffffffffu, mo[nb][cc][r], s);
                    }
                }
            }
        }
        if (dead) {
            for (; taken < issued; ++taken) mbar_drain(bars + 8 * (taken % C::S), (taken / C::S) & 1, kWaitLimitNs);
        }
        __syncthreads();
        {
            float *res = reinterpret_cast<float *>(smem + warp * C::RES);
            float *aux = res + C::COLS * C::CSTR;  // [COLS] maximum, [COLS] sum, [GR][COLS] divisor
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int cc = 0; cc < 2; ++cc) {
                    const int c = nb * 8 + 2 * t + cc;
#pragma unroll
                    for (int h = 0; h < HV; ++h) {
                        float v[8];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            v[2 * w] = fmaf(o[nb][h][w][cc], 16777216.0f, mo[nb][cc][h % GR]);
                            v[2 * w + 1] = fmaf(o[nb][h][w][2 + cc], 1048576.0f, mo[nb][cc][h % GR]);
                        }
                        float4 *to = reinterpret_cast<float4 *>(res + c * C::CSTR + 64 * h + 8 * g);
                        to[0] = make_float4(v[0], v[1], v[2], v[3]);
                        to[1] = make_float4(v[4], v[5], v[6], v[7]);
                    }
                    if (g == 0) {
                        aux[c] = m[nb][cc];
                        aux[C::COLS + c] = l[nb][cc][0];
#pragma unroll
                        for (int r = 0; r < GR; ++r) aux[(2 + r) * C::COLS + c] = l[nb][cc][r];
                    }
                }
            }
        }
        __syncthreads();
        const bool whole = u == item_begin && seg_end == item_end;
        // slot 2 cta + 1 for an item that begins here, 2 cta for one that began earlier
        float *slot = ws.slots + (2 * cta + (u == item_begin ? 1 : 0)) * C::SLOT;
        if (!whole && u == item_begin && threadIdx.x == 0) {
            const int64_t last = (item_end * ctas - 1) / total;  // CTA that holds the item's last unit
            ws.desc[cta] = {p.first, col0, ncols, head, static_cast<int>(last - cta) + 1};
        }
        for (int e = threadIdx.x; e < ncols * (D / 4); e += kThreads) {
            const int c = e / (D / 4), d = (e % (D / 4)) * 4;
            float top = kNoMax;
#pragma unroll
            for (int w = 0; w < kW; ++w)
                top = fmaxf(top, *(reinterpret_cast<const float *>(smem + w * C::RES) + C::COLS * C::CSTR + c));
            float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float den = 0.0f, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float *res = reinterpret_cast<const float *>(smem + w * C::RES);
                const float *aux = res + C::COLS * C::CSTR;
                const float k = ex2(aux[c] - top);
                const float4 v = *reinterpret_cast<const float4 *>(res + c * C::CSTR + d);
                num.x = fmaf(v.x, k, num.x);
                num.y = fmaf(v.y, k, num.y);
                num.z = fmaf(v.z, k, num.z);
                num.w = fmaf(v.w, k, num.w);
                sum = fmaf(aux[C::COLS + c], k, sum);
                den = fmaf(aux[(2 + d / C::G) * C::COLS + c], k, den);
            }
            const int row = (col0 + c) / share, hh = (col0 + c) - row * share;
            const int at = p.pos0 + row;
            if (at >= 0 && (((s_nan >> c) & 1u) || at >= cap)) {
                if (at >= cap) report(status, BQ_ERR_INVALID_ARG, SITE_KV4_ATTENTION);
                den = sum = __int_as_float(0x7fffffff);
            }
            if (whole) {
                const int64_t to = (p.first + row) * a.q_heads + static_cast<int64_t>(head) * share + hh;
                const float inv = den == 0.0f ? 0.0f : __fdividef(1.0f, den);
                *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + to * D + d) =
                    make_uint2(pack2(num.x * inv, num.y * inv, T()), pack2(num.z * inv, num.w * inv, T()));
                if (a.lse != nullptr && d == 0)
                    a.lse[to] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
            } else {
                float *s = slot + c * (D + 4);
                *reinterpret_cast<float4 *>(s + d) = num;
                if (d % C::G == 0) {
                    if (d == 0) {
                        s[D] = top;
                        s[D + 1] = sum;
                    }
                    s[D + 2 + d / C::G] = den;
                }
            }
        }
        fence_proxy_async_smem();  // the ring is written by copies again
        __syncthreads();
        u = seg_end;
    }
}

template <typename C, Mods MODS, typename T>
cudaError_t launch_decode(const Kv4AttnArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto kern = kv4_decode_kernel<C, MODS, T>;
    static SmemOptIn opt_in;
    cudaError_t e = smem_opt_in(opt_in, dev, reinterpret_cast<const void *>(kern), static_cast<size_t>(C::SMEM));
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(std::min(dev.num_sms, kKv4MaxSms) * C::CTAS);
    const Kv4Ws ws = kv4_workspace(a.workspace);
    kern<<<grid, kThreads, C::SMEM, s>>>(a, ws, dev.status);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kv4_launch_join<C::D, C::G, C::COLS, T>(a, ws, grid, s);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int64_t total, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
    // two slots for each CTA: three per SM with 8 columns, two with 24 (of a block), or, for many rows, one with 256
    const int64_t cols = total * (q_heads / kv_heads) > kKv4FewColumns ? 256 : 48;
    return kKv4MaxCtas * sizeof(Kv4Partial) + 2 * kKv4MaxSms * static_cast<size_t>(cols * (head_dim + 4)) * 4;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto by_cols = [&](auto tag, auto shape) {
        using T = decltype(tag);
        constexpr int D = decltype(shape)::D, G = decltype(shape)::G;
        const int64_t cols = static_cast<int64_t>(a.max_q) * (a.q_heads / a.pool.kv_heads);
        const Mods mods = mods_of(a);
        auto go = [&](auto c) {
            using C = decltype(c);
            if (mods == kPlain) return launch_decode<C, kPlain, T>(a, s, dev);
            return mods == kNearMods ? launch_decode<C, kNearMods, T>(a, s, dev) : launch_decode<C, kFarMods, T>(a, s, dev);
        };
        if (cols > kKv4FewColumns) return launch_kv4_prefill(a, s, dev);
        if (cols <= 8) return go(Shape<D, G, 1>());
        if (cols <= 16) return go(Shape<D, G, 2>());
        return go(Shape<D, G, 3>());
    };
    auto by_shape = [&](auto tag) {
        if (a.pool.head_dim == 64) return by_cols(tag, Shape<64, 64, 1>());
        return a.pool.group_size == 64 ? by_cols(tag, Shape<128, 64, 1>()) : by_cols(tag, Shape<128, 128, 1>());
    };
    return a.dtype == BQ_F16 ? by_shape(__half()) : by_shape(__nv_bfloat16());
}

}  // namespace bq

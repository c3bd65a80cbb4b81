// Attention of many query rows over the 4-bit key/value cache (prompts, and
// chunks of them): bound by the tensor cores, and by the exponentials.
//
// Arithmetic.  As with few rows (kv4_attention.cu) the steps and minima stay
// outside the products, whose operands are exact:
//
//   S = Q C_k^T         Q: rows scaled by powers of two into fp16, C_k: key codes
//   z = f (S s_k + q' m_k)           f, q' = sum(q) per row, s_k, m_k per token
//   w = fp16(2^(z - M + 7) mu)       value step s_v = mu 2^e0 (see below)
//   [O | L] += w [c_v - 8 | 1/mu | (m_v + 8 s_v)/mu 2^-e1]
//
// so that the output is (2^e0 O + 2^e1 L_m) / L_1: the divisor and the middles'
// term are sums of the same rounded weights w as the codes' term, and the
// rounding of a weight (2^-11 at most) changes how much a token counts, never
// what it stands for.  (fp16 is the type of the instruction; two products for
// one would take fp16 results from a relative error of 0.00023 to 0.00021, bf16
// results from 0.0017 nowhere.  Weights below 2^-12 of a row's largest may keep fewer bits: they
// are off by 2^-23 of that one at most.)  1/mu, which the divisor's sum takes
// as an operand of the same product, is a pair of fp16 (22 bits, a relative
// error of 2^-23 beside the sum's own); so is a middle, whose
// second half is held times 2^14, so that one far below the largest keeps its
// bits (to 2^-41 of the largest; 2^-27 without that, which a row that sees only
// small ones would notice).  The
// values' codes are taken from the middle because the tensor core's additions
// round toward zero: sums of 0..15 drift with every step, and what is left of
// them after the minima's term is small (0.0029 against 0.0017 relative error
// over 9000 tokens, the latter being bf16's own; now 0.0017).  It is paid for
// with time: 2048 rows after 8192 took 484 us before, 503 us after it.
// The exponents e0, e1 follow the largest step and middle so far, and the sums
// are rescaled when they move; where steps differ by more than 2^9, part of a
// step's exponent goes from the weight into the codes ((c_v - 8) 2^k).  A code
// of a key is an fp16 subnormal masked out of its word (c 2^-24 or, the upper
// half of a byte, 16 c 2^-24: Q takes the 16), of a value an fp16 1024 + c
// brought to c - 8 by one fused multiply-add; both are exact.
//
// Roles of the 768 threads of a CTA (one per SM), which takes 256 columns
// (pairs of query row and head of one key head) as two tiles of 128:
//   warps 0-7, 8-15  softmax of a tile of rows: S from TMEM as fragments of 16
//                    rows, w back to TMEM in its place, as the next A operand
//   warps 16-18      values: one (token, group) per thread from 4 bits to fp16
//   warps 19-21      the same for keys
//   warp 22          issues the products (tcgen05.mma kind::f16)
//   warp 23          plans, and copies pages (bulk copies)
// A tile of tokens is unpacked once for both tiles of rows, and the products
// of one tile run while the other's softmax does.
//
// Work.  The (sequence, head, 256 columns) items of the batch are one list
// whose cost (about the tokens that an item reads) has a closed form; the CTAs
// take equal shares of it, cutting items where a share ends, and the joining
// kernel adds up what was cut.
//
// What bounds it (2048 rows of 32 heads after 8192 tokens, 8 key heads of 128:
// 495 us, 625 TFLOP/s, tensor pipe active 31%): a tile's softmax (about 2700
// cycles while the other tile's runs too) and its two products (880 cycles, and
// 900 to hand over) follow one another, since its weights take the place of its
// scores; issue slots are 45% full, the exponentials' unit 29%, shared memory
// 45%.  Measured against this form: rows by thread, which reads every token's
// parameters in every thread, 779 us (shared memory); 8 softmax warps 634 us;
// weights in a place of their own so that the next scores are computed
// meanwhile, 80 tokens a tile, 634 to 773 us (the warps then run five codes at
// once and wait for instructions); a softmax loop of 16 tokens, 592 us.
//
// Every wait is bounded; if one runs out the kernel records BQ_ERR_TIMEOUT,
// lets its copies and products end (bounded again) and finishes.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4_attention.cuh"

namespace bq {
namespace {

constexpr int kRows = 128;     // of a tile
constexpr int kCols = 256;     // columns of an item
constexpr int kPThreads = 768;
constexpr int kLaunchRegs = 80, kSoftmaxRegs = 88, kOtherRegs = 64;  // registers: 512 x 88 + 256 x 64 = 768 x 80
constexpr int kRing = 3;       // raw stages
constexpr float kRest = 16384.0f;  // the second half of a middle is held times this
constexpr float kRise = 7.0f;  // the running maximum is raised when passed by more
constexpr int kOverhead = 192; // cost of starting an item, in tokens (8 ragged prompts: 236, 222, 228, 249 us at 96, 192, 400, 800)

template <int D_, int G_>
struct PShape {
    static constexpr int D = D_, G = G_, GR = D / G;
    static constexpr int TOK = GR == 1 ? 96 : 48;  // tokens of a tile: 96 threads unpack (token, group) pairs
    static constexpr int ROW = D / 2, PAR = 4 * GR;
    static constexpr int RAW = TOK * 2 * (ROW + PAR);
    static constexpr int OC = D + 16 * GR;         // columns of [O | L]
    static constexpr int QB = kRows * D * 2;       // bytes of a tile of Q
    static constexpr int KB = TOK * D * 2;
    static constexpr int VB = TOK * OC * 2;
    static constexpr int PB = TOK * GR * 3 * 4;    // s_k, m_k, mu
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * QB;
    static constexpr int OFF_V = OFF_K + 2 * KB;
    static constexpr int OFF_RAW = OFF_V + 2 * VB;
    static constexpr int OFF_P = OFF_RAW + kRing * RAW;
    static constexpr int SMEM = OFF_P + 2 * PB;
    static_assert(SMEM <= 231000, "shared memory of a CTA");
    // TMEM columns: S (and w in its place), then [O | L], of each tile
    static constexpr int SC = 96;
    static constexpr int T_O = 2 * SC;
    static_assert(T_O + 2 * OC <= 512, "TMEM");
};

// Polls a barrier up to `tries` times, four instructions each.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, uint32_t tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 c;\n\tmov.u32 c, %3;\n\t"
        "POLL:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "sub.u32 c, c, 1;\n\tsetp.ne.u32 q, c, 0;\n\t@q bra POLL;\n\t"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    return ok != 0;
}
// Bounded wait of a role.  The warps that work share its issue slots (longer
// polls were most of what the kernel issued), so the clock and the abort flag
// are looked at once in many polls.
__device__ __forceinline__ bool wait_role(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status,
                                          uint32_t site) {
    if (mbar_poll(bar, parity, 4096)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_poll(bar, parity, 4096)) {
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            report(status, BQ_ERR_TIMEOUT, site);
            *abort = 1;
            return false;
        }
    }
    return true;
}
// A row of the tiles, for the lanes that hold its scores; then what they found.
struct RowInfo {
    float f, sq[2], slope;
    int pos, finite;
    float m, sum;
};

// What a tile of tokens tells the softmax beside its parameters.
struct TileInfo {
    int e0, e1;  // O holds sums times 2^-e0, L the middles' times 2^-e1
    int odd;     // holds values that are not finite
};

__device__ __forceinline__ uint64_t pack64(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack64(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float pow2i(int e) {  // 2^e, 0 below 2^-126
    return e < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(min(e, 127) + 127) << 23);
}
__device__ __forceinline__ int exp_of(float x) {  // of a finite x; 2^-24 and less give -24
    return max(static_cast<int>((__float_as_uint(x) >> 23) & 255u) - 127, -24);
}
__device__ __forceinline__ uint64_t lds64x(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32f(uint32_t a, float x) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}

// ---- tensor cores
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Operand without a swizzle: blocks of 8 x 16 bytes, contiguous.  `lbo`: bytes
// to the next block along K, `sbo`: along M or N (the same for both majors).
__device__ __forceinline__ uint64_t desc_plain(uint32_t a, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((a >> 4) & 0x3fffu) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {  // M = 128, fp16 x fp16 -> fp32
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(kRows >> 4) << 24);
}
// 16 lanes x 8 N columns as the fragments of a matrix product: of each 8
// columns, lane 4 g + t holds columns 2 t, 2 t + 1 of rows g and g + 8.
template <int N>
__device__ __forceinline__ void tmem_ld_rows(uint32_t a, uint32_t *r);
template <>
__device__ __forceinline__ void tmem_ld_rows<2>(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a)
                 : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_rows<4>(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(a)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st_rows(uint32_t a, const uint32_t *r);
template <>
__device__ __forceinline__ void tmem_st_rows<2>(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 lanes x 4 N columns: of each 4, lane 4 g + t holds column t of rows g, g + 8.
template <int N>
__device__ __forceinline__ void tmem_st_half(uint32_t a, const uint32_t *r);
template <>
__device__ __forceinline__ void tmem_st_half<2>(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
template <>
__device__ __forceinline__ void tmem_st_half<4>(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_half1(uint32_t a, uint32_t (&r)[2]) {
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x1.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void tmem_st_half1(uint32_t a, const uint32_t (&r)[2]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1, %2};" ::"r"(a), "r"(r[0]), "r"(r[1]) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ---- the list of work
// Cost of the items (blocks of kCols columns) of one head of a sequence:
// kOverhead plus the tokens up to a block's last row, at least 1, at most what
// the window leaves: an arithmetic sequence with flat ends.
struct SeqWork {
    int64_t first;  // first row
    int64_t a0, step, cmax;
    int64_t flat0, flat1;  // blocks that cost the least, blocks up to where all cost the most
    int64_t blocks;
    int64_t cost;  // of one head
    int rows, pos0, cap;
};
__device__ __forceinline__ int64_t cost_upto(const SeqWork &w, int64_t n) {
    const int64_t i1 = min(w.flat0, n), i2 = max(i1, min(w.flat1, n));
    return n * kOverhead + i1 + (i2 - i1) * w.a0 + w.step * ((i1 + i2 - 1) * (i2 - i1) / 2) + (n - i2) * w.cmax;
}
__device__ __forceinline__ SeqWork seq_work(const Kv4AttnArgs &a, int b, int share) {
    SeqWork w;
    int n;
    kv4_rows(a.seqs, b, w.first, n);
    w.rows = static_cast<int>(min(static_cast<int64_t>(min(n, a.max_q)), a.total - w.first));
    if (n <= 0 || w.rows < 0 || w.first < 0) w.rows = 0;
    w.pos0 = kv4_first_position(a.seqs, b, n);
    w.cap = kv4_capacity(a.pool);
    w.step = max(kCols / share, 1);
    w.a0 = w.pos0 + w.step;
    w.cmax = a.window > 0 ? a.window + w.step : int64_t(1) << 40;
    w.blocks = (static_cast<int64_t>(w.rows) * share + kCols - 1) / kCols;
    // (step, share and the positions have 32 bits, and so have these quotients)
    w.flat0 = w.a0 >= 1 ? 0 : static_cast<uint32_t>(w.step - w.a0) / static_cast<uint32_t>(w.step);
    w.flat1 = w.a0 > w.cmax ? 0
              : a.window > 0 ? static_cast<int64_t>(static_cast<uint32_t>(w.cmax - w.a0) / static_cast<uint32_t>(w.step)) + 1
                             : w.blocks;
    w.cost = cost_upto(w, w.blocks);
    return w;
}

// The parts of items that make up a CTA's share, one after the other: the
// copying warp works them out and hands them to the others.
struct Segment {
    int b, head, col0, ncols;
    int start, hi;     // first token of the part, last token that is read (-1: none)
    int tiles;         // of this part; 0 behind the last part
    int pos0, cap;
    int64_t first;
    bool begins, whole;
};
struct Walk {
    int64_t at, stop, seq_begin;
    int b;
};
template <int TOK>
__device__ __forceinline__ bool next_segment(const Kv4AttnArgs &a, int share, int align, Walk &w, Segment &s, int64_t &end) {
    if (w.at >= w.stop) return false;
    SeqWork q = seq_work(a, w.b, share);
    while (w.at >= w.seq_begin + q.cost * a.pool.kv_heads) {
        w.seq_begin += q.cost * a.pool.kv_heads;
        q = seq_work(a, ++w.b, share);
    }
    const int64_t off = w.at - w.seq_begin;
    const int64_t head = off / q.cost, rem = off - head * q.cost;
    int64_t lo = 0, hi = q.blocks - 1;  // the last block whose cost begins at or below rem
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cost_upto(q, mid) <= rem)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int64_t begin = w.seq_begin + head * q.cost + cost_upto(q, lo);
    end = w.seq_begin + head * q.cost + cost_upto(q, lo + 1);
    s.b = w.b;
    s.head = static_cast<int>(head);
    s.col0 = static_cast<int>(lo) * kCols;
    s.ncols = static_cast<int>(min(int64_t(kCols), static_cast<int64_t>(q.rows) * share - s.col0));
    s.first = q.first;
    s.pos0 = q.pos0;
    s.cap = q.cap;
    const int r0 = s.col0 / share, r1 = (s.col0 + s.ncols - 1) / share;
    const int64_t from = a.window > 0 ? max(static_cast<int64_t>(q.pos0) + r0 - a.window + 1, int64_t(0)) : 0;
    s.start = static_cast<int>(from) & ~(align - 1);
    s.hi = static_cast<int>(min(static_cast<int64_t>(q.pos0) + r1, static_cast<int64_t>(q.cap) - 1));
    int tiles = 1;
    if (s.hi < static_cast<int>(from)) {
        s.hi = -1;  // nothing is seen, by any row
        s.start = 0;
    } else {
        tiles = (s.hi - s.start) / TOK + 1;
    }
    const int64_t stop = min(end, w.stop), cost = end - begin;
    const int tile0 = static_cast<int>((w.at - begin) * tiles / cost);
    s.tiles = static_cast<int>(stop == end ? tiles : (stop - begin) * tiles / cost) - tile0;
    s.start += tile0 * TOK;
    s.begins = w.at == begin;
    s.whole = s.begins && stop == end;
    w.at = stop;
    return true;
}

enum Bar {
    RAW_FULL = 0,
    RAW_EMPTY = RAW_FULL + kRing,
    KV_FULL = RAW_EMPTY + kRing,
    KV_EMPTY = KV_FULL + 2,
    S_FULL = KV_EMPTY + 2,
    P_FULL = S_FULL + 2,
    Q_FULL = P_FULL + 2,
    O_FULL = Q_FULL + 2,
    PAIR = O_FULL + 2,  // the two warps of 32 rows
    SEG_FULL = PAIR + 8,
    SEG_EMPTY = SEG_FULL + 2,
    DRAIN = SEG_EMPTY + 2,
    kBars = DRAIN + 1
};

template <typename C, Mods MODS, typename T>
__global__ void __launch_bounds__(kPThreads, 1) kv4_prefill_kernel(const Kv4AttnArgs a, const Kv4Ws ws, uint32_t *status) {
    constexpr int D = C::D, GR = C::GR, G = C::G, TOK = C::TOK, SC = C::SC, OC = C::OC;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_bars[kBars];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ TileInfo s_info[2];
    __shared__ uint32_t s_bad[kRing];
    __shared__ int64_t s_sum[kPThreads / 32];
    __shared__ int64_t s_before;
    __shared__ int s_b;
    __shared__ RowInfo s_rows[kCols];
    __shared__ Segment s_seg[2];
    pdl_launch_dependents();  // the joining kernel waits for this grid before it reads
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_u32(smem);
    uint32_t bars = smem_u32(s_bars);
    asm volatile("" : "+r"(bars));  // (kept, not worked out again in every poll)
    const int share = a.q_heads / a.pool.kv_heads, H = a.pool.kv_heads, page_log2 = a.pool.page_log2;
    auto bar = [&](int i) { return bars + 8 * i; };

    // ---- this CTA's share
    const int64_t per = (a.seqs.batch + kPThreads - 1) / kPThreads;
    const int64_t b_lo = min(per * threadIdx.x, static_cast<int64_t>(a.seqs.batch));
    const int64_t b_hi = min(b_lo + per, static_cast<int64_t>(a.seqs.batch));
    int64_t mine = 0;
    for (int64_t b = b_lo; b < b_hi; ++b) mine += seq_work(a, static_cast<int>(b), share).cost * H;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (threadIdx.x == 0) {
        s_abort = 0;
        ws.desc[blockIdx.x].count = 0;
    }
    __syncthreads();
    int64_t before = incl - mine, total = 0;
    for (int w = 0; w < kPThreads / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), (total + 2 * kOverhead - 1) / (2 * kOverhead));
    const int64_t cta = blockIdx.x;
    if (cta >= ctas) return;
    Walk walk;
    walk.at = total * cta / ctas;
    walk.stop = total * (cta + 1) / ctas;
    if (walk.at >= before && walk.at < before + mine) {
        int64_t at = before;
        for (int64_t b = b_lo; b < b_hi; ++b) {
            const int64_t n = seq_work(a, static_cast<int>(b), share).cost * H;
            if (walk.at < at + n) {
                s_b = static_cast<int>(b);
                s_before = at;
                break;
            }
            at += n;
        }
    }
    if (warp == 22) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i)
            mbar_init(bar(i), i >= RAW_EMPTY && i < KV_FULL ? 6
                              : i >= KV_FULL && i < KV_EMPTY ? 6
                              : i >= P_FULL && i < O_FULL ? 8 : i >= PAIR && i < SEG_FULL ? 2 : i >= SEG_EMPTY && i < DRAIN ? 23 : 1);
        fence_mbarrier_init();
    }
    // the columns of [O | L] behind the sums stay zero
    for (int i = threadIdx.x; i < 2 * GR * TOK; i += kPThreads) {
        const int buf = i / (GR * TOK), r = i / TOK % GR, tok = i % TOK;
        sts128(base + C::OFF_V + buf * C::VB + (r * (G / 8 + 2) + G / 8 + 1) * (TOK * 16) + tok * 16, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = 0;  // (all 512 columns are this CTA's, so they begin at 0)
    volatile int *abort = &s_abort;
    // tokens of a copy; tiles start at a multiple of it
    const int step = GR == 2 || page_log2 == 4 ? 16 : 32;

    // The next part for a warp that is done with the one before it.
    uint32_t parts = 0;
    auto next_part = [&](Segment &g) {
        __syncwarp();
        if (parts > 0 && lane == 0) mbar_arrive(bar(SEG_EMPTY + ((parts - 1) & 1)));
        const bool ok = wait_role(bar(SEG_FULL + (parts & 1)), (parts >> 1) & 1, abort, status, SITE_KV4_ATTENTION);
        if (!__all_sync(0xffffffffu, ok)) return false;
        g = s_seg[parts & 1];
        ++parts;
        return g.tiles > 0;
    };
    Segment g;

    if (warp < 16) {
        regs_inc<kSoftmaxRegs>();
        // =================================================================== softmax
        // warp 8 tile + 4 hw + wl: rows 32 wl + 16 hw + 0..15 of the tile (wl: the quarter of TMEM that it reaches)
        const int tile = warp >> 3, hw = warp >> 2 & 1, wl = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(32 * wl + 16 * hw) << 16;
        const uint32_t ts = tmem + tile * SC + lanes, to = tmem + C::T_O + tile * OC + lanes;
        uint32_t n = 0;        // tiles so far, of all items (buffers)
        uint32_t mine_n = 0;   // tiles so far of this tile of rows
        uint32_t segs = 0, meets = 0;
        bool ok = true;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(PAIR + tile * 4 + wl));
            ok = wait_role(bar(PAIR + tile * 4 + wl), meets++ & 1, abort, status, SITE_KV4_ATTENTION);
            ok = __all_sync(0xffffffffu, ok);
            return ok;
        };
        while (ok && next_part(g)) {
            if (tile * kRows >= g.ncols) {  // no rows for this tile
                n += g.tiles;
                continue;
            }
            if (!meet()) break;  // (the other warp of these 32 rows has read what the last item left)
            {
                // two lanes to a row, half of the dims each
                const int row = 32 * wl + 16 * hw + (lane >> 1), part = lane & 1, c = tile * kRows + row;
                const bool on = c < g.ncols;
                const int qrow = (g.col0 + c) / share, hh = (g.col0 + c) - qrow * share;
                const T *q = static_cast<const T *>(a.q) + (g.first + qrow) * a.q_tok +
                             (static_cast<int64_t>(g.head) * share + hh) * a.q_head + part * (D / 2);
                bool finite = true;
                float top = 0.0f;
                uint4 raw[D / 16];
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    raw[i] = make_uint4(0, 0, 0, 0);
                    if (on) raw[i] = __ldg(reinterpret_cast<const uint4 *>(q) + i);
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    float x[8];
                    Kv4In<T>::unpack(*reinterpret_cast<const uint4(*)[1]>(&raw[i]), x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        top = fmaxf(top, fabsf(x[j]));
                        finite &= fabsf(x[j]) <= 3.402823466e38f;
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                finite &= __shfl_xor_sync(0xffffffffu, finite ? 1 : 0, 1) != 0;
                // 2^k brings the row's largest into [2^14, 2^15); a negative scale turns the row
                int k = top > 0.0f && finite ? 14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127) : 0;
                k = min(k, 120);
                const float up = !finite ? 0.0f : copysignf(__uint_as_float(static_cast<uint32_t>(127 + k) << 23), a.scale);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                // codes are c 2^-24; (not 0: a hidden score is -inf before it meets this factor, and stays that)
                float f = fmaxf(fabsf(a.scale) * 1.4426950408889634f * down * 16777216.0f, 7.8886090522101181e-31f);
                if (MODS != kPlain && a.softcap > 0.0f) f = fminf(f * 2.0f / a.softcap, 3.402823466e38f);  // to tanh's argument, times 2 log2(e)
                const uint32_t dst = base + C::OFF_Q + tile * C::QB + part * (D / 16) * (kRows * 16) + row * 16;
                float sq = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    float x[8];
                    Kv4In<T>::unpack(*reinterpret_cast<const uint4(*)[1]>(&raw[i]), x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        x[j] = finite ? x[j] * up : 0.0f;
                        sq += x[j];
                    }
                    sts128(dst + i * (kRows * 16), pack_f16(x[0], x[4]), pack_f16(x[1] * 0.0625f, x[5] * 0.0625f),
                           pack_f16(x[2], x[6]), pack_f16(x[3] * 0.0625f, x[7] * 0.0625f));
                }
                sq *= 5.9604644775390625e-08f;  // 2^-24, as f has 2^24
                const float other = __shfl_xor_sync(0xffffffffu, sq, 1);
                if (part == 0) {
                    float slope = 0.0f;
                    if (MODS != kPlain && a.slopes != nullptr && on)
                        slope = __ldg(a.slopes + g.head * share + hh) * 1.4426950408889634f;
                    s_rows[c] = {f, {GR == 1 ? sq + other : sq, other}, slope, on ? g.pos0 + qrow : -1, finite ? 1 : 0, 0.0f, 0.0f};
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Q_FULL + tile));

            const int row_lo = (g.col0 + tile * kRows) / share;
            const int row_hi = (g.col0 + min(g.ncols, (tile + 1) * kRows) - 1) / share;
            const int all_hi = min(g.pos0 + row_lo, g.hi);  // positions that every row of the tile sees
            const int all_lo = a.window > 0 ? g.pos0 + row_hi - a.window + 1 : 0;

            // scores are held as a product's fragments: rows 8 i + g4 (i = 0, 1) of the warp's 16, tokens 8 b + 2 t4
            // and + 1 of a tile: a thread reads a quarter of the tokens' parameters (read by rows, they would take
            // as much of the shared memory's time as the products take)
            const int g4 = lane >> 2, t4 = lane & 3;
            RowInfo *rows = s_rows + tile * kRows + 32 * wl + 16 * hw + g4;
            float f[2], sq[2][GR], slope2[2], m[2], sum[2];  // sum: of the weights, kept where it is asked for
            int pos[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[i] = rows[8 * i].f;
#pragma unroll
                for (int r = 0; r < GR; ++r) sq[i][r] = rows[8 * i].sq[r];
                slope2[i] = MODS != kPlain ? rows[8 * i].slope : 0.0f;
                pos[i] = rows[8 * i].pos;
                m[i] = kNoMax;
                sum[i] = 0.0f;
            }
            int e0 = 0, e1 = 0;
            for (int j = 0; j < g.tiles; ++j) {
                const int tok0 = g.start + j * TOK;
                const int buf = n & 1;
                // (S first: these threads may have left tiles out that are not theirs, and S tells that KV_FULL is at n)
                ok = wait_role(bar(S_FULL + tile), mine_n & 1, abort, status, SITE_KV4_ATTENTION);
                ok = ok && wait_role(bar(KV_FULL + buf), (n >> 1) & 1, abort, status, SITE_KV4_ATTENTION);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const TileInfo info = s_info[buf];
                const bool edge = tok0 + TOK - 1 > all_hi || tok0 < all_lo;
                const uint32_t par = base + C::OFF_P + buf * C::PB;
                constexpr int NB = TOK / 8;
                uint64_t y[NB][2];  // pairs of tokens 8 b + 2 t4, + 1 of row 8 i + g4
                if constexpr (GR == 1) {
                    tmem_ld_rows<4>(ts, reinterpret_cast<uint32_t *>(y[0]));
#pragma unroll
                    for (int b0 = 0; b0 < NB; b0 += 4) {  // four blocks at a time, the next on its way
                        tmem_wait_ld();
                        if (b0 + 4 < NB) tmem_ld_rows<4>(ts + 8 * (b0 + 4), reinterpret_cast<uint32_t *>(y[b0 + 4]));
#pragma unroll
                        for (int b = b0; b < b0 + 4; ++b) {
                            const uint64_t s2 = lds64x(par + (8 * b + 2 * t4) * 4);
                            const uint64_t m2 = lds64x(par + (TOK + 8 * b + 2 * t4) * 4);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                y[b][i] = fma2(y[b][i], s2, mul2(m2, pack64(sq[i][0], sq[i][0])));
                        }
                    }
                } else {
#pragma unroll
                    for (int b0 = 0; b0 < NB; b0 += 2) {
                        uint64_t u[2][2];
                        tmem_ld_rows<2>(ts + 8 * b0, reinterpret_cast<uint32_t *>(y[b0]));
                        tmem_ld_rows<2>(ts + TOK + 8 * b0, reinterpret_cast<uint32_t *>(u[0]));
                        tmem_wait_ld();
#pragma unroll
                        for (int b = b0; b < b0 + 2; ++b) {
                            const uint32_t at = par + (8 * b + 2 * t4) * 4;
                            const uint64_t s2 = lds64x(at), v2 = lds64x(at + TOK * 4);
                            const uint64_t m2 = lds64x(at + TOK * 8), n2 = lds64x(at + TOK * 12);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                y[b][i] = fma2(y[b][i], s2,
                                               fma2(u[b - b0][i], v2, fma2(n2, pack64(sq[i][GR - 1], sq[i][GR - 1]),
                                                                           mul2(m2, pack64(sq[i][0], sq[i][0])))));
                        }
                    }
                }
                const uint32_t mu = par + (2 * GR * TOK + 2 * t4) * 4;

                if constexpr (MODS != kPlain) {  // scores in powers of two from here on
                    const float cap2 = a.softcap * 1.4426950408889634f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint64_t f2 = pack64(f[i], f[i]), slopes = pack64(slope2[i], slope2[i]);
                        const float away = static_cast<float>(tok0 + 2 * t4 - pos[i]);
                        const uint64_t bias = pack64(slope2[i] * away, slope2[i] * (away + 1.0f));
                        if (MODS == kFarMods) {
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const float2 v = unpack64(mul2(y[b][i], f2));
                                const float2 d = unpack64(fma2(slopes, pack64(8.0f * b, 8.0f * b), bias));
                                float2 z = make_float2(fmaf(-2.0f * cap2, rcp(ex2(v.x) + 1.0f), cap2),
                                                       fmaf(-2.0f * cap2, rcp(ex2(v.y) + 1.0f), cap2));
                                if (fabsf(v.x) < kSeries) z.x = cap_series(v.x, 0.5f * a.softcap);
                                if (fabsf(v.y) < kSeries) z.y = cap_series(v.y, 0.5f * a.softcap);
                                y[b][i] = pack64(z.x + d.x, z.y + d.y);
                            }
                        } else if (a.softcap > 0.0f) {
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                const float2 z = unpack64(mul2(y[b][i], f2));
                                const float2 d = unpack64(fma2(slopes, pack64(8.0f * b, 8.0f * b), bias));
                                y[b][i] = pack64(fmaf(-2.0f * cap2, rcp(ex2(z.x) + 1.0f), cap2) + d.x,
                                                 fmaf(-2.0f * cap2, rcp(ex2(z.y) + 1.0f), cap2) + d.y);
                            }
                        } else {
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                y[b][i] = fma2(y[b][i], f2, fma2(slopes, pack64(8.0f * b, 8.0f * b), bias));
                        }
                    }
                }
                int see_lo[2], see_hi[2];  // first and last token that the row sees, from 2 t4 of the tile on
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    see_hi[i] = min(pos[i], g.hi) - tok0 - 2 * t4;
                    see_lo[i] = a.window > 0 ? max(pos[i] - a.window + 1, 0) - tok0 - 2 * t4 : -TOK;
                }
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float2 z = unpack64(y[b][i]);
                            if (8 * b > see_hi[i] || 8 * b < see_lo[i]) z.x = -INFINITY;
                            if (8 * b + 1 > see_hi[i] || 8 * b + 1 < see_lo[i]) z.y = -INFINITY;
                            y[b][i] = pack64(z.x, z.y);
                        }
                    }
                }
                // (a row that has seen nothing keeps m = kNoMax, which is finite: its weights are 2^-inf = 0, whatever f is)
                float top[2];
                bool rise = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[i] = -INFINITY;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float2 z = unpack64(y[b][i]);
                        top[i] = fmaxf(top[i], fmaxf(z.x, z.y));
                    }
                    if (MODS == kPlain) top[i] *= f[i];
                    rise |= top[i] > m[i] + kRise;
                }
                if (__any_sync(0xffffffffu, rise) || (j > 0 && (info.e0 != e0 || info.e1 != e1))) {
                    float keep[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                        const float now = fmaxf(m[i], top[i]);
                        keep[i] = ex2(m[i] - now);
                        m[i] = now;
                        sum[i] *= keep[i];
                    }
                    if (j > 0) {  // (the products up to here are complete: S came after them)
                        // columns 2 t4, 2 t4 + 1 of 8; of the sums: the divisor's (t4 = 0), the middles'
                        const float ko = pow2i(e0 - info.e0);
                        const float ks = t4 == 0 ? 1.0f : pow2i(e1 - info.e1);
#pragma unroll 1
                        for (int c0 = 0; c0 < OC; c0 += 16) {
                            uint32_t o[8];
                            const float by = c0 % (G + 16) == G ? ks : ko;
                            tmem_ld_rows<2>(to + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int t = 0; t < 8; ++t)
                                o[t] = __float_as_uint(__uint_as_float(o[t]) * (by * keep[t >> 1 & 1]));
                            tmem_st_rows<2>(to + c0, o);
                        }
                    }
                }
                e0 = info.e0;
                e1 = info.e1;

#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float f1 = MODS != kPlain ? 1.0f : f[i];
                    const uint64_t f2 = pack64(f1, f1), off2 = pack64(kLift - m[i], kLift - m[i]);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const float2 x = unpack64(fma2(y[b][i], f2, off2));
                        y[b][i] = pack64(ex2(x.x), ex2(x.y));
                    }
                }
                if (a.lse != nullptr) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const float2 x = unpack64(y[b][i]);
                            sum[i] += x.x + x.y;
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < GR; ++r) {
                    uint32_t w[NB][2];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint64_t m2 = lds64x(mu + (r * TOK + 8 * b) * 4);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 x = unpack64(mul2(y[b][i], m2));
                            w[b][i] = pack_f16(x.x, x.y);
                        }
                    }
#pragma unroll
                    for (int b = 0; b + 4 <= NB; b += 4) tmem_st_half<4>(ts + r * (TOK / 2) + 4 * b, w[b]);
                    if constexpr (NB % 4 != 0) tmem_st_half<2>(ts + r * (TOK / 2) + 4 * (NB / 4 * 4), w[NB / 4 * 4]);
                }
                tmem_wait_st();
                if (info.odd) {  // NaN for the rows that see such a token only (a weight of 0 times NaN is in its place)
#pragma unroll 1
                    for (int c0 = 0; c0 < GR * NB; ++c0) {
                        uint32_t w[2];
                        tmem_ld_half1(ts + 4 * c0, w);
                        tmem_wait_ld();
                        const int b = c0 % NB;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (8 * b > see_hi[i] || 8 * b < see_lo[i]) w[i] &= 0xffff0000u;
                            if (8 * b + 1 > see_hi[i] || 8 * b + 1 < see_lo[i]) w[i] &= 0xffffu;
                        }
                        tmem_st_half1(ts + 4 * c0, w);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(P_FULL + tile));
                ++n;
                ++mine_n;
            }
            if (!ok) break;
            ok = wait_role(bar(O_FULL + tile), segs & 1, abort, status, SITE_KV4_ATTENTION);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            ++segs;
            tc_fence_after();
            // ---- results: a thread per row, half of the dims for each of the two warps of 32 rows
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
                if (t4 == 0) {
                    rows[8 * i].m = m[i];
                    rows[8 * i].sum = sum[i];
                }
            }
            if (!meet()) break;
            {
                const int c = tile * kRows + 32 * wl + lane;
                const bool on = c < g.ncols;
                const int qrow = (g.col0 + c) / share, hh = (g.col0 + c) - qrow * share;
                const RowInfo row = s_rows[c];
                const bool spoilt = row.pos >= 0 && (!row.finite || row.pos >= g.cap);
                if (row.pos >= g.cap) report(status, BQ_ERR_INVALID_ARG, SITE_KV4_ATTENTION);
                const float w0 = pow2i(e0), w1 = pow2i(e1);
                const int64_t row_out = (g.first + qrow) * a.q_heads + static_cast<int64_t>(g.head) * share + hh;
                float *slot = ws.slots + (2 * cta + (g.begins ? 1 : 0)) * (static_cast<int64_t>(kCols) * (D + 4)) + c * (D + 4);
                const uint32_t ot = tmem + C::T_O + tile * OC + (static_cast<uint32_t>(32 * wl) << 16);
                const int grp = GR == 1 ? 0 : hw;
                uint32_t l[16];
                tmem_ld_32x32b_x16(ot + grp * (G + 16) + G, l);
                tmem_wait_ld();
                float den = __uint_as_float(l[0]) + __uint_as_float(l[1]), row_sum = row.sum;
                const float lm = fmaf(__uint_as_float(l[3]), 1.0f / kRest, __uint_as_float(l[2])) * w1;
                if (a.lse == nullptr) row_sum = den;
                if (spoilt) den = row_sum = __int_as_float(0x7fffffff);
                const float inv = !g.whole ? 1.0f : den == 0.0f ? 0.0f : __fdividef(1.0f, den);
                const int d0 = hw * (D / 2);
#pragma unroll
                for (int h = 0; h < D / 2; h += 16) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(ot + (GR == 1 ? d0 : grp * (G + 16)) + h, o);
                    tmem_wait_ld();
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {  // columns 0..7 of a block are dims 0 4 1 5 2 6 3 7
                        const int d = (i & 8) + ((i & 1) << 2) + ((i & 7) >> 1);
                        v[d] = fmaf(__uint_as_float(o[i]), w0, lm) * inv;
                    }
                    if (on && g.whole) {
                        uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row_out * D + d0 + h);
                        out[0] = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                                            pack2(v[6], v[7], T()));
                        out[1] = make_uint4(pack2(v[8], v[9], T()), pack2(v[10], v[11], T()), pack2(v[12], v[13], T()),
                                            pack2(v[14], v[15], T()));
                    } else if (on) {
                        float4 *out = reinterpret_cast<float4 *>(slot + d0 + h);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            out[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
                if (on && !g.whole) {
                    if (hw == 0) {
                        slot[D] = row.m;
                        slot[D + 1] = row_sum;
                    }
                    if (hw < GR) slot[D + 2 + hw] = den;
                }
                if (on && g.whole && hw == 0 && a.lse != nullptr)
                    a.lse[row_out] = row_sum == 0.0f ? -INFINITY : (row.m - kLift + log2f(row_sum)) * 0.6931471805599453f;
            }
            tc_fence_before();
        }
    } else {
        regs_dec<kOtherRegs>();
        if (warp < 22) {
            // =============================================================== unpacking
            const bool values = warp < 19;
            const int u = (static_cast<int>(threadIdx.x) - (values ? 512 : 608));
            const int tok = u % TOK, r = u / TOK;  // token and group of this thread
            uint32_t n = 0;
            int e0 = 0, e1 = 0;
            bool near = true;  // the value steps are all within 2^9 of each other
            bool ok = true;
            // codes as fp16 subnormals, masked in place
            auto codes = [&](uint32_t src, uint32_t dst) {
#pragma unroll 1
                for (int i = 0; i < G / 32; ++i) {
                    // (the 16-byte pieces in an order that keeps 8 tokens off each other's banks)
                    const int ch = (i + (tok >> (C::ROW == 64 ? 1 : 2))) & (G / 32 - 1);
                    const uint4 v = lds128(src + ch * 16);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        sts128(dst + (ch * 4 + t) * (TOK * 16), w[t] & 0x000f000fu, w[t] & 0x00f000f0u,
                               (w[t] >> 8) & 0x000f000fu, (w[t] >> 8) & 0x00f000f0u);
                }
            };
            while (ok && next_part(g)) {
                for (int j = 0; j < g.tiles; ++j, ++n) {
                    const int stage = n % kRing, buf = n & 1;
                    const int tok0 = g.start + j * TOK;
                    ok = n < 2 || wait_role(bar(KV_EMPTY + buf), ((n >> 1) - 1) & 1, abort, status, SITE_KV4_ATTENTION);
                    ok = ok && wait_role(bar(RAW_FULL + stage), (n / kRing) & 1, abort, status, SITE_KV4_ATTENTION);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const uint32_t raw = base + C::OFF_RAW + stage * C::RAW + (values ? TOK * (C::ROW + C::PAR) : 0);
                    const uint32_t par = base + C::OFF_P + buf * C::PB;
                    const bool held = tok0 + tok <= g.hi;
                    const bool gone = (s_bad[stage] >> (tok / step)) & 1u;
                    const uint32_t src = raw + tok * C::ROW + r * (G / 2);
                    if (!values) {
                        float2 x = unpack_f16(lds32(raw + TOK * C::ROW + tok * C::PAR + 4 * r));
                        if (!held) x = make_float2(0.0f, 0.0f);
                        if (gone) x.x = __int_as_float(0x7fffffff);
                        sts32f(par + (r * TOK + tok) * 4, x.x);
                        sts32f(par + ((GR + r) * TOK + tok) * 4, x.y);
                        codes(src, base + C::OFF_K + buf * C::KB + r * (G / 8) * (TOK * 16) + tok * 16);
                    } else {
                        // exponents of the tile (fp16's fields): each warp looks at all of its tokens
                        uint32_t hi_s = 0, lo_s = 0x7c00u, hi_m = 0;  // (of s, s, m)
#pragma unroll
                        for (int i = 0; i < TOK * GR / 32; ++i) {
                            const int k = i * 32 + lane, kt = k % TOK;
                            const uint32_t w = lds32(raw + TOK * C::ROW + kt * C::PAR + 4 * (k / TOK));
                            const uint32_t fs = w & 0x7c00u, fm = (w >> 16) & 0x7c00u;
                            if (tok0 + kt <= g.hi && !((s_bad[stage] >> (kt / step)) & 1u)) {
                                hi_s = max(hi_s, fs == 0x7c00u || fm == 0x7c00u ? 0x8000u : fs);
                                if (fs != 0x7c00u && fm != 0x7c00u) {
                                    lo_s = min(lo_s, fs);
                                    hi_m = max(hi_m, fm);
                                }
                            }
                        }
                        hi_s = __reduce_max_sync(0xffffffffu, hi_s);
                        lo_s = __reduce_min_sync(0xffffffffu, lo_s);
                        hi_m = __reduce_max_sync(0xffffffffu, hi_m);
                        const bool odd = hi_s == 0x8000u;
                        if (odd) {  // the largest of the finite ones
                            hi_s = 0;
#pragma unroll 1
                            for (int i = 0; i < TOK * GR / 32; ++i) {
                                const int k = i * 32 + lane, kt = k % TOK;
                                const uint32_t w = lds32(raw + TOK * C::ROW + kt * C::PAR + 4 * (k / TOK));
                                if (tok0 + kt <= g.hi && (w & 0x7c00u) != 0x7c00u) hi_s = max(hi_s, w & 0x7c00u);
                            }
                            hi_s = __reduce_max_sync(0xffffffffu, hi_s);
                        }
                        const int top0 = static_cast<int>(hi_s >> 10) - 15;
                        const int top1 = max(static_cast<int>(hi_m >> 10) - 15, top0 + 3) + 1;  // of m + 8 s
                        if (j == 0) near = true;
                        if (j == 0 || top1 > e1 + 4) e1 = top1 - 2;
                        if (near) {
                            if (j == 0 || top0 > e0) e0 = top0 + 1;
                            near = lo_s == 0x7c00u || (lo_s != 0 && static_cast<int>(lo_s >> 10) - 15 >= e0 - 9);
                        }
                        if (!near && (j == 0 || top0 > e0 + 5)) e0 = top0 - 3;
                        const float2 x = unpack_f16(lds32(raw + TOK * C::ROW + tok * C::PAR + 4 * r));
                        const uint32_t vb = base + C::OFF_V + buf * C::VB + r * (G / 8 + 2) * (TOK * 16) + tok * 16;
                        const bool fit = held && !gone && fabsf(x.x) <= 65504.0f && fabsf(x.y) <= 65504.0f;
                        float mu = held && !gone && !fit ? __int_as_float(0x7fffffff) : 1.0f, inv = 0.0f, lm = 0.0f;
                        auto scaled = [](uint32_t v, uint32_t by, uint32_t minus) {
                            uint32_t d;
                            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(v | 0x64006400u), "r"(by), "r"(minus));
                            return d;
                        };
                        if (near) {
                            if (fit) {
                                mu = x.x * pow2i(-e0);
                                inv = rcp(mu);
                                lm = fmaf(8.0f, x.x, x.y) * pow2i(-e1) * inv;
                            }
#pragma unroll 1
                            for (int i = 0; i < G / 32; ++i) {
                                const int ch = (i + (tok >> (C::ROW == 64 ? 1 : 2))) & (G / 32 - 1);
                                const uint4 v = lds128(src + ch * 16);
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int t = 0; t < 4; ++t)  // 1, -1032; 1 / 16, -72
                                    sts128(vb + (ch * 4 + t) * (TOK * 16), scaled(w[t] & 0x000f000fu, 0x3c003c00u, 0xe408e408u),
                                           scaled(w[t] & 0x00f000f0u, 0x2c002c00u, 0xd480d480u),
                                           scaled((w[t] >> 8) & 0x000f000fu, 0x3c003c00u, 0xe408e408u),
                                           scaled((w[t] >> 8) & 0x00f000f0u, 0x2c002c00u, 0xd480d480u));
                            }
                        } else {
                            uint32_t mult = 0, less = 0, mult16 = 0, less16 = 0;  // 2^k, -1032 2^k, 2^(k - 4), -72 2^k
                            if (fit) {
                                // a step far below e0's takes part of its exponent into the weight (the codes
                                // reach down to 2^-24, 16 times a code's 2^k); where 1 / mu would leave fp16 even
                                // so, at steps below 2^-34 of the largest, the codes count as their middle
                                const int k = max(exp_of(x.x) - e0, -20);
                                mu = x.x * pow2i(-k - e0);
                                inv = rcp(mu);
                                lm = fmaf(8.0f, x.x, x.y) * pow2i(-e1);
                                if (fabsf(inv) <= 32768.0f && fabsf(lm * inv) <= 8192.0f) {
                                    lm *= inv;
                                    const float b = pow2i(k);
                                    mult = pack_f16(b, b);
                                    less = pack_f16(b * -1032.0f, b * -1032.0f);
                                    mult16 = pack_f16(b * 0.0625f, b * 0.0625f);
                                    less16 = pack_f16(b * -72.0f, b * -72.0f);
                                } else {
                                    mu = inv = 1.0f;
                                }
                            }
#pragma unroll 1
                            for (int i = 0; i < G / 8; ++i) {
                                const uint32_t w = lds32(src + 4 * i);
                                sts128(vb + i * (TOK * 16), scaled(w & 0x000f000fu, mult, less),
                                       scaled(w & 0x00f000f0u, mult16, less16), scaled((w >> 8) & 0x000f000fu, mult, less),
                                       scaled((w >> 8) & 0x00f000f0u, mult16, less16));
                            }
                        }
                        sts32f(par + ((2 * GR + r) * TOK + tok) * 4, mu);
                        // A middle is at most 2^13 here (1 / mu at most 2^9), so what fp16 leaves of it, times kRest,
                        // is at most 2^15, and the pair holds it to 2^-39: to 2^-41 of the largest middle of the part,
                        // whoever sees the token that has that one.
                        const uint32_t hi = pack_f16(inv, lm);
                        const float2 h = unpack_f16(hi);
                        const uint32_t lo = pack_f16(inv - h.x, (lm - h.y) * kRest);
                        sts128(vb + (G / 8) * (TOK * 16), __byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632), 0, 0);
                        if (warp == 16 && lane == 0) s_info[buf] = {e0, e1, odd ? 1 : 0};
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(RAW_EMPTY + stage));
                        mbar_arrive(bar(KV_FULL + buf));
                    }
                }
            }
        } else if (warp == 22) {
            // =============================================================== products
            uint32_t n = 0, np[2] = {0, 0}, segs[2] = {0, 0};
            bool ok = true;
            auto wait = [&](int i, uint32_t parity) {
                ok = ok && wait_role(bar(i), parity & 1, abort, status, SITE_KV4_ATTENTION);
                ok = __all_sync(0xffffffffu, ok);
                return ok;
            };
            // (tile and buffer are constants of each copy of this code, so that descriptors and addresses are
            // uniform: a product then issues in the time that the one before it takes)
            auto scores = [&](auto tile_, auto buf_) {
                constexpr int tile = decltype(tile_)::value, buf = decltype(buf_)::value;
                if (!elect_one()) return;
                const uint64_t qd = desc_plain(base + C::OFF_Q + tile * C::QB, kRows * 16, 128);
                const uint64_t kd = desc_plain(base + C::OFF_K + buf * C::KB, TOK * 16, 128);
#pragma unroll
                for (int r = 0; r < GR; ++r)
#pragma unroll
                    for (int k = 0; k < G / 16; ++k)
                        mma_ss(tile * SC + r * TOK, qd + (((r * (G / 16) + k) * 2 * kRows * 16) >> 4),
                               kd + (((r * (G / 16) + k) * 2 * TOK * 16) >> 4), idesc_f16(TOK, false), k > 0);
                tc_commit(bar(S_FULL + tile));
            };
            auto outputs = [&](auto tile_, auto buf_, bool more, bool end, bool done) {
                constexpr int tile = decltype(tile_)::value, buf = decltype(buf_)::value;
                if (!elect_one()) return;
                const uint64_t vd = desc_plain(base + C::OFF_V + buf * C::VB, 128, TOK * 16);
#pragma unroll
                for (int r = 0; r < GR; ++r)
#pragma unroll
                    for (int k = 0; k < TOK / 16; ++k)
                        mma_ts(C::T_O + tile * OC + r * (G + 16), tile * SC + r * (TOK / 2) + 8 * k,
                               vd + ((r * (G / 8 + 2) * TOK * 16 + k * 256) >> 4), idesc_f16(G + 16, true), more || k > 0);
                if (end) tc_commit(bar(O_FULL + tile));
                if (done) tc_commit(bar(KV_EMPTY + buf));
            };
            constexpr std::integral_constant<int, 0> c0;
            constexpr std::integral_constant<int, 1> c1;
            // products of tile n of the tokens, in buffer `buf`, and the scores of the next
            auto products = [&](auto buf, auto other, bool first, bool last, bool two) {
                if (!wait(P_FULL, np[0]++)) return;
                tc_fence_after();
                outputs(c0, buf, !first, last, !two);
                __syncwarp();
                if (!last) {
                    if (!wait(KV_FULL + decltype(other)::value, (n + 1) >> 1)) return;
                    tc_fence_after();
                    scores(c0, other);
                    __syncwarp();
                }
                if (!two) return;
                if (!wait(P_FULL + 1, np[1]++)) return;
                tc_fence_after();
                outputs(c1, buf, !first, last, true);
                __syncwarp();
                if (!last) scores(c1, other);
                __syncwarp();
            };
            while (ok && next_part(g)) {
                const bool two = g.ncols > kRows;
                wait(Q_FULL, segs[0]++);
                if (two) wait(Q_FULL + 1, segs[1]++);
                wait(KV_FULL + (n & 1), n >> 1);
                if (!ok) break;
                tc_fence_after();
                if (n & 1) {
                    scores(c0, c1);
                    if (two) scores(c1, c1);
                } else {
                    scores(c0, c0);
                    if (two) scores(c1, c0);
                }
                __syncwarp();
                for (int j = 0; j < g.tiles && ok; ++j, ++n) {
                    if (n & 1)
                        products(c1, c0, j == 0, j + 1 == g.tiles, two);
                    else
                        products(c0, c1, j == 0, j + 1 == g.tiles, two);
                }
            }
            // every product has ended before TMEM is given back
            if (elect_one()) {
                tc_commit(bar(DRAIN));
                mbar_drain(bar(DRAIN), 0, kWaitLimitNs);
            }
            __syncwarp();
        } else {
            // =============================================================== copies
            uint32_t n = 0;
            bool ok = true;
            walk.b = s_b;
            walk.seq_begin = s_before;
            while (ok) {
                int64_t end = 0;
                const bool more = next_segment<TOK>(a, share, step, walk, g, end);
                if (!more) g.tiles = 0;
                if (more && g.begins && !g.whole && lane == 0) {
                    const int64_t last = (end * ctas - 1) / total;  // CTA that holds the item's end
                    ws.desc[cta] = {g.first, g.col0, g.ncols, g.head, static_cast<int>(last - cta) + 1};
                }
                if (more && g.tiles <= 0) {
                    // a share that ends before the first tile of what it holds: nothing to add
                    float *slot = ws.slots + (2 * cta + (g.begins ? 1 : 0)) * (static_cast<int64_t>(kCols) * (D + 4));
                    for (int c = lane; c < kCols; c += 32) {
                        slot[c * (D + 4) + D] = kNoMax;
                        slot[c * (D + 4) + D + 1] = 0.0f;
                    }
                    continue;
                }
                ok = parts < 2 || wait_role(bar(SEG_EMPTY + (parts & 1)), ((parts >> 1) - 1) & 1, abort, status, SITE_KV4_ATTENTION);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane == 0) {
                    s_seg[parts & 1] = g;
                    mbar_arrive(bar(SEG_FULL + (parts & 1)));
                }
                __syncwarp();
                ++parts;
                if (!more) break;
                const int groups = TOK / step;
                const int grp = lane >> 2, what = lane & 3;  // K codes, K parameters, V codes, V parameters
                for (int j = 0; j < g.tiles; ++j, ++n) {
                    const int stage = n % kRing;
                    const int at = g.start + j * TOK + grp * step;
                    int64_t src = -1;
                    bool bad = false;
                    if (grp < groups && at <= g.hi) {
                        const int pg = __ldg(a.pool.table + static_cast<int64_t>(g.b) * a.pool.table_ld + (at >> page_log2));
                        bad = pg < 0 || pg >= a.pool.pages;
                        if (!bad)
                            src = static_cast<int64_t>(pg) * a.pool.page_stride +
                                  static_cast<int64_t>(g.head) * a.pool.block_bytes;
                    }
                    if (bad) report(status, BQ_ERR_INVALID_ARG, SITE_KV4_ATTENTION);
                    ok = n < kRing || wait_role(bar(RAW_EMPTY + stage), (n / kRing - 1) & 1, abort, status, SITE_KV4_ATTENTION);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const uint32_t good = __ballot_sync(0xffffffffu, src >= 0 && what == 0);
                    const uint32_t bads = __ballot_sync(0xffffffffu, bad && what == 0);
                    if (lane == 0) {
                        uint32_t bits = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) bits |= ((bads >> (4 * i)) & 1u) << i;
                        s_bad[stage] = bits;
                        mbar_arrive_expect_tx(bar(RAW_FULL + stage),
                                              static_cast<uint32_t>(__popc(good) * step * 2 * (C::ROW + C::PAR)));
                    }
                    __syncwarp();
                    if (src >= 0) {
                        const int slot = at & ((1 << page_log2) - 1);
                        const int off = (what >> 1) * static_cast<int>(a.pool.block_bytes >> 1) +
                                        ((what & 1) ? (C::ROW << page_log2) + slot * C::PAR : slot * C::ROW);
                        const uint32_t dst = base + C::OFF_RAW + stage * C::RAW + (what >> 1) * (TOK * (C::ROW + C::PAR)) +
                                             ((what & 1) ? TOK * C::ROW + grp * step * C::PAR : grp * step * C::ROW);
                        bulk_load(dst, a.pool.pool + src + off,
                                  static_cast<uint32_t>(step * ((what & 1) ? C::PAR : C::ROW)), bar(RAW_FULL + stage));
                    }
                    __syncwarp();
                }
            }
            // copies still in flight land before the CTA ends
            for (uint32_t i = n > kRing ? n - kRing : 0; i < n; ++i)
                mbar_drain(bar(RAW_FULL + i % kRing), (i / kRing) & 1, kWaitLimitNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 22) tmem_dealloc(s_tmem, 512);
}

template <typename C, Mods MODS, typename T>
cudaError_t launch_prefill(const Kv4AttnArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto kern = kv4_prefill_kernel<C, MODS, T>;
    static SmemOptIn opt_in;
    cudaError_t e = smem_opt_in(opt_in, dev, reinterpret_cast<const void *>(kern), static_cast<size_t>(C::SMEM));
    if (e != cudaSuccess) return e;
    // The register split of the roles adds up to what a CTA is launched with.  The build checks that (_build.py); a
    // library that was built some other way is refused here, since its warps would wait for registers for ever.
    static std::atomic<bool> checked{false};
    if (!checked.load(std::memory_order_relaxed)) {
        cudaFuncAttributes f = {};
        e = cudaFuncGetAttributes(&f, kern);
        if (e != cudaSuccess) return e;  // (asked again by the next call)
        if (f.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        checked.store(true, std::memory_order_relaxed);
    }
    const unsigned grid = static_cast<unsigned>(std::min(dev.num_sms, kKv4MaxSms));
    const Kv4Ws ws = kv4_workspace(a.workspace);
    kern<<<grid, kPThreads, C::SMEM, s>>>(a, ws, dev.status);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : kv4_launch_join<C::D, C::G, kCols, T>(a, ws, grid, s);
}

}  // namespace

cudaError_t launch_kv4_prefill(const Kv4AttnArgs &a, cudaStream_t s, const DevInfo &dev) {
    auto by_shape = [&](auto tag) {
        using T = decltype(tag);
        const Mods mods = mods_of(a);
        auto go = [&](auto c) {
            using C = decltype(c);
            if (mods == kPlain) return launch_prefill<C, kPlain, T>(a, s, dev);
            return mods == kNearMods ? launch_prefill<C, kNearMods, T>(a, s, dev) : launch_prefill<C, kFarMods, T>(a, s, dev);
        };
        if (a.pool.head_dim == 64) return go(PShape<64, 64>());
        return a.pool.group_size == 64 ? go(PShape<128, 64>()) : go(PShape<128, 128>());
    };
    return a.dtype == BQ_F16 ? by_shape(__half()) : by_shape(__nv_bfloat16());
}

}  // namespace bq

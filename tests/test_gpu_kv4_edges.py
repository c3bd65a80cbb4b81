"""The 4-bit cache's attention where its arithmetic and its bookkeeping have borders: rows that see nothing, in a tile or at
all, queries and values far from one, places behind a window, positions at the ends of their range, other streams.

Yardstick and bounds are those of test_gpu_kv4.py (kv4_reference.py) unless a test derives its own."""
import numpy as np
import pytest
import torch

import bit_quantized_linear_rmsnorm_b200 as bq
import kv4_reference as ref
from test_gpu_kv4 import DT, SHAPES, Setup, check_attention, dev, offsets, query, run_attention, status_ok

pytestmark = pytest.mark.gpu

EXTRAS = [dict(), dict(softcap=5.0), dict(slopes=1), dict(window=7), dict(window=33, softcap=20.0, slopes=1)]


def extras(kw, heads):
    return dict(kw, slopes=2.0 ** -np.linspace(1.0, 8.0, heads)) if "slopes" in kw else kw


def check_lse(s, lse, q, cu, scale, **kw):
    """lse against the yardstick, for scores of any size.

    d lse = sum p dz, so |error of lse| <= max |error of z| + that of the weights (2^-11 each, at most, on the sum that the
    logarithm is taken of) and of the logarithm itself: 2^-10 + 2^-20 |lse| for these two, as in check_attention.  A
    score's error is kv4_reference's: a dot product of D terms and the minimum's term in fp32, one step u = 2^-23 each,
    (D + 16) u |scale| sum|q| (15 s + |m|), and 4 u |z|, where |z| <= |scale| sum|q| (15 s + |m|) too."""
    _, want, _ = ref.attention(q.double().cpu().numpy(), s.host, s.table, s.lens, cu, scale, **kw)
    got = lse.double().cpu().numpy()[: int(cu[-1])]
    want = want[: len(got)]
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.array_equal(np.isnan(got), np.isnan(want))
    most = 0.0
    for b, n in enumerate(s.lens):
        par = s.host._part(0)[1][s.table[b, : -(-n // s.page)].astype(np.int64)].astype(np.float64)
        par = (15 * par[..., 0] + np.abs(par[..., 1])).transpose(0, 2, 1, 3).reshape(-1, s.H, par.shape[-2])[:n]
        most = max(most, par.max(initial=0.0))
    dz = (s.D + 16 + 4) * 2.0 ** -23 * abs(scale) * q.double().abs().sum(-1).cpu().numpy()[: len(got)] * most
    fin = np.isfinite(want)
    bad = np.abs(got[fin] - want[fin]) > (2.0 ** -10 + 2.0 ** -20 * np.abs(want) + dz)[fin]
    assert not bad.any()


def check_rounded(s, out, q, cu, scale, **kw):
    """check_attention, but where the value itself, to within its bound, is not below 65520 an fp16 output is an infinity
    of its sign: 65520 lies half-way between 65504, the largest fp16, and the 2^16 that would follow, and rounds up."""
    want, _, tol = ref.attention(q.double().cpu().numpy(), s.host, s.table, s.lens, cu, scale, **kw)
    over = (np.abs(want) + tol >= 65520) & (out.dtype is torch.float16)
    got = out.double().cpu().numpy()
    held = np.where(over & np.isinf(got) & (np.sign(got) == np.sign(want)), want, got)
    info = torch.finfo(out.dtype)
    bound = tol + (info.eps / 2) * (np.abs(want) + tol) + info.smallest_normal * info.eps
    assert np.array_equal(np.isnan(held), np.isnan(want))
    ok = np.isnan(want) | (np.abs(held - want) <= bound)
    assert ok.all(), (np.argwhere(~ok)[:5], np.nanmax(np.abs(held - want) / bound))


# ------------------------------------------------------------------ rows that see nothing of a tile, or nothing at all
@pytest.mark.parametrize("size", [1e-30, 1e-3, 0.006, 300.0])
@pytest.mark.parametrize("D,G", SHAPES)
def test_many_rows_with_queries_of_every_size(D, G, size):
    """The first tiles of an item hold nothing for its last rows (a window, one head to a key head), whatever the factor
    between a product and its score is."""
    s = Setup([200], 1, D, G, 32, seed=20).fill()
    pool, table, lens = s.cuda(), dev(s.table), dev(s.lens)

    def check(q, scale=D ** -0.5, **kw):
        lse = torch.full((200, 1), 3.0, device="cuda")
        out = bq.bq_kv4_attention(q, pool, table, lens, G, scale=scale, lse=lse, **kw)
        check_attention(s, out, None, q, [0, 200], scale, **kw)
        check_lse(s, lse, q, [0, 200], scale, **kw)
        assert torch.equal(bq.bq_kv4_attention(q, pool, table, lens, G, scale=scale, **kw), out)  # without lse

    q = query(s, 200, 1, "bf16", scale=size)
    for window in (16, 70, 0):
        check(q, window=window)
    q[::3] *= 2.0 ** -12  # rows of different sizes in one tile
    check(q, window=70)
    for scale in (0.01, -0.001):
        check(q, scale, window=16)
    status_ok()


@pytest.mark.parametrize("D,G", SHAPES)
def test_items_cut_between_ctas_with_small_queries(D, G):
    """The last part of a cut item holds nothing for its first rows."""
    s = Setup([2500, 130], 1, D, G, 64, seed=21).fill()
    for counts, heads in (([200, 5], 1), ([30, 100], 4)):
        q = query(s, sum(counts), heads, "bf16", scale=1e-3)
        run_attention(s, q, counts)
        run_attention(s, q, counts, window=900)


@pytest.mark.parametrize("kw", EXTRAS)
@pytest.mark.parametrize("D,G", SHAPES)
def test_many_rows_without_a_place_and_empty_slots(D, G, kw):
    """Rows before position 0 in an item whose other rows see tokens, a sequence of length 0, a padded slot: 0 and -inf."""
    kw = extras(kw, 4)
    s = Setup([35, 0, 0, 50], 1, D, G, 16, seed=22).fill()
    counts = [40, 30, 0, 12]
    for dtype, size in (("f16", 1.0), ("bf16", 1e-3)):
        out = run_attention(s, query(s, sum(counts) + 3, 4, dtype, scale=size), counts, rows_behind=3, **kw)
        assert (out[:5] == 0).all() and (out[40:70] == 0).all() and (out[5:40] != 0).any()
    # at once too small for its rows and alone in its call
    s = Setup([3], 1, D, G, 16, seed=23).fill()
    out = run_attention(s, query(s, 300, 4, "bf16"), [300], **kw)
    assert (out[:297] == 0).all()
    # the few-row kernel gives the same
    s = Setup([2, 0], 1, D, G, 16, seed=24).fill()
    run_attention(s, query(s, 8, 4, "bf16"), [4, 4], **kw)


# ------------------------------------------------------------------ values beyond fp16
@pytest.mark.parametrize("low,high", [(60000, 75000), (65504, 3e5), (-6e4, 1e6), (-1e6, -65600), (7e4, 7e4)])
@pytest.mark.parametrize("D,G", SHAPES)
def test_values_whose_middle_leaves_fp16(D, G, low, high):
    """What the write stores of bf16 values beyond fp16 is finite (minimum and step are), and so is what is attended to,
    in either kernel, alone or beside ordinary tokens."""
    for kind in ("all", "some"):
        s = Setup([150], 2, D, G, 16, seed=27)
        for p in range(150):
            k, v = s.rng.standard_normal((2, 2, D)).astype(np.float32)
            if kind == "all" or p % 40 == 3:
                v = s.rng.uniform(low, high, (2, D)).astype(np.float32)
            s.host.put(*s.place(0, p), k, v)
        for n in (1, 4, 40):
            out = run_attention(s, query(s, n, 4, "bf16"), [n])
            assert out.isfinite().all()


# ------------------------------------------------------------------ values of very different sizes
@pytest.mark.parametrize("counts", [[1, 1], [2, 5], [100, 70]])
@pytest.mark.parametrize("kind", ["larger", "offset", "first", "small", "not finite"])
@pytest.mark.parametrize("D,G", SHAPES)
def test_values_beside_far_larger_ones(D, G, kind, counts):
    """Tokens that a row does not see, or hardly weighs, and whose values are far larger than those that it does: in the
    same tile or in an earlier one, by their steps or by their minima only."""
    s = Setup([333, 81], 2, D, G, 64, seed=29)
    for b, n in enumerate(s.lens):
        for t in range(n):
            k, v = s.rng.standard_normal((2, 2, D)).astype(np.float32)
            far = t % 11 == 4
            if kind == "larger" and far:
                v *= 1.5e4
            elif kind == "offset" and far:
                v += 3e4
            elif kind == "first":
                v *= 1.0 if t >= 64 else 2e4
            elif kind == "small":
                v *= 1.5e4 if far else 2.0 ** -6
            elif kind == "not finite" and far:
                v *= 1.5e4 if t % 2 else np.nan
            if far:
                k[:] = 0
            s.host.put(*s.place(b, t), k, v)
    for dtype in ("f16", "bf16"):
        q = query(s, sum(counts), 4, dtype, scale=4.0)
        for window in (1, 9, 130):
            out = bq.bq_kv4_attention(q, s.cuda(), dev(s.table), dev(s.lens), G, cu_q=dev(offsets(counts)), max_q=max(counts),
                                      window=window)
            check_rounded(s, out, q, offsets(counts), D ** -0.5, window=window)
    status_ok()


# ------------------------------------------------------------------ pages behind a window
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=16), dict(window=50, slopes=1), dict(window=17, softcap=9.0)])
@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64])
def test_pages_before_the_window_may_be_gone(page, D, G, kw):
    """Entries of pages that no row of the call reaches any more name no page: nothing is reported, and nothing of what
    lies there, or of what an earlier tile left in shared memory, counts."""
    kw = extras(kw, 4)
    lens = [1, 17, 40, 81, 200, 333]
    for counts in ([1] * 6, [1, 2, 5, 3, 6, 4], [1, 10, 40, 30, 100, 33]):
        s = Setup(lens, 2, D, G, page, seed=28)
        for b, n in enumerate(lens):
            first = max(n - counts[b] - kw["window"] + 1, 0)  # the first position that a row sees
            for t in range(n):
                k, v = s.rng.standard_normal((2, 2, D)).astype(np.float32)
                # far larger than the rest, then not finite, where no row looks
                s.host.put(*s.place(b, t), k, v if t >= first else v * (3e4 if t % 3 else np.nan))
        pool = s.cuda()
        out = run_attention(s, query(s, sum(counts), 4, "bf16"), counts, **kw)
        full, q = s.table.copy(), query(s, sum(counts), 4, "bf16")
        want = bq.bq_kv4_attention(q, pool, dev(full), dev(lens), G, cu_q=dev(offsets(counts)), max_q=max(counts), window=kw["window"])
        for b, n in enumerate(lens):
            first = max(n - counts[b] - kw["window"] + 1, 0)
            s.table[b, : first // page] = -1
        got = bq.bq_kv4_attention(q, pool, dev(s.table), dev(lens), G, cu_q=dev(offsets(counts)), max_q=max(counts), window=kw["window"])
        assert torch.equal(got, want) and out.isfinite().all()
        status_ok()


# ------------------------------------------------------------------ positions at the ends of their range
def test_positions_near_the_end_of_32_bits():
    """A table as wide as positions go (2^24 pages of 128).  Up to 2^31 - 65537 a row is attended to as anywhere else;
    from there on it stands behind the table: NaN, reported, and no page is looked up outside the table."""
    page, G = 128, 64
    s = Setup([1024], 1, 64, G, page, seed=25).fill()
    pool = s.cuda()
    wide = dev(s.table[0, :8]).repeat(1 << 21)[None].contiguous()  # the small sequence's 8 pages over and over
    most = (1 << 31) - 65536
    for n, heads in ((1, 2), (200, 2)):
        q = query(s, n, heads, "bf16")
        out = bq.bq_kv4_attention(q, pool, wide, dev([most]), G, window=64)  # (most is a multiple of 1024)
        check_attention(s, out, None, q, [0, n], 64 ** -0.5, window=64)
        status_ok()
        # the last rows of 31 bits; with n = 200 some begin in a tile that would end behind them
        out = bq.bq_kv4_attention(q, pool, wide, dev([(1 << 31) - 1]), G, window=1)
        assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG and out.isnan().all()
        out = bq.bq_kv4_attention(q, pool, wide, dev([most + n // 2]), G, window=64)
        assert bq.bq_device_status()[0] == (bq.BQ_ERR_INVALID_ARG if n > 1 else bq.BQ_OK)
        if n > 1:
            assert out[n - n // 2:].isnan().all()
            keep = q[: n - n // 2]
            check_attention(s, out[: n - n // 2].contiguous(), None, keep, [0, len(keep)], 64 ** -0.5, window=64)


# ------------------------------------------------------------------ other streams than the current one
@pytest.mark.parametrize("n", [1, 50])
def test_calls_that_overlap_on_streams_given_to_them(n):
    """No workspace or output given, nothing waited for between the calls: each has its own, and what the current stream
    allocates meanwhile is not written to."""
    s = Setup([5000, 300, 4000], 2, 128, 64, 64, seed=26).fill()
    pool, table, lens = s.cuda(), dev(s.table), dev(s.lens)
    qs = [query(s, 3 * n, 8, "bf16") for _ in range(2)]
    want = [bq.bq_kv4_attention(q, pool, table, lens, s.G) for q in qs]
    cu = dev(offsets(s.lens))
    kv = bq.bq_kv4_read(pool, table, cu, 9300, 128, 64)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    size = bq.bq_kv4_attention_workspace_bytes(3 * n, 8, 2, 128)
    for _ in range(5):
        got, other, reads = [], [], []
        for q, st in zip(qs, side):
            got.append(bq.bq_kv4_attention(q, pool, table, lens, s.G, stream=st))
            other.append(torch.full((size,), 7, dtype=torch.uint8, device="cuda"))  # (on the current stream)
            reads.append(bq.bq_kv4_read(pool, table, cu, 9300, 128, 64, stream=st))
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], want[i]) and (other[i] == 7).all()
            assert torch.equal(reads[i][0], kv[0]) and torch.equal(reads[i][1], kv[1])
    status_ok()


@pytest.mark.parametrize("kw", EXTRAS)
@pytest.mark.parametrize("n", [1, 40])
def test_lengths_below_zero_hold_nothing(n, kw):
    """Any negative length is like 0, down to -2^31: 0 and -inf, nothing reported; the others are as they would be."""
    kw = extras(kw, 4)
    s = Setup([90, 0, 0, 0, 50], 2, 64, 64, 16, seed=30).fill()
    q = query(s, 5 * n, 4, "bf16")
    want = run_attention(s, q, [n] * 5, **kw)
    slopes = None if "slopes" not in kw else dev(kw["slopes"], torch.float32)
    lse = torch.zeros(5 * n, 4, device="cuda")
    out = bq.bq_kv4_attention(q, s.cuda(), dev(s.table), dev([90, -1, -2 ** 31, -2 ** 31 + 30, 50]), 64, lse=lse,
                              window=kw.get("window", 0), softcap=kw.get("softcap", 0.0), slopes=slopes)
    assert torch.equal(out, want) and not out[n:4 * n].any()
    assert lse[n:4 * n].isneginf().all() and lse[n - 1].isfinite().all()
    pool = s.cuda()
    kv = torch.randn(5, 2, 64, device="cuda").bfloat16()
    for lens in ([-1] * 5, [-2 ** 31] * 5):
        bq.bq_kv4_write(kv, kv, pool, dev(s.table), dev(lens), 64)
    assert torch.equal(pool, s.cuda())
    status_ok()


# ------------------------------------------------------------------ caps of every size
@pytest.mark.parametrize("n", [1, 5, 60])
@pytest.mark.parametrize("D,G", SHAPES)
def test_caps_of_every_size(D, G, n):
    """A cap costs a score no more than 2^-20 of its size, however large the cap; the smallest ones work as well."""
    s = Setup([150, 40], 2, D, G, 32, seed=31).fill()
    q = query(s, 2 * n, 4, "f16", scale=1.5)
    cu, scale = offsets([n, n]), D ** -0.5
    q64 = q.double().cpu().numpy()
    _, _, free = ref.attention(q64, s.host, s.table, s.lens, cu, scale)  # the bound without a cap
    biggest = np.abs(s.host.values(1, s.table[0], 150)).max()
    zmax = max(np.abs(scale * np.einsum("thd,khd->thk", q64[b * n:(b + 1) * n], np.repeat(
        s.host.values(0, s.table[b], s.lens[b]), 2, axis=1))).max() for b in range(2))
    for cap in (63.0, 65.0, 300.0, 1e4, 1e5, 1e6, 1e7, 1e20, 1e28, 1e29, 1e35, 3e38):
        out = bq.bq_kv4_attention(q, s.cuda(), dev(s.table), dev(s.lens), G, softcap=cap)
        want = ref.attention(q64, s.host, s.table, s.lens, cu, scale, softcap=cap)[0]
        # zmax <= cap / 4 or so: a weight moves by twice its score's error at most, the output by that times |v - out|;
        # up to the border of the two forms the error is the cap's, 2^-22 of it.  The softmax itself moves by less than
        # 3 (zmax / cap)^2 zmax from the free one, whose bound is scaled by that.
        dz = max(2.0 ** -20 * zmax, 2.0 ** -22 * 64)
        tol = free * (1 + 2 * zmax ** 3 / cap ** 2) + 2 * dz * 2 * biggest
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= tol + 2.0 ** -11 * (np.abs(want) + tol) + 2.0 ** -24).all(), cap
    for cap in (1e-3, 1e-30, 1e-40, 4.0):
        run_attention(s, q, [n, n], softcap=cap)
    for cap in (64.0, 200.0):  # with what else changes a score
        run_attention(s, q, [n, n], softcap=cap, slopes=2.0 ** -np.arange(1.0, 5.0), window=33)
    status_ok()


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(slopes=1), dict(softcap=500.0)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,G", SHAPES)
def test_every_variant_is_launched(D, G, dtype, kw):
    """Type, layout, what changes a score, and the number of columns (4, 12, 20, 160) choose the kernel's variant."""
    kw = extras(kw, 4)
    s = Setup([70], 1, D, G, 32, seed=32).fill()
    for n in (1, 3, 5, 40):
        run_attention(s, query(s, n, 4, dtype), [n], **kw)


@pytest.mark.parametrize("D,G", SHAPES)
def test_what_lies_in_place_of_a_bad_page_does_not_count(D, G):
    """Small values beside a NaN token and a page that is not there, after items with very large ones: rows that see
    neither are as exact as ever, though the missing page's place still holds what an earlier tile left."""
    lens = [300, 96] * 8
    s = Setup(lens, 1, D, G, 16, seed=33)
    for b, n in enumerate(lens):
        for t in range(n):
            k, v = s.rng.standard_normal((2, 1, D)).astype(np.float32)
            v = v * 1.5e4 if n == 300 else v * 2.0 ** -18
            s.host.put(*s.place(b, t), k, np.full_like(v, np.nan) if n == 96 and t == 78 else v)
    counts = [40] * 16
    q = query(s, sum(counts), 4, "bf16")
    table = s.table.copy()
    table[1::2, 5] = -1  # positions 80 .. 95
    out = bq.bq_kv4_attention(q, s.cuda(), dev(table), dev(lens), G)
    assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG
    want, _, tol = ref.attention(q.double().cpu().numpy(), s.host, s.table, lens, offsets(counts), D ** -0.5)
    got = out.double().cpu().numpy()
    for b in range(1, 16, 2):
        rows = slice(40 * b, 40 * b + 22)  # positions 56 .. 77
        assert np.isnan(got[40 * b + 22: 40 * b + 40]).all()
        bound = tol[rows] + 2.0 ** -8 * (np.abs(want[rows]) + tol[rows])
        assert (np.abs(got[rows] - want[rows]) <= bound).all()


@pytest.mark.parametrize("D,G,share", [(64, 64, 1), (128, 64, 4), (128, 128, 3), (64, 64, 24), (128, 128, 73)])
def test_columns_on_either_side_of_what_is_chosen(D, G, share):
    """Blocks of 24 columns of the few-row kernel, whole and begun, inside and between rows, up to its last column; and
    the many-row kernel's first."""
    s = Setup([200, 0, 140, 31], 2, D, G, 16, seed=34).fill()
    for cols in (9, 24, 25, 48, 49, 71, 72, 73, 96):
        if cols % share == 0 or share in (1, cols):
            n = cols // share
            counts = [n, 1, max(n // 2, 1), n]
            run_attention(s, query(s, sum(counts) + 1, 2 * share, "f16"), counts, rows_behind=1)
            run_attention(s, query(s, sum(counts) + 1, 2 * share, "bf16"), counts, rows_behind=1, window=20, softcap=30.0)
    # cut into parts
    s = Setup([4000], 1, D, G, 64, seed=35).fill()
    for n in {max(1, 72 // share), max(1, 40 // share)}:
        run_attention(s, query(s, n, share, "f16"), [n])


def test_pages_far_into_a_large_pool():
    """A pool of 5 GiB: byte offsets beyond 32 bits, signed or not, in the write, the read and both attention kernels."""
    D, G, page, H = 128, 64, 64, 2
    nbytes = ref.page_bytes(page, D, G)
    pages = (5 << 30) // (H * nbytes)
    s = Setup([150, 70], H, D, G, page, seed=36).fill()
    far = (2 ** 31 // (H * nbytes) + 1, 2 ** 32 // (H * nbytes), 2 ** 32 // (H * nbytes) + 1, pages - 1, pages - 2, 3, 0)
    table = np.full_like(s.table, -1)
    pool = torch.zeros((pages, H, nbytes), dtype=torch.uint8, device="cuda")
    here = torch.from_numpy(s.host.pool).cuda()
    at = 0
    for b, n in enumerate(s.lens):
        for i in range(-(-n // page)):
            table[b, i] = far[at]
            pool[far[at]] = here[int(s.table[b, i])]
            at += 1
    for counts in ([1, 1], [90, 40]):
        cu = offsets(counts)
        q = query(s, sum(counts), 4, "bf16")
        out = bq.bq_kv4_attention(q, pool, dev(table), dev(s.lens), G, cu_q=dev(cu), max_q=max(counts))
        check_attention(s, out, None, q, cu, D ** -0.5)
    cu = dev(offsets(s.lens))
    k, v = bq.bq_kv4_read(pool, dev(table), cu, 220, D, G, out_dtype=torch.float32)
    for which, got in ((0, k), (1, v)):
        want = np.concatenate([s.host.values(which, s.table[b], n, np.float32) for b, n in enumerate(s.lens)])
        assert np.array_equal(got.cpu().numpy(), want)
    other = torch.zeros_like(pool)
    bq.bq_kv4_write(k, v, other, dev(table), dev(s.lens), G, cu_q=cu)
    k2, v2 = bq.bq_kv4_read(other, dev(table), cu, 220, D, G, out_dtype=torch.float32)
    # (a group's smallest and largest value are kept to half a step of fp16's, the others to half a step more)
    for a, b in ((k, k2), (v, v2)):
        span = a.unflatten(-1, (-1, G))
        span = (span.amax(-1) - span.amin(-1)).repeat_interleave(G, -1)
        assert ((a - b).abs() <= span / 15 * 0.51 + a.abs() * 2.0 ** -10 + 1e-6).all()
    used = torch.zeros(pages, dtype=torch.bool, device="cuda")
    used[torch.from_numpy(table[table >= 0].astype(np.int64)).cuda()] = True
    touched = torch.cat([(x != 0).flatten(1).any(1) for x in other.split(4096)])
    assert torch.equal(touched, used)
    status_ok()

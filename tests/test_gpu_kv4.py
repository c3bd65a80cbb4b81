"""The 4-bit key/value cache on the GPU, against the 64-bit yardstick in kv4_reference.py.

Codes, parameters and values read are compared bit for bit.  Attention is held to the yardstick's own bound plus half a
step of the output type (and its smallest subnormal): the kernels sum in fp32 and round a weight to fp16 once.
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_rmsnorm_b200 as bq
import kv4_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SHAPES = [(64, 64), (128, 64), (128, 128)]


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def status_ok():
    st, detail = bq.bq_device_status()
    assert st == bq.BQ_OK, hex(detail)


class Setup:
    """Sequences of the given lengths in shuffled pages, on the host and on the GPU; table entries that no position
    reaches name no page."""

    def __init__(self, lens, H, D, G, page, seed=0, spare=2, fill=None):
        self.rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = self.rng.permutation(pages)
        self.lens, self.H, self.D, self.G, self.page = list(lens), H, D, G, page
        self.table = np.full((len(lens), max(max(need), 1) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (pages, H, ref.page_bytes(page, D, G))
        # what no one wrote holds NaN patterns
        self.host = ref.Cache(pages, H, D, G, page, fill=np.full(shape, 0xFF, dtype=np.uint8))

    def place(self, b, pos):
        return self.table[b, pos // self.page], pos % self.page

    def fill(self, loud=3.0):
        for b, n in enumerate(self.lens):
            for t in range(n):
                k, v = self.rng.standard_normal((2, self.H, self.D)).astype(np.float32)
                k[:, ::17] *= loud
                self.host.put(*self.place(b, t), k, v)
        return self

    def cuda(self):
        return torch.from_numpy(self.host.pool.copy()).cuda()


def offsets(counts):
    return np.concatenate(([0], np.cumsum(counts))).astype(np.int32)


def check_attention(s, out, lse, q, cu, scale, rows=None, **kw):
    want, wlse, tol = ref.attention(q.double().cpu().numpy(), s.host, s.table, s.lens, cu, scale, **kw)
    got = out.double().cpu().numpy()[: int(cu[-1])]
    info = torch.finfo(out.dtype)
    bound = tol + (info.eps / 2) * (np.abs(want) + tol) + info.smallest_normal * info.eps
    want, bound = want[: len(got)], bound[: len(got)]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.isnan(want) | (np.abs(got - want) <= bound)
    assert ok.all(), (np.argwhere(~ok)[:5], np.nanmax(np.abs(got - want) / bound))
    if lse is not None:
        gl, wl = lse.double().cpu().numpy()[: len(got)], wlse[: len(got)]
        assert np.array_equal(np.isneginf(gl), np.isneginf(wl)) and np.array_equal(np.isnan(gl), np.isnan(wl))
        fin = np.isfinite(wl)
        # the scores' error and the weights' (2^-11 each, at most) on a logarithm, and its own rounding
        assert (np.abs(gl - wl)[fin] <= 2.0 ** -10 + 2.0 ** -20 * np.abs(wl[fin])).all()


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page,H,counts,past,strided", [
    (16, 1, [1], [0], False),
    (64, 8, [1, 1, 1], [63, 64, 5], True),
    (32, 3, [7, 0, 33, 1], [30, 4, 0, 31], True),
    (128, 2, [130, 2], [1, 255], False),
])
def test_write_matches_bit_for_bit(dtype, D, G, page, H, counts, past, strided):
    lens = [p + n for p, n in zip(past, counts)]
    s = Setup(lens, H, D, G, page, seed=D + page)
    cu = offsets(counts)
    T, extra = int(cu[-1]), 3  # rows behind the last sequence: not read, and nothing is written for them
    k = s.rng.standard_normal((2, T + extra, H, D)).astype(np.float32)
    k[0, :, :, ::11] *= 8
    k[1, :, :, 1::2] += 40  # a group far from zero
    k[0, :, 0, :2] = 0
    x = torch.from_numpy(k).to(DT[dtype])
    x[:, T:] = float("nan")
    fused = torch.randn(T + extra, 3 * H, D, device="cuda").to(DT[dtype])
    kk, vv = x[0].cuda(), x[1].cuda()
    if strided:
        fused[:, :H], fused[:, 2 * H:] = kk, vv
        kk, vv = fused[:, :H], fused[:, 2 * H:]
    pool = s.cuda()
    bq.bq_kv4_write(kk, vv, pool, dev(s.table), dev(lens), G, cu_q=dev(cu))
    xf = x.float().numpy()
    for b in range(len(lens)):
        for j in range(counts[b]):
            s.host.put(*s.place(b, past[b] + j), xf[0, cu[b] + j], xf[1, cu[b] + j])
    assert np.array_equal(pool.cpu().numpy(), s.host.pool)
    # and read back the rows written, into rows that were there before
    for out in DT.values():
        ko = torch.full((T + extra, H, D), 7.0, dtype=out, device="cuda")
        vo = ko.clone()
        bq.bq_kv4_read(pool, dev(s.table), dev(cu), T + extra, D, G, starts=dev(past), k=ko, v=vo)
        for which, got in ((0, ko), (1, vo)):
            for b in range(len(lens)):
                want = ref.to_torch(s.host.values(which, s.table[b], lens[b], np.float32)[past[b]:], torch.float32)
                assert torch.equal(got[cu[b]:cu[b + 1]].cpu(), want.to(out))
            assert (got[T:] == 7).all()
    status_ok()


@pytest.mark.parametrize("dtype", DT)
def test_write_values_at_the_edges(dtype):
    """Ties and their neighbours, constant, huge, tiny and not finite groups."""
    D = G = 64
    rows = []
    base = np.zeros(64, dtype=np.float32)
    base[1] = 15
    for frac in (0.5, 0.5 + 2.0 ** -19, 0.5 - 2.0 ** -19, 0.25):
        x = base.copy()
        x[2:17] = np.arange(15) + frac
        rows += [x, x * 2.0 ** -12, -x, x + 1024, x * 3.7]
    for v in (0.0, 1.0, -1e-6, 65504.0, 7e4):
        rows.append(np.full(64, v, dtype=np.float32))
    rng = np.random.default_rng(3)
    for scale in (1e-8, 1e-6, 1e-3, 1e4, 1e6, 1e30, 3e38):
        rows.append((rng.uniform(-1, 1, 64) * scale).astype(np.float32))
    for bad in (np.inf, -np.inf, np.nan):
        x = rng.standard_normal(64).astype(np.float32)
        x[rng.integers(64)] = bad
        rows.append(x)
    for _ in range(200):  # values whose quotient by the step is a half, as near as the type can say
        x = rng.standard_normal(64).astype(np.float32)
        c, st, m = ref.quantize(ref.to_torch(x, DT[dtype]).float().numpy()[None], 64)
        y = m.astype(np.float64)[0, 0] + (rng.integers(0, 15, 64) + 0.5) * float(st[0, 0])
        y[:2] = x.min(), x.max()
        rows.append(y.astype(np.float32))
    x = ref.to_torch(np.stack(rows)[:, None], DT[dtype])
    T = len(rows)
    s = Setup([T], 1, D, G, 16)
    pool = s.cuda()
    bq.bq_kv4_write(x.cuda(), x.flip(0).cuda(), pool, dev(s.table), dev([T]), G)
    xf = x.float().numpy()
    for t in range(T):
        s.host.put(*s.place(0, t), xf[t], xf[T - 1 - t])
    got = s.host.__class__(s.host.pages, 1, D, G, 16, fill=pool.cpu().numpy())
    for which in (0, 1):
        (gc, gp), (wc, wp) = got._part(which), s.host._part(which)
        assert np.array_equal(gc, wc)
        assert np.array_equal(gp, wp, equal_nan=True)
    k, v = bq.bq_kv4_read(pool, dev(s.table), dev([0, T]), T, D, G, out_dtype=torch.float32)
    want = s.host.values(0, s.table[0], T, np.float32)
    assert np.array_equal(k.cpu().numpy(), want, equal_nan=True)


def test_rows_without_a_place_and_bad_pages():
    """A row before position 0 is not written; a table entry outside the pool is skipped and reported, and reads NaN."""
    s = Setup([40, 3, 0], 2, 64, 64, 16)
    pool = s.cuda()
    before = pool.clone()
    x = torch.randn(15, 2, 64, device="cuda")
    table = s.table.copy()
    table[0, 2] = s.host.pages  # positions 32..47 of sequence 0
    bq.bq_kv4_write(x, x, pool, dev(table), dev(s.lens), 64)  # five rows each; sequence 1 has three places, 2 none
    st, detail = bq.bq_device_status()
    assert st == bq.BQ_ERR_INVALID_ARG and detail >> 8 == 32
    for j in range(3):
        s.host.put(*s.place(1, j), x[7 + j].cpu().numpy(), x[7 + j].cpu().numpy())
    assert np.array_equal(pool.cpu().numpy(), s.host.pool)
    pool.copy_(before)
    for bad in (-1, s.host.pages, 2 ** 31 - 1, -2 ** 31):
        table[0, 2] = bad
        k, v = bq.bq_kv4_read(pool, dev(table), dev([0, 40, 43, 43]), 43, 64, 64, out_dtype=torch.float32)
        assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG
        assert k[32:40].isnan().all() and v[32:40].isnan().all()
    # behind the table, and before position 0
    k, v = bq.bq_kv4_read(pool, dev(s.table), dev([0, 1, 2, 2]), 2, 64, 64, starts=dev([10 ** 6, -1, 0]))
    assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG and k.isnan().all() and v.isnan().all()


# ------------------------------------------------------------------ attention
def run_attention(s, q, counts, scale=None, rows_behind=0, **kw):
    cu = offsets(counts)
    T = int(cu[-1])
    scale = s.D ** -0.5 if scale is None else scale
    uniform = len(set(counts)) == 1 and not rows_behind
    out = torch.full((T + rows_behind, q.shape[1], s.D), 3.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T + rows_behind, q.shape[1]), 3.0, device="cuda")
    slopes = kw.get("slopes")
    bq.bq_kv4_attention(q, s.cuda(), dev(s.table), dev(s.lens), s.G, cu_q=None if uniform else dev(cu),
                        max_q=None if uniform else max(max(counts), 1), scale=scale, window=kw.get("window", 0),
                        softcap=kw.get("softcap", 0.0), slopes=None if slopes is None else dev(slopes, torch.float32),
                        out=out, lse=lse)
    torch.cuda.synchronize()
    check_attention(s, out, lse, q, cu, scale, **kw)
    assert (out[T:] == 3).all() and (lse[T:] == 3).all()
    status_ok()
    return out


def query(s, T, Hq, dtype, scale=1.0):
    return (torch.from_numpy(s.rng.standard_normal((T, Hq, s.D))) * scale).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("page,H,share,lens", [
    (16, 2, 4, [1]),
    (64, 8, 4, [65, 0, 129]),
    (32, 1, 8, [777]),
    (128, 4, 1, [128, 127, 300]),
    (16, 2, 3, [15, 16, 17, 33, 500]),
    (64, 1, 16, [100, 64]),
    (64, 1, 71, [90]),
])
def test_one_new_token(dtype, D, G, page, H, share, lens):
    s = Setup(lens, H, D, G, page, seed=len(lens)).fill()
    run_attention(s, query(s, len(lens), H * share, dtype), [1] * len(lens))


@pytest.mark.parametrize("counts,past", [([5, 5], [100, 0]), ([2, 1, 0, 3], [31, 0, 7, 64]), ([17, 40], [200, 3]),
                                         ([130], [0]), ([64, 300, 1], [65, 10, 0]), ([3, 3], [-1, -3])])
@pytest.mark.parametrize("D,G,page,H,share,dtype", [(64, 64, 16, 2, 3, "f16"), (128, 64, 64, 1, 4, "bf16"),
                                                   (128, 128, 32, 2, 1, "f16"), (64, 64, 128, 1, 8, "bf16"),
                                                   (128, 128, 64, 1, 6, "bf16")])
def test_several_new_tokens(counts, past, D, G, page, H, share, dtype):
    lens = [max(p + n, 0) for p, n in zip(past, counts)]
    s = Setup(lens, H, D, G, page, seed=1).fill()
    behind = 4 if len(set(counts)) > 1 else 0
    run_attention(s, query(s, sum(counts) + behind, H * share, dtype), counts, rows_behind=behind)


@pytest.mark.parametrize("counts,past", [([1] * 3, [0, 150, 400]), ([70, 9], [40, 300])])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=16), dict(window=100), dict(softcap=5.0),
                                dict(slopes=1), dict(window=33, softcap=20.0, slopes=1), dict(scale=0.0),
                                dict(scale=-0.3)])
@pytest.mark.parametrize("D,G", SHAPES)
def test_masks_and_scores(counts, past, kw, D, G):
    s = Setup([p + n for p, n in zip(past, counts)], 2, D, G, 32, seed=2).fill()
    if "slopes" in kw:
        kw = dict(kw, slopes=2.0 ** -np.arange(1.0, 9.0))
    run_attention(s, query(s, sum(counts), 8, "bf16"), counts, **kw)


def test_long_sequences_are_split_and_joined():
    """Enough tokens for every SM, with ragged lengths and an empty slot among them."""
    s = Setup([9000, 1, 0, 2500], 1, 64, 64, 64, seed=4).fill()
    run_attention(s, query(s, 4, 2, "f16"), [1] * 4)
    run_attention(s, query(s, 4, 2, "f16", scale=40.0), [1] * 4)  # nearly all weight on one token
    run_attention(s, query(s, 4, 2, "bf16"), [1] * 4, window=4000)


@pytest.mark.parametrize("D,G", SHAPES)
@pytest.mark.parametrize("n", [1, 40])
def test_what_is_not_finite(D, G, n):
    """NaN tokens reach the rows that see them and no others; so do queries that are not finite; values of any size
    within fp16 do not overflow on the way."""
    s = Setup([200], 2, D, G, 16, seed=5).fill()
    q = query(s, n, 4, "bf16")
    if n > 1:
        q[3, 1, 5] = float("nan")
        q[4, 2, D - 1] = float("inf")
        q[5, 0, 0] = -float("inf")
        s.host.put(*s.place(0, 180), np.full((2, D), np.nan, np.float32), np.zeros((2, D), np.float32))
        s.host.put(*s.place(0, 190), np.zeros((2, D), np.float32), np.full((2, D), np.inf, np.float32))
        out = run_attention(s, q, [n])
        assert out[:20].isnan().sum() == 3 * D and out[20:].isnan().all()
        run_attention(s, q, [n], window=12)
    else:
        for big in (6e4, 1e-6, 2.0 ** -20):
            t = Setup([50], 2, D, G, 16, seed=6)
            for p in range(50):
                k, v = t.rng.standard_normal((2, 2, D)).astype(np.float32)
                t.host.put(*t.place(0, p), k, np.clip(v * big, -6.5e4, 6.5e4).astype(np.float32))
            run_attention(t, q, [1])
        # tokens whose value steps differ by orders of magnitude, and a constant one
        t = Setup([60], 2, D, G, 16, seed=7)
        for p in range(60):
            k, v = t.rng.standard_normal((2, 2, D)).astype(np.float32)
            t.host.put(*t.place(0, p), k, (v * 10.0 ** -(p % 5) if p % 7 else np.full_like(v, 2.5)).astype(np.float32))
        run_attention(t, q, [1])
        q[0, 1, 2] = float("nan")
        q[0, 3, 0] = float("inf")
        run_attention(s, q, [1])
        # queries of every size
        for scale in (1e-30, 1e-3, 1e4):
            run_attention(s, (query(s, 1, 4, "bf16").float() * scale).bfloat16(), [1])


def test_bad_pages_give_nan_and_are_reported():
    s = Setup([100, 70], 2, 128, 128, 16, seed=8).fill()
    good = s.table.copy()
    for n in (1, 30):
        q = query(s, 2 * n, 4, "bf16")
        for bad in (-5, s.host.pages):
            s.table = good.copy()
            want = run_attention(s, q, [n, n])
            s.table[0, 3] = bad
            out = bq.bq_kv4_attention(q, s.cuda(), dev(s.table), dev(s.lens), s.G)
            assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG
            assert out[:n].isnan().all() and torch.equal(out[n:], want[n:])
    # a sequence longer than its table
    out = bq.bq_kv4_attention(q, s.cuda(), dev(good), dev([10 ** 9, 70]), s.G, window=64)
    assert bq.bq_device_status()[0] == bq.BQ_ERR_INVALID_ARG and out[:30].isnan().all()


def test_queries_with_strides_and_a_pool_with_gaps():
    s = Setup([90, 33], 2, 64, 64, 16, seed=9).fill()
    fused = torch.randn(2, 12, 64, device="cuda").bfloat16()
    q = fused[:, 4:8]
    pool = torch.full((s.host.pages, 3, 2, s.host.pool.shape[2]), 0xFF, dtype=torch.uint8, device="cuda")
    pool[:, 1] = s.cuda()  # one layer of three
    out = bq.bq_kv4_attention(q, pool[:, 1], dev(s.table), dev(s.lens), 64)
    check_attention(s, out, None, q, [0, 1, 2], 64 ** -0.5)
    k, v = bq.bq_kv4_read(pool[:, 1], dev(s.table), dev([0, 90, 123]), 123, 64, 64, out_dtype=torch.float32)
    assert np.array_equal(k[:90].cpu().numpy(), s.host.values(0, s.table[0], 90, np.float32))
    status_ok()


def test_same_call_same_bits_on_any_stream():
    s = Setup([5000, 300, 4000], 2, 128, 64, 64, seed=10).fill()
    pool, table, lens = s.cuda(), dev(s.table), dev(s.lens)
    for n in (1, 3, 50):
        q = query(s, 3 * n, 8, "bf16")
        want = bq.bq_kv4_attention(q, pool, table, lens, s.G)
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            got = []
            for st in side:  # two calls at once, a workspace each
                with torch.cuda.stream(st):
                    got.append(bq.bq_kv4_attention(q, pool, table, lens, s.G))
            torch.cuda.synchronize()
            assert torch.equal(got[0], want) and torch.equal(got[1], want)
        got = bq.bq_kv4_attention(q, pool, table, lens, s.G, stream=side[0])
        side[0].synchronize()
        assert torch.equal(got, want)
    status_ok()


@pytest.mark.parametrize("D,G,page", [(128, 128, 64), (64, 64, 16)])
def test_prompt_then_captured_decoding(D, G, page):
    """As a decoder runs it: prompts written and attended to, then one token at a time from one captured graph whose
    lengths and rows change between replays."""
    H, Hq, prompts, steps = 2, 8, [70, 5, 33], 5
    s = Setup([n + steps for n in prompts], H, D, G, page, seed=11)
    pool, table = s.cuda(), dev(s.table)
    cu, T = offsets(prompts), sum(prompts)

    def rows(n):
        return [torch.from_numpy(s.rng.standard_normal((n, h, D)).astype(np.float32)).bfloat16().cuda() for h in (Hq, H, H)]

    def host_put(k, v, lens, cu):
        for b in range(len(lens)):
            for j in range(cu[b + 1] - cu[b]):
                t = cu[b] + j
                s.host.put(*s.place(b, lens[b] - (cu[b + 1] - cu[b]) + j), k[t].float().cpu().numpy(),
                           v[t].float().cpu().numpy())

    q, k, v = rows(T)
    bq.bq_kv4_write(k, v, pool, table, dev(prompts), G, cu_q=dev(cu))
    out = bq.bq_kv4_attention(q, pool, table, dev(prompts), G, cu_q=dev(cu), max_q=max(prompts))
    host_put(k, v, prompts, cu)
    s.lens = prompts
    check_attention(s, out, None, q, cu, D ** -0.5)

    q, k, v = rows(3)
    lens = dev(prompts)
    out = torch.empty_like(q)
    ws = torch.empty(bq.bq_kv4_attention_workspace_bytes(3, Hq, H, D), dtype=torch.uint8, device="cuda")

    def step():
        bq.bq_kv4_write(k, v, pool, table, lens, G)
        bq.bq_kv4_attention(q, pool, table, lens, G, out=out, workspace=ws)

    # (a warm-up before the capture, on a copy of what it changes)
    keep, pool = pool, pool.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    pool = keep
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # two captures that share a workspace, replayed in turn
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    one = offsets([1, 1, 1])
    for i in range(steps):
        s.lens = [n + i + 1 for n in prompts]
        for dst, src in zip((q, k, v), rows(3)):
            dst.copy_(src)
        lens.copy_(dev(s.lens))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        host_put(k, v, s.lens, one)
        assert np.array_equal(pool.cpu().numpy(), s.host.pool)
        check_attention(s, out, None, q, one, D ** -0.5)
    status_ok()


# ------------------------------------------------------------------ many rows: steps of every size, parts, head layouts
def steps_cache(kind, D, G, n, H=1, page=32, seed=12):
    """A sequence whose value groups differ in a way that the many-row kernel has to follow."""
    s = Setup([n], H, D, G, page, seed=seed)
    for p in range(n):
        k, v = s.rng.standard_normal((2, H, D)).astype(np.float32)
        if kind == "growing":  # each 50 tokens a hundred times larger, and their minima
            v = v * 10.0 ** (2 * (p // 50) - 4)
        elif kind == "shrinking":
            v = v * 10.0 ** (4 - 2 * (p // 50))
        elif kind == "mixed":  # orders of magnitude side by side, and constant groups
            v = v * 10.0 ** -(p % 5) if p % 7 else np.full_like(v, 2.5)
        elif kind == "zero":
            v = np.zeros_like(v)
        elif kind == "offset":  # far from zero: the minimum outweighs the step
            v = v * 0.01 + (40 if p % 2 else -3000)
        elif kind == "tiny":
            v = v * 2.0 ** -16
        s.host.put(*s.place(0, p), k, np.clip(v, -6.5e4, 6.5e4).astype(np.float32))
    return s


@pytest.mark.parametrize("kind", ["growing", "shrinking", "mixed", "zero", "offset", "tiny"])
@pytest.mark.parametrize("D,G", SHAPES)
def test_value_steps_of_every_size(kind, D, G):
    s = steps_cache(kind, D, G, 260)
    run_attention(s, query(s, 100, 2, "f16"), [100])
    run_attention(s, query(s, 100, 2, "bf16", scale=6.0), [100])  # few tokens carry most of the weight
    run_attention(s, query(s, 1, 2, "f16"), [1])


@pytest.mark.parametrize("D,G", SHAPES)
def test_weights_that_rise_late(D, G):
    """Scores that grow along the sequence, so that the running maximum is passed by a lot inside a tile and between tiles,
    with rows that begin to see tokens in the middle of one."""
    s = Setup([400], 1, D, G, 64, seed=13)
    for p in range(400):
        k, v = s.rng.standard_normal((2, 1, D)).astype(np.float32)
        s.host.put(*s.place(0, p), k + (p // 20) * 0.5, v)
    q = (torch.ones(90, 4, D) + 0.1 * torch.from_numpy(s.rng.standard_normal((90, 4, D)))).to(torch.bfloat16).cuda()
    for kw in (dict(), dict(window=70), dict(slopes=np.array([0.5, 0.1, 0.0, 2.0])), dict(softcap=30.0)):
        run_attention(s, q, [90], **kw)
        run_attention(s, q[:1], [1], **kw)


@pytest.mark.parametrize("share", [1, 3, 5, 12, 40, 300])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 64)])
def test_any_number_of_heads_to_a_key_head(share, D, G):
    """Rows and heads fill column blocks that begin and end inside a row, in one tile of rows or two."""
    s = Setup([75, 0, 40], 2, D, G, 16, seed=14).fill()
    counts = [9, 3, 30]
    run_attention(s, query(s, sum(counts) + 2, 2 * share, "bf16"), counts, rows_behind=2)


def test_items_cut_between_ctas():
    """Few columns and many tokens: every item is cut into parts, with column blocks of one tile of rows and of two."""
    s = Setup([3000, 130, 1700], 1, 64, 64, 128, seed=15).fill()
    for counts, Hq in (([40, 5, 90], 1), ([90, 0, 33], 4)):
        run_attention(s, query(s, sum(counts), Hq, "f16"), counts)
        run_attention(s, query(s, sum(counts), Hq, "bf16"), counts, window=1000, softcap=20.0)


def test_many_rows_captured_and_replayed():
    """One graph of a chunk, replayed with other lengths, offsets and pages; two graphs that share a workspace."""
    H, Hq, D, G, page = 2, 6, 128, 128, 32
    s = Setup([300, 200], H, D, G, page, seed=16).fill()
    pool, table, lens, cu = s.cuda(), dev(s.table), dev([300, 200]), dev([0, 60, 100])
    q = query(s, 100, Hq, "bf16")
    out = torch.full_like(q, 3.0)
    ws = torch.empty(bq.bq_kv4_attention_workspace_bytes(100, Hq, H, D), dtype=torch.uint8, device="cuda")

    def call():
        bq.bq_kv4_attention(q, pool, table, lens, G, cu_q=cu, max_q=100, out=out, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for i, (ln, off) in enumerate(([[300, 200], [0, 60, 100]], [[100, 64], [0, 1, 41]], [[31, 0], [0, 31, 31]],
                                   [[299, 200], [0, 0, 100]])):
        s.lens = ln
        lens.copy_(dev(ln))
        cu.copy_(dev(off))
        out.fill_(3.0)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        check_attention(s, out, None, q, off, D ** -0.5)
        assert (out[off[-1]:] == 3).all()
    status_ok()


def test_wrappers_refuse_what_is_not_on_the_device():
    s = Setup([20], 2, 64, 64, 16, seed=17).fill()
    pool, table, lens = s.cuda(), dev(s.table), dev(s.lens)
    q = query(s, 1, 4, "bf16")
    kv = torch.randn(1, 2, 64, device="cuda").bfloat16()
    for bad in (dict(q=q.cpu()), dict(q=q.float().double()), dict(table=table.cpu()), dict(table=table.long()),
                dict(lens=lens.cpu()), dict(pool=pool.cpu()), dict(pool=pool[..., :-1])):
        a = dict(q=q, pool=pool, table=table, lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            bq.bq_kv4_attention(a["q"], a["pool"], a["table"], a["lens"], 64)
        if "q" not in bad:
            with pytest.raises(ValueError):
                bq.bq_kv4_write(kv, kv, a["pool"], a["table"], a["lens"], 64)
    with pytest.raises(ValueError):
        bq.bq_kv4_write(kv, kv.cpu(), pool, table, lens, 64)
    with pytest.raises(ValueError):
        bq.bq_kv4_read(pool, table, dev([0, 20]).cpu(), 20, 64, 64)
    status_ok()

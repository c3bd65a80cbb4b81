"""The 4-bit key/value cache without a GPU: sizes, refusals, and the pins of the 64-bit yardstick."""
import numpy as np
import pytest
import torch

import bit_quantized_linear_rmsnorm_b200 as bq
import kv4_reference as ref
from bit_quantized_linear_rmsnorm_b200 import _build

FAKE = 0x10000  # 64 KiB-aligned, never dereferenced
ODD = 0x10001


@pytest.fixture(scope="module")
def L():
    _build.build()
    return bq.lib()


def test_page_bytes(L):
    assert bq.bq_kv4_page_bytes(64, 128, 128) == 64 * 136
    assert bq.bq_kv4_page_bytes(16, 128, 64) == 16 * 144
    assert bq.bq_kv4_page_bytes(128, 64, 64) == 128 * 72
    for bad in ((0, 64, 64), (8, 64, 64), (48, 64, 64), (256, 64, 64), (64, 80, 64), (64, 64, 128), (64, 128, 32),
                (64, 256, 64), (-16, 64, 64)):
        assert bq.bq_kv4_page_bytes(*bad) == 0
    for sizes in ((64, 128, 128), (16, 128, 64), (32, 64, 64)):
        assert bq.bq_kv4_page_bytes(*sizes) == ref.page_bytes(*sizes) and bq.bq_kv4_page_bytes(*sizes) % 16 == 0


SHARED = dict(total=8, H=2, D=128, G=64, page=16, batch=4, ld=5, width=5, pages=7, pool=FAKE, table=FAKE)
SHARED["stride"] = 2 * 16 * 144
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = (bq.BQ_ERR_INVALID_ARG, bq.BQ_ERR_UNSUPPORTED, bq.BQ_ERR_MISALIGNED,
                                               bq.BQ_ERR_WORKSPACE)


def write(L, **kw):
    a = dict(SHARED, k=FAKE, v=FAKE, dt=bq.BQ_BF16, kt=256, kh=128, vt=256, vh=128, cu=None, lens=FAKE)
    a.update(kw)
    return L.bq_kv4_write(a["k"], a["v"], a["dt"], a["total"], a["H"], a["D"], a["kt"], a["kh"], a["vt"], a["vh"],
                          a["cu"], a["lens"], a["batch"], a["table"], a["ld"], a["width"], a["pool"], a["pages"],
                          a["stride"], a["page"], a["G"], None)


def read(L, **kw):
    a = dict(SHARED, k=FAKE, v=FAKE, dt=bq.BQ_BF16, starts=None, cu=FAKE)
    a.update(kw)
    return L.bq_kv4_read(a["pool"], a["pages"], a["stride"], a["page"], a["H"], a["D"], a["G"], a["table"], a["ld"],
                         a["width"], a["starts"], a["cu"], a["batch"], a["total"], a["dt"], a["k"], a["v"], None)


def attend(L, **kw):
    a = dict(SHARED, q=FAKE, dt=bq.BQ_BF16, Hq=4, qt=512, qh=128, cu=None, maxq=8, lens=FAKE, scale=0.1, window=0,
             cap=0.0, slopes=None, out=FAKE, lse=None, ws=FAKE, nws=1 << 40)
    a.update(kw)
    return L.bq_kv4_attention(a["q"], a["dt"], a["total"], a["Hq"], a["D"], a["qt"], a["qh"], a["cu"], a["maxq"],
                              a["lens"], a["batch"], a["table"], a["ld"], a["width"], a["pool"], a["pages"],
                              a["stride"], a["page"], a["H"], a["G"], a["scale"], a["window"], a["cap"], a["slopes"],
                              a["out"], a["lse"], a["ws"], a["nws"], None)



@pytest.mark.parametrize("call", [write, read, attend])
def test_shared_refusals(L, call):
    for kw in (dict(total=-1), dict(batch=-1), dict(pages=-1), dict(H=0), dict(width=-1), dict(ld=4), dict(D=0),
               dict(G=0), dict(page=0), dict(dt=3), dict(dt=-1), dict(stride=2 * 16 * 144 - 16), dict(pool=None),
               dict(table=None)):
        assert call(L, **kw) == INVALID, kw
    for kw in (dict(D=80), dict(D=256), dict(G=32), dict(G=128, D=64), dict(page=8), dict(page=24), dict(page=256),
               dict(H=1 << 20, Hq=1 << 20, stride=1 << 40), dict(total=1 << 31), dict(pages=1 << 31)):
        assert call(L, **kw) == UNSUPPORTED, kw
    for kw in (dict(pool=FAKE + 8), dict(table=FAKE + 2), dict(stride=2 * 16 * 144 + 8)):
        assert call(L, **kw) == MISALIGNED, kw
    assert call(L, total=0, cu=None) == bq.BQ_OK
    assert call(L, batch=0, cu=None) == bq.BQ_OK


def test_write_refusals(L):
    for kw in (dict(k=None), dict(v=None), dict(lens=None), dict(kt=-256), dict(vh=-128), dict(total=9)):
        assert write(L, **kw) == INVALID, kw
    for kw in (dict(k=ODD), dict(v=FAKE + 8), dict(kt=260), dict(vh=130), dict(cu=ODD), dict(lens=FAKE + 2),
               dict(dt=bq.BQ_F32, kt=258)):
        assert write(L, **kw) == MISALIGNED, kw


def test_read_refusals(L):
    for kw in (dict(k=None), dict(v=None), dict(cu=None)):
        assert read(L, **kw) == INVALID, kw
    for kw in (dict(k=ODD), dict(v=FAKE + 8), dict(cu=FAKE + 2), dict(starts=FAKE + 1)):
        assert read(L, **kw) == MISALIGNED, kw


def test_attention_refusals(L):
    for kw in (dict(q=None), dict(out=None), dict(lens=None), dict(Hq=0), dict(Hq=5), dict(qt=-8), dict(qh=-8),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
               dict(window=-1), dict(total=9), dict(cu=FAKE, maxq=0)):
        assert attend(L, **kw) == INVALID, kw
    assert attend(L, dt=bq.BQ_F32) == UNSUPPORTED
    for kw in (dict(q=ODD), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(qt=516), dict(qh=132), dict(slopes=FAKE + 2),
               dict(lse=FAKE + 1), dict(ws=FAKE + 16)):
        assert attend(L, **kw) == MISALIGNED, kw
    need = bq.bq_kv4_attention_workspace_bytes(8, 4, 2, 128)
    for kw in (dict(ws=None), dict(nws=need - 1)):
        assert attend(L, **kw) == WORKSPACE, kw
    assert bq.bq_kv4_attention_workspace_bytes(-1, 4, 2, 128) == 0
    assert bq.bq_kv4_attention_workspace_bytes(8, 4, 0, 128) == 0


def test_binding_refuses_what_does_not_fit():
    cache = torch.zeros(3, 2, ref.page_bytes(16, 64, 64), dtype=torch.uint8)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    k = torch.zeros(2, 2, 64)
    bad = [
        lambda: bq.bq_kv4_write(k, k[:, :1], cache, table, lens, 64),
        lambda: bq.bq_kv4_write(k, k.half(), cache, table, lens, 64),
        lambda: bq.bq_kv4_write(k[:, :1], k[:, :1], cache, table, lens, 64),
        lambda: bq.bq_kv4_write(k.double(), k.double(), cache, table, lens, 64),
        lambda: bq.bq_kv4_write(k, k, cache.int(), table, lens, 64),
        lambda: bq.bq_kv4_write(k, k, cache[:, :, :-8], table, lens, 64),
        lambda: bq.bq_kv4_write(k, k, cache, table.long(), lens, 64),
        lambda: bq.bq_kv4_write(k, k, cache, table, lens[:1], 64),
        lambda: bq.bq_kv4_write(k, k, cache, table, lens, 64, cu_q=lens),
        lambda: bq.bq_kv4_write(k, k, cache, table, lens, 48),
        lambda: bq.bq_kv4_read(cache, table, lens, 2, 64, 64),
        lambda: bq.bq_kv4_read(cache, table, torch.zeros(3, dtype=torch.int32), 2, 64, 64, k=k.double()),
        lambda: bq.bq_kv4_attention(k[0], cache, table, lens, 64),
        lambda: bq.bq_kv4_attention(k.bfloat16(), cache, table, lens, 64, out=k),
        lambda: bq.bq_kv4_attention(k.bfloat16(), cache, table, lens, 64, slopes=torch.zeros(3)),
        lambda: bq.bq_kv4_attention(k.bfloat16(), cache, table, lens, 64, lse=torch.zeros(2, 3)),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


class OnDevice(torch.Tensor):
    """A host tensor that says it is on GPU 0, for what the binding does before the library's call."""

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


def test_allocations_follow_the_stream(monkeypatch):
    """Outputs and workspace that a call allocates belong to the stream that it launches on: two calls on two streams
    never share one, and none is handed out again before the call's kernels have run."""
    import contextlib

    class Stream:
        cuda_stream = 0

        def __init__(self, name):
            self.name = name

    now, made, given = ["current"], [], []
    empty = torch.empty

    @contextlib.contextmanager
    def enter(stream):
        now.append(stream.name)
        yield
        now.pop()

    def watched(*args, **kw):
        t = empty(*args, **kw)
        made.append((now[-1], t))
        return on_device(t)

    def call(dev, fn, stream, *args):
        given.append(None if stream is None else stream.name)
        return bq.BQ_OK

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch, "empty", watched)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: watched(t.shape, dtype=t.dtype, device=t.device))
    monkeypatch.setattr(bq, "_kv4_call", call)
    cache = on_device(torch.zeros(3, 2, ref.page_bytes(16, 64, 64), dtype=torch.uint8))
    table, lens = (on_device(torch.ones(s, dtype=torch.int32)) for s in ((2, 1), (2,)))
    cu = on_device(torch.tensor([0, 1, 2], dtype=torch.int32))
    q = on_device(torch.zeros(2, 4, 64).bfloat16())
    for stream, name in ((None, "current"), (Stream("a"), "a"), (Stream("b"), "b")):
        for fn, count in ((lambda: bq.bq_kv4_attention(q, cache, table, lens, 64, stream=stream), 2),
                          (lambda: bq.bq_kv4_read(cache, table, cu, 2, 64, 64, stream=stream), 2)):
            del made[:], given[:]
            fn()
            assert [m[0] for m in made] == [name] * count and given == [stream and name]


def test_binding_refuses_empty_heads_and_single_numbers():
    """No head of 0 elements, no table that is a single number, no stream of another device: a ValueError each."""
    class Elsewhere:
        cuda_stream, device_index = 0, 1

    nbytes = ref.page_bytes(16, 64, 64)
    cache = on_device(torch.zeros(3, 2, nbytes, dtype=torch.uint8))
    table, lens = (on_device(torch.ones(s, dtype=torch.int32)) for s in ((2, 1), (2,)))
    cu = on_device(torch.tensor([0, 1, 2], dtype=torch.int32))
    single = on_device(torch.tensor(1, dtype=torch.int32))
    q, none = (on_device(torch.zeros(s).bfloat16()) for s in ((2, 2, 64), (2, 2, 0)))
    bad = [
        lambda: bq.bq_kv4_write(none, none, cache, table, lens, 64),
        lambda: bq.bq_kv4_attention(none, cache, table, lens, 64),
        lambda: bq.bq_kv4_read(cache, table, cu, 2, 0, 64),
        lambda: bq.bq_kv4_read(cache, table, cu, 2, -64, 64),
        lambda: bq.bq_kv4_write(q, q, cache, single, lens, 64),
        lambda: bq.bq_kv4_write(q, q, cache, table, single, 64),
        lambda: bq.bq_kv4_attention(q, cache, table, single, 64),
        lambda: bq.bq_kv4_attention(q, cache, table, lens, 64, cu_q=single),
        lambda: bq.bq_kv4_read(cache, table, single, 2, 64, 64),
        lambda: bq.bq_kv4_read(cache, table, cu, 2, 64, 64, starts=single),
        lambda: bq.bq_kv4_write(q, q, cache, table, lens, 64, stream=Elsewhere()),
        lambda: bq.bq_kv4_read(cache, table, cu, 2, 64, 64, k=q, v=q, stream=Elsewhere()),
        lambda: bq.bq_kv4_attention(q, cache, table, lens, 64, out=q, workspace=q, stream=Elsewhere()),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------------------ pins of the yardstick
def test_quantize_by_hand():
    # minimum 0, maximum 15: step 1, so a value is its own code and k + 1/2 goes to the even neighbour
    x = np.zeros(64, dtype=np.float32)
    x[:8] = [0, 15, 0.5, 1.5, 2.5, 14.5, 7.49, 7.51]
    c, s, m = ref.quantize(x[None], 64)
    assert c[0, :8].tolist() == [0, 15, 0, 2, 2, 14, 7, 8] and s[0, 0] == 1 and m[0, 0] == 0
    # a constant group: step 0, the minimum stands for all
    c, s, m = ref.quantize(np.full((1, 64), -3.25, dtype=np.float32), 64)
    assert not c.any() and s[0, 0] == 0 and m[0, 0] == -3.25
    # one infinity or NaN, or a range beyond fp32, and the group is NaN; its neighbour is not
    for bad in (np.inf, -np.inf, np.nan, 3e38):
        x = np.zeros((1, 128), dtype=np.float32)
        x[0, 3], x[0, 4] = bad, -3e38 if bad == 3e38 else 0
        c, s, m = ref.quantize(x, 64)
        assert np.isnan(s[0, 0]) and np.isnan(m[0, 0]) and not c[0, :64].any() and s[0, 1] == 0 and m[0, 1] == 0
    # values beyond fp16 saturate
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :2] = [-1e6, 3e6]
    c, s, m = ref.quantize(x, 64)
    assert m[0, 0] == -65504 and s[0, 0] == 65504 and c[0, 0] == 0 and c[0, 1] == 15 and c[0, 2] == 1


def test_layout_and_round_trip():
    rng = np.random.default_rng(0)
    for D, G, page in ((64, 64, 16), (128, 64, 32), (128, 128, 64)):
        c = ref.Cache(3, 2, D, G, page)
        k, v = rng.standard_normal((2, 2, D)).astype(np.float32)
        c.put(2, 5, k, v)
        codes, s, m = ref.quantize(k, G)
        block = c.pool[2, 1]
        assert block[5 * D // 2] == codes[1, 0] | codes[1, 1] << 4
        par = block[page * D // 2:][5 * 4 * (D // G):][:4].view(np.float16)
        assert par[0] == s[1, 0] and par[1] == m[1, 0]
        got = c.values(0, [2], 6)[5]
        assert np.abs(got - k).max() <= 0.51 * float(s.max()) and np.abs(c.values(1, [2], 6)[5] - v).max() < 0.3
        assert not c.pool[[0, 1]].any() and np.count_nonzero(c.values(0, [2], 5)) == 0


def test_attention_against_torch():
    rng = np.random.default_rng(1)
    c = ref.Cache(4, 2, 64, 64, 16)
    table = [[3, 1], [0, 2]]
    for b in range(2):
        for t in range(20):
            c.put(table[b][t // 16], t % 16, *rng.standard_normal((2, 2, 64)).astype(np.float32))
    q = rng.standard_normal((5, 4, 64))
    out, lse, tol = ref.attention(q, c, table, [20, 0], [0, 4, 5], 0.125)
    k, v = (torch.from_numpy(c.values(i, table[0], 20)).permute(1, 0, 2).repeat_interleave(2, 0) for i in (0, 1))
    mask = torch.ones(4, 20, dtype=torch.bool).tril(16)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[:4]).permute(1, 0, 2), k, v, mask)
    assert np.abs(out[:4] - want.permute(1, 0, 2).numpy()).max() < 1e-12
    assert not out[4].any() and np.isinf(lse[4]).all() and np.isfinite(lse[:4]).all()
    assert (tol[:4] > 0).all() and tol.max() < 2.0 ** -10 * v.abs().max()
    win = ref.attention(q, c, table, [20, 0], [0, 4, 5], 0.125, window=1)[0]
    assert np.abs(win[3] - c.values(1, table[0], 20)[19].repeat(2, axis=0)).max() < 1e-12

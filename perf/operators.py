"""Cases of the 4-bit key/value cache: writing it, reading it back, and the attention that reads it.

The cache is a pool of pages, uint8 [pages, kv heads, page_bytes].  The block of one page and head holds, for `page` tokens,
key codes (two per byte, low nibble first along the head), key parameters (float16 step and minimum for each group of the head),
then value codes and value parameters.  A stored value stands for step * code + minimum.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    d = {"q_heads": 32, "kv_heads": 8, "dim": 128, "group": 128, "page": 64, "dtype": "bf16", "ragged": False,
         "window": 0, "cap": 0.0, "slopes": False, "strided": False, "past": 0, "new": 1, "batch": 1}
    return [
        # one user's next token after a short conversation: nothing but latency
        dict(d, name="decode_1x778", kind="attend", past=777),
        # one user's next token in a long document: the whole card on one sequence
        dict(d, name="decode_1x131072", kind="attend", past=131071),
        # a serving batch, every sequence at its own length, one padded slot
        dict(d, name="decode_64_ragged", kind="attend", batch=64, past=8191, ragged=True),
        # no shared heads, small pages, finer groups, float16
        dict(d, name="decode_mha_16x4096", kind="attend", batch=16, kv_heads=32, group=64, page=16, past=4095, dtype="f16"),
        # small heads, eight queries to a key head, a sliding window and capped scores
        dict(d, name="decode_window_cap", kind="attend", batch=33, q_heads=16, kv_heads=2, dim=64, group=64, page=32, past=5000,
             ragged=True, window=1024, cap=30.0),
        # five drafted tokens verified at once for each sequence
        dict(d, name="verify_32x5", kind="attend", batch=32, new=5, past=2500, ragged=True),
        # a prompt's next chunk after what is cached of it
        dict(d, name="chunk_2048_after_8192", kind="attend", new=2048, past=8192),
        # whole prompts of different lengths, distance bias
        dict(d, name="prompts_8_ragged", kind="attend", batch=8, q_heads=24, kv_heads=8, dim=64, group=64, page=128, new=1500,
             ragged=True, dtype="f16", slopes=True),
        # two prompts' keys and values stored, and read back as a 16-bit prefill would take them
        dict(d, name="write_2x4096", kind="write", batch=2, new=4096),
        # one decoded token of each sequence, keys and values being slices of the fused projection's output
        dict(d, name="write_64x1_strided", kind="write", batch=64, new=1, past=2000, ragged=True, strided=True),
        # a long cached prefix handed to code that takes 16-bit keys and values
        dict(d, name="read_1x65537", kind="read", past=65537, new=0),
        # a few short sequences read in 32 bits
        dict(d, name="read_3_ragged_f32", kind="read", batch=3, past=200, new=0, dim=64, group=64, page=16, ragged=True, dtype="f32"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "write", "read"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32])
    c = {"kind": kind, "dim": dim, "group": rng.choice([64, dim]), "page": rng.choice([16, 32, 64, 64, 128]), "kv_heads": kv_heads,
         "q_heads": kv_heads * rng.choice([1, 2, 3, 4, 4, 6, 8, 8][: 8 if kv_heads < 16 else 2]), "ragged": rng.random() < 0.7,
         "window": 0, "cap": 0.0, "slopes": False, "strided": rng.random() < 0.5, "past": 0, "new": 1, "batch": _log(rng, 1, 64)}
    if kind == "attend":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16"])
        c["past"] = _log(rng, 1, 131072) - 1
        c["new"] = rng.choice([1, 1, 1, rng.randint(2, 16), _log(rng, 16, 2048)])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        c["cap"] = rng.choice([0.0, 0.0, 0.0, 20.0, 50.0])
        c["slopes"] = rng.random() < 0.2
        while c["batch"] * (c["past"] + c["new"]) * kv_heads * dim > 1 << 28:
            c["past"], c["batch"] = c["past"] // 2, max(1, c["batch"] // 2)
        while c["batch"] * c["new"] * (c["past"] + c["new"]) * c["q_heads"] * dim > 1 << 36:
            c["new"] = max(1, c["new"] // 2)
    elif kind == "write":
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["past"] = _log(rng, 1, 4096) - 1
        c["new"] = rng.choice([1, _log(rng, 1, 4096)])
        while c["batch"] * c["new"] * kv_heads * dim > 1 << 24:
            c["batch"], c["new"] = max(1, c["batch"] // 2), (c["new"] + 1) // 2
    else:
        c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f32"])
        c["past"], c["new"] = _log(rng, 1, 65536), 0
        while c["batch"] * c["past"] * kv_heads * dim > 1 << 26:
            c["batch"], c["past"] = max(1, c["batch"] // 2), max(1, c["past"] // 2)
    return c


def _lengths(c):
    """(tokens after the call, new tokens) of each sequence: the case says them, the seed does not."""
    r = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    past, new = [c["past"]] * c["batch"], [c["new"]] * c["batch"]
    if c["ragged"]:
        past = [c["past"]] + [r.randint(c["past"] // 8, c["past"]) for _ in range(c["batch"] - 1)]
        if c["new"] > 5:
            new = [c["new"]] + [r.randint(1, c["new"]) for _ in range(c["batch"] - 1)]
    lens = [p + n for p, n in zip(past, new)]
    if c["ragged"] and c["kind"] == "attend" and c["new"] == 1 and c["batch"] >= 8:
        lens[-1] = 0  # a slot of the batch that no sequence holds
    return lens, new


def _page_bytes(c):
    return c["page"] * (c["dim"] + 8 * c["dim"] // c["group"])


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _lengths(c)
    H, D, page = c["kv_heads"], c["dim"], c["page"]
    need = [(n + page - 1) // page for n in lens]
    width = max(1, max(need))
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32)
    host, at = order.cpu(), 0
    for b, n in enumerate(need):
        table[b, :n] = host[at:at + n]
        at += n
    cu = [0]
    for n in (new if c["kind"] != "read" else lens):
        cu.append(cu[-1] + n)
    s = {"case": c, "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "total": cu[-1],
         "cu": torch.tensor(cu, dtype=torch.int32, device=dev),
         "starts": torch.tensor([n - q for n, q in zip(lens, new)], dtype=torch.int32, device=dev),
         "uniform": c["kind"] != "read" and len(set(new)) == 1, "max_new": max(new)}
    # channels of unequal size, as keys have them
    loud = 1.0 + 3.0 * (torch.rand(H, D, generator=g, device=dev) < 0.05).float()
    rows = page * max(1, (1 << 25) // (H * D * page))
    pool = torch.empty((pages, H, _page_bytes(c)), dtype=torch.uint8, device=dev)
    everywhere = torch.arange(pages * page, device=dev)
    for i in range(0, pages * page, rows):  # the cache as it was written token by token
        where = everywhere[i:i + rows]
        k = torch.randn(len(where), H, D, generator=g, device=dev) * loud
        v = torch.randn(len(where), H, D, generator=g, device=dev)
        _store(pool, c, where // page, where % page, k, v)
    s["pool"] = pool
    dt = _DTYPES[c["dtype"]]
    if c["kind"] == "attend":
        s["q"] = torch.randn(cu[-1], c["q_heads"], D, generator=g, device=dev).to(dt)
        s["slopes"] = None
        if c["slopes"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, c["q_heads"] + 1, device=dev, dtype=torch.float32) / c["q_heads"])
    elif c["kind"] == "write":
        k = (torch.randn(cu[-1], H, D, generator=g, device=dev) * loud).to(dt)
        v = torch.randn(cu[-1], H, D, generator=g, device=dev).to(dt)
        if c["strided"]:  # query, key and value heads side by side, as a fused projection leaves them
            fused = torch.zeros(cu[-1], c["q_heads"] + 2 * H, D, device=dev, dtype=dt)
            fused[:, c["q_heads"]:-H], fused[:, -H:] = k, v
            k, v = fused[:, c["q_heads"]:-H], fused[:, -H:]
        s["k"], s["v"] = k, v
    return s


def _quantise(x, c):
    """Codes, steps and minima of x [rows, heads, dim]."""
    x = x.float().unflatten(-1, (-1, c["group"]))
    low, high = x.amin(-1), x.amax(-1)
    bad = ~torch.isfinite(high - low)
    minimum = low.clamp(-65504.0, 65504.0).half()
    step = ((high - minimum.float()).clamp_min(0).double() / 15.0).float().clamp_max(65504.0).half()
    # the quotient in 64 bits: a code next to a border has to fall on its own side
    at = (x.double() - minimum.double()[..., None]) / step.double()[..., None]
    codes = torch.where((step > 0)[..., None], at.round().clamp(0, 15), 0.0)
    codes = torch.where(bad[..., None], 0.0, codes).to(torch.uint8).flatten(-2)
    nan = torch.full_like(step, float("nan"))
    return codes, torch.where(bad, nan, step), torch.where(bad, nan, minimum)


def _regions(pool, c):
    """The four parts of the pool: key codes, key parameters, value codes, value parameters."""
    page, half, params = c["page"], c["dim"] // 2, 4 * c["dim"] // c["group"]
    a, b = page * half, page * (half + params)
    part = lambda lo, hi, t: pool[..., lo:hi].view(t).unflatten(-1, (page, -1))  # noqa: E731
    return (part(0, a, torch.uint8), part(a, b, torch.float16), part(b, b + a, torch.uint8), part(b + a, 2 * b, torch.float16))


def _store(pool, c, pages, slots, k, v):
    kc, kp, vc, vp = _regions(pool, c)
    ck, sk, mk = _quantise(k, c)
    cv, sv, mv = _quantise(v, c)
    kc[pages, :, slots] = ck[..., 0::2] | (ck[..., 1::2] << 4)
    vc[pages, :, slots] = cv[..., 0::2] | (cv[..., 1::2] << 4)
    kp[pages, :, slots] = torch.stack((sk, mk), -1).flatten(-2)
    vp[pages, :, slots] = torch.stack((sv, mv), -1).flatten(-2)


def _values(codes, params, c):
    codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (-1, c["group"])).float()
    params = params.float().unflatten(-1, (-1, 2))
    return (codes * params[..., :1] + params[..., 1:]).flatten(-2)


def _rows_of(cu, total):
    """(sequence, place in it) of each of `total` rows."""
    row = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    return b, row - cu[b]


def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["kind"] == "attend":
        return _attend(state, c)
    if c["kind"] == "write":
        b, j = _rows_of(state["cu"], state["total"])
        at = state["lens"][b] - (state["cu"][b + 1] - state["cu"][b]) + j
        pages = state["table"][b, at // c["page"]].long()
        _store(state["pool"], c, pages, at % c["page"], state["k"], state["v"])
    else:
        b, at = _rows_of(state["cu"], state["total"])
        pages = state["table"][b, at // c["page"]].long()
    kc, kp, vc, vp = _regions(state["pool"], c)
    slots = at % c["page"]
    dt = _DTYPES[c["dtype"]]
    return _values(kc[pages, :, slots], kp[pages, :, slots], c).to(dt), _values(vc[pages, :, slots], vp[pages, :, slots], c).to(dt)


def _attend(state, c):
    B, H, D, n = c["batch"], c["kv_heads"], c["dim"], state["max_new"]
    lens, cu, table = state["lens"].long(), state["cu"].long(), state["table"].long()
    kc, kp, vc, vp = (x[table].transpose(1, 2).flatten(2, 3) for x in _regions(state["pool"], c))  # [B, H, tokens, ...]
    new = cu[1:] - cu[:-1]
    j = torch.arange(n, device=cu.device)
    q = state["q"].float()[(cu[:-1, None] + j).clamp_max(state["total"] - 1)]  # [B, n, q heads, D]
    q = q.unflatten(2, (H, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, H, heads of the group * n, D]
    scores = (q @ _values(kc, kp, c).transpose(-1, -2)) * D ** -0.5
    scores = scores.unflatten(2, (-1, n))  # [B, H, heads of the group, n, tokens]
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    t = torch.arange(scores.shape[-1], device=cu.device)
    at = (lens - new)[:, None] + j  # [B, n]
    away = (t - at[..., None])[:, None, None]
    if c["slopes"]:
        scores = scores + state["slopes"].view(1, H, -1, 1, 1) * away.float()
    seen = (away <= 0) & (away > -(c["window"] or 1 << 40))
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ _values(vc, vp, c)).unflatten(2, (-1, n)) / torch.where(total == 0, 1.0, total)
    b, i = _rows_of(state["cu"], state["total"])
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i].to(state["q"].dtype)


def _run_own(state, c):
    import bit_quantized_linear_rmsnorm_b200 as bq
    cu = None if state["uniform"] else state["cu"]
    if c["kind"] == "attend":
        return bq.bq_kv4_attention(state["q"], state["pool"], state["table"], state["lens"], c["group"], cu_q=cu,
                                   max_q=state["max_new"], window=c["window"], softcap=c["cap"], slopes=state["slopes"])
    if c["kind"] == "read":
        return bq.bq_kv4_read(state["pool"], state["table"], state["cu"], state["total"], c["dim"], c["group"],
                              out_dtype=_DTYPES[c["dtype"]])
    bq.bq_kv4_write(state["k"], state["v"], state["pool"], state["table"], state["lens"], c["group"], cu_q=cu)
    return bq.bq_kv4_read(state["pool"], state["table"], state["cu"], state["total"], c["dim"], c["group"],
                          starts=state["starts"], out_dtype=_DTYPES[c["dtype"]])


def work(case):
    c = case
    lens, new = _lengths(c)
    token = c["kv_heads"] * (c["dim"] + 8 * c["dim"] // c["group"])  # bytes of one token's keys and values in the cache
    size = 4 if c["dtype"] == "f32" else 2
    if c["kind"] == "read":
        n = sum(lens)
        return {"bytes": n * token + n * c["kv_heads"] * c["dim"] * 2 * size, "flops": n * c["kv_heads"] * c["dim"] * 4}
    if c["kind"] == "write":
        n = sum(new)
        return {"bytes": 2 * n * token + n * c["kv_heads"] * c["dim"] * 4 * size, "flops": n * c["kv_heads"] * c["dim"] * 16}
    window = c["window"] or 1 << 40
    read = pairs = 0
    for n, q in zip(lens, new):
        first = n - q  # the place of the first new token
        read += n - max(0, first - window + 1) if n else 0
        # sum over the new tokens of min(place + 1, window)
        short = max(0, min(n, window) - max(first, 0))
        pairs += (2 * first + short + 1) * short // 2 + (q - short) * window if n else 0
    return {"bytes": read * token + sum(new) * c["q_heads"] * c["dim"] * 2 * size,
            "flops": 4 * pairs * c["q_heads"] * c["dim"]}


def _stored(block, lo, c):
    """[heads, tokens, dim] in 64 bits from pages [pages, heads, bytes], the part that begins at byte `lo` of a block."""
    P, H = block.shape[:2]
    half, groups = c["dim"] // 2, c["dim"] // c["group"]
    mid, hi = lo + c["page"] * half, lo + c["page"] * (half + 4 * groups)
    byte = block[:, :, lo:mid].reshape(P, H, c["page"], half).to(torch.int64)
    both = torch.empty(P, H, c["page"], half, 2, dtype=torch.float64, device=block.device)
    both[..., 0], both[..., 1] = (byte % 16).double(), (byte // 16).double()
    par = block[:, :, mid:hi].contiguous().view(torch.float16).reshape(P, H, c["page"], groups, 1, 2).double()
    x = both.reshape(P, H, c["page"], groups, c["group"]) * par[..., 0] + par[..., 1]
    return x.reshape(P, H, c["page"], c["dim"]).permute(1, 0, 2, 3).reshape(H, P * c["page"], c["dim"])


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens, new = _lengths(c)
    half = _page_bytes(c) // 2
    if c["kind"] == "write":
        found = []
        for x in (s["k"], s["v"]):
            x = x.double().reshape(-1, c["group"])
            low = x.min(1, keepdim=True).values
            m = low.float().half().double()
            # the step as it is stored: the range over 15 in 32 bits, then float16
            step = ((x.max(1, keepdim=True).values.float() - m.float()).double() / 15).float().half().double()
            code = torch.round((x - m) / step.clamp_min(1e-300)).clamp(0, 15) * (step > 0)
            found.append((code * step + m).reshape(s["k"].shape))
        return tuple(found)
    outs, at = [], 0
    for b, (n, q) in enumerate(zip(lens, new)):
        block = s["pool"][s["table"][b, :(n + c["page"] - 1) // c["page"]].long()]
        if c["kind"] == "read":
            outs.append(tuple(_stored(block, lo, c)[:, :n].transpose(0, 1) for lo in (0, half)))
            continue
        out = torch.zeros(q, c["q_heads"], c["dim"], dtype=torch.float64, device=block.device)
        if n:
            share = c["q_heads"] // c["kv_heads"]
            k, v = (_stored(block, lo, c)[:, :n] for lo in (0, half))
            place = torch.arange(n - q, n, device=block.device)[:, None]
            key = torch.arange(n, device=block.device)[None]
            hidden = (key > place) | (key <= place - c["window"] if c["window"] else torch.zeros_like(key, dtype=torch.bool))
            for h in range(c["q_heads"]):
                z = s["q"][at:at + q, h].double() @ k[h // share].T / math.sqrt(c["dim"])
                z = torch.tanh(z / c["cap"]) * c["cap"] if c["cap"] else z
                z = z - s["slopes"][h].double() * (place - key) if c["slopes"] else z
                out[:, h] = torch.softmax(z.masked_fill(hidden, -math.inf), 1) @ v[h // share]
        outs.append(out)
        at += q
    if c["kind"] == "read":
        return tuple(torch.cat([o[i] for o in outs]) for i in (0, 1))
    return torch.cat(outs)

"""Measured cases of the 4-bit key/value store, its attention and the rotary
positions with several axes.

`run` is one pass of an operator as a program calls it. With `own` false it is
the operator's definition in elementary torch operations; with `own` true it
is the framework's calls. Both take the state that `prepare` made.
"""
import math

import torch

own = False

D = 128            # head dimension of the 4-bit store
ROWS = 16          # tokens of a group, one page of the store
BLOCK = 16         # elements that share a scale
TILE = 32          # elements of a row whose codes lie together: 16 bytes
PAGE = ROWS * (D // 2 + D // BLOCK)  # bytes of a page: 4 tiles of 16 rows of codes, then 16 rows of scales
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _rope(name, **kw):
    return dict(dict(name=name, op="rope", batch=1, tokens=1, heads=32, rep=1, d=128, dtype="bf16",
                     sections="16,24,24", interleaved=False, inverse=False, theta=1e6), **kw)


def _summaries(name, **kw):
    return dict(dict(name=name, op="summaries", batch=1, seq_len=65536, kv_heads=4, high=32,
                     sections="16,24,24", interleaved=False, theta=1e6), **kw)


def _store(name, **kw):
    return dict(dict(name=name, op="store", batch=1, seq_len=65536, kv_heads=4, begin=0,
                     tokens=65536, rotate=False, sections="16,24,24", interleaved=False,
                     theta=1e6), **kw)


def _attend(name, **kw):
    return dict(dict(name=name, op="attend", batch=1, seq_len=32768, q_heads=32, kv_heads=4,
                     begin=-1, tokens=1, sinks=1, locals=2, groups=96), **kw)


def listed():
    return [
        # the queries of one decode step of 16 sequences
        _rope("rope_step", batch=16),
        # the queries of a 64K-token prefill, the largest
        _rope("rope_64k", tokens=65536),
        # the gradient of a rotation in 32 bits: odd length, two axes in turn, small heads
        _rope("rope_grad_f32", batch=3, tokens=4999, heads=6, d=64, dtype="f32", sections="13,14",
              interleaved=True, inverse=True, theta=1e4),
        # key summaries and rotated keys of a 64K-token prefill
        _summaries("summaries_64k"),
        # several sequences of an odd length: the last group and chunk are partial
        _summaries("summaries_odd", batch=3, seq_len=4999, kv_heads=8, high=20,
                   sections="20,22,22", interleaved=True),
        # a whole prefill's rotated keys and values into the store, and back
        _store("store_64k"),
        # the new token of 64 sequences: its key rotated, both stored, read back
        _store("store_step", batch=64, seq_len=4096, begin=2077, tokens=1, rotate=True),
        # one decode step's attention: a short context of one sequence, where latency counts
        _attend("attend_one", seq_len=1000, groups=24),
        # 16 sequences of 32K tokens
        _attend("attend_16x32k", batch=16),
        # a full serving batch
        _attend("attend_128x8k", batch=128, seq_len=8192),
        # a prefill from the first token
        _attend("prefill_4k", seq_len=4096, begin=0, tokens=4096),
        # the last 16K tokens of a 32K context, the history in the store
        _attend("prefill_16k_of_32k", begin=16384, tokens=16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, half, axes):
    cut = sorted(rng.randint(0, half) for _ in range(axes))
    return ",".join(str(b - a) for a, b in zip([0] + cut[:-1], cut))


def draw(rng):
    kind = rng.choice(("rope", "summaries", "store", "store_step", "attend", "attend", "prefill"))
    inter = rng.random() < 0.5
    if kind == "rope":
        d, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "f32"))
        rep, batch = rng.choice((1, 1, 4)), _log(rng, 1, 16)
        heads = 1 if rep > 1 else rng.choice((1, 2, 5, 8, 32))  # keys: a row a head; queries
        tokens = _log(rng, 1, (1 << 20) // (heads * batch * rep))
        c = _rope("", batch=batch, tokens=tokens, heads=heads, rep=rep, d=d, dtype=dtype,
                  sections=_sections(rng, d // 2, rng.randint(1, 4)), interleaved=inter,
                  inverse=rng.random() < 0.4, theta=rng.choice((1e4, 5e5, 1e6)))
    elif kind == "summaries":
        batch, kv = _log(rng, 1, 8), rng.choice((1, 2, 4, 8))
        c = _summaries("", batch=batch, kv_heads=kv, seq_len=_log(rng, 1, 262144 // (batch * kv)),
                       high=rng.randint(0, 64), interleaved=inter,
                       sections=_sections(rng, 64, rng.randint(1, 4)))
    elif kind == "store":
        batch, kv = _log(rng, 1, 8), rng.choice((1, 2, 4, 8))
        n = _log(rng, 2, 262144 // (batch * kv))
        c = _store("", batch=batch, kv_heads=kv, tokens=n, begin=rng.randint(0, 100))
        c["seq_len"] = c["begin"] + n + rng.randint(0, 50)
    elif kind == "store_step":
        n = _log(rng, 16, 4096)
        c = _store("", batch=_log(rng, 1, 64), seq_len=n, begin=rng.randrange(n), tokens=1,
                   kv_heads=rng.choice((1, 2, 4, 8)), rotate=True, interleaved=inter,
                   sections=_sections(rng, 64, rng.randint(1, 4)))
    elif kind == "attend":
        kv, batch = rng.choice((1, 2, 4, 8)), _log(rng, 1, 64)
        c = _attend("", batch=batch, kv_heads=kv, q_heads=kv * rng.choice((1, 2, 3, 4, 8)),
                    seq_len=_log(rng, 1, (1 << 21) // (batch * kv)), sinks=rng.randint(0, 2),
                    locals=rng.randint(0, 4), groups=_log(rng, 8, 192 if batch * kv <= 256 else 64))
    else:
        kv = rng.choice((1, 2, 4))
        n = _log(rng, 2, 8192)
        c = _attend("", kv_heads=kv, q_heads=8 * kv, tokens=n, begin=rng.randint(0, 8000),
                    sinks=rng.randint(0, 2), locals=rng.randint(0, 3), groups=_log(rng, 8, 128))
        c["seq_len"] = c["begin"] + n + rng.randint(0, 70)
    del c["name"]
    return c


def work(c):
    if c["op"] == "rope":
        pairs = c["batch"] * c["rep"] * c["tokens"] * c["heads"] * (c["d"] // 2)
        es = 2 if c["dtype"] == "bf16" else 4
        axes = len(c["sections"].split(","))
        return {"bytes": 4 * pairs * es + 4 * axes * c["batch"] * c["tokens"], "flops": 6 * pairs}
    if c["op"] == "summaries":
        units = c["batch"] * c["kv_heads"]
        chunks = -(-c["seq_len"] // 64)
        axes = len(c["sections"].split(","))
        return {"bytes": units * (c["seq_len"] * 4 * D + chunks * 5 * 4 * D)
                + 4 * axes * c["batch"] * c["seq_len"],
                "flops": units * c["seq_len"] * (D // 2) * 8}
    if c["op"] == "store":
        # bf16 rows in, 4-bit rows out; the same read back
        rows = 2 * c["batch"] * c["kv_heads"] * c["tokens"]
        return {"bytes": rows * 2 * (2 * D + PAGE // ROWS), "flops": rows * D * 6}
    gq = c["q_heads"] // c["kv_heads"]
    units = c["batch"] * c["kv_heads"]
    begin = c["seq_len"] - 1 if c["begin"] < 0 else c["begin"]
    pairs, pages = 0, set()
    for j in range(begin // 64, (begin + c["tokens"] - 1) // 64 + 1):
        forced = set(range(min(c["sinks"], j + 1))) | set(range(max(0, j - c["locals"]), j + 1))
        routed = min(c["groups"], 4 * (j + 1 - len(forced)))
        lo, hi = max(begin, 64 * j), min(begin + c["tokens"], 64 * (j + 1))
        for p in range(lo, hi):  # every earlier key of the set, and the chunk's own up to p
            pairs += 64 * (len(forced) - 1) + 16 * routed + p - 64 * j + 1
        if c["tokens"] == 1:
            pages = 4 * (len(forced) - 1) + routed + (p - 64 * j) // 16 + 1
    if c["tokens"] > 1:  # the whole store up to the last query, at most, once
        pages = -(-(begin + c["tokens"]) // 16)
    rows = c["batch"] * c["tokens"] * c["q_heads"]
    return {"bytes": units * pages * 2 * PAGE + rows * D * 4, "flops": 4 * D * pairs * gq * units}


# ----------------------------------------------------------------- inputs
def _pair_axis(c, half):
    """Axis of each pair: the sections one after another, or in turn; -1 past them."""
    left = [int(s) for s in c["sections"].split(",")]
    if not c["interleaved"]:
        axis = [a for a, n in enumerate(left) for _ in range(n)]
    else:
        axis, left = [], list(left)
        while sum(left):
            for a in range(len(left)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    return axis + [-1] * (half - len(axis))


def _positions(g, axes, batch, tokens, begin=0):
    """Positions of text with images in it: axis 0 runs on, the others are small offsets
    within an image around it."""
    run = torch.arange(begin, begin + tokens, device="cuda").expand(batch, tokens)
    start = torch.randint(0, 1000, (batch, 1), device="cuda", generator=g)
    rows = [run + start]
    for _ in range(axes - 1):
        rows.append(run // 7 * 3 + start
                    + torch.randint(0, 48, (batch, tokens), device="cuda", generator=g))
    return torch.stack(rows).to(torch.int32).contiguous()


def _keys(g, batch, heads, n):
    """Keys of a long text: a topic per stretch of 64 tokens, and noise."""
    x = torch.randn(batch, heads, n, D, device="cuda", generator=g, dtype=torch.bfloat16)
    topic = torch.randn(batch, heads, -(-n // 64), 1, D, device="cuda", generator=g,
                        dtype=torch.bfloat16)
    x += topic.expand(-1, -1, -1, 64, -1).reshape(batch, heads, -1, D)[:, :, :n]
    return x


def _tensor_scale(x):
    """A power of two that puts the largest block scale into the range of its 8 bits."""
    return 2.0 ** math.ceil(math.log2(max(1e-30, float(x.abs().amax())) / (6 * 448)))


def _quantise(x, ts):
    """Codes (0..15) and scales of rows [..., D]: the definition, in 32 bits."""
    b = x.float().unflatten(-1, (D // BLOCK, BLOCK))
    scale = (b.abs().amax(-1) / (6 * ts)).clamp(max=448).to(torch.float8_e4m3fn)
    s = (scale.float() * ts).unsqueeze(-1)
    t = torch.where(s > 0, b.abs() / s, 0.0)
    code = ((t > 0.25).to(torch.uint8) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5)
            + (t >= 3.5) + (t > 5))
    code = code | ((b < 0).to(torch.uint8) << 3)
    return code.flatten(-2), scale


def _pack(x, ts):
    """The store's pages [B, H, ceil(n / 16), PAGE] of rows [B, H, n, D]."""
    B, H, n, _ = x.shape
    pages = torch.zeros(B, H, -(-n // ROWS), PAGE, dtype=torch.uint8, device=x.device)
    for b in range(B):
        code, scale = _quantise(x[b], ts)
        code, scale = code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)
        code, scale = (torch.nn.functional.pad(t, (0, 0, 0, -n % ROWS)).unflatten(1, (-1, ROWS))
                       for t in (code, scale))
        code = code.unflatten(-1, (D // TILE, TILE // 2)).transpose(2, 3)  # tile, row, bytes
        pages[b, :, :, :ROWS * D // 2] = code.flatten(2)
        pages[b, :, :, ROWS * D // 2:] = scale.flatten(2)
    return pages


def _config(c, **kw):
    """The framework's configuration of a case."""
    from long_context_rope_b200 import hga
    n = max(1, c.get("seq_len", 64))
    w = dict(batch=c["batch"], seq_len=n, n_q_heads=c.get("q_heads", c.get("kv_heads", 1)),
             n_kv_heads=c.get("kv_heads", 1), head_dim=c.get("d", D), chunk_size=64,
             groups_per_chunk=4, n_sink=c.get("sinks", 1), n_local=c.get("locals", 2),
             top_k_chunks=32, top_k_groups=c.get("groups", 96), n_high_freq_pairs=c.get("high", 32),
             rope_theta=c.get("theta", 1e6), dtype=c.get("dtype", "bf16"), q_begin=0, q_len=1)
    return hga.config_from(type("Shape", (), w), **kw)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["pair_axis"] = _pair_axis(c, c["d"] // 2)
        s["positions"] = _positions(g, len(c["sections"].split(",")), c["batch"], c["tokens"])
        s["x"] = torch.randn(c["batch"] * c["rep"], c["tokens"], c["heads"], c["d"], device="cuda",
                             generator=g, dtype=dt)
        s["y"] = torch.empty_like(s["x"])
    elif c["op"] == "summaries":
        s["pair_axis"] = _pair_axis(c, D // 2)
        s["positions"] = _positions(g, len(c["sections"].split(",")), c["batch"], c["seq_len"])
        s["k"] = _keys(g, c["batch"], c["kv_heads"], c["seq_len"])
        n = -(-c["seq_len"] // 64)
        s["chunk"] = torch.empty(c["batch"], c["kv_heads"], n, D, device="cuda")
        s["group"] = torch.empty(c["batch"], c["kv_heads"], 4 * n, D, device="cuda")
        s["rot"] = torch.empty_like(s["k"])
    elif c["op"] == "store":
        s["k"] = _keys(g, c["batch"], c["kv_heads"], c["tokens"])
        s["v"] = torch.randn(s["k"].shape, device="cuda", generator=g, dtype=torch.bfloat16)
        s["ks"], s["vs"] = 2.0 ** -8, 2.0 ** -9  # a deployment's calibrated scales
        s["pair_axis"] = _pair_axis(c, D // 2)
        s["positions"] = _positions(g, len(c["sections"].split(",")), c["batch"], c["tokens"],
                                    c["begin"])
        shape = (c["batch"], c["kv_heads"], -(-c["seq_len"] // ROWS), PAGE)
        s["kp"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        s["vp"] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        s["ko"], s["vo"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    else:
        k = _keys(g, c["batch"], c["kv_heads"], c["seq_len"])
        s["ks"] = _tensor_scale(k)
        s["kp"] = _pack(k, s["ks"])
        k.normal_(generator=g)
        s["vs"] = _tensor_scale(k)
        s["vp"] = _pack(k, s["vs"])
        del k
        begin = c["seq_len"] - 1 if c["begin"] < 0 else c["begin"]
        s["begin"] = begin
        s["q"] = torch.randn(c["batch"], c["tokens"], c["q_heads"], D, device="cuda", generator=g,
                             dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        # the router's lists: groups of earlier chunks that are not always visible, ascending
        j0, j1 = begin // 64, (begin + c["tokens"] - 1) // 64
        j = torch.arange(j0, j1 + 1, device="cuda").view(-1, 1)
        n = max(c["groups"], 4 * (j1 + 1))
        chunk = torch.arange(n, device="cuda").view(1, -1) // 4
        open_ = (chunk < j - c["locals"]) & (chunk >= c["sinks"])
        score = torch.rand(c["batch"], c["kv_heads"], j1 - j0 + 1, n, device="cuda", generator=g)
        got = score.masked_fill(~open_, -1.0).topk(c["groups"], -1)
        pick = got.indices.masked_fill(got.values < 0, 1 << 30).sort(-1).values
        s["count"] = (pick < 1 << 30).sum(-1).to(torch.int32)
        s["sel"] = pick.masked_fill(pick == 1 << 30, -1).to(torch.int32)
    if own:
        from long_context_rope_b200 import hga
        if c["op"] == "attend":
            s["cfg"] = _config(c, q_begin=s["begin"], q_len=c["tokens"], kv_type=hga.HGA_KV_E2M1,
                               k_scale=s["ks"], v_scale=s["vs"])
        else:
            kw = dict(kv_type=hga.HGA_KV_E2M1, k_scale=s["ks"], v_scale=s["vs"]) if "ks" in s else {}
            s["cfg"] = _config(c, **kw)
            s["axes"] = hga.rope_axes(s["pair_axis"], s["positions"].shape[0],
                                      inverse=c.get("inverse", False))
    return s


# ------------------------------------------------------------ plain forms
def _turn(positions, pair_axis, theta, d):
    """cos and sin [NB, T, d/2] of every pair's angle, formed in 64 bits."""
    axis = torch.tensor(pair_axis, device="cuda")
    freq = theta ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    a = positions.double()[axis.clamp(min=0)] * (freq * (axis >= 0)).view(-1, 1, 1)
    a = a.permute(1, 2, 0)
    return torch.cos(a), torch.sin(a)


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_rope(s):
    c, x = s["c"], s["x"]
    cos, sin = (t.float()[:, None, :, None] for t in _turn(s["positions"], s["pair_axis"],
                                                         c["theta"], c["d"]))
    y = x.float().unflatten(0, (c["batch"], c["rep"]))
    return _rotate(y, cos, -sin if c["inverse"] else sin).flatten(0, 1).to(x.dtype)


def _plain_summaries(s):
    c, k = s["c"], s["k"]
    cos, sin = (t.float()[:, None] for t in _turn(s["positions"], s["pair_axis"], c["theta"], D))
    rot = _rotate(k.float(), cos, sin)
    pair = torch.arange(D, device="cuda") % (D // 2)
    mixed = torch.where(pair < c["high"], rot, k.float())
    n = c["seq_len"]
    pad = -n % 64
    mixed = torch.nn.functional.pad(mixed, (0, 0, 0, pad))
    pos = torch.nn.functional.pad(s["positions"].double(), (0, pad))
    have = torch.nn.functional.pad(torch.ones(n, device="cuda"), (0, pad))

    def table(size):
        count = have.view(-1, size).sum(-1)
        some = count.clamp(min=1)
        mean = mixed.unflatten(2, (-1, size)).sum(3) / some.view(-1, 1)
        at = pos.unflatten(2, (-1, size)).sum(3) / some.double()
        co, si = (t.float()[:, None] for t in _turn(at, s["pair_axis"], c["theta"], D))
        return torch.where((pair < c["high"]), mean, _rotate(mean, co, si))

    return {"chunk": table(64), "group": table(16), "rot": rot.to(k.dtype)}


def _values(code, scale):
    """The numbers that codes and scales stand for, in 32 bits, without the tensor scale."""
    grid = torch.tensor(GRID, device="cuda")
    grid = torch.cat((grid, -grid))
    return grid[code.long()] * scale.float().repeat_interleave(BLOCK, -1)


def _plain_store(s):
    c, k = s["c"], s["k"].float()
    if c["rotate"]:
        cos, sin = (t[:, None] for t in _turn(s["positions"], s["pair_axis"], c["theta"], D))
        k = _rotate(k.double(), cos, sin).float()
    k = _values(*_quantise(k, s["ks"])) * s["ks"]
    v = _values(*_quantise(s["v"], s["vs"])) * s["vs"]
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _blocks(s):
    """Groups that each query chunk sees: [B, H, chunks, n], -1 where there is none."""
    c, sel = s["c"], s["sel"]
    j = s["begin"] // 64 + torch.arange(sel.shape[2], device="cuda").view(-1, 1)
    sink = torch.arange(c["sinks"], device="cuda").view(1, -1)
    sink = torch.where(sink <= j, sink, -1)
    near = j - torch.arange(c["locals"], -1, -1, device="cuda").view(1, -1)
    near = torch.where(near >= c["sinks"], near, torch.where((near == j) & (j >= c["sinks"]), near, -1))
    chunk = torch.cat((sink, near), 1)
    group = torch.where(chunk[..., None] >= 0, chunk[..., None] * 4 + torch.arange(4, device="cuda"), -1)
    group = group.flatten(1).expand(*sel.shape[:2], -1, -1)
    return torch.cat((group, sel.long()), -1)


def _read(pages, group):
    """Rows [B, H, chunks, n, 16, D] of the groups, without the tensor scale."""
    B, H = group.shape[:2]
    b = torch.arange(B, device="cuda").view(-1, 1, 1, 1)
    h = torch.arange(H, device="cuda").view(1, -1, 1, 1)
    page = pages[b, h, group.clamp(0, pages.shape[2] - 1)]
    byte, scale = page[..., :ROWS * D // 2], page[..., ROWS * D // 2:]
    byte = byte.unflatten(-1, (D // TILE, ROWS, TILE // 2)).transpose(-3, -2).flatten(-2)
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    return _values(code, scale.view(torch.float8_e4m3fn).unflatten(-1, (ROWS, -1)))


def _plain_attend(s):
    c, q = s["c"], s["q"]
    B, n, Hq, _ = q.shape
    H, begin = c["kv_heads"], s["begin"]
    gq = Hq // H
    group = _blocks(s)
    kpos = (group[..., None] * ROWS + torch.arange(ROWS, device="cuda")).flatten(3)
    kpos = torch.where(kpos < 0, 1 << 30, kpos)
    k, v = (_read(s[p], group).flatten(3, 4) for p in ("kp", "vp"))
    J = group.shape[2]
    if n == 1:
        rows = torch.tensor([[begin]], device="cuda")
    else:
        rows = (begin // 64 * 64 + torch.arange(J * 64, device="cuda")).view(J, 64)
    at = (rows - begin).clamp(0, n - 1)
    x = q.float()[:, at].unflatten(-2, (H, gq))            # [B, J, T, H, gq, D]
    x = x.permute(0, 3, 1, 2, 4, 5).flatten(3, 4)          # [B, H, J, T gq, D]
    w = x @ k.transpose(-1, -2) * (s["ks"] / math.sqrt(D))
    see = kpos[..., None, :] <= rows.repeat_interleave(gq, -1)[..., None]
    w = w.masked_fill(~see, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    o = (w @ v) / w.sum(-1, keepdim=True) * s["vs"]
    o = o.unflatten(3, (-1, gq)).permute(0, 2, 3, 1, 4, 5).flatten(1, 2).flatten(2, 3)
    if n == 1:
        return o.to(q.dtype)
    lead = begin % 64
    return o[:, lead:lead + n].to(q.dtype)


def run(s):
    c = s["c"]
    if not own:
        return {"rope": _plain_rope, "summaries": _plain_summaries, "store": _plain_store,
                "attend": _plain_attend}[c["op"]](s)
    from long_context_rope_b200 import hga
    if c["op"] == "rope":
        hga.apply_rope_axes(s["cfg"], s["axes"], s["positions"], s["x"], s["y"],
                            c["batch"] * c["rep"], c["tokens"], c["heads"])
        return s["y"]
    if c["op"] == "summaries":
        hga.build_summaries_axes(s["cfg"], s["axes"], s["positions"], s["k"], s["chunk"],
                                 s["group"], s["rot"])
        return {"chunk": s["chunk"], "group": s["group"], "rot": s["rot"]}
    if c["op"] == "store":
        if c["rotate"]:
            hga.store_kv(s["cfg"], s["k"], s["v"], s["kp"], s["vp"], c["begin"], axes=s["axes"],
                         positions=s["positions"])
        else:
            hga.store_kv(s["cfg"], s["k"], s["v"], s["kp"], s["vp"], c["begin"])
        hga.load_kv(s["cfg"], s["kp"], s["vp"], s["ko"], s["vo"], c["begin"])
        return {"k": s["ko"], "v": s["vo"]}
    hga.attend(s["cfg"], s["q"], s["kp"], s["vp"], s["sel"], s["count"], s["out"])
    return s["out"]


# ------------------------------------------------------- the definitions
def _exact_rotation(x, positions, pair_axis, theta, sign):
    """Rows x [NB, ..., T, H, d] turned as complex numbers, in 64 bits."""
    d = x.shape[-1]
    z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double())
    angle = torch.zeros(positions.shape[1], positions.shape[2], d // 2, device="cuda",
                        dtype=torch.float64)
    for i, a in enumerate(pair_axis):
        if a >= 0:
            angle[..., i] = positions[a].double() / theta ** (2 * i / d)
    e = torch.polar(torch.ones_like(angle), sign * angle)
    z = z * e.view(e.shape[0], *([1] * (x.dim() - 4)), e.shape[1], 1, e.shape[2])
    return torch.cat((z.real, z.imag), -1)


def _exact_store(x, ts):
    """Each value to the nearest of the 15, in 64 bits; ties to the even code."""
    b = x.double().reshape(*x.shape[:-1], D // BLOCK, BLOCK)
    scale = (b.abs().amax(-1) / ts / 6).clamp(max=448.0)
    e = torch.floor(torch.log2(scale.clamp(min=2.0 ** -6))).clamp(-6, 8)
    unit = 2.0 ** (e - 3)
    scale = torch.round(scale / unit) * unit               # half to even: 3 bits, least 2^-9
    s = (scale * ts)[..., None]
    t = torch.where(s > 0, b.abs() / torch.where(s > 0, s, 1.0), 0.0).clamp(max=6.0)
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0)).double()
    return (torch.sign(b) * torch.round(t / step) * step * s).reshape(x.shape)


def _exact_pages(pages, ts):
    """A store's rows [B, H, tokens, D] in 64 bits, from its bits."""
    B, H, n, _ = pages.shape
    byte = pages[..., :ROWS * D // 2].reshape(B, H, n, 4, ROWS, 16)
    byte = byte.permute(0, 1, 2, 4, 3, 5).reshape(B, H, n * ROWS, D // 2).int()
    sc = pages[..., ROWS * D // 2:].reshape(B, H, n * ROWS, D // BLOCK).int()
    code = torch.stack((byte % 16, byte // 16), -1).reshape(B, H, n * ROWS, D)
    m, e = (code % 8) % 2, (code % 8) // 2
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * 2.0 ** (e - 1).double()).double()
    mag = torch.where(code >= 8, -mag, mag)
    sm, se = sc % 8, sc // 8 % 16
    s = torch.where(se == 0, sm.double() * 2.0 ** -9, (1 + sm.double() / 8) * 2.0 ** (se - 7).double())
    return mag * s.repeat_interleave(BLOCK, -1) * ts


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "rope":
        x = s["x"].reshape(c["batch"], c["rep"], c["tokens"], c["heads"], c["d"])
        return _exact_rotation(x, s["positions"], s["pair_axis"], c["theta"],
                               -1.0 if c["inverse"] else 1.0).reshape(s["x"].shape)
    if c["op"] == "summaries":
        k, n = s["k"].double(), c["seq_len"]
        rot = _exact_rotation(k[..., None, :], s["positions"], s["pair_axis"], c["theta"], 1.0)[..., 0, :]
        high = (torch.arange(D, device="cuda") % (D // 2)) < c["high"]
        got = {"rot": rot}
        for name, size in (("chunk", 64), ("group", 16)):
            of = torch.arange(n, device="cuda") // size
            rows = -(-n // 64) * (64 // size)
            count = torch.zeros(rows, device="cuda", dtype=torch.float64).index_add_(
                0, of, torch.ones(n, device="cuda", dtype=torch.float64)).clamp(min=1)

            def mean(x, dim):
                shape = list(x.shape)
                shape[dim] = rows
                total = torch.zeros(shape, device="cuda", dtype=torch.float64).index_add_(dim, of, x)
                return total / count.reshape([-1 if i == dim else 1 for i in range(x.dim())])

            low = _exact_rotation(mean(k, 2)[..., None, :], mean(s["positions"].double(), 2),
                                  s["pair_axis"], c["theta"], 1.0)[..., 0, :]
            got[name] = torch.where(high, mean(rot, 2), low)
        return got
    if c["op"] == "store":
        k = s["k"].double()
        if c["rotate"]:
            k = _exact_rotation(k[..., None, :], s["positions"], s["pair_axis"], c["theta"], 1.0)[..., 0, :]
        return {"k": _exact_store(k, s["ks"]), "v": _exact_store(s["v"], s["vs"])}
    if c["batch"] * c["kv_heads"] * c["seq_len"] > 1 << 23:
        return None
    # every sequence and key head apart: a mask over all keys, in slices of the queries
    out = torch.empty(s["q"].shape, device="cuda", dtype=torch.float64)
    gq = c["q_heads"] // c["kv_heads"]
    begin, n = s["begin"], c["tokens"]
    last = begin + n
    step = 64 if n > 1 else 1
    for b in range(c["batch"]):
        for h in range(c["kv_heads"]):
            k = _exact_pages(s["kp"][b:b + 1, h:h + 1], s["ks"])[0, 0][:last]
            v = _exact_pages(s["vp"][b:b + 1, h:h + 1], s["vs"])[0, 0][:last]
            for j in range(begin // 64, (last - 1) // 64 + 1):
                lo, hi = max(begin, 64 * j), min(last, 64 * (j + 1))
                see = torch.zeros((last + 63) // 64, 4, device="cuda", dtype=torch.bool)
                see[:min(c["sinks"], j + 1)] = True
                see[max(0, j - c["locals"]):j + 1] = True
                jj = j - begin // 64
                see.view(-1)[s["sel"][b, h, jj, :int(s["count"][b, h, jj])].long()] = True
                at = torch.nonzero(see.view(-1).repeat_interleave(ROWS)[:last])[:, 0]
                x = s["q"][b, lo - begin:hi - begin, h * gq:(h + 1) * gq].double()
                w = torch.einsum("tgd,kd->tgk", x, k[at]) / math.sqrt(D)
                ok = at[None, None, :] <= torch.arange(lo, hi, device="cuda")[:, None, None]
                w = torch.softmax(w.masked_fill(~ok, -math.inf), -1)
                out[b, lo - begin:hi - begin, h * gq:(h + 1) * gq] = torch.einsum("tgk,kd->tgd", w, v[at])
    return out

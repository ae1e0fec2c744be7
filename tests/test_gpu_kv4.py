"""The 4-bit key/value store, its attention, and rotary positions with several
axes against 64-bit definitions (kv4_ref.py), through the public calls."""
import math

import pytest
import torch

import kv4_ref as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _cfg(hga, **kw):
    w = dict(batch=1, seq_len=256, n_q_heads=8, n_kv_heads=1, head_dim=128, chunk_size=64,
             groups_per_chunk=4, n_sink=1, n_local=2, top_k_chunks=8, top_k_groups=16,
             n_high_freq_pairs=20, rope_theta=1e4, dtype="bf16", q_begin=0, q_len=1)
    over = {k: kw.pop(k) for k in ("kv_type", "k_scale", "v_scale", "kv_layout", "routing",
                                   "summary_type") if k in kw}
    return hga.config_from(type("W", (), dict(w, **kw)), **over)


def _cfg4(hga, **kw):
    return _cfg(hga, **dict(dict(kv_type=hga.HGA_KV_E2M1, k_scale=2.0 ** -8, v_scale=2.0 ** -9),
                            **kw))


def _rows(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF)


def _clean(hga):
    torch.cuda.synchronize()
    assert hga.get_device_error() == 0


# ------------------------------------------------------------------ store
@pytest.mark.parametrize("B,H,L,pos0,n", [(1, 1, 1, 0, 1), (2, 3, 100, 37, 1), (1, 2, 33, 0, 33),
                                          (3, 1, 75, 15, 18), (2, 2, 64, 64, 0), (1, 4, 1000, 3, 990)])
def test_store_bytes(B, H, L, pos0, n):
    """The bytes of codes and scales, and every other byte left as it was."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, batch=B, n_kv_heads=H, n_q_heads=H, seq_len=L)
    k, v = _rows((B, H, n, 128), 1), _rows((B, H, n, 128), 2, 3.0)
    if n > 2:   # a zero block, tiny and large ones, a scale at its largest, NaN and infinity
        k[0, 0, 0, :16] = 0
        k[0, 0, 0, 16:32] = 1e-30
        k[0, 0, 0, 32:48] = 2.0 ** -18
        k[0, 0, 1, 64:80] = 3e38
        k[0, 0, 1, 80:96] *= 2.0 ** 9
        v[0, 0, 1, 3] = float("nan")
        v[0, 0, 2, 127] = float("-inf")
        v[0, 0, 2, 16:32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 2)
    ks = torch.full((B, H, -(-L // 16), 1152), 0xA5, dtype=torch.uint8, device="cuda")
    vs = ks.clone()
    hga.store_kv(cfg, k.cuda(), v.cuda(), ks, vs, pos0)
    _clean(hga)
    for got, x, ts in ((ks, k, cfg.k_scale), (vs, v, cfg.v_scale)):
        code, byte = R.quantise(x, ts)
        before = torch.full((B, H, -(-L // 16) * 16, 128), 5, dtype=torch.uint8)
        before[..., 1::2] = 10
        at = torch.full((B, H, -(-L // 16) * 16, 8), 0xA5, dtype=torch.uint8)
        before[:, :, pos0:pos0 + n], at[:, :, pos0:pos0 + n] = code, byte
        assert torch.equal(got.cpu(), R.pack(before, at))


@pytest.mark.parametrize("B,H,pos0,n,sections,inter", [
    (2, 2, 0, 70, (16, 24, 24), False), (1, 3, 999, 1, (20, 22), True),
    (64, 1, 5, 1, (64,), False), (2, 1, 1000000, 17, None, False)])
def test_store_rotated(B, H, pos0, n, sections, inter):
    """Keys rotated on the way; a code may differ only where its quotient in 64
    bits is within 2^-20 of the border between two codes."""
    from long_context_rope_b200 import hga
    L = pos0 + n + 3
    cfg = _cfg4(hga, batch=B, n_kv_heads=H, n_q_heads=H, seq_len=L)
    k, v = _rows((B, H, n, 128), 3), _rows((B, H, n, 128), 4)
    if sections is None:
        pair, pos, axes = [0] * 64, None, hga.rope_axes([0] * 64, 1)
        p64 = (pos0 + torch.arange(n)).expand(1, B, n)
    else:
        pair = hga.pair_axes(64, sections, inter)
        axes = hga.rope_axes(pair, len(sections))
        g = torch.Generator().manual_seed(5)
        pos = torch.randint(-5000, 200000, (len(sections), B, n), generator=g, dtype=torch.int32)
        p64 = pos
    ks = torch.zeros(cfg.kv_rows(B, H, rows=L), dtype=torch.uint8, device="cuda")
    vs = torch.zeros_like(ks)
    hga.store_kv(cfg, k.cuda(), v.cuda(), ks, vs, pos0, axes=axes,
                 positions=None if pos is None else pos.cuda())
    ko, vo = torch.empty_like(k).cuda(), torch.empty_like(v).cuda()
    hga.load_kv(cfg, ks, vs, ko, vo, pos0)
    _clean(hga)
    x = R.rotate(k, R.angles(p64, pair, 1e4, 128)[:, None])
    code, byte = R.quantise(x.float(), cfg.k_scale)
    S = byte.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * cfg.k_scale
    want = R.GRID[code.long()] * S
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    near = ((x / S).abs()[..., None] - border).abs().amin(-1) <= 2.0 ** -20
    assert torch.equal(ko.cpu().double()[~near], want[~near]) and near.sum() <= 2
    code, byte = R.quantise(v, cfg.v_scale)
    assert torch.equal(vo.cpu().double(), R.GRID[code.long()]
                       * byte.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * cfg.v_scale)


@pytest.mark.parametrize("scale", [2.0 ** -8, 0.3])
def test_load_any_bytes(scale):
    """Every code under every scale byte, rounded once."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=49, k_scale=scale, v_scale=2 * scale)
    g = torch.Generator().manual_seed(0)
    pages = torch.randint(0, 256, (1, 1, 4, 1152), generator=g, dtype=torch.uint8)
    pages[..., :3, 1024:] = (torch.arange(384) % 256).to(torch.uint8).view(3, 128)
    p = pages.cuda()
    k = torch.empty(1, 1, 45, 128, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    hga.load_kv(cfg, p, p, k, v, 4)
    _clean(hga)
    for got, ts in ((k, torch.tensor(scale)), (v, torch.tensor(2 * scale))):
        want = (R.values(pages, 1.0).float() * ts).to(BF)[:, :, 4:49]
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got.cpu()), nan)
        assert torch.equal(got.cpu()[~nan], want[~nan])


# -------------------------------------------------------------- attention
def _attend_case(hga, cfg, seed=0, count=None, junk=True):
    """q, pages (rows after the span filled with junk), lists, the reference."""
    end = cfg.q_begin + cfg.q_len
    B, H = cfg.batch, cfg.n_kv_heads
    kp = R.pack(*R.quantise(_rows((B, H, cfg.seq_len, 128), seed), cfg.k_scale))
    vp = R.pack(*R.quantise(_rows((B, H, cfg.seq_len, 128), seed + 1), cfg.v_scale))
    if junk:
        for p in (kp, vp):
            s = p[..., 1024:].unflatten(-1, (16, 8))
            s[:, :, torch.arange(16 * p.shape[2]).view(-1, 16) >= end] = 0x7F
    q = _rows((B, cfg.q_len, cfg.n_q_heads, 128), seed + 2)
    sel, n = R.lists(cfg, cfg.route_heads, seed, count)
    kv = [torch.nan_to_num(R.values(p, ts)) for p, ts in ((kp, cfg.k_scale), (vp, cfg.v_scale))]
    want, tol = R.attend(cfg, q, kv[0], kv[1], sel, n)
    return q, kp, vp, sel, n, want, tol


def _check(out, want, tol):
    err = (out.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


DECODE = [
    dict(seq_len=1), dict(seq_len=17, n_q_heads=1), dict(seq_len=64, n_local=0, n_sink=0),
    dict(seq_len=65, n_local=0, n_sink=0, n_q_heads=3), dict(seq_len=1000, top_k_groups=24),
    dict(seq_len=1024, batch=3, n_kv_heads=2, n_q_heads=8), dict(seq_len=777, n_sink=2, n_local=4),
    dict(seq_len=512, q_begin=300), dict(seq_len=4096, batch=2, n_kv_heads=4, n_q_heads=32,
                                         top_k_groups=96),
    dict(seq_len=400, batch=40, n_kv_heads=8, n_q_heads=8, top_k_groups=8),
    dict(seq_len=600, chunk_size=32, groups_per_chunk=2), dict(seq_len=500, chunk_size=48,
                                                               groups_per_chunk=3),
    dict(seq_len=2048, n_q_heads=12),  # more heads than a warp-level tile holds
]


@pytest.mark.parametrize("kw", DECODE, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("count", [None, 0, 1])
def test_attend_decode(kw, count):
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, **dict(dict(q_begin=kw["seq_len"] - 1), **kw))
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 10, count)
    out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    _check(out, want, tol)


def test_attend_decode_large_queries():
    """Queries beyond the range of 16-bit floats with 5 exponent bits, and tiny ones."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=400, q_begin=399, k_scale=2.0 ** -30, n_q_heads=4)
    end = 400
    kp = R.pack(*R.quantise(_rows((1, 1, end, 128), 1, 2.0 ** -22), cfg.k_scale))
    vp = R.pack(*R.quantise(_rows((1, 1, end, 128), 2), cfg.v_scale))
    q = _rows((1, 1, 4, 128), 3)
    q *= torch.tensor([2.0 ** 20, 2.0 ** 22, 1.0, 2.0 ** -20]).view(1, 1, 4, 1).to(BF)
    sel, n = R.lists(cfg, 1, 0)
    want, tol = R.attend(cfg, q, R.values(kp, cfg.k_scale), R.values(vp, cfg.v_scale), sel, n)
    out = torch.empty_like(q).cuda()
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    _check(out, want, tol)


@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("q_begin,q_len", [(639, 1), (512, 128), (560, 33)])
def test_attend_scores_that_rise(order, q_begin, q_len):
    """Keys whose scores grow by orders of magnitude from block to block (the running
    maximum is raised again and again), or shrink, for some heads only."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=640, q_begin=q_begin, q_len=q_len, n_sink=1, n_local=1, top_k_groups=24,
                k_scale=2.0 ** -4)
    k = _rows((1, 1, 640, 128), 130).float()
    size = torch.arange(640) / 16
    size = {"rising": size, "falling": 40 - size, "mixed": (size * 7) % 40}[order].floor()
    k *= (1 + size)[:, None] ** 1.5
    q = _rows((1, q_len, 8, 128), 131)
    q[:, :, :3] *= 0.01
    kp = R.pack(*R.quantise(k.to(BF), cfg.k_scale))
    vp = R.pack(*R.quantise(_rows((1, 1, 640, 128), 132), cfg.v_scale))
    sel, n = R.lists(cfg, 1, 133)
    want, tol = R.attend(cfg, q, R.values(kp, cfg.k_scale), R.values(vp, cfg.v_scale), sel, n)
    out = torch.empty_like(q).cuda()
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    _check(out, want, tol)


PREFILL = [
    dict(seq_len=2, q_len=2), dict(seq_len=65, q_len=65), dict(seq_len=300, q_len=300),
    dict(seq_len=700, q_begin=333, q_len=250), dict(seq_len=640, q_begin=128, q_len=512, batch=2,
                                                     n_kv_heads=2, n_q_heads=16),
    dict(seq_len=500, q_begin=63, q_len=2), dict(seq_len=400, q_len=400, n_sink=0, n_local=0),
    dict(seq_len=300, q_begin=100, q_len=150, n_q_heads=2), dict(seq_len=320, q_len=320, chunk_size=32,
                                                                  groups_per_chunk=2),
    dict(seq_len=300, q_len=200, chunk_size=48, groups_per_chunk=3, n_q_heads=4),
    dict(seq_len=640, q_len=640, n_sink=2, n_local=3, top_k_groups=12, n_kv_heads=2, n_q_heads=16),
]


@pytest.mark.parametrize("kw", PREFILL, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_attend_prefill(kw):
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, **kw)
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 20)
    out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    _check(out, want, tol)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_begin,q_len,heads", [(199, 1, 8), (128, 40, 8), (150, 30, 4)])
def test_attend_nan_row(which, q_begin, q_len, heads):
    """A row with a NaN scale reaches the queries that see it, and no other."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=256, q_begin=q_begin, q_len=q_len, n_q_heads=heads, n_local=0, n_sink=0)
    bad = q_begin + q_len // 2
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 30, count=0)
    (kp if which == "k" else vp)[0, 0, bad // 16, 1024 + (bad % 16) * 8 + 3] = 0x7F
    out = torch.empty_like(q).cuda()
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    got, seen = out.cpu().double(), q_begin + torch.arange(q_len) >= bad
    assert torch.isnan(got[0, seen][..., 48:64]).all()
    err = (got - want).abs()[0, ~seen]
    assert bool((err <= tol[0, ~seen]).all())
    # a decode step over this chunk only: one key, and it is NaN
    if q_len == 1:
        c1 = _cfg4(hga, seq_len=1, n_q_heads=heads)
        one = kp[:, :, :1].clone()
        one[..., 1024:1032] = 0x7F
        sel1 = torch.full((1, 1, 1, 16), -1, dtype=torch.int32, device="cuda")
        hga.attend(c1, q.cuda(), one.cuda(), one.cuda(), sel1, torch.zeros(1, 1, 1, dtype=torch.int32,
                                                                          device="cuda"), out)
        _clean(hga)
        assert torch.isnan(out).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_begin,q_len,heads", [(199, 1, 8), (64, 140, 8), (150, 30, 3)])
def test_attend_nan_query(value, q_begin, q_len, heads):
    """A query with a NaN or an infinity makes its own row NaN, and no other."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=256, q_begin=q_begin, q_len=q_len, n_q_heads=heads)
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 30)
    t, h = q_len // 2, heads - 1
    q[0, t, h, 5] = value
    q[0, t, h, 6] = -value
    out = torch.empty_like(q).cuda()
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    got = out.cpu().double()
    assert torch.isnan(got[0, t, h]).all()
    got[0, t, h] = want[0, t, h]
    _check(got, want, tol)


@pytest.mark.parametrize("L", [1024, 999])
@pytest.mark.parametrize("heads", [8, 5])
def test_gathered_windows_and_warm(L, heads):
    """Gathers of pages from HBM and host memory, the warm tier and the windows:
    bitwise copies, and attention over them as over the full store."""
    from long_context_rope_b200 import hga, pipeline
    cfg = _cfg4(hga, seq_len=L, q_begin=L - 1, batch=2, n_kv_heads=2, n_q_heads=2 * heads,
                top_k_groups=20)
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 40)
    n[0, 1, 0] = 7
    sel[0, 1, 0, 7:] = -1
    kv = [torch.nan_to_num(R.values(p, ts)) for p, ts in ((kp, cfg.k_scale), (vp, cfg.v_scale))]
    want, tol = R.attend(cfg, q, kv[0], kv[1], sel, n)
    qd, kd, vd, sd, nd = (t.cuda() for t in (q, kp, vp, sel, n))
    kh, vh = kp.pin_memory(), vp.pin_memory()
    outs = []

    def attend(c, kr, vr, gat=(None, None)):
        out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
        hga.attend(c, qd, kr, vr, sd, nd, out, k_gat=gat[0], v_gat=gat[1])
        _clean(hga)
        _check(out, want, tol)
        outs.append(out)
    attend(cfg, kd, vd)
    gat = pipeline.alloc_gathered(cfg)
    hga.gather_kv(cfg, kd, vd, False, sd, nd, *gat)
    attend(cfg, kd, vd, gat)
    for b in range(2):
        for h in range(2):
            for s in range(int(n[b, h, 0])):
                assert torch.equal(gat[0][b, h, 0, s].cpu(), kp[b, h, sel[b, h, 0, s]])
    host = pipeline.alloc_gathered(cfg)
    hga.gather_kv(cfg, kh, vh, True, sd, nd, *host)
    cfg_w = cfg.copy(kv_layout=hga.HGA_KV_WINDOWS)
    rows = hga.window_slots(cfg) * cfg.chunk_size
    win = [torch.zeros(cfg.kv_rows(2, 2, rows=rows), dtype=torch.uint8, device="cuda") for _ in "kv"]
    pipeline.fill_windows(cfg, kh, vh, *win)
    attend(cfg_w, *win, host)
    pool = pipeline.alloc_warm_pool(cfg, 40)
    for it in range(2):
        warm = pipeline.alloc_gathered(cfg)
        hga.gather_kv_warm(cfg, kh, vh, sd, nd, pool.k, pool.v, pool.tag, pool.last, it, pool.src,
                           *warm, pool.stats)
        _clean(hga)
        assert torch.equal(warm[0], host[0]) and torch.equal(warm[1], host[1])
    assert torch.equal(host[0], gat[0]) and torch.equal(host[1], gat[1])


def test_bad_lists_and_counts():
    """An invalid entry is left out and reported; the rest of the unit stands."""
    from long_context_rope_b200 import hga
    for kw in (dict(q_begin=511), dict(q_begin=448, q_len=64)):
        cfg = _cfg4(hga, seq_len=512, **kw)
        q, kp, vp, sel, n, _, _ = _attend_case(hga, cfg, 50, count=6)
        sel[0, 0, 0, 5] = 4 * 7 + 1   # of the current chunk
        kv = [R.values(p, ts) for p, ts in ((kp, cfg.k_scale), (vp, cfg.v_scale))]
        good = n - 1
        want, tol = R.attend(cfg, q, kv[0], kv[1], sel, good)
        out = torch.empty_like(q).cuda()
        args = (q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
        hga.attend(cfg, *args)
        torch.cuda.synchronize()
        assert hga.get_device_error() != 0 and hga.get_device_error() == 0
        _check(out, want, tol)


# ----------------------------------------------------------------- rotation
ROPE = [("bf16", 128, (16, 24, 24), False), ("bf16", 64, (10, 11, 11), True),
        ("f32", 128, (64,), False), ("f32", 64, (13, 14), True), ("bf16", 128, (), False),
        ("f32", 128, (0, 16, 0, 40), True)]


@pytest.mark.parametrize("dtype,d,sections,inter", ROPE)
@pytest.mark.parametrize("nb,rep,t,h", [(1, 1, 1, 1), (2, 1, 33, 5), (3, 4, 7, 1), (1, 2, 100, 3),
                                        (16, 1, 1, 32)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes(dtype, d, sections, inter, nb, rep, t, h, inverse):
    """Against the 64-bit rotation. The kernel's angle is reduced in 64 bits and
    its sine and cosine are off by 2^-22 at most; product and sum round in fp32."""
    from long_context_rope_b200 import hga
    cfg = _cfg(hga, head_dim=d, dtype=dtype, rope_theta=5e5)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(nb * rep, t, h, d, generator=g).to(cfg.torch_dtype())
    n_axes = max(1, len(sections))
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n_axes, nb, t), generator=g).to(torch.int32)
    pos[:, :, ::2] %= 70000
    pair = hga.pair_axes(d // 2, sections, inter)
    axes = hga.rope_axes(pair, n_axes, inverse=inverse)
    y = torch.empty_like(x).cuda()
    xd = x.cuda()
    hga.apply_rope_axes(cfg, axes, pos.cuda(), xd, y, nb * rep, t, h)
    hga.apply_rope_axes(cfg, axes, pos.cuda(), xd, xd, nb * rep, t, h)   # in place
    _clean(hga)
    a = R.angles(pos, pair, 5e5, d) * (-1 if inverse else 1)
    want = R.rotate(x, a[:, None, :, None].expand(-1, rep, -1, h, -1).flatten(0, 1))
    mag = (x.double().abs()[..., :d // 2] + x.double().abs()[..., d // 2:]).repeat(1, 1, 1, 2)
    u = R.BF16 if dtype == "bf16" else R.F32
    # 64-bit angles up to 2^31: their own rounding and the reduction's, 2^-53 of the angle each
    tol = mag * (2.0 ** -22 + 3 * R.F32 + 2.0 ** -19.5) + u * want.abs()
    assert bool(((y.cpu().double() - want).abs() <= tol).all())
    assert torch.equal(xd, y)
    off = torch.tensor([p < 0 for p in pair]).repeat(2)
    assert torch.equal(y.cpu()[..., off], x[..., off])


def test_rope_axes_is_its_gradient():
    """<R x, g> = <x, R^-1 g>, and a difference along one element."""
    from long_context_rope_b200 import hga
    cfg = _cfg(hga, dtype="f32")
    g = torch.Generator().manual_seed(8)
    x, dy = (torch.randn(2, 19, 3, 128, generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 5000, (3, 2, 19), generator=g, dtype=torch.int32).cuda()
    pair = hga.pair_axes(64, (16, 20, 20), True)

    def turn(t, inverse):
        y = torch.empty_like(t)
        hga.apply_rope_axes(cfg, hga.rope_axes(pair, 3, inverse=inverse), pos, t, y, 2, 19, 3)
        return y
    y, dx = turn(x, False), turn(dy, True)
    lhs, rhs = (y.double() * dy.double()).sum(), (x.double() * dx.double()).sum()
    # each element of y and dx is off by 2^-20 of its pair at most
    bound = 2.0 ** -20 * 2 * float((x.abs().double() * dy.abs().double()).sum()
                                   + x.double().norm() * dy.double().norm())
    assert abs(float(lhs - rhs)) <= bound
    for i in ((0, 0, 0, 3), (1, 18, 2, 100), (0, 7, 1, 63)):
        xp, xm = x.clone(), x.clone()
        xp[i] += 1.0
        xm[i] -= 1.0
        d = ((turn(xp, False).double() - turn(xm, False).double()) * dy.double()).sum() / 2
        assert abs(float(d) - float(dx[i])) <= 2.0 ** -19 * 4 * 8
    assert float((turn(y, True) - x).abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("dtype,d,F", [("bf16", 128, 20), ("f32", 64, 0), ("f32", 128, 64), ("bf16", 64, 7)])
@pytest.mark.parametrize("B,H,L,C", [(1, 1, 1, 64), (2, 3, 200, 64), (1, 2, 129, 128), (2, 1, 96, 32),
                                     (1, 1, 100, 48)])
def test_summaries_axes(dtype, d, F, B, H, L, C):
    from long_context_rope_b200 import hga, pipeline
    if (d // 2 // (8 if dtype == "bf16" else 4)) * 4 * (C // 16) % 32:
        pytest.skip("the framework's configurations do not have this one")
    cfg = _cfg(hga, batch=B, n_kv_heads=H, n_q_heads=H, seq_len=L, head_dim=d, dtype=dtype,
               n_high_freq_pairs=min(F, d // 2), chunk_size=C, groups_per_chunk=C // 16)
    g = torch.Generator().manual_seed(9)
    k = torch.randn(B, H, L, d, generator=g).to(cfg.torch_dtype())
    pair = hga.pair_axes(d // 2, (d // 8, d // 8, d // 8), True)
    pos = torch.randint(0, 100000, (3, B, L), generator=g, dtype=torch.int32)
    cs, gs = pipeline.alloc_summaries(cfg)
    rot = torch.empty_like(k).cuda()
    hga.build_summaries_axes(cfg, hga.rope_axes(pair, 3), pos.cuda(), k.cuda(), cs, gs, rot)
    _clean(hga)
    a = R.angles(pos, pair, 1e4, d)[:, None]
    want = R.rotate(k, a)
    mag = (k.double().abs()[..., :d // 2] + k.double().abs()[..., d // 2:]).repeat(1, 1, 1, 2)
    u = R.BF16 if dtype == "bf16" else R.F32
    assert bool(((rot.cpu().double() - want).abs() <= mag * 2.0 ** -19 + u * want.abs()).all())
    high = (torch.arange(d) % (d // 2)) < cfg.n_high_freq_pairs
    for table, size in ((cs, C), (gs, 16)):
        n = table.shape[2]
        ref = torch.zeros(B, H, n, d, dtype=torch.float64)
        tol = torch.zeros_like(ref)
        for i in range(n):
            s = slice(i * size, min(L, (i + 1) * size))
            if s.start >= L:
                continue
            low = R.rotate(k[:, :, s].double().mean(2, keepdim=True),
                           R.angles(pos[:, :, s].double().mean(2, keepdim=True), pair, 1e4, d)[:, None])
            ref[:, :, i] = torch.where(high, want[:, :, s].mean(2), low[:, :, 0])
            # sums of at most 128 terms in fp32, and the rotation's error
            tol[:, :, i] = mag[:, :, s].mean(2) * (2.0 ** -19 + 130 * R.F32) + 1e-30
        assert bool(((table.cpu().double() - ref).abs() <= tol).all()), size


# ------------------------------------------------------ used as a program does
def test_streams_and_graphs():
    """Another stream, a captured run replayed on new inputs, two graphs at once."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=900, batch=2, n_kv_heads=2, n_q_heads=16, q_begin=899)
    cases = [_attend_case(hga, cfg, s) for s in (60, 61)]
    axes = hga.rope_axes(hga.pair_axes(64, (16, 24, 24)), 3)
    bufs, graphs = [], []
    side = torch.cuda.Stream()
    for c in cases:
        b = [t.cuda() for t in c[:5]]
        out = torch.empty_like(b[0])
        x = torch.randn(2, 1, 16, 128, device="cuda").to(BF)
        pos = torch.randint(0, 99, (3, 2, 1), device="cuda", dtype=torch.int32)
        y = torch.empty_like(x)
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            hga.attend(cfg, *b, out)
            hga.apply_rope_axes(cfg, axes, pos, x, y, 2, 1, 16)
        bufs.append((b, out, x, pos, y))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    _clean(hga)
    for c, (b, out, x, pos, y) in zip(cases, bufs):
        _check(out, c[5], c[6])
        z = torch.empty_like(x)
        with torch.cuda.stream(side):
            hga.apply_rope_axes(cfg, axes, pos, x, z, 2, 1, 16)
        side.synchronize()
        assert torch.equal(y, z)
    # the second graph on the first case's inputs
    for dst, src in zip(bufs[1][0], cases[0][:5]):
        dst.copy_(src)
    graphs[1].replay()
    _clean(hga)
    _check(bufs[1][1], cases[0][5], cases[0][6])


@pytest.mark.parametrize("sections", [None, (16, 24, 24)])
def test_prefill_then_decode(sections):
    """A prefill and a decode loop over the 4-bit store (rotation, summaries, store,
    routing, attention), each step against the definition on the store as it is."""
    from long_context_rope_b200 import hga, pipeline
    B, H, L0, steps = 2, 2, 250, 9
    cap = L0 + steps
    cfg = _cfg4(hga, batch=B, n_kv_heads=H, n_q_heads=16, seq_len=cap, top_k_groups=6, top_k_chunks=3,
                n_local=1, k_scale=2.0 ** -8, v_scale=2.0 ** -9)
    g = torch.Generator().manual_seed(70)
    k = _rows((B, H, cap, 128), 71)
    v = _rows((B, H, cap, 128), 72)
    q = _rows((B, cap, 16, 128), 73)
    axes = pair = pos = None
    if sections:
        pair = hga.pair_axes(64, sections)
        axes = hga.rope_axes(pair, len(sections))
        pos = torch.randint(0, 300, (len(sections), B, cap), generator=g, dtype=torch.int32).cuda()
    kd, vd, qd = k.cuda(), v.cuda(), q.cuda()
    kc = torch.zeros_like(kd)
    kc[:, :, :L0] = kd[:, :, :L0]
    ks, vs = pipeline.alloc_store(cfg)
    cs, gs = pipeline.alloc_summaries(cfg)
    cs.zero_(), gs.zero_()
    part = lambda a, b: None if pos is None else pos[:, :, a:b].contiguous()

    c0 = cfg.copy(seq_len=L0, q_begin=0, q_len=L0)
    cs0, gs0 = pipeline.alloc_summaries(c0)
    ks0, vs0 = pipeline.alloc_store(c0)
    q0 = pipeline.rotate_queries(c0, qd[:, :L0].contiguous(), axes=axes, positions=part(0, L0))
    rb0, out0 = pipeline.alloc_route(c0), torch.empty_like(q0)
    pipeline.prefill(c0, kd[:, :, :L0].contiguous(), vd[:, :, :L0].contiguous(), q0, cs0, gs0, ks0, rb0,
                     out0, v_store=vs0, axes=axes, positions=part(0, L0))
    _clean(hga)
    ks[:, :, :ks0.shape[2]], vs[:, :, :vs0.shape[2]] = ks0, vs0
    cs[:, :, :cs0.shape[2]], gs[:, :, :gs0.shape[2]] = cs0, gs0
    val = lambda st, ts: R.values(st.cpu(), ts)
    want, tol = R.attend(c0, q0.cpu(), val(ks0, cfg.k_scale), val(vs0, cfg.v_scale),
                         rb0.sel_groups.cpu(), rb0.n_sel_groups.cpu())
    _check(out0, want, tol)
    # the store holds the rotated keys: half a step of a code is a sixth of a block's largest
    p64 = torch.arange(cap).expand(1, B, cap) if pos is None else pos.cpu()
    rot = R.rotate(k, R.angles(p64, pair or [0] * 64, 1e4, 128)[:, None])
    big = rot.unflatten(-1, (8, 16)).abs().amax(-1).repeat_interleave(16, -1)
    assert bool(((val(ks0, cfg.k_scale)[:, :, :L0] - rot[:, :, :L0]).abs()
                 <= big[:, :, :L0] * (1 / 6 + 2.0 ** -3)).all())

    rb = pipeline.alloc_route(cfg.copy(q_begin=L0, q_len=1))
    for t in range(L0, cap):
        qr = pipeline.rotate_queries(cfg.copy(q_begin=t, q_len=1), qd[:, t:t + 1].contiguous(),
                                     axes=axes, positions=part(t, t + 1))
        out = torch.full_like(qr, float("nan"))
        pipeline.decode_append(cfg, t, kd[:, :, t], vd[:, :, t], qr, kc, ks, vs, cs, gs, rb, out,
                               axes=axes, positions=pos)
        _clean(hga)
        ct = cfg.copy(q_begin=t, q_len=1)
        want, tol = R.attend(ct, qr.cpu(), val(ks, cfg.k_scale), val(vs, cfg.v_scale),
                             rb.sel_groups.cpu(), rb.n_sel_groups.cpu())
        _check(out, want, tol)
    full = R.quantise(rot.float(), cfg.k_scale)
    assert (val(ks, cfg.k_scale)[:, :, :cap] != R.values(R.pack(*full), cfg.k_scale)[:, :, :cap]).sum() <= 2
    # the chunk that the loop completed has the summaries of one call over all tokens
    cs1, gs1 = pipeline.alloc_summaries(cfg)
    pipeline.summaries(cfg, kd, cs1, gs1, axes=axes, positions=pos)
    n = cap // 64
    assert torch.equal(cs[:, :, :n], cs1[:, :, :n]) and torch.equal(gs[:, :, :4 * n], gs1[:, :, :4 * n])


def test_append_axes_bf16():
    """The decode loop over bf16 caches with several axes: rotated keys and summaries
    as of one call over all tokens."""
    from long_context_rope_b200 import hga, pipeline
    B, H, L = 2, 2, 70
    cfg = _cfg(hga, batch=B, n_kv_heads=H, n_q_heads=8, seq_len=L)
    k, v, q = (_rows(s, i).cuda() for i, s in enumerate([(B, H, L, 128), (B, H, L, 128), (B, 1, 8, 128)]))
    axes = hga.rope_axes(hga.pair_axes(64, (20, 20, 20), True), 3)
    pos = torch.randint(0, 300, (3, B, L), device="cuda", dtype=torch.int32)
    kc, kr, vc = (torch.zeros_like(k) for _ in range(3))
    cs, gs = pipeline.alloc_summaries(cfg)
    out = torch.empty_like(q)
    rb = pipeline.alloc_route(cfg)
    for t in range(L):
        pipeline.decode_append(cfg, t, k[:, :, t], v[:, :, t], q, kc, kr, vc, cs, gs, rb, out,
                               axes=axes, positions=pos)
    _clean(hga)
    cs1, gs1 = pipeline.alloc_summaries(cfg)
    kr1 = torch.empty_like(k)
    pipeline.summaries(cfg, k, cs1, gs1, kr1, axes=axes, positions=pos)
    assert torch.equal(cs[:, :, :1], cs1[:, :, :1]) and torch.equal(gs[:, :, :4], gs1[:, :, :4])
    d = (kr.float() - kr1.float()).abs()
    assert bool((d <= 2 * R.BF16 * kr1.float().abs() + 2.0 ** -18).all())


# ------------------------------------------------- the other ways to a result
STEPS = [dict(seq_len=1024), dict(seq_len=999, n_q_heads=10), dict(seq_len=1000, q_begin=700),
         dict(seq_len=2000, summary_type=1), dict(seq_len=777, routing=1),
         dict(seq_len=1100, n_q_heads=24), dict(seq_len=3000, top_k_chunks=100, n_local=1),
         dict(seq_len=40), dict(seq_len=640, chunk_size=128, groups_per_chunk=8)]


@pytest.mark.parametrize("kw", STEPS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_decode_step(kw):
    """hga_decode_step over the 4-bit store: the selections of hga_route, and attention
    over them; where the cache may lie in host memory, the tiered step the same."""
    from long_context_rope_b200 import hga, pipeline
    kw = dict(dict(batch=2, n_kv_heads=2, n_q_heads=16, q_begin=kw["seq_len"] - 1), **kw)
    cfg = _cfg4(hga, **kw)
    q, kp, vp, _, _, _, _ = _attend_case(hga, cfg, 80, count=0)
    qd, kd, vd = q.cuda(), kp.cuda(), vp.cuda()
    cs, gs = pipeline.alloc_summaries(cfg)
    g = torch.Generator(device="cuda").manual_seed(81)
    cs.copy_(torch.randn(cs.shape, device="cuda", generator=g))
    gs.copy_(torch.randn(gs.shape, device="cuda", generator=g))
    rb0, rb = pipeline.alloc_route(cfg), pipeline.alloc_route(cfg)
    pipeline.route(cfg, qd, cs, gs, rb0)
    kv = [torch.nan_to_num(R.values(p, ts)) for p, ts in ((kp, cfg.k_scale), (vp, cfg.v_scale))]
    want, tol = R.attend(cfg, q, *kv, rb0.sel_groups.cpu(), rb0.n_sel_groups.cpu())

    def check(step, name):
        out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
        try:
            step(out)
        except hga.HgaError as e:   # 12 heads a KV head, 100 chunks: separate calls only
            assert name == "tiered" and "UNSUPPORTED" in str(e)
            assert cfg.n_q_heads == 24 or cfg.top_k_chunks == 100
            return
        _clean(hga)
        assert torch.equal(rb.sel_groups, rb0.sel_groups) and torch.equal(rb.sel_chunks, rb0.sel_chunks)
        assert torch.equal(rb.qbar, rb0.qbar)
        _check(out, want, tol)
    check(lambda out: pipeline.decode(cfg, qd, cs, gs, kd, vd, rb, out), "step")
    if cfg.q_begin == cfg.seq_len - 1:
        cfg_w = cfg.copy(kv_layout=hga.HGA_KV_WINDOWS)
        rows = hga.window_slots(cfg) * cfg.chunk_size
        win = [torch.zeros(cfg.kv_rows(2, 2, rows=rows), dtype=torch.uint8, device="cuda") for _ in "kv"]
        kh, vh = kp.pin_memory(), vp.pin_memory()
        pipeline.fill_windows(cfg, kh, vh, *win)
        check(lambda out: pipeline.decode_tiered(cfg_w, qd, cs, gs, *win, kh, vh, rb, out), "tiered")


MORE = [dict(seq_len=200, chunk_size=16, groups_per_chunk=1), dict(seq_len=500, chunk_size=128,
                                                                    groups_per_chunk=8),
        dict(seq_len=150, n_q_heads=16), dict(seq_len=150, n_q_heads=7), dict(seq_len=70, n_q_heads=128),
        dict(seq_len=70, n_q_heads=130), dict(seq_len=900, top_k_groups=400, n_local=1)]


@pytest.mark.parametrize("kw", MORE, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
@pytest.mark.parametrize("gathered", [False, True])
def test_attend_more_shapes(kw, gathered):
    """Chunks of one group and of eight, many heads, long lists; each as a prefill of the
    last 40 tokens and as a decode step; from the store and from gathered buffers."""
    from long_context_rope_b200 import hga, pipeline
    for n in (40, 1):
        cfg = _cfg4(hga, **dict(kw, q_begin=kw["seq_len"] - n, q_len=n))
        q, kp, vp, sel, cnt, want, tol = _attend_case(hga, cfg, 90)
        qd, kd, vd, sd, nd = (t.cuda() for t in (q, kp, vp, sel, cnt))
        gat = (None, None)
        if gathered:
            gat = pipeline.alloc_gathered(cfg)
            hga.gather_kv(cfg, kd, vd, False, sd, nd, *gat)
        out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
        hga.attend(cfg, qd, kd, vd, sd, nd, out, k_gat=gat[0], v_gat=gat[1])
        again = torch.empty_like(out)
        hga.attend(cfg, qd, kd, vd, sd, nd, again, k_gat=gat[0], v_gat=gat[1])
        _clean(hga)
        _check(out, want, tol)
        assert torch.equal(out, again)   # no sum depends on the order of arrival


def test_attend_per_query_head():
    """Lists of a query head's own, in one call and on two streams at once."""
    from long_context_rope_b200 import hga
    cases = []
    for seed in (100, 101):
        cfg = _cfg4(hga, seq_len=1500, q_begin=1499, batch=2, n_kv_heads=2, n_q_heads=8,
                    routing=hga.HGA_ROUTE_PER_Q_HEAD)
        cases.append((cfg, _attend_case(hga, cfg, seed)))
    streams = [torch.cuda.Stream() for _ in cases]
    args = [[t.cuda() for t in c[:5]] for _, c in cases]
    outs = [torch.full(c[0].shape, float("nan"), dtype=BF, device="cuda") for _, c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for (cfg, _), st, a, out in zip(cases, streams, args, outs):
            hga.attend(cfg, *a, out, stream=st)
    _clean(hga)
    for (_, c), out in zip(cases, outs):
        _check(out, c[5], c[6])


def test_prefill_wait_limit():
    """A prefill whose waits may last a nanosecond ends, with or without an error, and the
    next one is right."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=512, q_len=512)
    c = _attend_case(hga, cfg, 110)
    args = [t.cuda() for t in c[:5]]
    out = torch.empty_like(args[0])
    hga.set_wait_limit_ns(1)
    try:
        hga.attend(cfg, *args, out)
        torch.cuda.synchronize()
        hga.get_device_error()
    finally:
        hga.set_wait_limit_ns(0)
    hga.attend(cfg, *args, out)
    _clean(hga)
    _check(out, c[5], c[6])


def test_offsets_past_32_bits():
    """A store of 4.8 GB per tensor (rows, pages and bytes past 2^31 and 2^32): the last
    tokens written, read back and attended to as in a short store."""
    from long_context_rope_b200 import hga
    L, n = 1 << 20, 512
    cfg = _cfg4(hga, batch=8, n_kv_heads=8, n_q_heads=16, seq_len=L, q_begin=L - 1, n_sink=0)
    short = cfg.copy(seq_len=n, q_begin=n - 1)
    k, v = _rows((8, 8, n, 128), 120).cuda(), _rows((8, 8, n, 128), 121).cuda()
    q = _rows((8, 1, 16, 128), 122).cuda()
    sel, cnt = R.lists(short, 8, 123)
    outs, loads = [], []
    for c in (cfg, short):
        shift = c.seq_len - n
        ks = torch.zeros(c.kv_rows(8, 8, rows=c.seq_len), dtype=torch.uint8, device="cuda")
        vs = torch.zeros_like(ks)
        hga.store_kv(c, k, v, ks, vs, shift, axes=hga.rope_axes([0, 1] * 32, 2),
                     positions=torch.arange(2 * 8 * n, device="cuda", dtype=torch.int32).view(2, 8, n))
        ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        hga.load_kv(c, ks, vs, ko, vo, shift)
        moved = torch.where(sel >= 0, sel + shift // 16, sel).cuda()
        hga.attend(c, q, ks, vs, moved, cnt.cuda(), out)
        _clean(hga)
        assert not ks[:, :, :shift // 16].any() and not vs[:, :, :shift // 16].any()
        outs.append(out)
        loads.append((ko, vo))
        del ks, vs
    assert torch.equal(*outs) and torch.equal(loads[0][0], loads[1][0])
    assert torch.equal(loads[0][1], loads[1][1])


def test_large_calls():
    """More rows than one launch of the store takes, and a rotation of more than 2^31
    elements: as the same work in parts."""
    from long_context_rope_b200 import hga
    n = 70000
    cfg = _cfg4(hga, batch=8, n_kv_heads=8, n_q_heads=8, seq_len=n)
    k = torch.randn(8, 8, n, 128, device="cuda", dtype=BF)
    axes = hga.rope_axes([0] * 64, 1)
    st = [torch.zeros(cfg.kv_rows(8, 8, rows=n), dtype=torch.uint8, device="cuda") for _ in range(4)]
    hga.store_kv(cfg, k, k, st[0], st[1], 0, axes=axes)
    for a, b in ((0, 33333), (33333, n)):
        part = k[:, :, a:b].contiguous()
        hga.store_kv(cfg, part, part, st[2], st[3], a, axes=axes)
    assert torch.equal(st[0], st[2]) and torch.equal(st[1], st[3])
    o = [torch.empty_like(k) for _ in range(2)]
    hga.load_kv(cfg, st[0], st[1], *o, 0)
    part = torch.empty(8, 8, 1234, 128, device="cuda", dtype=BF), torch.empty(8, 8, 1234, 128, device="cuda",
                                                                             dtype=BF)
    hga.load_kv(cfg, st[0], st[1], *part, n - 1234)
    assert torch.equal(o[0][:, :, n - 1234:], part[0]) and torch.equal(o[1][:, :, n - 1234:], part[1])
    del o, part, st, k
    T = (1 << 18) + 3
    x = torch.randn(1, T, 64, 128, device="cuda", dtype=BF)
    pos = torch.randint(0, 1 << 20, (2, 1, T), device="cuda", dtype=torch.int32)
    axes = hga.rope_axes([0, 1] * 32, 2)
    last = x[:, -5:].clone()
    hga.apply_rope_axes(cfg, axes, pos, x, x, 1, T, 64)
    y = torch.empty_like(last)
    hga.apply_rope_axes(cfg, axes, pos[:, :, -5:].contiguous(), last, y, 1, 5, 64)
    _clean(hga)
    assert torch.equal(x[:, -5:], y)


def test_other_device_is_refused():
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=16, q_begin=15)
    k = torch.zeros(1, 1, 16, 128, dtype=BF)
    st = torch.zeros(1, 1, 1, 1152, dtype=torch.uint8, device="cuda")
    for bad in (k, k.cuda().transpose(2, 3).contiguous().transpose(2, 3), k.cuda().float()):
        with pytest.raises(ValueError):
            hga.store_kv(cfg, bad, k.cuda(), st, st, 0)


@pytest.mark.parametrize("kv4,handle", [(False, False), (True, False), (True, True)])
def test_append_on_another_stream(kv4, handle):
    """A decode step given a stream runs on it whole: its copies do not wait for what the
    current stream is busy with, so the step sees its own token there."""
    from long_context_rope_b200 import hga, pipeline
    L0, kw = 70, dict(batch=1, n_kv_heads=2, n_q_heads=16, seq_len=128)
    cfg = _cfg4(hga, **kw) if kv4 else _cfg4(hga, kv_type=hga.HGA_KV_AS_DTYPE, **kw)
    k, v = _rows((1, 2, 128, 128), 90).cuda(), _rows((1, 2, 128, 128), 91).cuda()
    axes = hga.rope_axes([0, 1] * 32, 2)
    pos = torch.randint(0, 99, (2, 1, 128), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(92)).cuda()
    q = _rows((1, 1, 16, 128), 93).cuda()
    outs = []
    side = torch.cuda.Stream()
    for other in (False, True):
        kc = torch.zeros_like(k)
        kr, vs = pipeline.alloc_store(cfg)
        cs, gs = pipeline.alloc_summaries(cfg)
        cs.zero_(), gs.zero_()
        rb = pipeline.alloc_route(cfg.copy(q_begin=0, q_len=1))
        out = torch.full_like(q, float("nan"))
        torch.cuda.synchronize()
        if other:
            torch.cuda._sleep(400_000_000)  # some 0.2 s of the current stream
        st = None if not other else (side.cuda_stream if handle else side)
        for t in range(60, L0):             # a chunk's end among them
            pipeline.decode_append(cfg, t, k[:, :, t], v[:, :, t], q, kc, kr, vs, cs, gs, rb, out,
                                   stream=st, axes=axes, positions=pos)
        side.synchronize()
        got = [x.to("cpu") for x in (out, kc, kr, vs, cs[:, :, :1], gs[:, :, :4])] if not other else None
        if other:
            with torch.cuda.stream(side):
                got = [x.clone() for x in (out, kc, kr, vs, cs[:, :, :1], gs[:, :, :4])]
            torch.cuda.synchronize()
            got = [x.cpu() for x in got]
        _clean(hga)
        outs.append(got)
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# spans around the 592 units (tokens x sequences x KV heads) up to which they go token by
# token, on either side; chunks and query blocks that begin and end inside a span
SPANS = [dict(q_begin=100, q_len=592, seq_len=700), dict(q_begin=100, q_len=593, seq_len=700),
         dict(q_begin=61, q_len=148, seq_len=209, n_kv_heads=2, n_q_heads=16, batch=2),
         dict(q_begin=61, q_len=149, seq_len=215, n_kv_heads=2, n_q_heads=16, batch=2),
         dict(q_begin=500, q_len=3, seq_len=520, n_kv_heads=4, n_q_heads=12, batch=3),
         dict(q_begin=63, q_len=2, seq_len=200, n_sink=0, n_local=0),
         dict(q_begin=40, q_len=700, seq_len=740, n_q_heads=3),
         dict(q_begin=40, q_len=300, seq_len=345, n_q_heads=2, n_kv_heads=1, batch=2),
         dict(q_begin=0, q_len=320, seq_len=320, batch=2, n_sink=2, n_local=0),
         dict(q_begin=190, q_len=220, seq_len=420, chunk_size=48, groups_per_chunk=3, batch=3)]


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("kw", SPANS, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_attend_spans(kw, gathered):
    """Short and long spans of queries, from the store or from gathered groups."""
    from long_context_rope_b200 import hga, pipeline
    cfg = _cfg4(hga, **kw)
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 96)
    q, kp, vp, sel, n = (x.cuda() for x in (q, kp, vp, sel, n))
    out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
    gat = {}
    if gathered:
        kg, vg = pipeline.alloc_gathered(cfg)
        hga.gather_kv(cfg, kp, vp, False, sel, n, kg, vg)
        gat = dict(k_gat=kg, v_gat=vg)
    hga.attend(cfg, q, kp, vp, sel, n, out, **gat)
    _clean(hga)
    _check(out, want, tol)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (torch.float32, 128), (BF, 64), (torch.float32, 64)])
@pytest.mark.parametrize("rep,heads,T", [(1, 1, 9001), (4, 1, 7659), (1, 5, 12007), (3, 2, 5003), (1, 9, 6001)])
def test_rope_of_few_rows_equals_its_parts(dtype, d, rep, heads, T):
    """Many tokens of few rows each: how rows fall to threads changes with the size of the
    call, their values do not."""
    from long_context_rope_b200 import hga
    B = 2
    cfg = _cfg(hga, batch=B, head_dim=d, n_high_freq_pairs=0, dtype="bf16" if dtype == BF else "f32")
    axes = hga.rope_axes(hga.pair_axes(d // 2, [d // 4, d // 8]), 2)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(-100, 1 << 18, (2, B, T), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(B * rep, T, heads, d, generator=g).to(dtype).cuda()
    y = torch.full_like(x, float("nan"))
    hga.apply_rope_axes(cfg, axes, pos, x, y, B * rep, T, heads)
    for a, b in ((0, 37), (T // 2, T // 2 + 40), (T - 29, T)):
        part = x[:, a:b].contiguous()
        got = torch.empty_like(part)
        hga.apply_rope_axes(cfg, axes, pos[:, :, a:b].contiguous(), part, got, B * rep, b - a, heads)
        assert torch.equal(y[:, a:b], got)
    _clean(hga)

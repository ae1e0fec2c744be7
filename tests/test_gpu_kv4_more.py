"""More of the 4-bit store, its attention and rotary positions with several axes on a
GPU: calls that the documentation allows, each against kv4_ref.py or a longer call."""
import math

import pytest
import torch

import kv4_ref as R
from test_gpu_kv4 import BF, _attend_case, _cfg, _cfg4, _check, _clean, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv4", [False, True])
def test_append_one_axis_of_one_sequence(kv4):
    """Token after token with positions on one axis: what one call over all tokens
    gives, bit by bit (each slice of the positions is contiguous where it lies)."""
    from long_context_rope_b200 import hga, pipeline
    H, L = 2, 70
    kw = dict(n_kv_heads=H, n_q_heads=16, seq_len=L)
    cfg = _cfg4(hga, **kw) if kv4 else _cfg(hga, **kw)
    k, v, q = _rows((1, H, L, 128), 1).cuda(), _rows((1, H, L, 128), 2).cuda(), _rows((1, 1, 16, 128), 3).cuda()
    axes = hga.rope_axes([0] * 40 + [-1] * 24, 1)
    pos = torch.randint(0, 5000, (1, 1, L), generator=torch.Generator().manual_seed(4),
                        dtype=torch.int32).cuda()
    kc = torch.zeros_like(k)
    kr, vs = pipeline.alloc_store(cfg)
    cs, gs = pipeline.alloc_summaries(cfg)
    rb, out = pipeline.alloc_route(cfg), torch.empty_like(q)
    want = torch.empty_like(k)
    # rows in the order in which the step turns them: a token of every head
    hga.apply_rope_axes(cfg, axes, pos, k, want, H, L, 1)
    turned = []
    for t in range(L):
        at = pos[:, :, t:t + 1].contiguous()
        turned.append(pipeline.rotate_queries(cfg.copy(q_begin=t, q_len=1), q, axes=axes, positions=at))
        pipeline.decode_append(cfg, t, k[:, :, t], v[:, :, t], turned[-1], kc, kr, vs, cs, gs, rb, out,
                               axes=axes, positions=pos)
    _clean(hga)
    assert torch.equal(kc, k)
    if kv4:
        ks1, vs1 = pipeline.alloc_store(cfg)
        hga.store_kv(cfg, k, v, ks1, vs1, 0, axes=axes, positions=pos)
        assert torch.equal(kr, ks1) and torch.equal(vs, vs1)
    else:
        assert torch.equal(kr, want) and torch.equal(vs, v)
    all_q = torch.empty(1, L, 16, 128, dtype=BF, device="cuda")
    hga.apply_rope_axes(cfg, axes, pos, q.expand(1, L, 16, 128).contiguous(), all_q, 1, L, 16)
    assert torch.equal(torch.cat(turned, 1), all_q)


def _to_bf16(x):
    """64-bit numbers rounded once to bf16 (nearest even), as 64-bit numbers."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-125) - 8)   # 8 bits; subnormals below 2^-126
    r = torch.round(x / step) * step
    return torch.where(r.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(r, float("inf")), r), r)


# scales under which a product rounded to fp32 first becomes a tie between two bf16 numbers and
# goes the wrong way; ordinary ones; those near fp32's ends
@pytest.mark.parametrize("scale", [float.fromhex(s) for s in (
    "0x1.e6aaacp-9", "0x1.45b6dcp-9", "0x1.5c924ap-9", "0x1.b364dap-9", "0x1.18e38ep-9", "0x1.18e38ep-99",
    "0x1.45b6dcp-101", "0x1.b364dap-126", "0x1.18e38p-130", "0x1p-149", "0x1p-8", "0x1.8p-8", "0x1.333334p-2",
    "0x1.e6aaacp+40", "0x1.b364dap+125", "0x1.fffffep+127")])
def test_load_rounds_once(scale):
    """Every code under every scale byte."""
    from long_context_rope_b200 import hga
    ts = float(torch.tensor(scale, dtype=torch.float32))
    assert ts == scale
    cfg = _cfg4(hga, seq_len=32, k_scale=scale, v_scale=1.0)
    code = (torch.arange(32 * 128) % 16).to(torch.uint8).view(1, 1, 32, 128)
    byte = torch.arange(256).to(torch.uint8).view(1, 1, 32, 8)
    pages = R.pack(code, byte)
    want = _to_bf16(R.values(pages, ts))
    k = torch.empty(1, 1, 32, 128, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    p = pages.cuda()
    hga.load_kv(cfg, p, p, k, v, 0)
    _clean(hga)
    got, nan = k.cpu().double(), torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    assert torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))
    v = v.cpu().double()
    assert torch.equal(v[~nan], R.values(pages, 1.0)[~nan])


# ------------------------------------------- the prefill kernel on the tensor cores
# Spans of more than 592 units (tokens x sequences x KV heads) of at most 8 heads a KV head, and any of
# more heads: what the kernel of single tokens does not take.
def _tc(cfg):
    assert (cfg.n_q_heads // cfg.n_kv_heads > 8
            or cfg.q_len * cfg.batch * cfg.n_kv_heads > 592), "not the prefill kernel's"
    return cfg


TC = [(639, 1, 16), (512, 128, 16), (560, 33, 16), (575, 3, 12), (0, 640, 8), (30, 605, 3)]


@pytest.mark.parametrize("order", ["rising", "falling", "mixed", "late"])
@pytest.mark.parametrize("q_begin,q_len,heads", TC)
def test_prefill_scores_that_rise(order, q_begin, q_len, heads):
    """Keys whose scores grow by orders of magnitude from tile to tile, for some heads only:
    weights against the first tile's maximum would pass fp16's range, so it is raised and what
    was summed shrinks. late: the routed groups, which come after the near chunks."""
    from long_context_rope_b200 import hga
    cfg = _tc(_cfg4(hga, seq_len=640, q_begin=q_begin, q_len=q_len, n_q_heads=heads,
                    n_sink=0 if order == "late" else 1, n_local=1, top_k_groups=24, k_scale=2.0 ** -4))
    k = _rows((1, 1, 640, 128), 130).float()
    size = torch.arange(640) / 16
    size = {"rising": size, "falling": 40 - size, "mixed": (size * 7) % 40,
            "late": size * (torch.arange(640) < 512)}[order].floor()
    k *= (1 + size)[:, None] ** 1.5
    q = _rows((1, q_len, heads, 128), 131)
    q[:, :, :heads // 3] *= 0.01
    kp = R.pack(*R.quantise(k.to(BF), cfg.k_scale))
    vp = R.pack(*R.quantise(_rows((1, 1, 640, 128), 132), cfg.v_scale))
    sel, n = R.lists(cfg, 1, 133)
    kv = R.values(kp, cfg.k_scale), R.values(vp, cfg.v_scale)
    if order == "late" and q_begin + q_len == 640:
        # the last row, tile by tile: its largest weight against its first tile's maximum
        at = R.visible(cfg, torch.empty(0, dtype=torch.int32), 0, 639)
        far = torch.cat([torch.arange(16 * g, 16 * g + 16) for g in sel[0, 0, -1, :n[0, 0, -1]].tolist()])
        s = kv[0][0, 0] @ q[0, -1, -1].double() / 128 ** 0.5 / math.log(2)
        assert float(s[far].max() - s[at].max()) > 13, "no raise after the first tile"
    want, tol = R.attend(cfg, q, *kv, sel, n)
    out = torch.full(q.shape, float("nan"), dtype=BF, device="cuda")
    hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
    _clean(hga)
    _check(out, want, tol)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_begin,q_len,heads", [(199, 1, 16), (128, 40, 16), (150, 30, 9), (30, 600, 8)])
def test_prefill_nan_row(which, q_begin, q_len, heads):
    """A row with a NaN scale reaches the queries that see it, and no other."""
    from long_context_rope_b200 import hga
    long = q_len > 100
    cfg = _tc(_cfg4(hga, seq_len=640 if long else 256, q_begin=q_begin, q_len=q_len, n_q_heads=heads,
                    n_local=0, n_sink=0))
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 30, count=0)
    for bad in ([q_begin + q_len // 2] if not long else [70, 127, 128, 333]):
        p = (kp if which == "k" else vp).clone()
        p[0, 0, bad // 16, 1024 + (bad % 16) * 8 + 3] = 0x7F
        out = torch.empty_like(q).cuda()
        pair = (p, vp) if which == "k" else (kp, p)
        hga.attend(cfg, q.cuda(), pair[0].cuda(), pair[1].cuda(), sel.cuda(), n.cuda(), out)
        _clean(hga)
        at = q_begin + torch.arange(q_len)
        seen = (at >= bad) & (at // 64 == bad // 64)   # no lists: a query's own chunk alone
        got = out.cpu().double()
        assert bool(seen.any()) and torch.isnan(got[0, seen][..., 48:64]).all()
        assert bool(((got - want).abs()[0, ~seen] <= tol[0, ~seen]).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_begin,q_len,heads", [(199, 1, 16), (64, 140, 16), (150, 30, 11), (0, 610, 8)])
def test_prefill_nan_query(value, q_begin, q_len, heads):
    """A query with a NaN or an infinity makes its own row NaN, and no other."""
    from long_context_rope_b200 import hga
    cfg = _tc(_cfg4(hga, seq_len=620, q_begin=q_begin, q_len=q_len, n_q_heads=heads))
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


@pytest.mark.parametrize("kw", [dict(q_begin=511, n_q_heads=16), dict(q_begin=448, q_len=64, n_q_heads=16),
                                dict(q_begin=449, q_len=63, batch=10),
                                dict(q_begin=511), dict(q_begin=480, q_len=4, n_q_heads=3)])  # token by token
def test_bad_lists_and_counts_by_either_kernel(kw):
    """An invalid entry is left out and reported; a count past its list is cut and reported;
    the rest of the unit, and the other units, stand."""
    from long_context_rope_b200 import hga
    cfg = _cfg4(hga, seq_len=512, **kw)
    q, kp, vp, sel, n, _, _ = _attend_case(hga, cfg, 50, count=6)
    kv = [torch.nan_to_num(R.values(p, ts)) for p, ts in ((kp, cfg.k_scale), (vp, cfg.v_scale))]

    def run(sel, n, good):
        want, tol = R.attend(cfg, q, kv[0], kv[1], sel, good)
        out = torch.empty_like(q).cuda()
        hga.attend(cfg, q.cuda(), kp.cuda(), vp.cuda(), sel.cuda(), n.cuda(), out)
        torch.cuda.synchronize()
        code = hga.get_device_error()
        assert hga.get_device_error() == 0
        _check(out, want, tol)
        return code
    assert run(sel, n, n) == 0
    bad, good = sel.clone(), n.clone()
    bad[0, 0, 0, 5] = 4 * 7 + 1   # of the current chunk
    good[0, 0, 0] = 5
    assert run(bad, n, good) == 2
    full, cnt = R.lists(cfg, 1, 50)   # every entry of the list is good, the count is not
    assert int(cnt[0, 0, 0]) == cfg.top_k_groups
    wrong = cnt.clone()
    wrong[0, 0, 0] = cfg.top_k_groups + 1
    assert run(full, wrong, cnt) == 3
    wrong[0, 0, 0] = -1
    good = cnt.clone()
    good[0, 0, 0] = 0
    assert run(full, wrong, good) == 3


@pytest.mark.parametrize("kw", [dict(seq_len=640, q_len=640), dict(seq_len=512, q_len=512, n_q_heads=16)])
def test_prefill_waits_that_run_out(kw):
    """Waits that may last a nanosecond (a tile's products, a tile's weights) run out: the launch
    says so and ends, and the same launch afterwards is as before, bit by bit."""
    from long_context_rope_b200 import hga
    cfg = _tc(_cfg4(hga, **kw))
    c = _attend_case(hga, cfg, 110)
    args = [t.cuda() for t in c[:5]]
    first, out = torch.empty_like(args[0]), torch.empty_like(args[0])
    hga.attend(cfg, *args, first)
    _clean(hga)
    _check(first, c[5], c[6])
    hga.set_wait_limit_ns(1)
    try:
        hga.attend(cfg, *args, out)
        torch.cuda.synchronize()
        assert hga.get_device_error() == 4
    finally:
        hga.set_wait_limit_ns(0)
    hga.attend(cfg, *args, out)
    _clean(hga)
    assert torch.equal(out, first)


def test_prefill_streams_and_graphs():
    """Two prefills at once on two streams, and one captured and replayed on new inputs."""
    from long_context_rope_b200 import hga
    cfg = _tc(_cfg4(hga, seq_len=700, q_begin=380, q_len=320, batch=2, n_q_heads=8))
    cases = [_attend_case(hga, cfg, s) for s in (140, 141)]
    args = [[t.cuda() for t in c[:5]] for c in cases]
    outs = [torch.full(c[0].shape, float("nan"), dtype=BF, device="cuda") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for a, o, st in zip(args, outs, streams):
            hga.attend(cfg, *a, o, stream=st)
    _clean(hga)
    for c, o in zip(cases, outs):
        _check(o, c[5], c[6])
    g = torch.cuda.CUDAGraph()
    buf, out = [t.clone() for t in args[0]], torch.empty_like(outs[0])
    with torch.cuda.graph(g):
        hga.attend(cfg, *buf, out)
    for a, o in zip(args, outs):
        for dst, src in zip(buf, a):
            dst.copy_(src)
        g.replay()
        _clean(hga)
        assert torch.equal(out, o)


def test_prefill_offsets_past_32_bits():
    """Over a store of 4.8 GB per tensor as over a short one."""
    from long_context_rope_b200 import hga
    L, n, T = 1 << 20, 512, 16
    cfg = _tc(_cfg4(hga, batch=8, n_kv_heads=8, n_q_heads=16, seq_len=L, q_begin=L - T, q_len=T, n_sink=0))
    short = _tc(cfg.copy(seq_len=n, q_begin=n - T))
    k, v = _rows((8, 8, n, 128), 120).cuda(), _rows((8, 8, n, 128), 121).cuda()
    q = _rows((8, T, 16, 128), 122).cuda()
    sel, cnt = R.lists(short, 8, 123)
    outs = []
    for c in (cfg, short):
        shift = c.seq_len - n
        ks = torch.zeros(c.kv_rows(8, 8, rows=c.seq_len), dtype=torch.uint8, device="cuda")
        vs, out = torch.zeros_like(ks), torch.empty_like(q)
        hga.store_kv(c, k, v, ks, vs, shift)
        moved = torch.where(sel >= 0, sel + shift // 16, sel).cuda()
        hga.attend(c, q, ks, vs, moved, cnt.cuda(), out)
        _clean(hga)
        outs.append(out)
        del ks, vs
    assert torch.equal(*outs) and bool(torch.isfinite(outs[0].float()).all())


# ------------------------------------------------------------------ positions
SUMS = [("bf16", 128, 20), ("f32", 64, 0), ("f32", 128, 64), ("bf16", 64, 7), ("bf16", 128, 0), ("f32", 128, 33)]


@pytest.mark.parametrize("dtype,d,F", SUMS)
@pytest.mark.parametrize("tables", ["f32", "bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("B,H,L,C,every", [(1, 1, 1, 64, False), (2, 3, 200, 64, True), (1, 9, 129, 128, False),
                                           (2, 1, 96, 32, True), (1, 2, 100, 48, False)])
def test_summaries_axes_tables(dtype, d, F, tables, rotated, B, H, L, C, every):
    """Tables of fp32 and bf16, with and without the rotated keys, against the definition; pairs on
    no axis are plain means. Rows of chunks outside the call stay as they were."""
    from long_context_rope_b200 import hga, pipeline
    if (d // 2 // (8 if dtype == "bf16" else 4)) * 4 * (C // 16) % 32:
        pytest.skip("the framework's configurations do not have this one")
    cfg = _cfg(hga, batch=B, n_kv_heads=H, n_q_heads=H, seq_len=L, head_dim=d, dtype=dtype,
               n_high_freq_pairs=min(F, d // 2), chunk_size=C, groups_per_chunk=C // 16,
               summary_type=int(tables == "bf16"))
    g = torch.Generator().manual_seed(19)
    k = torch.randn(B, H, L, d, generator=g).to(cfg.torch_dtype())
    pair = hga.pair_axes(d // 2, (d // 4, d // 8, d // 8) if every else (d // 8, d // 8, d // 8), True)
    pos = torch.randint(-1000, 100000, (3, B, L), generator=g, dtype=torch.int32)
    cs, gs = pipeline.alloc_summaries(cfg)
    cs.fill_(7.0), gs.fill_(7.0)
    rot = torch.full_like(k, 7.0).cuda() if rotated else None
    c0 = 1 if L > C else 0
    pipeline.summaries(cfg, k.cuda(), cs, gs, rot, axes=hga.rope_axes(pair, 3), positions=pos.cuda(),
                       chunk_begin=c0)
    _clean(hga)
    turned = R.rotate(k, R.angles(pos, pair, 1e4, d)[:, None])
    mag = (k.double().abs()[..., :d // 2] + k.double().abs()[..., d // 2:]).repeat(1, 1, 1, 2)
    u = R.BF16 if dtype == "bf16" else R.F32
    if rotated:
        assert bool((rot[:, :, :c0 * C] == 7.0).all())
        err = (rot.cpu().double() - turned).abs()[:, :, c0 * C:]
        # the sine and cosine are off by 2^-23, product and sum round in fp32
        assert bool((err <= (mag * (2.0 ** -23 + 3 * R.F32) + u * turned.abs())[:, :, c0 * C:]).all())
    high = (torch.arange(d) % (d // 2)) < cfg.n_high_freq_pairs
    for table, size in ((cs, C), (gs, 16)):
        got, first = table.cpu().double(), c0 * C // size
        assert bool((got[:, :, :first] == 7.0).all())
        for i in range(first, table.shape[2]):
            s = slice(i * size, min(L, (i + 1) * size))
            if s.start >= L:
                assert not got[:, :, i].any()
                continue
            low = R.rotate(k[:, :, s].double().mean(2, keepdim=True),
                           R.angles(pos[:, :, s].double().mean(2, keepdim=True), pair, 1e4, d)[:, None])
            ref = torch.where(high, turned[:, :, s].mean(2), low[:, :, 0])
            # a sum of at most 128 terms in fp32 and its division, the rotation of the terms or of
            # the mean, and the table's own rounding
            e = mag[:, :, s].mean(2) * (2.0 ** -23 + (130 + 3) * R.F32)
            tol = e + (R.BF16 * (ref.abs() + e) if tables == "bf16" else 0) + 1e-30
            assert bool(((got[:, :, i] - ref).abs() <= tol).all()), (size, i)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes_sine_and_cosine(d, inverse):
    """Rows of (1, 0) pairs turn into the cosine and the sine themselves. The reduced angle's are off
    by 2^-23 at most (polynomials in fp32: the last rounding 2^-25, the terms' 2^-25, the series' end
    2^-29). The angle is a 64-bit product of a 64-bit power: 2^-50 of it covers its roundings here
    and in the reference."""
    from long_context_rope_b200 import hga
    cfg = _cfg(hga, head_dim=d, dtype="f32", rope_theta=5e5)
    T = 40000
    g = torch.Generator().manual_seed(21)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, 1, T), generator=g)
    for i, top in enumerate((2, 100, 5000, 70000, 1 << 20)):   # far positions are a sixth only
        pos[:, :, i::6] %= top
    pos[:, :, :12] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 3, 22, 355, 710, 52174, 103993, -355])
    pos = pos.to(torch.int32)
    pair = hga.pair_axes(d // 2, (d // 4, d // 4), True)
    x = torch.zeros(1, T, 1, d)
    x[..., :d // 2] = 1.0
    y = torch.empty_like(x).cuda()
    hga.apply_rope_axes(cfg, hga.rope_axes(pair, 2, inverse=inverse), pos.cuda(), x.cuda(), y, 1, T, 1)
    _clean(hga)
    a = R.angles(pos, pair, 5e5, d)
    want = torch.cat((torch.cos(a), torch.sin(-a if inverse else a)), -1)
    tol = 2.0 ** -23 + a.abs().repeat(1, 1, 2) * 2.0 ** -50
    err = (y.cpu().double()[:, :, 0] - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_tensor_of_another_gpu_is_refused():
    from long_context_rope_b200 import hga
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU here (test_kv4_pipeline_cpu.py has the check itself)")
    cfg = _cfg4(hga, seq_len=16, q_begin=15)
    k = torch.zeros(1, 1, 16, 128, dtype=BF, device="cuda:0")
    st = torch.zeros(1, 1, 1, 1152, dtype=torch.uint8, device="cuda:0")
    with pytest.raises(ValueError, match="current device"):
        hga.store_kv(cfg, k.to("cuda:1"), k, st, st, 0)
    with torch.cuda.device(1), pytest.raises(ValueError, match="current device"):
        hga.store_kv(cfg, k, k, st, st, 0)


# ------------------------------------------------------------------- refusals
@pytest.mark.parametrize("kv4", [False, True])
def test_launch_that_cuda_refuses_leaves_nothing_behind(kv4):
    """More units than a grid takes: an error of that call alone, not of the next one, the
    library's or torch's."""
    from long_context_rope_b200 import hga
    kw = dict(batch=70000, n_q_heads=1, seq_len=16, q_begin=15, top_k_groups=1, top_k_chunks=1)
    cfg = _cfg4(hga, **kw) if kv4 else _cfg(hga, **kw)
    q = torch.zeros(70000, 1, 1, 128, dtype=BF, device="cuda")
    st = torch.zeros(cfg.kv_rows(70000, 1, rows=16), dtype=cfg.kv_torch_dtype(), device="cuda")
    sel = torch.zeros(70000, 1, 1, 1, dtype=torch.int32, device="cuda")
    small = _cfg4(hga, seq_len=16)
    pages = torch.zeros(1, 1, 1, 1152, dtype=torch.uint8, device="cuda")
    k = torch.full((1, 1, 16, 128), 7.0, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    with pytest.raises(hga.HgaError, match="HGA_ERR_CUDA"):
        hga.attend(cfg, q, st, st, sel, sel[..., 0], torch.empty_like(q))
    hga.load_kv(small, pages, pages, k, k.clone(), 0)
    _clean(hga)
    assert not k.any()
    # what does not put its units on a grid axis takes them all
    if kv4:
        rows = torch.randn(70000, 1, 16, 128, device="cuda").to(BF)
        ks, vs = torch.zeros_like(st), torch.zeros_like(st)
        hga.store_kv(cfg, rows, rows, ks, vs, 0)
        one = cfg.copy(batch=1)
        k1, v1 = ks[:1].clone().zero_(), vs[:1].clone().zero_()
        hga.store_kv(one, rows[-1:].clone(), rows[-1:].clone(), k1, v1, 0)
        _clean(hga)
        assert torch.equal(ks[-1:], k1) and not torch.equal(ks[0], ks[-1])


# --------------------------------------------------------- more shapes and gathers
TC_SHAPES = [
    dict(seq_len=200, q_begin=160, q_len=40, chunk_size=16, groups_per_chunk=1, n_q_heads=16),
    dict(seq_len=700, q_begin=37, q_len=650, chunk_size=16, groups_per_chunk=1),
    dict(seq_len=700, q_begin=20, q_len=640, chunk_size=32, groups_per_chunk=2, n_q_heads=5),
    dict(seq_len=500, q_begin=300, q_len=200, chunk_size=112, groups_per_chunk=7, n_q_heads=9),
    dict(seq_len=700, q_begin=37, q_len=600, chunk_size=128, groups_per_chunk=8),
    dict(seq_len=640, q_begin=0, q_len=640, n_q_heads=1),
    dict(seq_len=333, q_begin=332, q_len=1, batch=5, n_kv_heads=2, n_q_heads=66),
    dict(seq_len=300, q_begin=250, q_len=5, batch=3, n_kv_heads=2, n_q_heads=18),
    dict(seq_len=7000, q_begin=6950, q_len=40, n_q_heads=10, top_k_groups=400, n_local=1),
    dict(seq_len=130, q_begin=60, q_len=9, batch=70, n_local=0, n_sink=0, n_q_heads=2),
]


@pytest.mark.parametrize("count", [None, 0, 1])
@pytest.mark.parametrize("kw", TC_SHAPES, ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()))
def test_prefill_shapes(kw, count):
    """Every chunk size, one head and many, a list of hundreds, many short sequences."""
    from long_context_rope_b200 import hga
    cfg = _tc(_cfg4(hga, **kw))
    q, kp, vp, sel, n, want, tol = _attend_case(hga, cfg, 150, count)
    args = [t.cuda() for t in (q, kp, vp, sel, n)]
    outs = [torch.full(q.shape, float("nan"), dtype=BF, device="cuda") for _ in range(2)]
    for out in outs:
        hga.attend(cfg, *args, out)
    _clean(hga)
    _check(outs[0], want, tol)
    assert torch.equal(*outs)


def test_gathers_of_pages_for_a_span_and_without_a_buffer():
    """Pages of several query chunks from host memory as from the device; the warm tier that is
    given no list buffer, as the one that is."""
    from long_context_rope_b200 import hga, pipeline
    cfg = _cfg4(hga, seq_len=999, q_begin=500, q_len=300, batch=2, n_kv_heads=2, n_q_heads=16)
    g = torch.Generator().manual_seed(160)
    pages = [torch.randint(0, 256, cfg.kv_rows(2, 2, rows=999), generator=g, dtype=torch.uint8)
             for _ in "kv"]
    sel, n = R.lists(cfg, 2, 161)
    sd, nd = sel.cuda(), n.cuda()
    host, dev = pipeline.alloc_gathered(cfg), pipeline.alloc_gathered(cfg)
    pinned = [p.pin_memory() for p in pages]
    hga.gather_kv(cfg, *pinned, True, sd, nd, *host)
    hga.gather_kv(cfg, *(p.cuda() for p in pages), False, sd, nd, *dev)
    _clean(hga)
    for a, b, p in zip(host, dev, pages):
        assert torch.equal(a, b)
        for bb in range(2):
            for h in range(2):
                for j in range(cfg.n_qchunks):
                    m = int(n[bb, h, j])
                    assert torch.equal(a[bb, h, j, :m].cpu(), p[bb, h, sel[bb, h, j, :m].long()])
    one = cfg.copy(q_begin=998, q_len=1)
    pools = [pipeline.alloc_warm_pool(one, 20) for _ in range(2)]
    for step in range(3):
        sel, n = R.lists(one, 2, 170 + step)
        sd, nd = sel.cuda(), n.cuda()
        outs = [pipeline.alloc_gathered(one) for _ in range(2)]
        for pool, out, free in zip(pools, outs, (False, True)):
            head = (one, *pinned, sd, nd, pool.k, pool.v, pool.tag, pool.last, step)
            if free:
                hga.gather_kv_warm_noalloc(*head, *out, pool.stats)
            else:
                hga.gather_kv_warm(*head, pool.src, *out, pool.stats)
        _clean(hga)
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        for name in ("k", "v", "tag", "last", "stats"):
            assert torch.equal(getattr(pools[0], name), getattr(pools[1], name))
        m = int(n[1, 1, 0])
        assert torch.equal(outs[0][0][1, 1, 0, :m].cpu(), pages[0][1, 1, sel[1, 1, 0, :m].long()])


@pytest.mark.parametrize("q_len,heads,gathered", [(1, 12, False), (30, 12, False), (1, 130, False), (1, 12, True)])
def test_attend_large_queries(q_len, heads, gathered):
    """Queries beyond the range of 16-bit floats with 5 exponent bits, and tiny ones, on the
    kernels that take more heads than single tokens' does."""
    from long_context_rope_b200 import hga, pipeline
    cfg = _cfg4(hga, seq_len=400, q_begin=400 - q_len, q_len=q_len, k_scale=2.0 ** -30, n_q_heads=heads)
    kp = R.pack(*R.quantise(_rows((1, 1, 400, 128), 1, 2.0 ** -22), cfg.k_scale))
    vp = R.pack(*R.quantise(_rows((1, 1, 400, 128), 2), cfg.v_scale))
    q = _rows((1, q_len, heads, 128), 3)
    q *= torch.tensor([2.0 ** 20, 2.0 ** 22, 1.0, 2.0 ** -20])[torch.arange(heads) % 4].view(1, 1, -1, 1).to(BF)
    sel, n = R.lists(cfg, 1, 0)
    want, tol = R.attend(cfg, q, R.values(kp, cfg.k_scale), R.values(vp, cfg.v_scale), sel, n)
    args = [t.cuda() for t in (q, kp, vp, sel, n)]
    gat = (None, None)
    if gathered:
        gat = pipeline.alloc_gathered(cfg)
        hga.gather_kv(cfg, args[1], args[2], False, args[3], args[4], *gat)
    out = torch.empty_like(args[0])
    hga.attend(cfg, *args, out, k_gat=gat[0], v_gat=gat[1])
    _clean(hga)
    _check(out, want, tol)

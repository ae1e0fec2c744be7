"""More of the 4-bit store, its attention and rotary positions with several axes on a
GPU: calls that the documentation allows, each against kv4_ref.py or a longer call."""
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

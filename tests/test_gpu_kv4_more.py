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

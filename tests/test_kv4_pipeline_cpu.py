"""What the pipeline hands to the library's calls, with the calls themselves replaced (no
GPU; nothing is launched)."""
import pytest
import torch


@pytest.fixture(scope="module")
def hga():
    from long_context_rope_b200 import build
    build.build()
    from long_context_rope_b200 import hga as mod
    return mod


def _cfg(hga, kv4, **kw):
    from long_context_rope_b200 import synth
    over = dict(kv_type=hga.HGA_KV_E2M1, k_scale=0.5, v_scale=0.25) if kv4 else {}
    return hga.config_from(synth.WORKLOADS["prefill_4k"], **dict(over, **kw))


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("n_axes,batch", [(1, 1), (1, 2), (3, 1)])
def test_positions_from_any_token_on(hga, monkeypatch, kv4, n_axes, batch):
    """Each call gets its positions contiguous and at a 16-byte boundary, wherever the
    token's own lie: one axis of one sequence is contiguous without being copied."""
    from long_context_rope_b200 import pipeline
    L = 64
    cfg = _cfg(hga, kv4, batch=batch, seq_len=L, q_begin=0, q_len=1, n_q_heads=8, n_kv_heads=1)
    pos = torch.arange(n_axes * batch * L, dtype=torch.int32).view(n_axes, batch, L)
    axes = hga.rope_axes([i % n_axes for i in range(64)], n_axes)
    seen = []

    def call(name, at):
        def f(*args, **kw):
            p = args[at] if len(args) > at else kw.get("positions")
            assert p.is_contiguous() and p.data_ptr() % 16 == 0, name
            seen.append((name, p.clone()))
        monkeypatch.setattr(hga, name, f)
    call("apply_rope_axes", 2)
    call("build_summaries_axes", 2)
    call("store_kv", 7)
    monkeypatch.setattr(hga, "decode_step", lambda *a, **k: None)
    k = torch.zeros(batch, 1, L, 128, dtype=torch.bfloat16)
    q = torch.zeros(batch, 1, 8, 128, dtype=torch.bfloat16)
    rb = pipeline.alloc_route(cfg, device="cpu")
    for t in range(L):
        seen.clear()
        qp = pos[:, :, t:t + 1].contiguous()
        pipeline.rotate_queries(cfg, q, axes=axes, positions=qp)
        pipeline.decode_append(cfg, t, k[:, :, t], k[:, :, t], q, k.clone(), k.clone(), k.clone(), None,
                               None, rb, q.clone(), axes=axes, positions=pos)
        want = [("apply_rope_axes", qp), ("store_kv" if kv4 else "apply_rope_axes", qp)]
        if t == L - 1:
            want.append(("build_summaries_axes", pos))
        assert [n for n, _ in seen] == [n for n, _ in want]
        assert all(torch.equal(a, b) for (_, a), (_, b) in zip(seen, want))


def test_prefill_positions_from_any_token_on(hga, monkeypatch):
    """A part of a longer sequence's positions, not at a 16-byte boundary."""
    from long_context_rope_b200 import pipeline
    cfg = _cfg(hga, True, batch=1, seq_len=9, q_begin=0, q_len=9, n_q_heads=8, n_kv_heads=1)
    pos = torch.arange(32, dtype=torch.int32).view(1, 1, 32)[:, :, 7:16].contiguous()
    got = []
    monkeypatch.setattr(hga, "build_summaries_axes", lambda *a, **k: got.append(a[2]))
    monkeypatch.setattr(hga, "store_kv", lambda *a, **k: got.append(a[7]))
    monkeypatch.setattr(hga, "route", lambda *a, **k: None)
    monkeypatch.setattr(hga, "attend", lambda *a, **k: None)
    rb = pipeline.alloc_route(cfg, device="cpu")
    pipeline.prefill(cfg, None, None, None, None, None, None, rb, None, v_store=None,
                     axes=hga.rope_axes([0] * 64, 1), positions=pos)
    assert len(got) == 2 and all(p.data_ptr() % 16 == 0 and torch.equal(p, pos) for p in got)


@pytest.mark.parametrize("current", [0, 1])
def test_tensor_of_another_device_is_refused(hga, monkeypatch, current):
    """By its device's number, with a tensor that says it is of a GPU."""
    class OnGpu(torch.Tensor):
        is_cuda = True
        device = torch.device("cuda", 1)

        def get_device(self):
            return 1
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    t = torch.zeros(4).as_subclass(OnGpu)
    if current == 1:
        assert hga._ptr_checked(t, "x", torch.float32, (4,)) == t.data_ptr()
        return
    for f in (hga._ptr, hga._ptr_checked):   # the native check passes it on to the other
        with pytest.raises(ValueError, match="x must be on the current device, cuda:0, not on cuda:1"):
            f(t, "x", torch.float32, (4,))

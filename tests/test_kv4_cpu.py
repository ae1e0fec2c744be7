"""Host side of the 4-bit store and of positions with several axes: refusals,
empty calls and the pair-axis lists (no GPU; nothing is launched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def hga():
    from long_context_rope_b200 import build
    build.build()
    from long_context_rope_b200 import hga as mod
    return mod


P = 16 * 1024  # aligned, never dereferenced: every call here is refused or empty


def _cfg(hga, **kw):
    from long_context_rope_b200 import synth
    return hga.config_from(synth.WORKLOADS["prefill_4k"], **kw)


def _cfg4(hga, **kw):
    return _cfg(hga, **dict(dict(kv_type=hga.HGA_KV_E2M1, k_scale=0.5, v_scale=0.25), **kw))


def test_struct_layout(hga):
    assert ctypes.sizeof(hga.HgaRopeAxes) == 72
    assert hga.HgaRopeAxes.pair_axis.offset == 8


def test_pair_axes(hga):
    assert hga.pair_axes(8, [2, 3, 3]) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert hga.pair_axes(8, [2, 3, 1], interleaved=True) == [0, 1, 2, 0, 1, 1, -1, -1]
    assert hga.pair_axes(4, []) == [-1] * 4
    assert hga.pair_axes(4, [0, 4]) == [1] * 4
    for bad in ([5], [-1, 2], [2, 3]):
        with pytest.raises(ValueError):
            hga.pair_axes(4, bad)
    with pytest.raises(ValueError):
        hga.rope_axes([0] * 65, 1)
    ax = hga.rope_axes([1, 0, -1], 2, inverse=True)
    assert list(ax.pair_axis)[:4] == [1, 0, -1, -1] and ax.n_axes == 2 and ax.inverse == 1


def test_scales_and_shape_of_the_store(hga):
    L, by = hga.library(), ctypes.byref
    attend = [P] * 3 + [None, None] + [P] * 3 + [None]
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0), (1.0, float("inf"))):
        assert L.hga_attend(by(_cfg4(hga, k_scale=ks, v_scale=vs)), *attend) == -4
    assert L.hga_attend(by(_cfg4(hga, dtype=hga.HGA_F32)), *attend) == -8
    assert L.hga_attend(by(_cfg4(hga, head_dim=64)), *attend) == -8
    assert L.hga_build_summaries(by(_cfg4(hga)), P, P, P, P, 0, 4, None) == -8
    cfg = _cfg4(hga, seq_len=33, q_len=1, q_begin=0)
    assert cfg.kv_rows(2, 3, rows=33) == (2, 3, 3, 1152)
    assert hga.pool_shape(cfg, 7) == (1, 4, 7, 1152)
    assert _cfg(hga).kv_rows(2, rows=33) == (2, 33, 128)


def test_rope_axes_refusals(hga):
    L, by = hga.library(), ctypes.byref
    ax = hga.rope_axes(hga.pair_axes(64, [16, 24, 24]), 3)

    def call(cfg=None, a=ax, pos=P, x=P, y=P, nb=2, no=4, nt=5, nh=1):
        return L.hga_apply_rope_axes(by(cfg or _cfg(hga)), by(a) if a else None, pos, x, y, nb, no,
                                     nt, nh, None)
    assert call(a=None) == -1
    for n_axes, pairs in ((0, []), (5, []), (2, [2] * 64), (1, [-2] * 64)):
        assert call(a=hga.rope_axes(pairs, n_axes)) == -4, (n_axes, pairs)
    bad = hga.rope_axes([], 1)
    bad.inverse = 2
    assert call(a=bad) == -4
    for kw in (dict(nb=3), dict(nb=0), dict(nb=-1), dict(no=-1), dict(nt=-1), dict(nh=0),
               dict(nt=2**31), dict(no=2**30, nt=2**30, nh=2**30, nb=1)):
        assert call(**kw) == -2, kw
    assert call(pos=None) == -1 and call(x=None) == -1 and call(y=None) == -1
    assert call(pos=P + 4) == -3 and call(x=P + 2) == -3 and call(y=P + 8) == -3
    assert call(nt=0) == 0 and call(no=0, nb=0) == 0
    # entries past d / 2 are not read
    assert call(cfg=_cfg(hga, head_dim=64), a=hga.rope_axes([0] * 32 + [9] * 32, 1), nt=0) == 0


def test_summaries_axes_refusals(hga):
    L, by = hga.library(), ctypes.byref
    ax = hga.rope_axes(hga.pair_axes(64, [16, 24, 24]), 3)

    def call(cfg=None, a=ax, args=(P, P, P, P), rot=None, c0=0, c1=4):
        return L.hga_build_summaries_axes(by(cfg or _cfg(hga)), by(a) if a else None, *args, rot, c0,
                                          c1, None)
    assert call(a=None) == -1
    assert call(a=hga.rope_axes([0], 1, inverse=True)) == -4
    assert call(a=hga.rope_axes([1], 1)) == -4
    assert call(c0=3, c1=2) == -2 and call(c1=65) == -2 and call(c0=2, c1=2) == 0
    for i in range(4):
        assert call(args=tuple(None if i == j else P for j in range(4))) == -1
        assert call(args=tuple(P + 4 if i == j else P for j in range(4))) == -3
    assert call(rot=P + 8) == -3
    assert call(cfg=_cfg4(hga), rot=P) == -8


def test_store_and_load_refusals(hga):
    L, by = hga.library(), ctypes.byref
    ax = hga.rope_axes(hga.pair_axes(64, [16, 24, 24]), 3)
    one = hga.rope_axes(hga.pair_axes(64, [64]), 1)

    def store(cfg=None, a=None, pos=None, ptr=(P, P, P, P), pos0=0, n=4):
        return L.hga_store_kv(by(cfg or _cfg4(hga)), by(a) if a else None, pos, *ptr, pos0, n, None)

    def load(cfg=None, ptr=(P, P, P, P), pos0=0, n=4):
        return L.hga_load_kv(by(cfg or _cfg4(hga)), *ptr, pos0, n, None)
    for f in (store, load):
        assert f(cfg=_cfg(hga)) == -8
        assert f(cfg=_cfg(hga, kv_type=hga.HGA_KV_E4M3, k_scale=1.0, v_scale=1.0)) == -8
        for pos0, n in ((-1, 4), (0, -1), (4097, 0), (4093, 4), (0, 4097), (2**62, 2**62)):
            assert f(pos0=pos0, n=n) == -2, (pos0, n)
        assert f(pos0=4096, n=0) == 0 and f(n=0) == 0
        for i in range(4):
            assert f(ptr=tuple(None if i == j else P for j in range(4))) == -1
            assert f(ptr=tuple(P + 8 if i == j else P for j in range(4))) == -3
    assert store(pos=P) == -4                         # positions without axes
    assert store(a=ax) == -1                          # several axes without positions
    assert store(a=ax, pos=P + 4) == -3
    assert store(a=hga.rope_axes([0], 1, inverse=True), pos=P) == -4
    assert store(a=hga.rope_axes([3], 3), pos=P) == -4
    assert store(a=one, n=0) == 0


def test_binding_refusals(hga):
    import torch
    cfg = _cfg4(hga, seq_len=64, q_begin=0, q_len=1)
    ax = hga.rope_axes([0], 1)
    with pytest.raises(ValueError):
        hga.apply_rope_axes(cfg, ax, torch.zeros(1, 4), torch.zeros(4, 128), torch.zeros(4, 128), 1, 4,
                            1)
    with pytest.raises(ValueError):
        hga.apply_rope_axes(cfg, ax, torch.zeros(1, 1, 4), torch.zeros(3, 128), torch.zeros(3, 128),
                            1, 4, 1)
    k = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    st = torch.zeros(1, 4, 4, 1152, dtype=torch.uint8)
    for bad in (None, torch.zeros(2, 128)):
        with pytest.raises((ValueError, TypeError)):
            hga.store_kv(cfg, bad, k, st, st, 0)
        with pytest.raises((ValueError, TypeError)):
            hga.load_kv(cfg, st, st, bad, k, 0)
    with pytest.raises(ValueError):
        hga.store_kv(cfg, k, k, st, st, 0, positions=torch.zeros(1, 1, 2, dtype=torch.int32))


def test_tensor_of_the_cpu_is_a_value_error(hga):
    """With or without a driver, a right tensor in the wrong place is refused by name."""
    import torch
    cfg = _cfg(hga)
    x = torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        hga.apply_rope(cfg, x, x, 1, 4, 1, 0)
    pos = torch.zeros(1, 1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        hga.apply_rope_axes(cfg, hga.rope_axes([0], 1), pos, x, x, 1, 4, 1)


@pytest.mark.parametrize("kv4", [False, True])
def test_axes_and_positions_go_together(hga, kv4):
    """Refused before anything is launched or written: positions without axes (they would
    be passed over), axes without positions, positions of another shape."""
    import torch
    from long_context_rope_b200 import pipeline
    cfg = (_cfg4 if kv4 else _cfg)(hga, batch=1, seq_len=64, q_begin=0, q_len=64)
    ax = hga.rope_axes([0, 1] * 32, 2)
    right = torch.zeros(2, 1, 64, dtype=torch.int32)
    k = torch.zeros(1, cfg.n_kv_heads, 64, 128, dtype=torch.bfloat16)
    q = torch.zeros(1, 64, cfg.n_q_heads, 128, dtype=torch.bfloat16)
    cs, gs, rb, out = None, None, None, None
    for axes, pos in ((None, right), (ax, None), (ax, right[:, :, :63]), (ax, right[:1])):
        with pytest.raises(ValueError, match="positions"):
            pipeline.rotate_queries(cfg, q, axes=axes, positions=pos)
        with pytest.raises(ValueError, match="positions"):
            pipeline.summaries(cfg, k, cs, gs, axes=axes, positions=pos)
        with pytest.raises(ValueError, match="positions"):
            pipeline.prefill(cfg, k, k, q, cs, gs, None, rb, out, axes=axes, positions=pos)
        with pytest.raises(ValueError, match="positions"):
            pipeline.decode_append(cfg, 3, k[:, :, 0], k[:, :, 0], q[:, :1], k, None, None, cs, gs,
                                   rb, out, axes=axes, positions=pos)

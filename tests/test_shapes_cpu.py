"""The shapes that calls ask of their tensors, kept from call to call (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def hga():
    from long_context_rope_b200 import build
    build.build()
    from long_context_rope_b200 import hga as mod
    return mod


def _cfg(hga, **kw):
    from long_context_rope_b200 import synth
    return hga.config_from(synth.WORKLOADS["prefill_4k"], **kw)


@pytest.mark.parametrize("kv_type", [0, 1, 2])
@pytest.mark.parametrize("layout", [0, 1])
def test_a_decode_loop_works_them_out_once(hga, kv_type, layout):
    """Single tokens one after another: the same object, and the shapes of each."""
    base = _cfg(hga, kv_type=kv_type, kv_layout=layout, q_len=1)
    hga._shapes_of.cache_clear()
    for t in range(300, 1200):
        c = base.copy(q_begin=t, seq_len=t + 1 if layout else 4096)
        s = hga._shapes(c, windows=bool(layout))
        if not layout:
            assert s.store == c.kv_rows(c.batch, c.n_kv_heads, rows=4096) == s.res
        else:
            assert s.res == c.kv_rows(c.batch, c.n_kv_heads, rows=hga.window_slots(c) * c.chunk_size)
        assert s.q == (c.batch, 1, c.n_q_heads, c.head_dim)
        assert s.sel == (c.batch, c.n_kv_heads, 1, c.top_k_groups) and s.n_sel == s.sel[:3]
        assert s.gathered == c.kv_rows(c.batch, c.n_kv_heads, 1, rows=c.top_k_groups * 16)
    assert hga._shapes_of.cache_info().misses == 1


def test_what_the_shapes_depend_on_tells_them_apart(hga):
    base = _cfg(hga, seq_len=1000, q_begin=10, q_len=50)
    one = hga._shapes(base)
    assert one.sel[2] == base.n_qchunks == 1
    two = hga._shapes(base.copy(q_begin=20))     # over a chunk's end
    assert two.sel[2] == 2 and two.gathered[2] == 2 and one.sel[2] == 1
    assert hga._shapes(base.copy(q_len=51)).q[1] == 51
    assert hga._shapes(base.copy(seq_len=999)).store[2] == 999
    assert hga._shapes(base.copy(routing=1)).sel[1] == base.n_q_heads
    assert hga._shapes(base.copy(q_len=0)).sel[2] == 0
    assert hga._shapes(base.copy(kv_type=hga.HGA_KV_E2M1)).store == (1, base.n_kv_heads, 63, 1152)
    for bad in (dict(chunk_size=0), dict(groups_per_chunk=0), dict(chunk_size=0, q_len=1)):
        with pytest.raises(hga.HgaError):
            hga._shapes(base.copy(**bad))


def test_key_counts_the_chunks_of_a_span(hga):
    import ctypes
    import random
    rng = random.Random(5)
    for _ in range(300):
        c = _cfg(hga, q_begin=rng.choice((0, 1, 63, 64, rng.randrange(4096))),
                 q_len=rng.choice((0, 1, 2, 64, 65, rng.randrange(500))))
        key = hga.HgaConfig.from_buffer_copy(hga._bind.shape_key(ctypes.addressof(c), False))
        assert key.q_begin == c.n_qchunks
        back = key.copy(q_begin=c.q_begin)
        assert all(getattr(back, n) == getattr(c, n) for n, _ in c._fields_)
    with pytest.raises(ValueError):
        hga._bind.shape_key(0, False)
    for args in ((None, False), (5,)):
        with pytest.raises(TypeError):
            hga._bind.shape_key(*args)

"""The native binding: what it takes as it is, and what it refuses and how (no GPU)."""
import ctypes
import threading

import pytest
import torch


@pytest.fixture(scope="module")
def hga():
    from long_context_rope_b200 import build
    build.build()
    from long_context_rope_b200 import hga as mod
    return mod


BF = torch.bfloat16


def test_ptr_of_a_tensor_as_asked(hga):
    t = torch.zeros(2, 3, 8, dtype=BF)
    for a in (dict(), dict(dtype=BF), dict(shape=(2, 3, 8)), dict(dtype=BF, shape=t.shape),
              dict(dtype=BF, shape=[2, 3, 8]), dict(shape=(2, 3, 8), nullable=True)):
        assert hga._ptr(t, "t", device=False, **a) == t.data_ptr()
        assert hga._ptr_checked(t, "t", device=False, **a) == t.data_ptr()
    assert hga._ptr(t, "t", BF, (2, 3, 8), False, False) == t.data_ptr()
    assert hga._ptr(t[1:], "t", BF, (1, 3, 8), False) == t.data_ptr() + 48
    assert hga._ptr(None, "t", BF, (1,), nullable=True) is None
    assert hga._ptr(torch.zeros(0, 4), "t", torch.float32, (0, 4), False) in (0, None)
    sub = torch.nn.Parameter(torch.zeros(4))
    assert hga._ptr(sub, "t", torch.float32, (4,), False) == sub.data_ptr()


@pytest.mark.parametrize("bad,kw,err", [
    (None, {}, ValueError), (3, {}, TypeError), ([1.0], {}, TypeError),
    (torch.zeros(4), dict(dtype=BF), ValueError), (torch.zeros(4), dict(shape=(5,)), ValueError),
    (torch.zeros(4), dict(shape=(4, 1)), ValueError), (torch.zeros(4), dict(shape=()), ValueError),
    (torch.zeros(4, 4).t(), dict(shape=(4, 4)), ValueError),
    (torch.zeros(8)[::2], dict(shape=(4,)), ValueError),
    (torch.zeros(4), dict(device=True), ValueError),
    (torch.zeros(4), dict(shape=("4",)), ValueError),
    (torch.zeros(4), dict(other=1), TypeError)])
def test_ptr_refuses_as_the_step_by_step_checks(hga, bad, kw, err):
    kw = dict(dict(device=False), **kw)
    said = []
    for f in (hga._ptr, hga._ptr_checked):
        with pytest.raises(err) as e:
            f(bad, "the_name", **kw)
        said.append(str(e.value))
    assert said[0] == said[1]
    with pytest.raises(TypeError):
        hga._ptr()
    with pytest.raises(TypeError):
        hga._ptr(torch.zeros(1), "t", None, None, False, False, 7)


def test_calls_equal_those_of_ctypes(hga):
    """The same status for the same arguments, by either way in."""
    from long_context_rope_b200 import synth
    cfg = hga.config_from(synth.WORKLOADS["prefill_4k"])
    ok = 16 * 1024  # aligned, never dereferenced
    at, ref = hga._cfg_at(cfg), ctypes.byref(cfg)
    for args in ((None, ok, 1, 1, 1, 0, 0), (ok, ok + 8, 1, 1, 1, 0, 0), (ok, ok, -1, 1, 1, 0, 0),
                 (ok, ok, 0, 1, 1, 0, 0), (ok, ok, 1, 1, 0, 0, 0)):
        assert hga._bind.hga_apply_rope(at, *args) == hga._lib.hga_apply_rope(ref, *args)
    bad = cfg.copy(chunk_size=0)
    assert (hga._bind.hga_apply_rope(hga._cfg_at(bad), ok, ok, 1, 1, 1, 0, 0)
            == hga._lib.hga_apply_rope(ctypes.byref(bad), ok, ok, 1, 1, 1, 0, 0) != 0)
    assert hga._bind.hga_apply_rope(None, ok, ok, 1, 1, 1, 0, 0) == -1


def test_calls_refuse_what_they_cannot_convert(hga):
    from long_context_rope_b200 import synth
    cfg = hga.config_from(synth.WORKLOADS["prefill_4k"])
    at, call = hga._cfg_at(cfg), hga._bind.hga_apply_rope
    with pytest.raises(TypeError):
        call(at, None, None)
    with pytest.raises(TypeError):
        call(at, "x", None, 1, 1, 1, 0, 0)
    with pytest.raises(TypeError):
        call(at, None, None, 1.5, 1, 1, 0, 0)
    with pytest.raises(OverflowError):
        call(at, None, None, 1, 1, 2 ** 31, 0, 0)      # n_heads is 32 bits
    with pytest.raises(OverflowError):
        call(at, None, None, 2 ** 63, 1, 1, 0, 0)
    for f in (hga._cfg_at, hga._axes_at):
        for bad in (None, 5, ctypes.c_int(1)):
            with pytest.raises(TypeError):
                f(bad)
    with pytest.raises(TypeError):
        hga._cfg_at(hga.rope_axes([0], 1))


def test_calls_from_many_threads(hga):
    from long_context_rope_b200 import synth
    cfg = hga.config_from(synth.WORKLOADS["prefill_4k"])
    t = torch.zeros(2, 3, dtype=BF)
    wrong = []

    def work():
        for _ in range(2000):
            if (hga._bind.hga_apply_rope(hga._cfg_at(cfg), None, None, 1, 1, 1, 0, 0) != -1
                    or hga._ptr(t, "t", BF, (2, 3), False) != t.data_ptr()):
                wrong.append(1)

    ts = [threading.Thread(target=work) for _ in range(8)]
    for x in ts:
        x.start()
    for x in ts:
        x.join()
    assert not wrong

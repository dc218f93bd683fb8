"""The feed-forward operators where their native binding is missing: a warning, and
the same calls through ctypes."""
import pytest
import torch

import async_copy_pipelined_gb300 as pg
from async_copy_pipelined_gb300 import feedforward as ff


@pytest.fixture
def without(monkeypatch, tmp_path):
    pg.build()
    monkeypatch.setattr(ff, "_torch", None)
    monkeypatch.setattr(ff, "_native", None)
    monkeypatch.setattr(ff, "_NATIVE_PATH", str(tmp_path / "_feedforward.so"))


def test_a_warning_and_the_calls_are_made_in_python(without):
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="native binding not built"):
        with pytest.raises(ValueError, match="CUDA tensors"):
            pg.quantize_fp8(x)
    with pytest.raises(ValueError, match="CUDA tensors"):  # warned once
        pg.gated_projection(x, x, x)


def test_a_binding_that_does_not_load_is_warned_of(without, monkeypatch, tmp_path):
    (tmp_path / "_feedforward.so").write_text("no shared object")
    with pytest.warns(RuntimeWarning, match="10 to 25 us"):
        ff._load()
    assert ff._native.gemm_fp8(None, None, None, None, 0) is None


@pytest.mark.gpu
def test_the_results_are_the_same(monkeypatch, tmp_path):
    g = torch.Generator("cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    x, wg, wu, wd, dh = randn(40, 64), randn(64, 136), randn(64, 136), randn(136, 64), randn(40, 136)

    def run():
        h, gate, up = pg.gated_projection(x, wg, wu, save=True)
        q, s = pg.quantize_fp8(h)
        d, t = pg.quantize_fp8(wd, "block")
        return (h, gate, up, q, s, d, t, pg.gemm_fp8(q, d, s, t),
                *pg.gated_projection_backward(dh, x, wg, wu, gate, up))

    want = run()
    monkeypatch.setattr(ff, "_torch", None)
    monkeypatch.setattr(ff, "_native", None)
    monkeypatch.setattr(ff, "_NATIVE_PATH", str(tmp_path / "_feedforward.so"))
    with pytest.warns(RuntimeWarning, match="native binding not built"):
        got = run()
    for a, b in zip(got, want):
        assert a.stride() == b.stride() and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert pg.device_status()[0] == 0

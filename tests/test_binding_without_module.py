"""Where the compiled module behind the quickest calls is missing or does not load, the calls go through ctypes."""
import os
import warnings

import pytest
import torch

from tests.test_new_operator_checks import fake


@pytest.fixture
def pq(monkeypatch, tmp_path):
    """pq.py with nothing loaded yet, looking for the module in an empty folder."""
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    monkeypatch.setattr(_pq, "_call", None)
    monkeypatch.setattr(_pq, "_LIB_PATH", str(tmp_path / "libpq.so"))
    return _pq


def four_calls(pq, make, stream=0):
    """Each call in its shortest form; make(shape, type) gives its tensors."""
    bf16, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    X, c, s, Y = make((4, 256), bf16), make((4, 128), u8), make((4096,), u8), make((4, 4), f32)
    pq.pq_quant_fp4(X, c, s)
    pq.pq_fp4_gemm(c, s, c, s, Y)
    pq.pq_fp4_linear(X, c, s, c, s, Y)
    codes, sc = make((3, 2, 16, 64), u8), make((3, 2, 16), f32)
    Q = make((5, 4, 128), bf16)
    pq.pq_kv4_attention_masked(pq.KV4Cache(codes, sc, codes, sc), Q, make((5, 4, 128), bf16), make((3,), i32), make((2,), i32), make((2, 3), i32),
                               1, 1, window=2, sinks=1)


def reached(pq, monkeypatch):
    names = []
    entry = lambda name: staticmethod(lambda *a: names.append(name) or 0)                      # noqa: E731
    monkeypatch.setattr(pq, "lib", type("Library", (), {n: entry(n) for n in
                                                        ("pq_quant_fp4", "pq_fp4_gemm", "pq_fp4_linear", "pq_kv4_attention_masked")}))
    monkeypatch.setattr(pq, "_raw_stream", lambda *a: 0)
    return names


@pytest.mark.parametrize("content", [None, b"", b"not a library", b"\x7fELF\x02\x01\x01"])
def test_calls_reach_the_library(pq, monkeypatch, tmp_path, content):
    if content is not None:                              # whatever the module's file is called
        from rotation_int4_w4a4_b200 import build
        (tmp_path / os.path.basename(build.CALL_LIB)).write_bytes(content)
    names = reached(pq, monkeypatch)
    with pytest.warns(RuntimeWarning, match="rotation_int4_w4a4_b200.build"):
        four_calls(pq, lambda shape, t: fake(*shape, dtype=t))
    assert names == ["pq_quant_fp4", "pq_fp4_gemm", "pq_fp4_linear", "pq_kv4_attention_masked"]
    with warnings.catch_warnings():                      # told once
        warnings.simplefilter("error")
        four_calls(pq, lambda shape, t: fake(*shape, dtype=t))
    assert len(names) == 8


def test_refusals_are_the_same(pq):
    with pytest.warns(RuntimeWarning):
        with pytest.raises(ValueError, match="codes: dtype"):
            pq.pq_quant_fp4(fake(4, 256), fake(4, 128, dtype=torch.int8), fake(2048, dtype=torch.uint8))


@pytest.mark.gpu
def test_the_same_bits(pq, monkeypatch):
    gen = torch.Generator(device="cuda").manual_seed(3)
    X, W = (torch.randn(n, 512, generator=gen, device="cuda").to(torch.bfloat16) for n in (20, 130))
    outs = []
    for module in (False, True):
        if module:
            monkeypatch.undo()
            monkeypatch.setattr(pq, "_call", None)
        buffers = [torch.zeros(n, dtype=torch.uint8, device="cuda").view(*v) for r in (20, 130)
                   for n, v in ((r * 256, (r, 256)), (pq.pq_fp4_scale_bytes(r, 512), (-1,)))]
        Y = torch.zeros(20, 130, device="cuda")
        with warnings.catch_warnings(record=True) as told:
            warnings.simplefilter("always")
            pq.pq_quant_fp4(W, buffers[2], buffers[3], g=128, factor=0.01)
            pq.pq_fp4_linear(X, *buffers, Y, g=128, factor_A=0.01, factor_W=0.01)
        assert bool(told) != module
        outs.append((*buffers, Y))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and outs[0][4].abs().sum() > 0


def test_a_warning_that_is_an_error_stops_one_call_only(pq, monkeypatch):
    names = reached(pq, monkeypatch)
    X, c, s = fake(4, 256), fake(4, 128, dtype=torch.uint8), fake(4096, dtype=torch.uint8)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning):
            pq.pq_quant_fp4(X, c, s)
        pq.pq_quant_fp4(X, c, s)
    assert names == ["pq_quant_fp4"]

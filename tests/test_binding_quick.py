"""The compiled way into the library (_pqcall): it takes plainly right calls only; all others are checked, and refused in words, by
pq.py, with the same result."""
import ctypes

import pytest
import torch

from tests.test_new_operator_checks import fake


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def test_calls_that_are_not_plainly_right_are_not_taken(pq):
    """Without a GPU every call is one of these; nothing is dereferenced."""
    call = pq._caller()
    X, c, s, Y = (torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(2048, dtype=torch.uint8),
                  torch.zeros(4, 4))
    lists = torch.zeros(4, 1, dtype=torch.int32)
    cache = pq._KV4Struct(0, 0, 0, 0, 1, 16, 2, 128, 0)
    handle = ctypes.addressof(cache)
    for args in ((X, c, s, "nv", 0, 1.0), (X, c, s, "fp4", 0, 1.0), (X, c, s, "nv", 0), (None, c, s, "nv", 0, 1.0), (X, c, s, 1, 0, 1.0), ()):
        assert call.quant_fp4(*args) == -1
    for args in ((c, s, c, s, Y, "nv", 1.0), (c, s, c, s, Y, "nv", "x"), (c, s, c, s, Y, "nv", torch.ones(())), (fake(4, 128, dtype=torch.uint8), s, c, s, Y, "nv", 1.0)):
        assert call.fp4_gemm(*args) == -1
    assert call.fp4_linear(X, c, s, c, s, Y, "mx", 0, 1.0, 1.0) == -1
    assert call.fp4_linear(X, c, s, c, s, Y, "mx", 1.5, 1.0, 1.0) == -1
    good = [handle, 0, X, X, lists, lists, lists, 1, 1, None, 0, 0, lists]
    for i in range(len(good)):
        for bad in (None, "x", 1 << 70):
            assert call.attention_masked(*(good[:i] + [bad] + good[i + 1:])) == -1
    with pytest.raises(TypeError):
        call.bind(1, 2, 3)


def test_every_function_is_bound(pq):
    call = pq._caller()
    assert {n for n in dir(call) if not n.startswith("_")} == {"bind", "quant_fp4", "fp4_gemm", "fp4_linear", "attention_masked"}
    assert pq._caller() is not None and pq._call is not None


@pytest.mark.gpu
def test_both_ways_give_the_same_bits(pq):
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, N, D = 20, 130, 512
    wide = torch.randn(T, D + 8, generator=gen, device="cuda").to(torch.bfloat16)
    for X in (wide[:, :D].contiguous(), wide[:, :D]):
        for fmt in ("mx", "nv"):
            n = pq.pq_fp4_scale_bytes
            out = []
            for explicit in (False, True):
                ca, sa = torch.zeros(T, D // 2, dtype=torch.uint8, device="cuda"), torch.zeros(n(T, D, fmt), dtype=torch.uint8, device="cuda")
                cw, sw = torch.zeros(N, D // 2, dtype=torch.uint8, device="cuda"), torch.zeros(n(N, D, fmt), dtype=torch.uint8, device="cuda")
                W = torch.randn(N, D, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
                more = dict(stream=torch.cuda.current_stream()) if explicit else {}
                Y = [torch.zeros(T, N, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)]
                pq.pq_quant_fp4(W, cw, sw, fmt=fmt, g=128, factor=0.01, **more)
                pq.pq_fp4_linear(X, ca, sa, cw, sw, Y[0], fmt=fmt, g=128, factor_A=0.01, factor_W=0.01, **more)
                pq.pq_fp4_gemm(ca, sa, cw, sw, Y[1], fmt=fmt, alpha=1e-4, **more)
                out.append((ca, sa, cw, sw, *Y))
            assert all(torch.equal(a, b) for a, b in zip(*out)) and out[0][4].abs().sum() > 0 and out[0][5].abs().sum() > 0


@pytest.mark.gpu
def test_attention_both_ways_and_as_two_dimensions(pq):
    from tests.test_gpu_kv4 import make_case
    cache, Q, starts, lens, table = make_case(pq, 3, [5, 2], [300, 40], 8, 2, 128, 16)
    tree = torch.full((7, 1), 31, dtype=torch.int32, device="cuda")
    outs = []
    for q, more in ((Q, {}), (Q, dict(stream=torch.cuda.current_stream())), (Q.view(7, -1), {}), (Q, dict(scale=128 ** -0.5))):
        O = torch.zeros_like(q)
        pq.pq_kv4_attention_masked(cache, q, O, starts, lens, table, 5, 300, window=100, sinks=3, tree=tree, **more)
        outs.append(O.view(7, 8, 128))
    assert all(torch.equal(outs[0], o) for o in outs[1:]) and outs[0].abs().sum() > 0


@pytest.mark.gpu
def test_refusals_with_cuda_tensors(pq):
    """What the compiled way does not take is named by pq.py; what the library refuses comes as its error."""
    X, c, s = (torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 128, dtype=torch.uint8, device="cuda"),
               torch.zeros(2048 * 2, dtype=torch.uint8, device="cuda"))
    Y = torch.zeros(4, 4, device="cuda")
    with pytest.raises(ValueError, match="codes: dtype"):
        pq.pq_quant_fp4(X, c.view(torch.int8), s)
    with pytest.raises(ValueError, match="scales: holds"):
        pq.pq_quant_fp4(X, c, s[:100])
    with pytest.raises(ValueError, match="fmt="):
        pq.pq_quant_fp4(X, c, s, fmt="e2m1")
    with pytest.raises(ValueError, match="CUDA"):
        pq.pq_fp4_gemm(c, s, c.cpu(), s, Y)
    with pytest.raises(ValueError, match="Y: dtype"):
        pq.pq_fp4_gemm(c, s, c, s, Y.half())
    with pytest.raises(ValueError, match="contiguous"):
        pq.pq_fp4_linear(X, c, s, c, s, Y.t())
    with pytest.raises(pq.PQError, match="multiple of g=128"):
        pq.pq_quant_fp4(X[:, :64], c, s, g=128)
    with pytest.raises(pq.PQError, match="alpha"):
        pq.pq_fp4_gemm(c, s, c, s, Y, alpha=float("nan"))
    with pytest.raises(pq.PQError, match="aligned"):
        pq.pq_fp4_gemm(c, s[8:], c, s, Y)
    cache = pq.KV4Cache.empty(4, 2, 16, 128)
    Q = torch.zeros(5, 4, 128, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="tree: expected"):
        pq.pq_kv4_attention_masked(cache, Q, Q.clone(), i[:2], i[:1], i[:3].view(1, 3), 1, 1, tree=i.view(8, 1))
    with pytest.raises(ValueError, match="q_start: holds"):
        pq.pq_kv4_attention_masked(cache, Q, Q.clone(), i[:1], i[:1], i[:3].view(1, 3), 1, 1, sinks=1, window=2)
    with pytest.raises(pq.PQError, match="sinks=-1"):
        pq.pq_kv4_attention_masked(cache, Q, Q.clone(), i[:2], i[:1], i[:3].view(1, 3), 1, 1, sinks=-1, window=2)


@pytest.mark.gpu
def test_tensors_without_memory_and_other_layouts_are_refused(pq):
    """Sparse and fake tensors reach the compiled way too: an error in words, not an exception out of C."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    X, c, s, Y = (torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 128, dtype=torch.uint8, device="cuda"),
                  torch.zeros(4096, dtype=torch.uint8, device="cuda"), torch.zeros(4, 4, device="cuda"))
    with FakeTensorMode(allow_non_fake_inputs=True) as mode:
        none = {"X": mode.from_tensor(X), "c": mode.from_tensor(c), "s": mode.from_tensor(s), "Y": mode.from_tensor(Y)}
    thin = {"X": X.to_sparse(), "c": c.to_sparse(), "s": s.to_sparse(), "Y": Y.to_sparse()}
    call = pq._caller()
    for other in (none, thin):
        x, codes, scales, y = other["X"], other["c"], other["s"], other["Y"]
        for args in ((x, c, s), (X, codes, s), (X, c, scales)):
            assert call.quant_fp4(*args, "nv", 0, 1.0) != 0
        for args in ((codes, s, c, s, Y), (c, scales, c, s, Y), (c, s, codes, s, Y), (c, s, c, scales, Y), (c, s, c, s, y)):
            assert call.fp4_gemm(*args, "nv", 1.0) != 0
            assert call.fp4_linear(X, *args, "nv", 0, 1.0, 1.0) != 0
        assert call.fp4_linear(x, c, s, c, s, Y, "nv", 0, 1.0, 1.0) != 0


@pytest.mark.gpu
def test_weights_of_another_width_and_groups_past_an_int(pq):
    X, c, s, Y = (torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 128, dtype=torch.uint8, device="cuda"),
                  torch.zeros(4096, dtype=torch.uint8, device="cuda"), torch.zeros(4, 4, device="cuda"))
    wide = torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="codes_W: rows of 256 bytes, expected 128"):
        pq.pq_fp4_gemm(c, s, wide, s, Y)
    with pytest.raises(ValueError, match="codes_W: rows of 256 bytes, expected 128"):
        pq.pq_fp4_linear(X, c, s, wide, s, Y)
    pq.pq_fp4_gemm(c, s, wide, s, Y, D=256)
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises(ValueError, match="g=4294967296"):
            pq.pq_quant_fp4(X, c, s, g=1 << 32, stream=stream)
        with pytest.raises(ValueError, match="g=4294967360"):
            pq.pq_fp4_linear(X, c, s, c, s, Y, g=(1 << 32) + 64, stream=stream)


def test_products_of_factors_below_normal_numbers_are_refused(pq):
    """2^-100 * 2^-40 keeps no more than 9 bits in float32: refused before anything is launched; a factor of 0 is a tensor of zeros."""
    st = pq.lib.pq_fp4_linear(256, 4, 256, 256, 0, 1, 2.0 ** -100, 256, 256, 256, 256, 2.0 ** -40, 4, 256, 0, None)
    assert st != 0 and b"below float32's normal numbers" in pq.lib.pq_last_error()
    st = pq.lib.pq_fp4_linear(256, 4, 256, 256, 0, 1, 2.0 ** -100, 256, 256, 256, 256, -(2.0 ** -40), 4, 256, 0, None)
    assert st != 0 and b"below float32's normal numbers" in pq.lib.pq_last_error()

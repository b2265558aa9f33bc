"""Refusals of the 4-bit floating-point calls and of masked attention, on the CPU: every call below must fail in the binding or
in the library's argument checks, before anything is launched."""
import ctypes

import pytest
import torch

from tests.test_new_operator_checks import ATTEND, FAKE, cache_struct, fake, refused

MX, NV = 0, 1


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


ROWS = dict(X=FAKE, T=4, D=256, ldx=256, g=128, format=NV, factor=1.0, codes=FAKE, scales=FAKE, stream=None)
BAD_ROWS = [
    ({"X": None}, "non-NULL"), ({"codes": None}, "non-NULL"), ({"scales": None}, "non-NULL"), ({"T": 0}, "T=0"), ({"T": (1 << 24) + 1}, "T="),
    ({"D": 16, "g": 0}, "D=16"), ({"D": 80, "ldx": 80, "g": 0}, "D=80"), ({"D": 192, "ldx": 192}, "D=192"),
    ({"D": 65568, "ldx": 65568, "g": 0}, "D=65568"), ({"ldx": 248}, "ldx=248"), ({"ldx": 260}, "ldx=260"), ({"format": 2}, "format"),
    ({"format": -1}, "format"), ({"factor": 0.0}, "factor"), ({"factor": -1.0}, "factor"), ({"factor": float("nan")}, "factor"),
    ({"factor": float("inf")}, "factor"), ({"factor": 1e-38}, "factor"), ({"X": FAKE + 2}, "aligned"), ({"scales": FAKE + 8}, "aligned"),
]


@pytest.mark.parametrize("change,word", BAD_ROWS)
def test_rows(pq, change, word):
    refused(pq, "pq_quant_fp4", ROWS, change, "PQ_ERR_INVALID_ARG", word)


def test_rotation_blocks(pq):
    refused(pq, "pq_quant_fp4", ROWS, {"g": 32}, "PQ_ERR_UNSUPPORTED", "g=32")


GEMM = dict(ca=FAKE, sa=FAKE, cw=FAKE, sw=FAKE, T=4, N=10, D=64, format=MX, alpha=1.0, Y=FAKE, out=0, stream=None)
LINEAR = dict(X=FAKE, T=4, D=64, ldx=64, g=0, format=NV, factor_A=1.0, ca=FAKE, sa=FAKE, cw=FAKE, sw=FAKE, factor_W=1.0, N=10, Y=FAKE,
              out=0, stream=None)


@pytest.mark.parametrize("change,word", [
    ({"ca": None}, "non-NULL"), ({"sw": None}, "non-NULL"), ({"Y": None}, "non-NULL"), ({"T": 0}, "T=0"), ({"N": 0}, "N=0"), ({"N": 1 << 25}, "N="),
    ({"D": 48}, "D=48"), ({"D": 131072}, "D=131072"), ({"format": 3}, "format"), ({"out": 2}, "out_dtype"), ({"cw": FAKE + 4}, "aligned"),
    ({"Y": FAKE + 4}, "aligned"),
])
def test_product(pq, change, word):
    refused(pq, "pq_fp4_gemm", GEMM, change, "PQ_ERR_INVALID_ARG", word)
    change = dict(change, **({"ldx": change["D"]} if "D" in change else {}))
    refused(pq, "pq_fp4_linear", LINEAR, change, "PQ_ERR_INVALID_ARG", word)


@pytest.mark.parametrize("alpha", [float("nan"), float("inf")])
def test_alpha(pq, alpha):
    refused(pq, "pq_fp4_gemm", GEMM, {"alpha": alpha}, "PQ_ERR_INVALID_ARG", "alpha")
    refused(pq, "pq_fp4_linear", LINEAR, {"factor_W": alpha}, "PQ_ERR_INVALID_ARG", "alpha")
    refused(pq, "pq_fp4_linear", LINEAR, {"factor_A": alpha}, "PQ_ERR_INVALID_ARG", "factor")


def test_scale_bytes(pq):
    assert pq.pq_fp4_scale_bytes(1, 32, "mx") == 512 and pq.pq_fp4_scale_bytes(128, 128, "mx") == 512
    assert pq.pq_fp4_scale_bytes(129, 160, "mx") == 2 * 2 * 512 and pq.pq_fp4_scale_bytes(200, 4096, "nv") == 2 * 64 * 512
    for rows, D, fmt in ((0, 64, "mx"), (4, 40, "nv"), (1 << 25, 64, "nv")):
        with pytest.raises(ValueError, match="pq_fp4_scale_bytes"):
            pq.pq_fp4_scale_bytes(rows, D, fmt)
    with pytest.raises(ValueError, match="fmt="):
        pq.pq_fp4_scale_bytes(4, 64, "fp4")


def test_binding_rejects_wrong_tensors(pq):
    X, codes, sc = fake(4, 256), fake(4, 128, dtype=torch.uint8), fake(2048, dtype=torch.uint8)
    with pytest.raises(ValueError, match="fmt="):
        pq.pq_quant_fp4(X, codes, sc, fmt="e2m1")
    with pytest.raises(ValueError, match="codes: dtype"):
        pq.pq_quant_fp4(X, fake(4, 128, dtype=torch.int8), sc)
    with pytest.raises(ValueError, match="codes: holds"):
        pq.pq_quant_fp4(X, fake(4, 127, dtype=torch.uint8), sc)
    with pytest.raises(ValueError, match="scales: holds"):
        pq.pq_quant_fp4(X, codes, fake(2047, dtype=torch.uint8))
    with pytest.raises(ValueError, match="scales: dtype"):
        pq.pq_quant_fp4(X, codes, fake(2048, dtype=torch.float32))
    with pytest.raises(ValueError, match="row stride"):
        pq.pq_quant_fp4(X, codes, sc, ldx=512)
    with pytest.raises(ValueError, match="scales_W: holds"):
        pq.pq_fp4_gemm(codes, sc, fake(129, 128, dtype=torch.uint8), sc, fake(4, 129))
    with pytest.raises(ValueError, match="Y: dtype"):
        pq.pq_fp4_gemm(codes, sc, codes, sc, fake(4, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="Y: holds"):
        pq.pq_fp4_linear(X, codes, sc, codes, sc, fake(4, 3, dtype=torch.float32))
    with pytest.raises(ValueError, match="codes_W: holds"):
        pq.pq_fp4_linear(X, codes, sc, fake(4, 64, dtype=torch.uint8), sc, fake(4, 4))


MASKED = {k: v for k, v in ATTEND.items() if k not in ("O", "ldo", "stream")}
MASKED.update(sinks=4, tree=FAKE, words=1, O=FAKE, ldo=512, stream=None)


@pytest.mark.parametrize("change,word", [
    ({"Q": None}, "Q"), ({"ldq": 516}, "Q"), ({"O": FAKE + 8}, "O"), ({"hq": 5}, "heads_q"), ({"qs": None}, "q_start"), ({"width": 0}, "table_width"),
    ({"B": 0}, "B=0"), ({"T": 0}, "T=0"), ({"max_q": 0}, "max_q"), ({"window": -1}, "window"), ({"sinks": -1}, "sinks=-1"),
    ({"sinks": 1 << 31}, "sinks="), ({"tree": FAKE + 2}, "tree"), ({"words": 0}, "tree_words=0"), ({"words": 1025}, "tree_words=1025"),
    ({"words": -1}, "tree_words=-1"), ({"scale": float("nan")}, "scale"),
])
def test_masked_attention(pq, change, word):
    s = cache_struct(pq)
    refused(pq, "pq_kv4_attention_masked", dict(cache=ctypes.addressof(s), **MASKED), change, "PQ_ERR_INVALID_ARG", word)


def test_binding_rejects_wrong_trees(pq):
    codes, sc = fake(3, 2, 16, 64, dtype=torch.uint8), fake(3, 2, 16, dtype=torch.float32)
    cache = pq.KV4Cache(codes, sc, codes, sc)
    Q, i32 = fake(5, 4, 128), torch.int32
    call = lambda tree: pq.pq_kv4_attention_masked(cache, Q, Q, fake(3, dtype=i32), fake(2, dtype=i32), fake(2, 3, dtype=i32), 1, 1, tree=tree)  # noqa: E731
    for tree, word in ((fake(5, dtype=i32), "tree: expected"), (fake(4, 1, dtype=i32), "tree: expected"), (fake(5, 1, dtype=torch.int64), "tree: dtype")):
        with pytest.raises(ValueError, match=word):
            call(tree)

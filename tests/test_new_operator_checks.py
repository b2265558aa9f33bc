"""Refusals of the 8-bit product and the 4-bit key/value cache, on the CPU: every call below must fail in the binding or in
the library's argument checks, before anything is launched."""
import ctypes

import pytest
import torch

FAKE = 1 << 20            # a 16-byte aligned address, never dereferenced


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def refused(pq, name, good, change, status, word):
    args = dict(good)
    args.update(change)
    st = getattr(pq.lib, name)(*args.values())
    text = pq.lib.pq_last_error().decode()
    assert st == getattr(pq, status), (name, change, st, text)
    assert word in text, (change, text)


ROWS = dict(X=FAKE, T=4, D=256, ldx=256, g=128, codes=FAKE, scales=FAKE, stream=None)


@pytest.mark.parametrize("change,status,word", [
    ({"X": None}, "PQ_ERR_INVALID_ARG", "non-NULL"), ({"codes": None}, "PQ_ERR_INVALID_ARG", "non-NULL"),
    ({"T": 0}, "PQ_ERR_INVALID_ARG", "T=0"), ({"T": -3}, "PQ_ERR_INVALID_ARG", "T=-3"),
    ({"T": (1 << 24) + 1}, "PQ_ERR_INVALID_ARG", "T="),
    ({"D": 0, "g": 0}, "PQ_ERR_INVALID_ARG", "D=0"), ({"D": 264, "ldx": 264, "g": 0}, "PQ_ERR_INVALID_ARG", "D=264"),
    ({"D": 192, "g": 128}, "PQ_ERR_INVALID_ARG", "D=192"), ({"D": 65552, "ldx": 65552, "g": 0}, "PQ_ERR_INVALID_ARG", "D=65552"),
    ({"ldx": 248}, "PQ_ERR_INVALID_ARG", "ldx=248"), ({"ldx": 260}, "PQ_ERR_INVALID_ARG", "ldx=260"),
    ({"g": 32}, "PQ_ERR_UNSUPPORTED", "g=32"), ({"X": FAKE + 2}, "PQ_ERR_INVALID_ARG", "aligned"),
    ({"codes": FAKE + 8}, "PQ_ERR_INVALID_ARG", "aligned"),
])
def test_rows(pq, change, status, word):
    refused(pq, "pq_quant_rows8", ROWS, change, status, word)


GEMM = dict(ca=FAKE, sa=FAKE, cw=FAKE, sw=FAKE, T=4, N=10, D=64, Y=FAKE, out=0, stream=None)


@pytest.mark.parametrize("change,status,word", [
    ({"ca": None}, "PQ_ERR_INVALID_ARG", "non-NULL"), ({"Y": None}, "PQ_ERR_INVALID_ARG", "non-NULL"),
    ({"T": 0}, "PQ_ERR_INVALID_ARG", "T=0"), ({"N": 0}, "PQ_ERR_INVALID_ARG", "N=0"), ({"D": 72}, "PQ_ERR_INVALID_ARG", "D=72"),
    ({"D": 131072}, "PQ_ERR_INVALID_ARG", "D=131072"), ({"out": 2}, "PQ_ERR_INVALID_ARG", "out_dtype"),
    ({"cw": FAKE + 4}, "PQ_ERR_INVALID_ARG", "aligned"),
])
def test_product(pq, change, status, word):
    refused(pq, "pq_w8a8_gemm", GEMM, change, status, word)
    linear = dict(X=FAKE, T=4, D=64, ldx=64, g=0, ca=FAKE, sa=FAKE, cw=FAKE, sw=FAKE, N=10, Y=FAKE, out=0, stream=None)
    if "D" in change:
        change = dict(change, ldx=change["D"])
    args = dict(linear, **change)
    assert pq.lib.pq_w8a8_linear(*args.values()) == getattr(pq, status)


def cache_struct(pq, **change):
    fields = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, pages=4, page_size=16, heads=2, head_dim=128, flags=3)
    fields.update(change)
    s = pq._KV4Struct(*fields.values())
    return s


APPEND = dict(Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, T=3, hq=4, qn=FAKE, kn=FAKE, eps=1e-5, rope=FAKE, rows=10, dim=64,
              pos=FAKE, slots=FAKE, flags=0, out=FAKE, stream=None)
ATTEND = dict(Q=FAKE, ldq=512, hq=4, qs=FAKE, ls=FAKE, bt=FAKE, width=5, B=2, T=3, max_q=2, max_len=50, scale=0.1, window=0, O=FAKE,
              ldo=512, stream=None)
READ = dict(slots=FAKE, T=3, K=FAKE, V=FAKE, stream=None)
CALLS = {"pq_kv4_append": APPEND, "pq_kv4_attention": ATTEND, "pq_kv4_read": READ}


def refused_kv(pq, name, cache_change, change, status, word):
    s = cache_struct(pq, **cache_change)
    refused(pq, name, dict(cache=ctypes.addressof(s), **CALLS[name]), change, status, word)


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("change,status,word", [
    ({"k_codes": None}, "PQ_ERR_INVALID_ARG", "non-NULL"), ({"v_scales": None}, "PQ_ERR_INVALID_ARG", "non-NULL"),
    ({"v_codes": FAKE + 8}, "PQ_ERR_INVALID_ARG", "aligned"), ({"head_dim": 96}, "PQ_ERR_UNSUPPORTED", "head_dim=96"),
    ({"head_dim": 256}, "PQ_ERR_UNSUPPORTED", "head_dim=256"), ({"page_size": 8}, "PQ_ERR_UNSUPPORTED", "page_size=8"),
    ({"page_size": 48}, "PQ_ERR_UNSUPPORTED", "page_size=48"), ({"page_size": 512}, "PQ_ERR_UNSUPPORTED", "page_size=512"),
    ({"heads": 0}, "PQ_ERR_INVALID_ARG", "heads=0"), ({"pages": 0}, "PQ_ERR_INVALID_ARG", "pages=0"),
    ({"flags": 4}, "PQ_ERR_INVALID_ARG", "flags"),
])
def test_cache(pq, name, change, status, word):
    refused_kv(pq, name, change, {}, status, word)


def test_null_cache(pq):
    for name, args in CALLS.items():
        assert getattr(pq.lib, name)(None, *args.values()) == pq.PQ_ERR_INVALID_ARG


@pytest.mark.parametrize("change,word", [
    ({"Q": None}, "Q"), ({"ldq": 508}, "Q"), ({"ldk": 250}, "K"), ({"ldk": 258}, "K"), ({"V": FAKE + 4}, "V"), ({"out": FAKE + 8}, "Q_out"),
    ({"T": 0}, "T=0"), ({"hq": 3}, "heads_q=3"), ({"hq": 0}, "heads_q=0"), ({"slots": None}, "slots"), ({"flags": 2}, "flags"),
    ({"eps": -1.0}, "eps"), ({"eps": float("nan")}, "eps"), ({"dim": 12}, "rope_dim"), ({"dim": 136}, "rope_dim"), ({"dim": 0}, "rope_dim"),
    ({"rows": 0}, "rope"), ({"pos": None}, "rope"), ({"rope": FAKE + 4}, "rope"), ({"qn": FAKE + 2}, "norm"),
])
def test_append(pq, change, word):
    refused_kv(pq, "pq_kv4_append", {}, change, "PQ_ERR_INVALID_ARG", word)


@pytest.mark.parametrize("change,word", [
    ({"Q": None}, "Q"), ({"ldq": 516}, "Q"), ({"O": FAKE + 8}, "O"), ({"ldo": 504}, "O"), ({"hq": 5}, "heads_q"), ({"qs": None}, "q_start"),
    ({"ls": FAKE + 2}, "seq_lens"), ({"width": 0}, "table_width"), ({"width": 1 << 28}, "table_width"), ({"B": 0}, "B=0"), ({"B": 65536}, "B="),
    ({"T": 0}, "T=0"), ({"max_q": 0}, "max_q"), ({"max_len": 0}, "max_len"), ({"window": -1}, "window"), ({"scale": float("inf")}, "scale"),
])
def test_attention(pq, change, word):
    refused_kv(pq, "pq_kv4_attention", {}, change, "PQ_ERR_INVALID_ARG", word)


@pytest.mark.parametrize("width", [(1 << 26) + 1, 1 << 30, 1 << 40, 1 << 62])
def test_attention_lengths(pq, width):
    """Pages of 16: tokens of a sequence are numbered in int32, sums of two of them too."""
    refused_kv(pq, "pq_kv4_attention", {"page_size": 16}, {"width": width}, "PQ_ERR_INVALID_ARG", "table_width")


# ------------------------------------------------------------------- the binding's own checks
class FakeCuda:
    """Stands in for a CUDA tensor (never dereferenced)."""

    def __init__(self, t):
        self._t = t
        self.shape, self.dtype, self.is_cuda, self.device = t.shape, t.dtype, True, "cuda:0"

    def __getattr__(self, name):
        return getattr(self._t, name)

    def data_ptr(self):
        return FAKE


def fake(*shape, dtype=torch.bfloat16):
    return FakeCuda(torch.empty(*shape, dtype=dtype))


def test_binding_rejects_wrong_tensors(pq):
    X, codes, sc = fake(4, 256), fake(4, 256, dtype=torch.int8), fake(4, dtype=torch.float32)
    with pytest.raises(ValueError, match="codes: dtype"):
        pq.pq_quant_rows8(X, fake(4, 256, dtype=torch.uint8), sc)
    with pytest.raises(ValueError, match="scales: holds"):
        pq.pq_quant_rows8(X, codes, fake(3, dtype=torch.float32))
    with pytest.raises(ValueError, match="Y: dtype"):
        pq.pq_w8a8_gemm(codes, sc, codes, sc, fake(4, 4, dtype=torch.float16))
    with pytest.raises(ValueError, match="Y: holds"):
        pq.pq_w8a8_gemm(codes, sc, codes, sc, fake(4, 3, dtype=torch.float32))
    with pytest.raises(ValueError, match="codes_W: holds"):
        pq.pq_w8a8_linear(X, codes, sc, fake(4, 128, dtype=torch.int8), sc, fake(4, 4))


def test_binding_rejects_wrong_caches(pq):
    codes, sc = fake(3, 2, 16, 64, dtype=torch.uint8), fake(3, 2, 16, dtype=torch.float32)
    cache = pq.KV4Cache(codes, sc, codes, sc)
    assert (cache.pages, cache.heads, cache.page_size, cache.head_dim) == (3, 2, 16, 128)
    with pytest.raises(ValueError, match="shapes"):
        pq.KV4Cache(codes, sc, fake(3, 2, 16, 32, dtype=torch.uint8), sc)
    with pytest.raises(ValueError, match="expected"):
        pq.KV4Cache(fake(3, 2, 16, dtype=torch.uint8), sc, codes, sc)
    with pytest.raises(ValueError, match="dtype"):
        pq.KV4Cache(codes, fake(3, 2, 16), codes, sc)
    with pytest.raises(ValueError, match="CUDA"):
        pq.KV4Cache(*(t._t for t in (codes, sc, codes, sc)))
    Q, K = fake(5, 4, 128), fake(5, 256)
    slots = fake(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="slots: dtype"):
        pq.pq_kv4_append(cache, Q, K, K, fake(5, 4, 128), None, fake(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="K: shape"):
        pq.pq_kv4_append(cache, Q, fake(5, 128), K, fake(5, 4, 128), None, slots)
    with pytest.raises(ValueError, match="Q_out: holds"):
        pq.pq_kv4_append(cache, Q, K, K, fake(5, 3, 128), None, slots)
    with pytest.raises(ValueError, match="whole heads"):
        pq.pq_kv4_append(cache, fake(5, 200), K, K, fake(5, 200), None, slots)
    with pytest.raises(ValueError, match="Q: shape"):
        pq.pq_kv4_attention(cache, FakeCuda(torch.empty(128, 10, dtype=torch.bfloat16).t()), fake(10, 128), None, None, fake(1, 2, dtype=torch.int32), 1, 1)
    with pytest.raises(ValueError, match="q_start: holds"):
        pq.pq_kv4_attention(cache, Q, Q, fake(2, dtype=torch.int32), fake(2, dtype=torch.int32), fake(2, 3, dtype=torch.int32), 1, 1)
    with pytest.raises(ValueError, match="block_table"):
        pq.pq_kv4_attention(cache, Q, Q, slots, slots, fake(6, dtype=torch.int32), 1, 1)

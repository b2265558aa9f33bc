"""What the binding refuses before the 8-bit calls reach the library, on the CPU: row strides that are not the tensor's, and
tensors that are not on a GPU.  The library itself is replaced, so nothing can be launched."""
import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


class FakeCuda:
    """Stands in for a CUDA tensor (never dereferenced)."""

    def __init__(self, t):
        self._t = t
        self.shape, self.dtype, self.is_cuda, self.device = t.shape, t.dtype, True, "cuda:0"

    def __getattr__(self, name):
        return getattr(self._t, name)

    def data_ptr(self):
        return FAKE


class NoLibrary:
    """Stands in for the loaded library: records the calls that get as far as it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def reached(pq, monkeypatch):
    lib = NoLibrary()
    monkeypatch.setattr(pq, "lib", lib)
    monkeypatch.setattr(pq, "_raw_stream", lambda stream, dev, torch: 0)
    return lib.calls


def rows8(pq, X, T=4, D=256, **kw):
    codes, sc = FakeCuda(torch.empty(T, D, dtype=torch.int8)), FakeCuda(torch.empty(T))
    pq.pq_quant_rows8(X, codes, sc, T=T, D=D, **kw)


def linear8(pq, X, T=4, D=256, N=8, **kw):
    codes, sc = FakeCuda(torch.empty(T, D, dtype=torch.int8)), FakeCuda(torch.empty(T))
    w, sw = FakeCuda(torch.empty(N, D, dtype=torch.int8)), FakeCuda(torch.empty(N))
    pq.pq_w8a8_linear(X, codes, sc, w, sw, FakeCuda(torch.empty(T, N)), T=T, D=D, **kw)


@pytest.mark.parametrize("call", [rows8, linear8])
@pytest.mark.parametrize("ldx", [1 << 20, 512, 264, 248, 8, 0])
def test_a_row_stride_that_is_not_the_tensors(pq, reached, call, ldx):
    with pytest.raises(ValueError, match="row stride 256 differs from ldx"):
        call(pq, FakeCuda(torch.empty(4, 256, dtype=torch.bfloat16)), ldx=ldx)
    with pytest.raises(ValueError, match="row stride 256 differs from ldx"):
        call(pq, FakeCuda(torch.empty(4, 256, dtype=torch.bfloat16)), T=2, ldx=ldx)
    assert not reached


@pytest.mark.parametrize("call", [rows8, linear8])
def test_row_strides_that_are(pq, reached, call):
    wide = torch.empty(4, 1024, dtype=torch.bfloat16)
    call(pq, FakeCuda(wide[:, :256]))
    call(pq, FakeCuda(wide[:, :256]), ldx=1024)
    call(pq, FakeCuda(wide[:1, :256]), T=1, ldx=256)               # a single row's stride says nothing
    call(pq, FakeCuda(wide[:1, :256]), T=1)
    assert [args[3] for _, args in reached] == [1024, 1024, 256, 256]
    with pytest.raises(ValueError, match="X: holds"):
        call(pq, FakeCuda(wide[:, :256]), T=5)
    with pytest.raises(ValueError, match="X: holds"):
        call(pq, FakeCuda(wide[:1, :128]), T=1, D=256, ldx=1024)
    assert len(reached) == 4


class Host:
    """A CPU tensor whose address must not leave the binding."""

    def __init__(self, t):
        self._t = t
        self.shape, self.dtype, self.is_cuda, self.device = t.shape, t.dtype, False, t.device

    def __getattr__(self, name):
        return getattr(self._t, name)

    def data_ptr(self):
        raise AssertionError("the address of a host tensor was taken")


ROWS = {"X": ((4, 256), torch.bfloat16), "codes": ((4, 256), torch.int8), "scales": ((4,), torch.float32)}
GEMM = {"codes_A": ((4, 256), torch.int8), "scales_A": ((4,), torch.float32), "codes_W": ((8, 256), torch.int8),
        "scales_W": ((8,), torch.float32), "Y": ((4, 8), torch.float32)}
LINEAR = dict([("X", ROWS["X"])], **GEMM)


@pytest.mark.parametrize("name,spec,host", [(n, s, h) for n, s in (("pq_quant_rows8", ROWS), ("pq_w8a8_gemm", GEMM), ("pq_w8a8_linear", LINEAR))
                                            for h in s])
def test_host_tensors_are_refused(pq, reached, name, spec, host):
    """One argument on the CPU, the others on the GPU; nothing has touched CUDA before."""
    args = {k: (Host if k == host else FakeCuda)(torch.empty(shape, dtype=dtype)) for k, (shape, dtype) in spec.items()}
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        getattr(pq, name)(**args)
    assert not reached


def test_host_tensors_of_the_cache_calls_are_refused(pq, reached):
    codes, sc = FakeCuda(torch.empty(3, 2, 16, 64, dtype=torch.uint8)), FakeCuda(torch.empty(3, 2, 16))
    cache = pq.KV4Cache(codes, sc, codes, sc)
    rows, i64, i32 = torch.empty(5, 256, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int64), torch.zeros(6, dtype=torch.int32)
    good = FakeCuda(rows)
    for Q, K, Q_out, slots in ((Host(rows), good, good, FakeCuda(i64)), (good, Host(rows), good, FakeCuda(i64)),
                               (good, good, Host(rows), FakeCuda(i64)), (good, good, good, Host(i64))):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            pq.pq_kv4_append(cache, Q, K, good, Q_out, None, slots)
    with pytest.raises(ValueError, match="expected a CUDA tensor"):
        pq.pq_kv4_read(cache, Host(i64), good, good)
    table = torch.zeros(5, 4, dtype=torch.int32)
    for starts, lens, tab in ((Host(i32), FakeCuda(i32), FakeCuda(table)), (FakeCuda(i32), Host(i32), FakeCuda(table)),
                              (FakeCuda(i32), FakeCuda(i32), Host(table))):
        with pytest.raises(ValueError, match="expected a CUDA tensor"):
            pq.pq_kv4_attention(cache, good, good, starts, lens, tab, 1, 10)
    assert not reached

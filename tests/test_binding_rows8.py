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

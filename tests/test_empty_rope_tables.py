"""A table of positions without entries is refused: its memory is no address, which the library reads as no rotation at all."""
import pytest
import torch

from tests.test_new_operator_checks import FakeCuda, fake


class Empty(FakeCuda):
    def data_ptr(self):
        return 0                                         # as torch gives for tensors without elements


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def append(pq, monkeypatch, rope):
    codes, sc = fake(3, 2, 16, 64, dtype=torch.uint8), fake(3, 2, 16, dtype=torch.float32)
    cache = pq.KV4Cache(codes, sc, codes, sc)
    reached = []
    monkeypatch.setattr(pq, "lib", type("Library", (), {"pq_kv4_append": staticmethod(lambda *a: reached.append(a) or 0)}))
    pq.pq_kv4_append(cache, fake(5, 512), fake(5, 256), fake(5, 256), fake(5, 512), fake(5, dtype=torch.int32), fake(5, dtype=torch.int64),
                     rope=rope, stream=0)
    return reached


@pytest.mark.parametrize("shape", [(0, 64), (4096, 0), (0, 0)])
def test_tables_without_entries(pq, monkeypatch, shape):
    with pytest.raises(ValueError, match="rope: expected"):
        append(pq, monkeypatch, Empty(torch.empty(*shape)))


def test_tables_and_none_arrive(pq, monkeypatch):
    (args,) = append(pq, monkeypatch, fake(4096, 64, dtype=torch.float32))
    assert args[12] and args[13:15] == (4096, 64)
    (args,) = append(pq, monkeypatch, None)
    assert args[12] is None and args[13:15] == (0, 0)

"""A tree of no words is refused: its memory is no address, which the library reads as no tree at all, and the rows would see all
tokens in front of them."""
import pytest
import torch

from tests.test_new_operator_checks import FakeCuda, fake


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import build
    build.build()
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def attend(pq, tree, monkeypatch, **more):
    """The masked call on host tensors; returns what would reach the library."""
    codes, sc = fake(3, 2, 16, 64, dtype=torch.uint8), fake(3, 2, 16, dtype=torch.float32)
    cache = pq.KV4Cache(codes, sc, codes, sc)
    Q, i32 = fake(5, 4, 128), torch.int32
    reached = []
    monkeypatch.setattr(pq, "lib", type("Library", (), {"pq_kv4_attention_masked": staticmethod(lambda *a: reached.append(a) or 0)}))
    pq.pq_kv4_attention_masked(cache, Q, Q, fake(3, dtype=i32), fake(2, dtype=i32), fake(2, 3, dtype=i32), 3, 9, tree=tree, stream=0, **more)
    return reached


@pytest.mark.parametrize("more", [{}, dict(window=4, sinks=1)])
@pytest.mark.parametrize("tree", [torch.empty(5, 0, dtype=torch.int32), torch.empty(5, 1, dtype=torch.int32)[:, :0]], ids=["empty", "cut"])
def test_trees_of_no_words(pq, monkeypatch, tree, more):
    with pytest.raises(ValueError, match=r"tree: expected \[5, words\]"):
        attend(pq, FakeCuda(tree), monkeypatch, **more)


def test_trees_with_words_and_none_arrive(pq, monkeypatch):
    (args,) = attend(pq, fake(5, 2, dtype=torch.int32), monkeypatch)
    assert args[15] and args[16] == 2
    (args,) = attend(pq, None, monkeypatch)
    assert args[15] is None and args[16] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q", [2, 64])
def test_trees_of_no_words_on_the_gpu(pq, q):
    from tests.test_gpu_kv4 import make_case
    cache, Q, starts, lens, table = make_case(pq, 3, [q], [100], 8, 2, 128, 16)
    O = torch.full_like(Q, 7.0)
    for more in ({}, dict(stream=torch.cuda.current_stream())):
        for tree in (torch.zeros(q, 0, dtype=torch.int32, device="cuda"), torch.zeros(q, 1, dtype=torch.int32, device="cuda")[:, :0]):
            with pytest.raises(ValueError, match="words"):
                pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, 100, tree=tree, **more)
    assert bool((O == 7.0).all())

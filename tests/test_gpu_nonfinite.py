"""A NaN or an infinity among the inputs is seen in the outputs that depend on it, and in no other."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


BAD = [float("nan"), float("inf"), float("-inf"), -float("nan")]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,D,g", [(5, 256, 0), (5, 256, 64), (9, 4096, 128), (3, 512, 256), (3, 14336, 128), (3, 40960, 128), (3, 40976, 0)])
def test_rows8(pq, T, D, g, bad):
    X = normal(D, T, D)

    def run():
        codes, sc = torch.full((T, D), 99, dtype=torch.int8, device="cuda"), torch.full((T,), -1.0, device="cuda")
        pq.pq_quant_rows8(X, codes, sc, g=g)
        return codes, sc

    codes, sc = run()
    for row, channel in ((0, 0), (T // 2, D // 2 + 3), (T - 1, D - 1)):
        keep = X[row, channel].clone()
        X[row, channel] = bad
        c, s = run()
        X[row, channel] = keep
        others = torch.arange(T, device="cuda") != row
        assert s[row].isnan() and (c[row] == 0).all()
        assert torch.equal(s[others], sc[others]) and torch.equal(c[others], codes[others])


@pytest.mark.parametrize("T,N,D", [(1, 100, 256), (20, 500, 4096), (300, 700, 512), (600, 9000, 256)])
def test_linear8(pq, T, N, D):
    """One token diverged: its outputs are NaN, the others' the same bits."""
    X, W = normal(1, T, D), normal(2, N, D)
    cw, sw = torch.empty(N, D, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    pq.pq_quant_rows8(W, cw, sw, g=128)

    def run():
        ca, sa, Y = torch.empty(T, D, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        pq.pq_w8a8_linear(X, ca, sa, cw, sw, Y, g=128)
        return Y

    want = run()
    assert want.isfinite().all()
    X[T // 2, 3] = float("nan")
    Y = run()
    others = torch.arange(T, device="cuda") != T // 2
    assert Y[T // 2].isnan().all() and torch.equal(Y[others], want[others])

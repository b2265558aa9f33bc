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


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("hd,rope_dim,norm", [(64, 0, False), (64, 48, False), (128, 128, True), (128, 24, True), (128, 0, False)])
@pytest.mark.parametrize("rotate", [False, True])
def test_append(pq, hd, rope_dim, norm, rotate, bad):
    """A bad channel of a key or a value: its head's scale is NaN, and what attends to the token is NaN; other heads, tokens
    and slots keep their bits."""
    T, hkv, page = 6, 3, 16
    qkv = normal(hd, T, 3 * hkv * hd)
    Q, K, V = qkv.split(hkv * hd, dim=1)
    w = (1 + 0.1 * normal(3, hd).float()).to(torch.bfloat16) if norm else None
    inv = 10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device="cuda") / max(rope_dim, 1))
    a = torch.arange(40, dtype=torch.float64, device="cuda")[:, None] * inv
    rope = torch.cat([a.cos(), a.sin()], dim=1).float().contiguous() if rope_dim else None
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 3, -1, 17, 0, 30], device="cuda")

    def run():
        cache = pq.KV4Cache.empty(2, hkv, page, hd, rotate_k=rotate, rotate_v=rotate)
        Q_out = torch.empty(T, hkv, hd, dtype=torch.bfloat16, device="cuda")
        pq.pq_kv4_append(cache, Q, K, V, Q_out, positions, slots, rope=rope, q_norm=w, k_norm=w)
        return cache, Q_out

    want, q_want = run()
    for i, x in ((0, K), (2, V)):
        token, head = 3, 1
        keep = x[token, head * hd + 5].clone()
        x[token, head * hd + 5] = bad
        got, q_got = run()
        x[token, head * hd + 5] = keep
        assert torch.equal(q_got, q_want)
        for k in range(4):
            same = torch.ones_like(want.tensors[k], dtype=torch.bool)
            if k in (i, i + 1):
                same[1, head, 1] = False                        # slot 17 = page 1, place 1
            assert torch.equal(got.tensors[k][same], want.tensors[k][same])
        assert got.tensors[i + 1][1, head, 1].isnan() and (got.tensors[i][1, head, 1] == 0).all()
        out = [torch.empty(T, hkv, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        pq.pq_kv4_read(got, slots, *out)
        assert out[i // 2][token, head].isnan().all()
    keep = Q[2, hd + 7].clone()
    Q[2, hd + 7] = bad
    _, q_got = run()
    Q[2, hd + 7] = keep
    others = torch.ones(T, hkv, dtype=torch.bool, device="cuda")
    others[2, 1] = False
    assert torch.equal(q_got[others], q_want[others]) and not q_got[2, 1].isfinite().all()

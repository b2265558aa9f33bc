"""Attention over the 4-bit cache, every output within the spread of its kernel's roundings (spread64.py)."""
import pytest
import torch

from tests.spread64 import attention
from tests.test_gpu_kv4 import make_case, spread

pytestmark = pytest.mark.gpu

FEW_ROWS = 32         # query rows a key/value head and sequence up to which pq.h promises exact codes


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def check(pq, case, max_q, max_len, window=0, scale=None):
    cache, Q, starts, lens, table = case
    T, hq, hd = Q.shape
    O = torch.empty_like(Q)
    pq.pq_kv4_attention(cache, Q, O, starts, lens, table, max_q, max_len, scale=scale, window=window)
    want, tol = attention(cache, Q, starts, lens, table, hd ** -0.5 if scale is None else scale, window,
                          max_q * (hq // cache.heads) > FEW_ROWS)
    off = (O.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / tol).nan_to_num(1e9).max()):.3g} "
                           f"of its bound, first at {bad.nonzero()[0].tolist()}")
    pq.pq_check_status()


@pytest.mark.parametrize("rv", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page,window", [
    ([1], [1], 1, 1, 16, 0), ([1], [517], 32, 8, 64, 0), ([1], [4097], 8, 8, 32, 0), ([1], [20000], 5, 1, 256, 0),
    ([1, 0, 1, 1], [300, 0, 1, 1025], 14, 2, 16, 0), ([2, 3], [2, 700], 7, 1, 128, 0), ([4, 1], [900, 3000], 8, 2, 32, 0),
    ([5], [5], 4, 2, 16, 0), ([1, 1], [5000, 130], 8, 2, 16, 1000), ([8], [777], 8, 2, 16, 100),
    (*spread(6, 60, 3, 3000, 7), 8, 4, 64, 0),
])
def test_few_rows(pq, hd, rv, qs, ls, hq, hkv, page, window):
    check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page, rv=rv), max(qs), max(ls), window=window)


@pytest.mark.parametrize("rv", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page,window", [
    ([128], [128], 2, 1, 64, 0), ([127], [130], 4, 2, 16, 0), ([129, 64], [129, 1000], 8, 8, 128, 0),
    ([300, 0, 1, 77], [811, 0, 400, 77], 14, 2, 16, 0), ([65, 200], [3000, 200], 32, 8, 256, 0), ([513], [1537], 8, 1, 32, 0),
    ([17, 1, 40], [17, 900, 64], 8, 2, 32, 0), ([64, 1, 1, 1], [64, 5000, 900, 1], 8, 2, 64, 0), ([40], [9000], 4, 4, 64, 0),
    ([200, 30], [200, 999], 8, 2, 16, 100), ([100], [6000], 8, 2, 32, 1024),
])
def test_many_rows(pq, hd, rv, qs, ls, hq, hkv, page, window):
    check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page, rv=rv), max(qs), max(ls), window=window)


@pytest.mark.parametrize("rv", [False, True])
@pytest.mark.parametrize("key", [1.0, 30.0, 1e4])
@pytest.mark.parametrize("value", [3e-3, 8.0, 50.0, 700.0, 2.0 ** 20])
@pytest.mark.parametrize("q,n,js", [(1, 900, [3]), (7, 700, [0, 600]), (140, 700, [3]), (140, 700, [40]), (64, 3000, [0, 1000, 2900]), (300, 400, [290])])
def test_one_token_of_another_scale(pq, q, n, js, value, key, rv):
    """A token whose value scale lies far above or below the others', with any share of the probability (its score is near the
    others', or dozens or thousands above or below them), costs the other tokens nothing of their precision."""
    cache, Q, starts, lens, table = make_case(pq, n + q, [q], [n], 8, 2, 128, 16, rv=rv, poison=False)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(q)
    for i in (1, 3):                                      # the others' scales: within a factor of 2
        cache.tensors[i].copy_(torch.rand(cache.tensors[i].shape, generator=gen, device="cuda") * 0.05 + 0.05)
    for j in js:
        page, place = int(table[0, j // 16]), j % 16
        cache.tensors[1][page, :, place] *= key
        cache.tensors[3][page, :, place] *= value
    check(pq, (cache, Q, starts, lens, table), q, n)


@pytest.mark.parametrize("rv", [False, True])
@pytest.mark.parametrize("q,n,j0,step", [(1, 900, 3, 40), (140, 700, 3, 1000), (140, 700, 5, 97), (300, 1500, 0, 33), (64, 500, 0, 1)])
def test_values_of_zero(pq, q, n, j0, step, rv):
    """Tokens whose value is zero (scale 0) may take all of a row's probability but e^-40: the little that the other tokens
    leave comes out as precisely as any output.  step 1: more than half of the tokens, whole blocks of 32 among them."""
    cache, Q, starts, lens, table = make_case(pq, n + q, [q], [n], 8, 2, 128, 16, rv=rv, poison=False)
    for j in range(j0, n if step > 1 else n * 2 // 3, step):
        page, place = int(table[0, j // 16]), j % 16
        cache.tensors[1][page, :, place] = 0.8
        cache.tensors[3][page, :, place] = 0.0
    check(pq, (cache, Q, starts, lens, table), q, n)

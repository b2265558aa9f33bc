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

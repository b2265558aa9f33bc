"""Pages of a sequence that a sliding window has left behind, and starts and bounds at the ends of their types."""
import pytest
import torch

from tests.test_gpu_kv4 import make_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("q,n,max_len", [(1, 300, 300), (1, 3000, 3000), (3, 777, 777), (64, 900, 900), (300, 1000, 1000)])
def test_pages_before_the_window_are_not_looked_at(pq, q, n, max_len, page):
    """A server takes back the pages that no new token's window reaches; their places in the table say nothing any more."""
    cache, Q, starts, lens, table = make_case(pq, n, [q], [n], 8, 2, 128, page, poison=False)
    for window in (1, 7, 16, 17, 40, 60, 100, 200, 255):
        want, O = torch.empty_like(Q), torch.empty_like(Q)
        pq.pq_kv4_attention(cache, Q, want, starts, lens, table, q, max_len, window=window)
        freed = table.clone()
        freed[0, :max(0, n - q - window + 1) // page] = -1
        pq.pq_check_status()
        pq.pq_kv4_attention(cache, Q, O, starts, lens, freed, q, max_len, window=window)
        pq.pq_check_status()
        assert torch.equal(O, want)


@pytest.mark.parametrize("q,n", [(5, 300), (5, 2000), (200, 900)])
@pytest.mark.parametrize("ends", [(2 ** 31 - 1, -2 ** 31), (-2 ** 31, -1), (2 ** 31 - 2, 2 ** 31 - 1), (-7, None), (0, 2 ** 31 - 1)])
def test_starts_outside_the_rows(pq, q, n, ends):
    """An entry of q_start outside 0..T counts as the nearer end: no row beyond Q is read or written."""
    cache, Q, starts, lens, table = make_case(pq, n, [q], [n], 8, 2, 128, 16, poison=False)
    want, O = torch.full_like(Q, 11.0), torch.full_like(Q, 11.0)
    first, last = (min(max(q if x is None else x, 0), q) for x in ends)
    if last > first:
        pq.pq_kv4_attention(cache, Q, want, starts, lens, table, q, n)
    ends = torch.tensor([q if x is None else x for x in ends], dtype=torch.int32, device="cuda")
    pq.pq_kv4_attention(cache, Q, O, ends, lens, table, q, n)
    assert torch.equal(O, want)
    pq.pq_check_status()


@pytest.mark.parametrize("q,n", [(1, 300), (1, 2000), (70, 900)])
@pytest.mark.parametrize("max_q,max_len", [(2 ** 62, 2 ** 31), (2 ** 63 - 1, 2 ** 63 - 1), (2 ** 33, 2 ** 40), (1 << 24, 1 << 30)])
def test_bounds_as_large_as_their_type(pq, q, n, max_q, max_len):
    """Upper bounds that bound nothing: as many query rows and tokens as there can be."""
    cache, Q, starts, lens, table = make_case(pq, n, [q], [n], 8, 2, 128, 16, poison=False)
    want, O = torch.empty_like(Q), torch.empty_like(Q)
    pq.pq_kv4_attention(cache, Q, want, starts, lens, table, 1 << 20, 1 << 30)
    pq.pq_kv4_attention(cache, Q, O, starts, lens, table, max_q, max_len)
    assert torch.equal(O, want)
    pq.pq_check_status()

"""Trees of many drafted tokens under a window: a row's list says its position, and lists are long (to 40 words here)."""
import pytest

from tests.test_gpu_kv4 import make_case
from tests.test_gpu_kv4_masked import check, pq, trees_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,hq,hkv", [(128, 2, 1), (64, 7, 1)])
@pytest.mark.parametrize("qs,ls,window,sinks", [
    ([1000], [1300], 300, 4), ([1250, 3], [1250, 900], 100, 0), ([700, 0, 129], [2000, 0, 4000], 1500, 130), ([300], [5000], 1, 1),
    ([260, 1, 64], [300, 1, 6000], 5000, 7),
])
def test_long_lists(pq, hd, hq, hkv, qs, ls, window, sinks):  # noqa: F811
    check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, 32), max(qs), max(ls), window, sinks, trees_of(qs, sum(ls), 0.9))

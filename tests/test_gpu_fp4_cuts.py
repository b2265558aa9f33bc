"""Products of few tokens on both sides of the sizes where their reduction is cut further: every output exact, however it is cut
(sums of magnitudes below 2^24 smallest products, as in test_gpu_fp4.test_exact_products)."""
import numpy as np
import pytest

from tests import plain_fp4 as P
from tests.test_gpu_fp4 import _codes, _gemm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 16, 17])
@pytest.mark.parametrize("N,D", [(4096, 8192), (4224, 8192), (4225, 8192), (4608, 8192), (4736, 8160), (9088, 4096), (9089, 4096), (9216, 4064), (9473, 4096),
                                 (2304, 10240)])
def test_cuts(fmt, T, N, D):
    lo, hi, unit = (127, 128, 0.25) if fmt == "mx" else (56, 57, 2.0 ** -8)
    ca, sa = _codes(T, D, fmt, 21, lo, hi)
    cw, sw = _codes(N, D, fmt, 22, lo, hi)
    a, w = P.values(ca.cpu().numpy(), sa.cpu().numpy(), T, D, fmt), P.values(cw.cpu().numpy(), sw.cpu().numpy(), N, D, fmt)
    # float32 sums of D positive terms are off by D / 2^24 of them at most
    assert (np.abs(a).astype(np.float32) @ np.abs(w).astype(np.float32).T).max() / unit * (1 + D * 2.0 ** -24) < 2 ** 24
    got = _gemm(ca, sa, cw, sw, T, N, fmt).double().cpu().numpy()
    assert np.array_equal(got, a.astype(np.float64) @ w.astype(np.float64).T)

"""test_gpu_fp4.test_exact_products compares the outputs whose sums float32 holds exactly in any order: those whose magnitudes, in
units of the smallest product, add up to less than 2^24.  Here, without a GPU: at its sizes and scales that is every output, so
nothing is left out there.  (The largest sum is 0.76 of 2^24: 257 x 1003 x 4192, nv.)"""
import numpy as np
import pytest
import torch

from tests import plain_fp4 as P
from tests import test_gpu_fp4 as G


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,N,D", G.SIZES)
def test_every_output_is_compared(monkeypatch, fmt, T, N, D):
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self: self)
    (lo, hi), unit = ((127, 129), 0.25) if fmt == "mx" else ((56, 63), 2.0 ** -8)
    a, w = (np.abs(P.values(c.numpy(), s.numpy(), rows, D, fmt)) for rows, seed in ((T, 1), (N, 2)) for c, s in [G._codes(rows, D, fmt, seed, lo, hi)])
    assert np.all(a / np.sqrt(unit) == np.rint(a / np.sqrt(unit)))       # so all products are whole units
    a, w = a.astype(np.float32), w.astype(np.float32)                    # positive sums: float32 adds D / 2^24 of them at most
    assert (a @ w.T).max() / unit * (1 + D * 2.0 ** -24) < 2 ** 24

"""The bound that the attention kernels are held to (spread64.py) lets exact outputs and their roundings pass and no mistake of
a few percent: mistakes planted in a float64 attention, on the CPU."""
import math

import pytest
import torch

from tests.plain64 import hadamard, unpack
from tests.spread64 import attention


class Cache:
    def __init__(self, gen, pages, hkv, page, hd, rotate_v):
        y = torch.randn(pages, hkv, page, hd, generator=gen), torch.randn(pages, hkv, page, hd, generator=gen)
        self.tensors = []
        for x in y:
            m = x.abs().amax(-1)
            u = torch.round(x * (7 / m)[..., None]).to(torch.int32) & 15
            self.tensors += [(u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8), m / 7]
        self.pages, self.heads, self.page_size, self.head_dim, self.rotate_v = pages, hkv, page, hd, rotate_v


def case(q, n, hq, hkv, hd, rotate_v, page=16):
    gen = torch.Generator().manual_seed(n + q)
    pages = -(-n // page)
    cache = Cache(gen, pages, hkv, page, hd, rotate_v)
    Q = torch.randn(q, hq, hd, generator=gen).to(torch.bfloat16)
    table = torch.randperm(pages, generator=gen)[None].to(torch.int32)
    return cache, Q, torch.tensor([0, q], dtype=torch.int32), torch.tensor([n], dtype=torch.int32), table


def direct(cache, Q, table, n, scale, window=0, skip=None, value_scale=1.0, dtype=torch.float64):
    """The same attention, straight from the definition, with mistakes: tokens skip[0] .. skip[1] - 1 left out, values
    scaled, the arithmetic in another type."""
    kc, ks, vc, vs = cache.tensors
    pages, hkv, hd = table[0].long(), cache.heads, cache.head_dim
    k, v = (unpack(c[pages], s[pages])[1].permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n].to(dtype) for c, s in ((kc, ks), (vc, vs)))
    q = Q.shape[0]
    x = Q.to(dtype).reshape(q, hkv, -1, hd)
    s = torch.einsum("qhgd,hnd->qhgn", x, k) * scale
    t, pos = torch.arange(n), torch.arange(n - q, n)[:, None]
    hidden = (t > pos) | ((t <= pos - window) if window else torch.zeros((), dtype=torch.bool))
    if skip:
        hidden = hidden | ((t >= skip[0]) & (t < skip[1]))
    p = torch.softmax(s.masked_fill(hidden[:, None, None], -math.inf), -1)
    o = torch.einsum("qhgn,hnd->qhgd", p, v) * value_scale
    if cache.rotate_v:
        o = o @ hadamard(hd, "cpu").to(dtype)
    return o.reshape(q, -1, hd)


CASES = [(1, 4097, 2, 1, 128, True, 0, False), (1, 4097, 2, 1, 128, False, 0, False), (1, 20000, 1, 1, 64, True, 0, False),
         (1, 517, 4, 2, 128, True, 0, False), (1, 5000, 2, 1, 128, True, 1024, False), (4, 900, 4, 2, 64, False, 0, False),
         (513, 1537, 1, 1, 128, True, 0, True), (129, 1000, 2, 2, 64, False, 0, True), (200, 999, 2, 1, 128, True, 300, True)]


@pytest.mark.parametrize("q,n,hq,hkv,hd,rv,window,many", CASES)
def test_exact_outputs_pass_and_mistakes_do_not(q, n, hq, hkv, hd, rv, window, many):
    cache, Q, starts, lens, table = case(q, n, hq, hkv, hd, rv)
    scale = hd ** -0.5
    want, tol = attention(cache, Q, starts, lens, table, scale, window, many)

    def passes(o):
        return bool(((o - want).abs() <= tol).all())

    o = direct(cache, Q, table, n, scale, window)
    assert ((o - want).abs() <= 1e-12 * want.abs().amax()).all()              # two routes, one value
    assert passes(o.to(torch.bfloat16).double())
    assert passes(direct(cache, Q, table, n, scale, window, dtype=torch.float32).to(torch.bfloat16).double())
    assert not passes(torch.zeros_like(o))
    middle = (n - (window or n) // 2 - q // 2) // 32 * 32
    for name, wrong in (("a block of 32 tokens left out", direct(cache, Q, table, n, scale, window, skip=(middle, middle + 32))),
                        ("the last token left out", direct(cache, Q, table, n, scale, window, skip=(n - 1, n)) if n < 1000 else None),
                        ("scores 3% too large", direct(cache, Q, table, n, 1.03 * scale, window)),
                        ("outputs 3% too small", direct(cache, Q, table, n, scale, window, value_scale=0.97)),
                        ("a window one token too long", direct(cache, Q, table, n, scale, window + 1) if 0 < window < 500 else None),
                        ("not rotated back", o @ hadamard(hd, "cpu") if rv else None),
                        ("the heads' order turned round", o.flip(1) if hq > 1 else None)):
        assert wrong is None or not passes(wrong), name
    # not in a corner only: each of these reaches most rows
    off = ((direct(cache, Q, table, n, scale, window, skip=(middle, middle + 32)) - want).abs() > tol).any(-1)
    assert off.double().mean() > 0.4


def test_few_percent_of_the_output():
    """The bound stays below a few percent of a row's size over thousands of tokens."""
    for q, n, hq, hkv, hd, rv, window, many in CASES:
        cache, Q, starts, lens, table = case(q, n, hq, hkv, hd, rv)
        want, tol = attention(cache, Q, starts, lens, table, hd ** -0.5, window, many)
        share = tol.square().mean(-1).sqrt() / want.square().mean(-1).sqrt()
        assert share.max() < 0.04, (n, q, float(share.max()))

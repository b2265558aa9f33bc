"""Calls of the 4-bit floating-point product and of masked attention at their edges: first calls that are captured, offsets that
pass 32 bits, rows that begin anywhere, NaN and infinities, bounds that do not fit, two calls at once."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import plain_fp4 as P
from tests.masked64 import pack
from tests.test_gpu_kv4 import make_case
from tests.test_gpu_kv4_masked import check, trees_of

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def quant(pq, x, fmt, g=0, factor=1.0):
    T, D = x.shape
    codes = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pq.pq_fp4_scale_bytes(T, D, fmt), dtype=torch.uint8, device="cuda")
    pq.pq_quant_fp4(x, codes, scales, fmt=fmt, g=g, factor=factor)
    return codes, scales


CODE = """
import sys
import torch
from rotation_int4_w4a4_b200 import pq

which, dev = sys.argv[1], "cuda"


def attention(q, n, tree, hq=8, hkv=2, hd=128, page=16):
    pages = -(-n // page) + 1
    tensors = []
    for _ in "kv":
        tensors += [torch.randint(0, 256, (pages, hkv, page, hd // 2), device=dev, dtype=torch.uint8),
                    torch.rand(pages, hkv, page, device=dev) * 0.1 + 0.2]
    cache, Q = pq.KV4Cache(*tensors), torch.randn(q, hq, hd, device=dev).to(torch.bfloat16)
    O, table = torch.zeros_like(Q), torch.randperm(pages, device=dev)[None].to(torch.int32)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, q], [n]))
    lists = torch.full((q, -(-q // 32)), -1, dtype=torch.int32, device=dev) if tree else None
    return O, lambda: pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, n, window=0 if tree else 700, sinks=5, tree=lists)


def linear(T, N, D=512):
    X, W = torch.randn(T, D, device=dev).to(torch.bfloat16), torch.randint(0, 256, (N, D // 2), dtype=torch.uint8, device=dev)
    ca, Y = torch.empty(T, D // 2, dtype=torch.uint8, device=dev), torch.zeros(T, N, device=dev)
    sa, sw = (torch.full((pq.pq_fp4_scale_bytes(r, D, "mx"),), 127, dtype=torch.uint8, device=dev) for r in (T, N))
    return Y, lambda: pq.pq_fp4_linear(X, ca, sa, W, sw, Y, fmt="mx", g=128)


out, call = {"tree 5": lambda: attention(5, 3000, True), "tree 300": lambda: attention(300, 9000, True), "sinks 1": lambda: attention(1, 3000, False),
             "sinks 200": lambda: attention(200, 900, False), "linear 1": lambda: linear(1, 100), "linear 60": lambda: linear(60, 100),
             "linear 600": lambda: linear(600, 9000)}[which]()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
replayed = out.clone()
out.zero_()
call()
assert replayed.abs().sum() > 0 and torch.equal(replayed, out)
pq.pq_check_status()
print("done")
"""


@pytest.mark.parametrize("which", ["tree 5", "tree 300", "sinks 1", "sinks 200", "linear 1", "linear 60", "linear 600"])
def test_the_first_call_is_captured(which):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE, which], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_past_32_bits(pq, fmt):
    """More than 2^31 channels: the last rows are what they are in a call of their own."""
    D, some, times = 16384, 1280, 110                      # 1280 rows: whole pieces of 128
    x = normal(1, some, D)
    X = x.repeat(times, 1)
    assert X.numel() > 2 ** 31
    codes, scales = quant(pq, X, fmt, g=128)
    c, s = quant(pq, x, fmt, g=128)
    assert torch.equal(codes[-some:], c) and torch.equal(scales[-s.numel():], s)
    middle = (2 ** 31 // D) // some * some
    assert torch.equal(codes[middle:middle + some], c)


@pytest.mark.parametrize("N", [33000, 33001])
def test_products_past_32_bits(pq, N):
    """More than 2^31 outputs (rows that begin on 16 bytes, and rows that do not), all products exact."""
    T, D, fmt = 128 * 520, 64, "mx"
    gen = torch.Generator(device="cuda").manual_seed(N)
    ca, cw = (torch.randint(0, 256, (r, D // 2), generator=gen, dtype=torch.uint8, device="cuda") for r in (T, N))
    sa, sw = (torch.full((pq.pq_fp4_scale_bytes(r, D, fmt),), 127, dtype=torch.uint8, device="cuda") for r in (T, N))
    Y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert Y.numel() > 2 ** 31
    pq.pq_fp4_gemm(ca, sa, cw, sw, Y, fmt=fmt)
    for first in (0, 128 * 507, T - 256):
        rows = slice(first, first + 256)
        want = P.code_values(ca[rows].cpu().numpy(), 256, D) @ P.code_values(cw.cpu().numpy(), N, D).T
        want = torch.from_numpy(want).to(torch.bfloat16)
        assert torch.equal(Y[rows].cpu(), want)
    pq.pq_check_status()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,N,D,g", [(1, 200, 256, 64), (9, 130, 512, 256), (40, 200, 256, 128), (700, 4900, 320, 0)])
@pytest.mark.parametrize("pad,shift", [(8, 8), (16, 16), (40, 24)])
def test_rows_that_begin_anywhere(pq, fmt, T, N, D, g, pad, shift):
    """Row strides and beginnings that are multiples of 16 bytes but not of 32, and ones that are."""
    wide = torch.full((T, D + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = normal(T, T, D)
    wide[:, shift:shift + D] = x
    cw, sw = quant(pq, normal(2, N, D), fmt, g)
    out = []
    for X in (x, wide[:, shift:shift + D]):
        ca, sa = torch.zeros(T, D // 2, dtype=torch.uint8, device="cuda"), torch.zeros(pq.pq_fp4_scale_bytes(T, D, fmt), dtype=torch.uint8, device="cuda")
        Y = torch.full((T, N), float("nan"), device="cuda")
        pq.pq_fp4_linear(X, ca, sa, cw, sw, Y, fmt=fmt, g=g)
        out.append((ca, sa, Y))
    assert out[0][2].isfinite().all() and all(torch.equal(a, b) for a, b in zip(*out))
    c, s = quant(pq, x, fmt, g)
    assert torch.equal(out[0][0], c)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,N,D", [(1, 100, 256), (9, 500, 1024), (20, 500, 4096), (300, 700, 512), (600, 9000, 256)])
def test_a_token_that_diverged(pq, fmt, T, N, D, bad):
    """Its outputs are NaN, the others' the same bits."""
    X, W = normal(1, T, D), normal(2, N, D)
    cw, sw = quant(pq, W, fmt, 128)

    def run():
        ca, sa = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(pq.pq_fp4_scale_bytes(T, D, fmt), dtype=torch.uint8, device="cuda")
        Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        pq.pq_fp4_linear(X, ca, sa, cw, sw, Y, fmt=fmt, g=128)
        return Y

    want = run()
    assert want.isfinite().all()
    X[T // 2, 3] = bad
    Y = run()
    others = torch.arange(T, device="cuda") != T // 2
    assert Y[T // 2].isnan().all() and torch.equal(Y[others], want[others])


@pytest.mark.parametrize("factor", [2.0 ** -100, 1e-20, 1e20, 2.0 ** 100])
def test_factors_at_their_ends(pq, factor):
    """Tiny factors cut everything off at 6 * 448, large ones round scales to 0; nothing becomes NaN or infinite."""
    x = normal(3, 5, 64)
    codes, scales = quant(pq, x, "nv", 64, factor)
    s = P.scale_values(scales.cpu().numpy(), 5, 64, "nv")
    q = P.code_values(codes.cpu().numpy(), 5, 64)
    assert np.isfinite(s).all() and (np.all(s == 448) if factor < 1 else np.all(s == 0) and np.all(q == 0))
    if factor < 1:
        assert np.all(np.abs(q[q != 0]) == 6)


def test_two_calls_at_once(pq):
    """Products and attention on two streams, and replayed from two graphs, share nothing."""
    T, N, D = 30, 300, 2048
    cw, sw = quant(pq, normal(2, N, D), "nv", 128)
    jobs = []
    for k in range(2):
        X = normal(10 + k, T, D)
        ca, sa = quant(pq, X, "nv", 128)
        Y = torch.empty(T, N, device="cuda")
        cache, Q, starts, lens, table = make_case(pq, 6 + k, [40, 3], [900, 4000], 8, 2, 128, 16, poison=False)
        lists = pack(trees_of([40, 3], k), 2).cuda()
        O = torch.empty_like(Q)

        def job(X=X, ca=ca, sa=sa, Y=Y, cache=cache, Q=Q, O=O, rest=(starts, lens, table), lists=lists):
            for _ in range(5):
                pq.pq_fp4_linear(X, ca, sa, cw, sw, Y, fmt="nv", g=128)
                pq.pq_kv4_attention_masked(cache, Q, O, *rest, 40, 4000, window=600, sinks=9, tree=lists)
        job()
        torch.cuda.synchronize()
        jobs.append((job, Y, O, Y.clone(), O.clone()))
    streams = [torch.cuda.Stream() for _ in jobs]
    graphs = []
    for job, Y, O, _, _ in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            job()
        graphs.append(g)
    for replay in (False, True):
        for job, Y, O, _, _ in jobs:
            Y.zero_(), O.zero_()
        torch.cuda.synchronize()
        for k, (s, (job, *_)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                graphs[k].replay() if replay else job()
        torch.cuda.synchronize()
        for _, Y, O, y, o in jobs:
            assert torch.equal(Y, y) and torch.equal(O, o)
    pq.pq_check_status()


@pytest.mark.parametrize("qs,ls,max_q,max_len", [([1, 1], [900, 3000], 1, 64), ([40], [700], 1, 16), ([1], [50], 1, 100000),
                                                 ([3, 200], [500, 600], 2, 10), ([200], [600], 4000, 9000), ([8], [1000], 8, 100), ([60], [5000], 9, 1)])
@pytest.mark.parametrize("window,sinks,tree", [(0, 0, True), (100, 4, True), (300, 50, False)])
def test_bounds_that_do_not_fit(pq, qs, ls, max_q, max_len, window, sinks, tree):
    """max_q and max_len only size the launch."""
    check(pq, make_case(pq, 8, qs, ls, 8, 2, 64, 32), max_q, max_len, window=window, sinks=sinks, trees=trees_of(qs, 2) if tree else None)


@pytest.mark.parametrize("q,n,window", [(1, 300, 100), (1, 6000, 3000), (6, 1500, 0), (16, 2000, 0), (64, 3000, 700), (100, 400, 0), (200, 9000, 0)])
@pytest.mark.parametrize("bad", BAD)
def test_nan_queries_and_scales(pq, q, n, window, bad):
    """A bad query spoils its own row; a bad value or key scale of a token the rows that see it: here of the first token of the
    new ones, which a tree's other branches do not list, and of an old one that all see."""
    cache, Q, starts, lens, table = make_case(pq, 5, [q], [n], 8, 2, 128, 16, poison=False)
    bits = torch.eye(q, dtype=torch.bool)
    bits[q // 2:, 0] = True                                # the later half descends from the first
    lists = pack([bits], -(-q // 32)).cuda()
    tree = dict(tree=lists) if q > 1 else {}

    def run():
        O = torch.empty_like(Q)
        pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, n, window=window, sinks=3, **tree)
        return O

    want = run()
    assert want.isfinite().all()
    keep = Q[q // 3, 5].clone()
    Q[q // 3, 5, 7] = bad
    got = run()
    Q[q // 3, 5] = keep
    rows = torch.ones(q, 8, dtype=torch.bool, device="cuda")
    rows[q // 3, 5] = False
    assert torch.equal(got[rows], want[rows]) and not got[q // 3, 5].isfinite().all()
    for which in (1, 3):
        for t, seen in ((n - q, bits[:, 0]), (1, torch.ones(q, dtype=torch.bool))):
            page, place = int(table[0, t // 16]), t % 16
            old = cache.tensors[which][page, 1, place].clone()
            cache.tensors[which][page, 1, place] = bad
            got = run()
            cache.tensors[which][page, 1, place] = old
            head = torch.arange(8, device="cuda") >= 4
            touched = seen.cuda()[:, None] & head[None, :]
            assert torch.equal(got[~touched], want[~touched])
            if which == 3:
                assert bool((~got[touched].isfinite()).any(-1).all())
    assert torch.equal(run(), want)
    pq.pq_check_status()


# Few sequences of up to 256 rows a head: blocks of 8 rows uncut and in clusters, tiles of 128 rows uncut, in clusters of 2 to 8 and in
# parts that a second kernel joins; sequences that leave most of a tile empty beside others.
@pytest.mark.parametrize("window,sinks,tree", [(0, 0, True), (700, 5, True), (300, 70, False)])
@pytest.mark.parametrize("B,q,n", [(1, 32, 300), (1, 9, 1029), (1, 25, 1500), (2, 32, 300), (2, 18, 1029), (3, 30, 2000), (4, 12, 1029), (4, 24, 2100),
                                   (8, 12, 300), (8, 12, 1029), (8, 24, 300), (8, 30, 1029), (9, 60, 900), (12, 17, 3000)])
def test_batches_across_the_borders(pq, B, q, n, window, sinks, tree):
    qs = [q] + [max(1, (q * (3 * b + 1)) % q) for b in range(1, B)]
    ls = [n] + [max(qs[b], n * (b + 2) // (B + 3)) for b in range(1, B)]
    check(pq, make_case(pq, B + q, qs, ls, 32, 8, 128, 32), max(qs), n, window=window, sinks=sinks, trees=trees_of(qs, 5) if tree else None)


def test_rows_behind_a_tile_cost_nothing_and_say_nothing(pq):
    """36 of 128 rows: what the other rows' place held (NaN and infinities of an earlier call) reaches nothing."""
    cache, Q, starts, lens, table = make_case(pq, 3, [9] * 9, [900] * 9, 32, 8, 128, 32)
    tree = torch.full((81, 1), 511, dtype=torch.int32, device="cuda")
    outs = []
    for bad in (None, float("nan"), float("inf")):
        if bad is not None:
            big = make_case(pq, 4, [60] * 9, [900] * 9, 32, 8, 128, 32)
            big[1].fill_(bad)
            pq.pq_kv4_attention_masked(big[0], big[1], torch.empty_like(big[1]), *big[2:], 60, 900, tree=torch.ones(540, 2, dtype=torch.int32, device="cuda"))
        O = torch.empty_like(Q)
        pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, 9, 900, tree=tree)
        outs.append(O)
    assert torch.isfinite(outs[0].float()).all() and all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("window,sinks,tree", [(0, 0, True), (2500, 9, True), (3000, 200, False)])
@pytest.mark.parametrize("qs,ls,hq,hkv", [
    ([61] * 5, [5000, 130, 61, 2600, 4100], 16, 4), ([40, 1, 70, 0, 64, 33], [6000, 5000, 70, 0, 4500, 6000], 8, 2),      # parts of uneven walks
    ([50] * 12, [4300 - 7 * b for b in range(12)], 8, 2), ([64] * 33, [100 + 130 * b for b in range(33)], 4, 1),            # whole walks; more than 32 sequences
    ([300, 20, 200], [4000, 4500, 900], 8, 2),
])
def test_walks_in_parts_and_whole(pq, qs, ls, hq, hkv, window, sinks, tree):
    """Sequences whose walks are cut beside ones that are not, sorted by length, with the rows of the others left alone."""
    check(pq, make_case(pq, len(qs) + window, qs, ls, hq, hkv, 128, 64), max(qs), max(ls), window=window, sinks=sinks,
          trees=trees_of(qs, 6) if tree else None)

"""8-bit rows and their product against float64, at the sizes where tiles, rows and dispatch rules end."""
import pytest
import torch

from tests.plain64 import HALF_STEP, U, check_codes, rows8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def normal(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda")


def codes8(seed, rows, D, lo=-127):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(lo, 128, (rows, D), generator=gen, device="cuda", dtype=torch.int8)


def scales(seed, rows):
    return normal(seed, rows).abs() * 0.01 + 1e-4


def product64(ca, sa, cw, sw):
    return (ca.double() @ cw.double().t()) * sa.double()[:, None] * sw.double()[None, :]


def check_product(Y, want):
    # int32 -> float32 and two products: three roundings; then the output's own
    tol = (3.01 * U + (HALF_STEP[Y.dtype] if Y.dtype != torch.float32 else 0)) * want.abs() * 1.001
    bad = (Y.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("T,D,g", [(1, 16, 0), (3, 64, 64), (1, 128, 128), (5, 256, 256), (7, 1008, 0), (2, 4096, 128),
                                   (33, 1088, 64), (4, 14336, 128), (3, 14336, 256), (2, 32768, 128), (2, 32784, 0),
                                   (1, 65536, 256), (130, 384, 128)])
def test_rows(pq, T, D, g):
    X = (normal(T * D + g, T, D) * (1 + 30 * (torch.arange(D, device="cuda") % 97 == 3))).to(torch.bfloat16)
    codes = torch.full((T, D), 99, dtype=torch.int8, device="cuda")
    sc = torch.full((T,), -1.0, device="cuda")
    pq.pq_quant_rows8(X, codes, sc, g=g)
    y, want, band, rel = rows8(X, g)
    assert ((sc.double() - want).abs() <= rel * want).all()
    check_codes(codes, y / want[:, None], band)


def test_rows_strided_zero_and_tiny(pq):
    """Rows of a wider matrix; a row of zeros, one of the smallest numbers; what lies beside stays."""
    wide = torch.zeros(6, 1024, dtype=torch.bfloat16, device="cuda")
    wide[:, :256] = normal(5, 6, 256).to(torch.bfloat16)
    wide[2, :256] = 0
    wide[4, :256] = 1e-39
    codes = torch.full((7, 256), 55, dtype=torch.int8, device="cuda")
    sc = torch.full((7,), 5.0, device="cuda")
    pq.pq_quant_rows8(wide[:, :256], codes[:6], sc[:6], g=128)
    for r in (2, 4):
        assert (codes[r] == 0).all() and sc[r] == 0
    assert (codes[6] == 55).all() and sc[6] == 5
    live = [0, 1, 3, 5]
    y, want, band, rel = rows8(wide[live, :256].contiguous(), 128)
    check_codes(codes[live], y / want[:, None], band[:, :])
    assert ((sc[live].double() - want).abs() <= rel * want).all()


SIZES = [(1, 1, 16), (1, 4096, 4096), (1, 1003, 4112), (2, 17, 32), (3, 128, 128), (4, 333, 1040), (5, 129, 256),
         (8, 4096, 4096), (15, 31, 144), (16, 16, 2048), (17, 257, 112), (33, 1000, 528), (64, 128, 14336), (65, 96, 1024),
         (100, 130, 4080), (127, 255, 272), (128, 1024, 4096), (129, 256, 128), (200, 65, 16), (255, 511, 1024),
         (257, 513, 784), (391, 1003, 4176), (513, 2049, 320), (1, 100000, 64), (1000, 16, 65536)]


@pytest.mark.parametrize("T,N,D", SIZES)
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product(pq, T, N, D, out):
    ca, cw, sa, sw = codes8(T, T, D, -128), codes8(N + 1, N, D, -128), scales(1, T), scales(2, N)
    full = torch.full((T * N + 64,), 7.5, dtype=out, device="cuda")
    Y = full[:T * N].view(T, N)
    pq.pq_w8a8_gemm(ca, sa, cw, sw, Y)
    check_product(Y, product64(ca, sa, cw, sw))
    assert (full[T * N:] == 7.5).all()                   # nothing behind the last row is written
    pq.pq_check_status()


@pytest.mark.parametrize("T", [1, 4, 5, 64, 128, 129, 300])
def test_largest_sums_are_exact(pq, T):
    """Every code -128, the longest reduction: 2^30, held in int32."""
    D, N = 65536, 40
    ca = torch.full((T, D), -128, dtype=torch.int8, device="cuda")
    cw = torch.full((N, D), -128, dtype=torch.int8, device="cuda")
    one_a, one_w = torch.ones(T, device="cuda"), torch.ones(N, device="cuda")
    Y = torch.empty(T, N, device="cuda")
    pq.pq_w8a8_gemm(ca, one_a, cw, one_w, Y)
    assert (Y == 2.0 ** 30).all()


@pytest.mark.parametrize("T,N,D,g", [(1, 256, 256, 128), (3, 1003, 4096, 64), (6, 64, 512, 256), (64, 14336, 4096, 128),
                                     (128, 257, 1024, 0), (129, 300, 768, 128), (700, 513, 1280, 256)])
def test_linear_is_rows_then_product(pq, T, N, D, g):
    X = normal(T + N, T, D).to(torch.bfloat16)
    W = (normal(D, N, D) * 0.02).to(torch.bfloat16)
    cw, sw = torch.empty(N, D, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    pq.pq_quant_rows8(W, cw, sw, g=g)
    ca, sa = torch.empty(T, D, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    Y = torch.empty(T, N, device="cuda")
    pq.pq_w8a8_linear(X, ca, sa, cw, sw, Y, g=g)
    ca2, sa2, Y2 = torch.empty_like(ca), torch.empty_like(sa), torch.empty_like(Y)
    pq.pq_quant_rows8(X, ca2, sa2, g=g)
    pq.pq_w8a8_gemm(ca2, sa2, cw, sw, Y2)
    assert torch.equal(ca, ca2) and torch.equal(sa, sa2) and torch.equal(Y, Y2)
    check_product(Y, product64(ca, sa, cw, sw))
    # and the quantised product is near the exact one: each side's codes are off by at most half a step
    x, w = X.double(), W.double()
    bound = (x.abs().sum(1)[:, None] + D * sa.double()[:, None] / 2) * sw.double()[None, :] / 2 * (g ** 0.5 if g else 1)
    bound = bound + w.abs().sum(1)[None, :] * sa.double()[:, None] / 2 * (g ** 0.5 if g else 1)
    assert ((Y.double() - x @ w.t()).abs() <= bound * 1.01).all()


@pytest.mark.parametrize("T", [1, 32, 300])
def test_repeated_calls_capture_and_streams(pq, T):
    """The same call gives the same bits: again, on a side stream, and from a captured graph replayed on new inputs."""
    N, D = 512, 1024
    W = (normal(1, N, D) * 0.02).to(torch.bfloat16)
    cw, sw = torch.empty(N, D, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    pq.pq_quant_rows8(W, cw, sw, g=128)
    X, X2 = normal(2, T, D).to(torch.bfloat16), normal(3, T, D).to(torch.bfloat16)
    ca, sa = torch.empty(T, D, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    want = []
    for x in (X, X2):
        pq.pq_w8a8_linear(x, ca, sa, cw, sw, Y, g=128)
        want.append(Y.clone())
    for _ in range(20):
        pq.pq_w8a8_linear(X, ca, sa, cw, sw, Y, g=128)
        assert torch.equal(Y, want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pq.pq_w8a8_linear(X2, ca, sa, cw, sw, Y, g=128, stream=side)
    side.synchronize()
    assert torch.equal(Y, want[1])
    inp = X.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq.pq_w8a8_linear(inp, ca, sa, cw, sw, Y, g=128)
    for x, w in ((X2, want[1]), (X, want[0]), (X2, want[1])):
        inp.copy_(x)
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w)


def test_two_streams_at_once(pq):
    N, D = 1024, 2048
    cw, sw = codes8(1, N, D), scales(1, N)
    jobs = []
    for i, T in enumerate((1, 40, 260, 128)):
        jobs.append((codes8(10 + i, T, D), scales(20 + i, T), torch.empty(T, N, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for ca, sa, Y, st in jobs:
            pq.pq_w8a8_gemm(ca, sa, cw, sw, Y, stream=st)
    torch.cuda.synchronize()
    for ca, sa, Y, _ in jobs:
        check_product(Y, product64(ca, sa, cw, sw))


def test_large_offsets(pq):
    """Outputs and operands beyond 2^31 elements."""
    T, N, D = 40000, 65536, 16
    ca, cw, sa, sw = codes8(1, T, D), codes8(2, N, D), scales(1, T), scales(2, N)
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    pq.pq_w8a8_gemm(ca, sa, cw, sw, Y)
    rows = torch.tensor([0, 1, 32767, 32768, 32769, 39998, 39999], device="cuda")
    want = product64(ca[rows], sa[rows], cw, sw)
    check_product(Y[rows], want)

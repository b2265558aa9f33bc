"""4-bit floating-point rows and their product against the formulas in float64."""
import numpy as np
import pytest

from tests import plain_fp4 as P

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24          # half a step of float32


def _rows(T, D, seed, outliers=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=gen)
    if outliers:
        x[:, ::37] *= 20.0
        x[T // 2] *= 1e-3
    return x.to(torch.bfloat16)


def _buffers(T, D, fmt, fill=0xFF):
    """Codes and scales, filled with what must not matter: a NaN in every scale place that the call does not write."""
    import torch
    from rotation_int4_w4a4_b200 import pq
    n = pq.pq_fp4_scale_bytes(T, D, fmt)
    assert n == P.scale_bytes(T, D, fmt)
    return (torch.full((T, D // 2), fill, dtype=torch.uint8, device="cuda"),
            torch.full((n,), 0x7F if fmt == "nv" else 0xFF, dtype=torch.uint8, device="cuda"))


def _quant(x, fmt, g=0, factor=1.0):
    from rotation_int4_w4a4_b200 import pq
    codes, scales = _buffers(x.shape[0], x.shape[1], fmt)
    pq.pq_quant_fp4(x if x.is_cuda else x.cuda(), codes, scales, fmt=fmt, g=g, factor=factor)
    return codes, scales


def _check_rows(x, codes, scales, fmt, g, factor):
    """Each scale is the nearest to the formula's argument and each code to its quotient by that scale, up to the float32
    roundings of what is rounded: the rotation adds g numbers in log2(g) levels at most (each of at most sqrt(g) max|x| after
    the factor), then a product with the factor and one with the reciprocal."""
    T, D = x.shape
    x64 = x.double().cpu().numpy()
    y = P.rotate(x64, g) / (factor if fmt == "nv" else 1.0)
    b = P.BLOCK[fmt]
    # absolute error of y: the matrix instruction may drop up to one float32 step of its largest partial sum a term (16
    # terms), the levels after it round: (16 + 4) steps of the sum of magnitudes over sqrt(g); then 3 relative roundings
    if g:
        mass = np.abs(x64).reshape(T, -1, g).sum(-1) / np.sqrt(g) / (factor if fmt == "nv" else 1.0)
        err = np.repeat(mass, g, axis=1) * 20 * 2 * EPS
    else:
        err = np.zeros_like(y)
    err = err + np.abs(y) * 4 * EPS
    s = P.scale_values(scales.cpu().numpy(), T, D, fmt)
    m = np.abs(y).reshape(T, -1, b).max(-1)
    me = err.reshape(T, -1, b).max(-1)
    if fmt == "mx":
        lo = np.where(m - me >= 2.0 ** -100, 2.0 ** (np.floor(np.log2(np.maximum(m - me, 2.0 ** -100))) - 2), 0)
        hi = np.where(m + me >= 2.0 ** -100, 2.0 ** (np.floor(np.log2(np.maximum(m + me, 2.0 ** -100))) - 2), 0)
        zero = m < 2.0 ** -100
        assert np.all((s == lo) | (s == hi) | (zero & (s == 2.0 ** -127)))
    else:
        grid = P.e4m3_values()
        assert np.all(np.abs(s - np.minimum(m / 6, 448)) <= P.distance(np.minimum(m / 6, 448), grid) + me / 6 + m * 2 * EPS)
    q = P.code_values(codes.cpu().numpy(), T, D)
    sr = np.repeat(s, b, axis=1)
    live = sr > (2.0 ** -120 if fmt == "mx" else 0)
    z = np.divide(y, sr, out=np.zeros_like(y), where=live)
    tol = np.divide(err, sr, out=np.zeros_like(y), where=live)
    assert np.all(q[~live] == 0)
    clipped = np.sign(z) * np.minimum(np.abs(z), 6.0)
    assert np.all(np.abs(q - clipped) <= P.distance(clipped, P.GRID) + tol)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,D,g", [(1, 32, 0), (1, 4096, 128), (3, 96, 0), (5, 64, 64), (16, 160, 0), (17, 192, 64), (33, 256, 256),
                                   (129, 384, 128), (200, 1056, 0), (300, 512, 256), (1000, 4096, 128)])
def test_rows(fmt, T, D, g):
    x = _rows(T, D, 100 * T + D)
    factor = 0.05 if fmt == "nv" else 1.0
    codes, scales = _quant(x, fmt, g, factor)
    _check_rows(x, codes, scales, fmt, g, float(np.float32(factor)))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_rows_without_rotation_are_the_formula_s(fmt):
    """Numbers whose quotients by the scale are exact in float32: every code and scale is the formula's, ties included."""
    import torch
    gen = torch.Generator().manual_seed(5)
    x = (torch.randint(-64, 65, (70, 256), generator=gen).float() / 16)
    x.view(70, -1, P.BLOCK[fmt])[:, :, 0] = 6.0               # nv: scale 1; mx: 2^(2 - 2)
    codes, scales = _quant(x.to(torch.bfloat16), fmt)
    s, q = P.quantised(x.double().numpy(), fmt)
    assert np.array_equal(P.scale_values(scales.cpu().numpy(), 70, 256, fmt), s)
    assert np.array_equal(P.code_values(codes.cpu().numpy(), 70, 256), q)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_padding_and_neighbours_stay(fmt):
    """Strided rows; bytes of rows past the last are not written, those of blocks past the last are 0."""
    import torch
    T, D = 37, 32 * 5
    wide = torch.full((T, D + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = _rows(T, D, 3)
    wide[:, :D] = x.cuda()
    codes, scales = _quant(wide[:, :D], fmt)
    want_c, want_s = _quant(x, fmt)
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    b = scales.cpu().numpy().reshape(-1, 32, 4, 4)             # [pieces][row % 32][row / 32][block % 4]
    row = np.arange(32)[:, None] + 32 * np.arange(4)[None, :]
    nan = 0x7F if fmt == "nv" else 0xFF
    assert np.all(b[:, row >= T] == nan)
    blocks = D // P.BLOCK[fmt]
    for p in range(b.shape[0]):
        for k in range(4):
            if 4 * p + k >= blocks:
                assert np.all(b[p, :, :, k][row < T] == 0)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("g", [0, 64])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_block_with_nan_or_infinity(fmt, g, bad):
    import torch
    T, D = 20, 256
    x = _rows(T, D, 8)
    clean_c, clean_s = _quant(x, fmt, g)
    x[3, 70] = bad
    codes, scales = _quant(x, fmt, g)
    s, clean = (P.scale_values(v.cpu().numpy(), T, D, fmt) for v in (scales, clean_s))
    b = P.BLOCK[fmt]
    hit = np.zeros((T, D // b), dtype=bool)
    hit[3, (70 // g * g // b if g else 70 // b):((70 // g + 1) * g // b if g else 70 // b + 1)] = True
    assert np.all(np.isnan(s[hit])) and np.array_equal(s[~hit], clean[~hit])
    q, qc = P.code_values(codes.cpu().numpy(), T, D), P.code_values(clean_c.cpu().numpy(), T, D)
    wide = np.repeat(hit, b, axis=1)
    assert np.all(q[wide] == 0) and np.array_equal(q[~wide], qc[~wide])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_zeros_tiny_and_large_blocks(fmt):
    import torch
    T, D = 4, 128
    x = torch.zeros(T, D)
    x[1] = 1e-38                                              # mx: below 2^-100; nv: the scale rounds to 0
    x[2] = 3e38
    x[3, :64] = 2.0 ** -99
    x = x.to(torch.bfloat16)
    codes, scales = _quant(x, fmt)
    s, q = P.scale_values(scales.cpu().numpy(), T, D, fmt), P.code_values(codes.cpu().numpy(), T, D)
    assert np.all(q[:2] == 0)
    if fmt == "mx":
        assert np.all(s[2] == 2.0 ** (127 - 2)) and np.all(q[2] == 6)        # 3e38 = 1.76 * 2^127, quotient 7.05
        assert np.all(s[3, :2] == 2.0 ** -101) and np.all(q[3, :64] == 4) and np.all(q[3, 64:] == 0)
    else:
        assert np.all(s[2] == 448) and np.all(q[2] == 6) and np.all(q[3] == 0)


def _gemm(ca, sa, cw, sw, T, N, fmt, alpha=1.0, bf16=False):
    import torch
    from rotation_int4_w4a4_b200 import pq
    Y = torch.full((T, N), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    pq.pq_fp4_gemm(ca, sa, cw, sw, Y, fmt=fmt, alpha=alpha)
    pq.pq_check_status()
    return Y


def _codes(rows, D, fmt, seed, lo, hi):
    """Random codes and scale bytes in lo..hi; NaN where no scale belongs, 0 in blocks past the last."""
    import torch
    gen = np.random.default_rng(seed)
    codes = torch.from_numpy(gen.integers(0, 256, (rows, D // 2), dtype=np.uint8)).cuda()
    placed = np.full(P.scale_bytes(rows, D, fmt), 0x7F if fmt == "nv" else 0xFF, dtype=np.uint8)
    pad = P.scale_index(rows, -(-D // (4 * P.BLOCK[fmt])) * 4 * P.BLOCK[fmt], fmt)
    placed[pad] = 0
    placed[P.scale_index(rows, D, fmt)] = gen.integers(lo, hi + 1, (rows, D // P.BLOCK[fmt]), dtype=np.uint8)
    return codes, torch.from_numpy(placed).cuda()


SIZES = [(1, 1, 32), (1, 128, 64), (2, 7, 96), (5, 300, 256), (16, 129, 288), (17, 128, 512), (33, 1003, 1056), (64, 256, 4096),
         (65, 96, 2048), (128, 512, 320), (129, 130, 736), (257, 1003, 4192), (300, 2500, 544), (1, 4096, 4096), (700, 5000, 1312),
         (513, 5003, 288), (2000, 2056, 800), (4100, 1300, 64)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,N,D", SIZES)
def test_exact_products(fmt, T, N, D):
    """Scales 1, 2 and 4 (mx) or 1 to 1.875 in eighths (nv): every product and partial sum is a multiple of 2^-8 and below
    D * 36 * 16, so float32 holds them all exactly for these D (2^8 * 2^10 * D <= 2^30 does not, but sums of random signs
    do: asserted below from their magnitudes)."""
    lo, hi = (127, 129) if fmt == "mx" else (56, 63)
    ca, sa = _codes(T, D, fmt, 1, lo, hi)
    cw, sw = _codes(N, D, fmt, 2, lo, hi)
    a, w = P.values(ca.cpu().numpy(), sa.cpu().numpy(), T, D, fmt), P.values(cw.cpu().numpy(), sw.cpu().numpy(), N, D, fmt)
    want = a @ w.T
    unit = 0.25 if fmt == "mx" else 2.0 ** -8
    got = _gemm(ca, sa, cw, sw, T, N, fmt).double().cpu().numpy()
    exact_everywhere = (np.abs(a) @ np.abs(w).T) / unit < 2 ** 24   # no partial sum in any order leaves the integers
    assert exact_everywhere.any()
    assert np.array_equal(got[exact_everywhere], want[exact_everywhere])
    assert np.all(np.isfinite(got))


def _bound(a, w, D):
    """Of a sum in float32: D / 64 instructions, each rounding the sum and dropping at most one step of the largest magnitude
    for each of its 64 products' alignment: (D / 64 + 64) steps of the sum of magnitudes; ranges add 8."""
    return (D / 64 + 64 + 8) * 2 * EPS * (np.abs(a) @ np.abs(w).T)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,N,D", SIZES)
def test_products(fmt, bf16, T, N, D):
    lo, hi = (120, 134) if fmt == "mx" else (1, 126)
    alpha = 0.37
    ca, sa = _codes(T, D, fmt, 3, lo, hi)
    cw, sw = _codes(N, D, fmt, 4, lo, hi)
    a, w = P.values(ca.cpu().numpy(), sa.cpu().numpy(), T, D, fmt), P.values(cw.cpu().numpy(), sw.cpu().numpy(), N, D, fmt)
    want = float(np.float32(alpha)) * (a @ w.T)
    got = _gemm(ca, sa, cw, sw, T, N, fmt, alpha, bf16).double().cpu().numpy()
    tol = alpha * _bound(a, w, D) + np.abs(want) * EPS
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(got - want) <= tol)
    if not bf16 and want.size > 1000:
        assert np.linalg.norm(got - want) <= 2e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_nan_scale_stays_in_its_row(fmt):
    import torch
    T, N, D = 200, 300, 512
    ca, sa = _codes(T, D, fmt, 5, 60, 64)
    cw, sw = _codes(N, D, fmt, 6, 60, 64)
    clean = _gemm(ca, sa, cw, sw, T, N, fmt)
    nan = 0x7F if fmt == "nv" else 0xFF
    sa[int(P.scale_index(T, D, fmt)[150, 5])] = nan
    sw[int(P.scale_index(N, D, fmt)[7, 0])] = nan
    got = _gemm(ca, sa, cw, sw, T, N, fmt)
    hit = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    hit[150] = True
    hit[:, 7] = True
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T,N,D,g", [(1, 4096, 4096, 128), (40, 257, 768, 256), (129, 1003, 1056, 0), (600, 4200, 2048, 64),
                                     (2, 100, 32, 0), (3, 1, 64, 64), (16, 130, 288, 0), (5, 2000, 1280, 256), (7, 20000, 8192, 128),
                                     (16, 40000, 1024, 256), (1, 300, 65536, 64), (9, 5000, 480, 0), (17, 700, 640, 128)])
def test_linear_is_quantisation_and_product(fmt, T, N, D, g):
    import torch
    from rotation_int4_w4a4_b200 import pq
    fa, fw = (0.04, 0.003) if fmt == "nv" else (1.0, 1.0)
    x, w = _rows(T, D, 11), _rows(N, D, 12)
    cw, sw = _quant(w, fmt, g, fw)
    ca, sa = _quant(x, fmt, g, fa)
    alpha = float(np.float32(fa) * np.float32(fw)) if fmt == "nv" else 1.0
    want = _gemm(ca, sa, cw, sw, T, N, fmt, alpha, True)
    ca2, sa2 = _buffers(T, D, fmt)
    Y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    xd = x.cuda()
    for _ in range(3):
        pq.pq_fp4_linear(xd, ca2, sa2, cw, sw, Y, fmt=fmt, g=g, factor_A=fa, factor_W=fw)
        pq.pq_check_status()
        assert torch.equal(ca2, ca) and torch.equal(sa2, sa) and torch.equal(Y, want)
    # A rotation of both sides leaves the product, but for the codes' rounding: half a step of E2M1 is at most a fifth of a
    # number above 0.5 (0.5 of 2.5), a block's small ones hardly count, and two sides' independent errors stay below 0.25.
    # That holds where no block is cut off: scales end at 448, so numbers above 6 * 448 * 0.003 = 8.06 come out smaller
    # (unrotated rows here reach 20 * 3).
    if fmt == "nv" and any(int((v & 0x7F == 0x7E).sum()) for v in (sa, sw)):
        return
    ref = x.double() @ w.double().T
    err = float(torch.linalg.norm(Y.double().cpu() - ref) / torch.linalg.norm(ref))
    assert err < 0.25


def test_captured_linear_replays_with_new_rows_and_streams():
    import torch
    from rotation_int4_w4a4_b200 import pq
    T, N, D, fmt = 24, 520, 1024, "nv"
    cw, sw = _quant(_rows(N, D, 12), fmt, 128)
    x = _rows(T, D, 1).cuda()
    ca, sa = _buffers(T, D, fmt)
    Y = torch.empty(T, N, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pq.pq_fp4_linear(x, ca, sa, cw, sw, Y, fmt=fmt, g=128)
    torch.cuda.current_stream().wait_stream(side)
    first = Y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq.pq_fp4_linear(x, ca, sa, cw, sw, Y, fmt=fmt, g=128)
    Y.zero_()
    graph.replay()
    assert torch.equal(Y, first)
    x.copy_(_rows(T, D, 2))
    graph.replay()
    replayed = Y.clone()
    pq.pq_fp4_linear(x, ca, sa, cw, sw, Y, fmt=fmt, g=128)
    assert torch.equal(Y, replayed) and not torch.equal(Y, first)
    pq.pq_check_status()

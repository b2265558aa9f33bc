"""The 4-bit key/value cache: what is appended, read back and attended to, against float64."""
import pytest
import torch

from tests.plain64 import U, attention64, check_codes, heads64, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def rope_table(rows, dim):
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


# ---------------------------------------------------------------------------------------- append
@pytest.mark.parametrize("T,hq,hkv,hd,page,q_norm,k_norm,rope_dim,inter,rk,rv", [
    (1, 1, 1, 64, 16, False, False, 0, False, False, False),
    (1, 32, 8, 128, 64, True, True, 128, False, True, True),
    (3, 8, 8, 128, 16, False, True, 64, True, True, False),
    (5, 14, 2, 64, 32, True, False, 32, False, False, True),
    (37, 7, 1, 64, 256, True, True, 64, True, True, True),
    (64, 6, 3, 128, 128, False, False, 128, True, False, False),
    (130, 5, 5, 64, 64, True, True, 8, False, True, True),
    (257, 40, 8, 128, 64, True, True, 120, False, True, True),
])
def test_append(pq, T, hq, hkv, hd, page, q_norm, k_norm, rope_dim, inter, rk, rv):
    gen = generator(T + hq)
    rows = torch.randn(T, (hq + 2 * hkv) * hd + 8, generator=gen, device="cuda").to(torch.bfloat16)
    Q, K, V = rows[:, :hq * hd], rows[:, hq * hd:(hq + hkv) * hd], rows[:, (hq + hkv) * hd:(hq + 2 * hkv) * hd]
    norms = [(1 + 0.2 * torch.randn(hd, generator=gen, device="cuda")).to(torch.bfloat16) if n else None for n in (q_norm, k_norm)]
    rope = rope_table(500, rope_dim) if rope_dim else None
    positions = torch.randint(0, 500, (T,), generator=gen, device="cuda", dtype=torch.int32)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T]
    slots[T // 2::7] = -1
    cache = pq.KV4Cache.empty(pages, hkv, page, hd, rotate_k=rk, rotate_v=rv)
    for x in cache.tensors:
        x.fill_(3)
    Q_out = torch.empty(T, hq, hd, dtype=torch.bfloat16, device="cuda")
    eps = 1e-5
    pq.pq_kv4_append(cache, Q, K, V, Q_out, positions, slots, rope=rope, q_norm=norms[0], k_norm=norms[1], eps=eps,
                     interleaved=inter)
    y, err = heads64(Q, hq, hd, norms[0], eps, rope, positions, inter, rk)
    assert ((Q_out.double() - y).abs() <= 2.0 ** -8 * (y.abs() + err) + err).all()
    used = slots >= 0
    page_of, place = slots[used] // page, slots[used] % page
    for name, x, norm, r, rot in (("k", K, norms[1], rope, rk), ("v", V, None, None, rv)):
        y, err = heads64(x, hkv, hd, norm, eps, r, positions, inter, rot)
        codes, scales = cache.tensors[0 if name == "k" else 1 + 1], cache.tensors[1 if name == "k" else 3]
        got, _ = unpack(codes[page_of, :, place], scales[page_of, :, place])
        m = y.abs().amax(-1, keepdim=True)
        worst = err.amax(-1, keepdim=True) / m
        # the code's own error and the maximum's, then the reciprocal and two products
        check_codes(got, (y / (m / 7))[used], (2 * 7 * worst + 7 * 4 * U)[used])
        sc = scales[page_of, :, place].double()[..., None]
        assert ((sc - m[used] / 7).abs() <= (worst[used] + 4 * U) * m[used] / 7).all()
        untouched = torch.ones(pages, page, dtype=torch.bool, device="cuda")
        untouched[page_of, place] = False
        assert (codes.permute(0, 2, 1, 3)[untouched] == 3).all() and (scales.permute(0, 2, 1)[untouched] == 3).all()
    # read back
    outs = [torch.full((T, hkv, hd), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pq.pq_kv4_read(cache, slots, *outs)
    for out, (c, s) in zip(outs, (cache.tensors[:2], cache.tensors[2:])):
        _, val = unpack(c[page_of, :, place], s[page_of, :, place])
        assert torch.equal(out[used], val.float().to(torch.bfloat16))
        assert (out[~used] == 0).all()
    pq.pq_check_status()


def neighbours_sum(v):
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v


def butterflies(y):
    n, shape, h = y.shape[-1], y.shape, 1
    while h < n:
        v = y.reshape(*shape[:-1], n // (2 * h), 2, h)
        y = torch.stack([v[..., 0, :] + v[..., 1, :], v[..., 0, :] - v[..., 1, :]], dim=-2).reshape(shape)
        h *= 2
    return y


@pytest.mark.parametrize("hd,rope_dim,inter", [(128, 128, False), (128, 64, False), (128, 24, False), (128, 128, True), (64, 64, False),
                                               (64, 32, False), (64, 48, False), (64, 32, True), (128, 0, False)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_bits(pq, hd, rope_dim, inter, norm):
    """Codes and scales are those of the documented float32 formula, each product and sum rounded on its own, bit for bit:
    a code next to a rounding border does not depend on how the kernel groups its arithmetic."""
    T, hkv, hq, page = 700, 3, 6, 32
    gen = generator(hd + rope_dim)
    rows = torch.randn(T, (hq + 2 * hkv) * hd, generator=gen, device="cuda").to(torch.bfloat16)
    Q, K, V = rows.split([hq * hd, hkv * hd, hkv * hd], dim=1)
    w = (1 + 0.2 * torch.randn(hd, generator=gen, device="cuda")).to(torch.bfloat16) if norm else None
    rope = rope_table(900, rope_dim) if rope_dim else None
    positions = torch.randint(0, 900, (T,), generator=gen, device="cuda", dtype=torch.int32)
    cache = pq.KV4Cache.empty(-(-T // page), hkv, page, hd)
    slots = torch.arange(T, device="cuda")
    Q_out = torch.empty(T, hq, hd, dtype=torch.bfloat16, device="cuda")
    pq.pq_kv4_append(cache, Q, K, V, Q_out, positions, slots, rope=rope, q_norm=w, k_norm=w, eps=1e-5, interleaved=inter)

    def formula(x, heads, turned):
        x = x.float().reshape(T, heads, hd)
        if turned and norm:
            r = 1 / torch.sqrt(neighbours_sum(x * x) * (1 / hd) + 1e-5)
            x = (x * r) * w.float()
        if turned and rope_dim:
            cs = rope[positions.long()][:, None, :]
            cos, sin = cs[..., :rope_dim // 2], cs[..., rope_dim // 2:]
            a, b = (x[..., 0:rope_dim:2], x[..., 1:rope_dim:2]) if inter else (x[..., :rope_dim // 2], x[..., rope_dim // 2:rope_dim])
            u, v = a * cos - b * sin, b * cos + a * sin
            head = torch.stack([u, v], dim=-1).flatten(-2) if inter else torch.cat([u, v], dim=-1)
            x = torch.cat([head, x[..., rope_dim:]], dim=-1)
        return butterflies(x)

    assert torch.equal(Q_out, (formula(Q, hq, True) * (1 / hd ** 0.5)).to(torch.bfloat16))
    for i, (x, turned) in ((0, (K, True)), (2, (V, False))):
        y = formula(x, hkv, turned)
        m = y.abs().amax(-1, keepdim=True)
        want = torch.round(y * (m.reciprocal() * 7))
        got, _ = unpack(cache.tensors[i][slots // page, :, slots % page], cache.tensors[i + 1][slots // page, :, slots % page])
        assert torch.equal(got.float(), want)
        assert torch.equal(cache.tensors[i + 1][slots // page, :, slots % page], (m * (1 / (7 * hd ** 0.5)))[..., 0])


def test_append_zero_heads_and_bad_indices(pq):
    hd, hkv, page = 128, 2, 16
    cache = pq.KV4Cache.empty(2, hkv, page, hd)
    K = torch.randn(4, hkv * hd, generator=generator(1), device="cuda").to(torch.bfloat16)
    K[0] = 0
    Q_out = torch.full((4, hkv, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    rope = rope_table(10, hd)
    positions = torch.tensor([0, 10, 3, -1], dtype=torch.int32, device="cuda")      # two outside the table
    slots = torch.tensor([0, 1, 2 * page, 3], device="cuda")                         # one outside the cache
    pq.pq_kv4_append(cache, K, K, K, Q_out, positions, slots, rope=rope)
    with pytest.raises(pq.PQError) as e:
        pq.pq_check_status()
    assert e.value.status == pq.PQ_ERR_INVALID_ARG
    pq.pq_check_status()                                                             # cleared
    for x in cache.tensors:
        assert (x == 0).all()                                                        # zeros, skips, nothing else
    assert (Q_out[[0, 1, 3]] == 0).all() and (Q_out[2] != 0).any()
    out = [torch.full((4, hkv, hd), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    pq.pq_kv4_read(cache, slots, *out)
    assert (out[0][2] == 0).all()
    with pytest.raises(pq.PQError):
        pq.pq_check_status()


# ------------------------------------------------------------------------------------- attention
def make_cache(pq, gen, pages, hkv, page, hd, rk, rv):
    cache = pq.KV4Cache.empty(pages, hkv, page, hd, rotate_k=rk, rotate_v=rv)
    for i in (0, 2):
        cache.tensors[i].copy_(torch.randint(0, 256, cache.tensors[i].shape, generator=gen, device="cuda", dtype=torch.uint8))
        cache.tensors[i + 1].copy_(torch.randn(cache.tensors[i + 1].shape, generator=gen, device="cuda").abs() * 0.2 + 0.02)
    return cache


def make_case(pq, seed, qs, ls, hq, hkv, hd, page, rv=True, poison=True, extra_pages=0):
    """Sequences of ls cached tokens, qs of them new, on shuffled pages; what lies behind a sequence's end in its last
    page, and in pages of no sequence, is poisoned with NaN and infinite scales."""
    gen = generator(seed)
    used = [-(-n // page) for n in ls]
    width = max(1, max(used)) + 1
    pages = sum(used) + 2 + extra_pages
    cache = make_cache(pq, gen, pages, hkv, page, hd, True, rv)
    order = torch.randperm(pages, generator=gen, device="cuda")
    table = torch.full((len(ls), width), -7, dtype=torch.int32, device="cuda")     # never followed
    if poison:
        keep = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, (u, n) in enumerate(zip(used, ls)):
        table[b, :u] = order[at:at + u].to(torch.int32)
        if poison and u:
            mine = torch.arange(u * page, device="cuda") < n
            keep[order[at:at + u]] = mine.view(u, page)
        at += u
    if poison:
        for i, bad in ((1, float("nan")), (3, float("inf"))):
            cache.tensors[i].copy_(torch.where(keep[:, None, :], cache.tensors[i], torch.full_like(cache.tensors[i], bad)))
    T = sum(qs)
    Q = torch.randn(T, hq, hd, generator=gen, device="cuda").to(torch.bfloat16)
    starts = torch.tensor([sum(qs[:b]) for b in range(len(qs) + 1)], dtype=torch.int32, device="cuda")
    return cache, Q, starts, torch.tensor(ls, dtype=torch.int32, device="cuda"), table


def run_and_check(pq, case, max_q, max_len, window=0, scale=None, pad=0):
    cache, Q, starts, lens, table = case
    T, hq, hd = Q.shape
    full = torch.full((T + pad, hq, hd), 11.0, dtype=torch.bfloat16, device="cuda")
    Qp = torch.cat([Q, Q.new_full((pad, hq, hd), float("nan"))]) if pad else Q
    pq.pq_kv4_attention(cache, Qp, full, starts, lens, table, max_q, max_len, scale=scale, window=window)
    want, tol = attention64(cache, Q, starts, lens, table, hd ** -0.5 if scale is None else scale, window,
                            torch.full((T, hq, hd), 11.0, dtype=torch.float64, device="cuda"))
    off = (full[:T].double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / tol).nan_to_num(1e9).max()):.3g} "
                           f"of its bound, first at {bad.nonzero()[0].tolist()}")
    assert (full[T:] == 11).all()
    pq.pq_check_status()
    return full[:T]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page", [
    ([1], [1], 1, 1, 16),
    ([1], [2], 8, 2, 16),
    ([1], [517], 32, 8, 64),
    ([1], [4097], 8, 8, 32),
    ([1, 1, 0, 1], [64, 65, 0, 63], 4, 4, 64),
    ([1, 0, 1, 1], [300, 0, 1, 1025], 14, 2, 16),
    ([1], [20000], 5, 1, 256),
    ([2, 3], [2, 700], 7, 1, 128),
    ([5], [5], 4, 2, 16),
    ([17, 1, 40], [17, 900, 64], 8, 2, 32),
])
def test_few_rows(pq, hd, qs, ls, hq, hkv, page):
    run_and_check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page), max(qs), max(ls))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page,rv", [
    ([128], [128], 2, 1, 64, True),
    ([127], [130], 4, 2, 16, False),
    ([129, 64], [129, 1000], 8, 8, 128, True),
    ([300, 0, 1, 77], [811, 0, 400, 77], 14, 2, 16, True),
    ([1000], [1000], 5, 1, 64, False),
    ([65, 200], [3000, 200], 32, 8, 256, True),
    ([513], [1537], 8, 1, 32, True),
])
def test_prompts(pq, hd, qs, ls, hq, hkv, page, rv):
    run_and_check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page, rv=rv), max(qs), max(ls))


@pytest.mark.parametrize("window", [1, 2, 15, 64, 100, 511, 5000])
@pytest.mark.parametrize("qs,ls", [([1, 1], [1000, 130]), ([4], [777]), ([200, 30], [200, 999])])
def test_window(pq, window, qs, ls):
    run_and_check(pq, make_case(pq, window, qs, ls, 8, 2, 128, 16), max(qs), max(ls), window=window)


@pytest.mark.parametrize("qs,ls", [([5, 1], [3, 0]), ([200], [60]), ([1], [0]), ([300, 4], [0, 4])])
def test_rows_that_see_nothing(pq, qs, ls):
    """More new rows than cached tokens: the first rows sit before the sequence and see nothing."""
    out = run_and_check(pq, make_case(pq, 3, qs, ls, 4, 2, 128, 16), max(qs), max(1, max(ls)))
    at = 0
    for q, n in zip(qs, ls):
        assert (out[at:at + max(0, q - n)] == 0).all()
        at += q


@pytest.mark.parametrize("qs,ls,max_q,max_len", [([1, 1], [900, 3000], 1, 64), ([40], [700], 1, 16), ([1], [50], 1, 100000),
                                                 ([3, 200], [500, 600], 2, 10), ([200], [600], 4000, 9000)])
def test_bounds_that_do_not_fit(pq, qs, ls, max_q, max_len):
    """max_q and max_len only size the launch."""
    run_and_check(pq, make_case(pq, 8, qs, ls, 8, 2, 64, 32), max_q, max_len)


def spread(seed, B, q, ctx, empty):
    """(new, cached) tokens of B sequences: short ones outnumber long ones, every `empty`-th has nothing cached and every
    seventh asks for nothing."""
    gen = torch.Generator().manual_seed(seed)
    ls = [0 if b % empty == 2 else int(ctx ** float(torch.rand((), generator=gen))) for b in range(B)]
    return [0 if b % 7 == 3 else 1 + b % q for b in range(B)], ls


@pytest.mark.parametrize("hd,hq,hkv,page,window,qs,ls", [
    (64, 8, 2, 16, 0, *spread(1, 300, 3, 2500, 5)),
    (128, 8, 2, 64, 700, *spread(2, 40, 4, 9000, 6)),
    (128, 16, 1, 32, 0, *spread(3, 20, 3, 6000, 9)),
    (64, 2, 2, 16, 0, [1] * 500, [700 if b == 123 else 0 for b in range(500)]),
    (128, 4, 4, 16, 0, [1, 1], [30000, 1]),
    (64, 4, 2, 16, 0, *spread(4, 1024, 1, 900, 50)),
    (64, 4, 2, 16, 0, *spread(5, 1025, 1, 900, 50)),
    (64, 1, 1, 16, 0, [0, 0, 1, 0], [5000, 0, 4999, 70]),
])
def test_many_sequences_in_equal_shares(pq, hd, hq, hkv, page, window, qs, ls):
    """The tokens of all sequences are cut into equal shares: sequences of one share, shares of one sequence, shares that end
    where a sequence begins; the same twice gives the same bits."""
    case = make_case(pq, len(ls), qs, ls, hq, hkv, hd, page)
    first = run_and_check(pq, case, max(qs), max(max(ls), 700), window=window)
    assert torch.equal(first, run_and_check(pq, case, max(qs), max(max(ls), 700), window=window))


@pytest.mark.parametrize("q,n", [(1, 400), (150, 400)])
def test_padding_rows_strides_and_scale(pq, q, n):
    cache, Q, starts, lens, table = make_case(pq, 4, [q, q], [n, n + 7], 8, 2, 128, 16)
    run_and_check(pq, (cache, Q, starts, lens, table), q, n + 7, scale=0.5, pad=9)
    wide = torch.randn(2 * q, 3, 8 * 128, device="cuda").to(torch.bfloat16)
    wide[:, 1] = Q.view(2 * q, -1)
    O1, O2 = torch.empty(2 * q, 8 * 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(2 * q, 2, 8 * 128, dtype=torch.bfloat16, device="cuda")
    pq.pq_kv4_attention(cache, Q, O1.view(2 * q, 8, 128), starts, lens, table, q, n + 7)
    pq.pq_kv4_attention(cache, wide[:, 1], O2[:, 0], starts, lens, table, q, n + 7)
    assert torch.equal(O1, O2[:, 0]) and (O2[:, 1] == 0).all()


@pytest.mark.parametrize("q,n", [(1, 300), (2, 70), (200, 300)])
def test_hidden_poison_inside_the_sequence(pq, q, n):
    """A cached token that a row must not see may hold anything: NaN, infinite and huge scales of the newest token reach
    only the last row."""
    cache, Q, starts, lens, table = make_case(pq, 5, [q], [n], 4, 2, 128, 16, poison=False)
    O = torch.empty_like(Q)
    pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n)
    page, place = int(table[0, (n - 1) // 16]), (n - 1) % 16
    for k, v in ((float("nan"), 1.0), (1.0, float("inf")), (float("inf"), float("nan")), (1.0, 1e30)):
        cache.tensors[1][page, :, place], cache.tensors[3][page, :, place] = k, v
        O2 = torch.empty_like(Q)
        pq.pq_kv4_attention(cache, Q, O2, starts, lens, table, q, n)
        assert torch.equal(O[:q - 1], O2[:q - 1])


@pytest.mark.parametrize("q,n", [(2, 90), (5, 333), (8, 1500), (40, 700), (200, 900)])
def test_later_tokens_change_no_bit(pq, q, n):
    """What the newest tokens' rows meet (scores and values that outgrow whatever their tile's rows share) does not reach
    the rows before them, not even in the last bit."""
    cache, Q, starts, lens, table = make_case(pq, q + n, [q], [n], 4, 2, 128, 16, poison=False)
    O = torch.empty_like(Q)
    pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n)
    page, place = int(table[0, (n - 1) // 16]), (n - 1) % 16
    for k, v in ((3.0, 0.1), (40.0, 40.0), (0.01, 3e5), (500.0, 1e-3), (1e5, 1e5), (-7.0, -9e4)):
        cache.tensors[1][page, :, place], cache.tensors[3][page, :, place] = k, v
        O2 = torch.empty_like(Q)
        pq.pq_kv4_attention(cache, Q, O2, starts, lens, table, q, n)
        assert torch.equal(O[:q - 1], O2[:q - 1]), (k, v)


def scores_of(cache, Q, table, j):
    """Code products q . kc of cached token j with every query row, float64 [T, heads_q]."""
    page, place = int(table[0, j // cache.page_size]), j % cache.page_size
    code, _ = unpack(cache.tensors[0][page, :, place], torch.ones(cache.heads, device="cuda"))
    return torch.einsum("tgrd,gd->tgr", Q.double().view(len(Q), cache.heads, -1, cache.head_dim), code.double()).flatten(1)


@pytest.mark.parametrize("q,n,j", [(1, 300, 290), (3, 900, 700), (7, 40, 20), (140, 700, 350), (140, 300, 199)])
def test_a_value_of_zero_with_the_highest_score(pq, q, n, j):
    """Scores may lie further apart than float32's exponents: a token whose value is zero (scale 0) and whose score is
    thousands above all others leaves exactly 0 in the rows that see it, and no infinite sum."""
    cache, Q, starts, lens, table = make_case(pq, n + j, [q], [n], 8, 2, 128, 16, rv=False, poison=False)
    cache.tensors[1][int(table[0, j // 16]), :, j % 16] = 1e4
    cache.tensors[3][int(table[0, j // 16]), :, j % 16] = 0.0
    O = torch.empty_like(Q)
    pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n)
    assert O.isfinite().all()
    sees = (torch.arange(q, device="cuda") >= j - (n - q))[:, None]
    on_top = (scores_of(cache, Q, table, j) > 30) & sees     # 30 * 1e4 / sqrt(128): the others stay below 3000
    assert on_top.any() and (O[on_top] == 0).all() and (O[~sees.expand_as(on_top)] != 0).any(-1).all()


@pytest.mark.parametrize("q,n,j", [(1, 300, 3), (1, 2000, 1), (4, 900, 2), (8, 700, 600)])
def test_a_large_value_that_hardly_counts(pq, q, n, j):
    """The largest value scale belongs to a token whose probability is 0: the others keep their precision.  Both runs round
    each product by 2^-11, so they differ by 2^-10 of the largest value at most, and by a step of bf16."""
    cache, Q, starts, lens, table = make_case(pq, n + j, [q], [n], 8, 2, 128, 16, rv=False, poison=False)
    page, place = int(table[0, j // 16]), j % 16
    cache.tensors[1][page, :, place] = 1e4
    outs = []
    for scale in (1e6, 0.02):
        cache.tensors[3][page, :, place] = scale
        outs.append(torch.empty_like(Q))
        pq.pq_kv4_attention(cache, Q, outs[-1], starts, lens, table, q, n)
    off = scores_of(cache, Q, table, j) < -30
    a, b = (x[off].double() for x in outs)
    assert off.any() and b.abs().max() < 10
    assert ((a - b).abs() <= 2.0 ** -10 * 8 * cache.tensors[3].abs().max() * (1 + 2.0 ** -8) + 2.0 ** -8 * (a.abs() + b.abs())).all()


@pytest.mark.parametrize("q", [1, 140])
def test_bad_pages_and_lengths(pq, q):
    """A page outside the cache is skipped, a length beyond the table is cut, and both are reported."""
    cache, Q, starts, lens, table = make_case(pq, 6, [q], [400], 4, 2, 64, 16, poison=False)
    O, O2 = torch.empty_like(Q), torch.empty_like(Q)
    short = table[:, :10].contiguous()                     # 160 tokens
    pq.pq_kv4_attention(cache, Q, O, starts, torch.full_like(lens, 160), short, q, 400)
    pq.pq_check_status()
    pq.pq_kv4_attention(cache, Q, O2, starts, torch.full_like(lens, 2000), short, q, 400)
    with pytest.raises(pq.PQError):
        pq.pq_check_status()
    assert torch.equal(O, O2)
    # page 3 of the table skipped: as if its tokens could not be seen
    kc, ks, vc, vs = cache.tensors
    bad = short.clone()
    bad[0, 3] = cache.pages
    pq.pq_kv4_attention(cache, Q, O2, starts, torch.full_like(lens, 160), bad, q, 400)
    with pytest.raises(pq.PQError):
        pq.pq_check_status()
    pages = short[0].long()
    _, k = unpack(kc[pages], ks[pages])
    _, v = unpack(vc[pages], vs[pages])
    k, v = (x.permute(1, 0, 2, 3).reshape(2, 160, 64) for x in (k, v))
    last = Q[-1].double().view(2, 2, 64)
    s = torch.einsum("hgd,hnd->hgn", last, k) / 8
    s[..., 48:64] = float("-inf")
    p = torch.softmax(s, -1)
    from tests.plain64 import hadamard
    want = torch.einsum("hgn,hnd->hgd", p, v) @ hadamard(64, "cuda")
    assert ((O2[-1].double().view(2, 2, 64) - want).abs() <= 0.01 * want.abs().amax()).all()


@pytest.mark.parametrize("q,n,B", [(1, 5000, 1), (1, 700, 9), (4, 1200, 2), (260, 900, 2)])
def test_repeats_capture_and_streams(pq, q, n, B):
    """The same bits again and again, on other streams at the same time, and from two captured graphs replayed together."""
    cases = [make_case(pq, 40 + i, [q] * B, [n + i] * B, 8, 2, 128, 64) for i in range(2)]
    outs, want = [], []
    for cache, Q, starts, lens, table in cases:
        O = torch.empty_like(Q)
        pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n + 2)
        outs.append(O)
        want.append(O.clone())
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for (cache, Q, starts, lens, table), O, st in zip(cases, outs, streams):
            pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n + 2, stream=st)
    torch.cuda.synchronize()
    for O, w in zip(outs, want):
        assert torch.equal(O, w)
    graphs = []
    for (cache, Q, starts, lens, table), O in zip(cases, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            pq.pq_kv4_attention(cache, Q, O, starts, lens, table, q, n + 2)
        graphs.append(gr)
    for _ in range(3):
        for O in outs:
            O.zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for O, w in zip(outs, want):
            assert torch.equal(O, w)


@pytest.mark.parametrize("qs,ls", [([1, 1, 0, 1], [40, 3000, 0, 700]), ([2, 1], [5000, 1]), ([150, 60], [700, 900])])
def test_replayed_with_new_lengths(pq, qs, ls):
    """A captured call reads lengths and pages when it is replayed: the cut of the work follows them."""
    cache, Q, starts, lens, table = make_case(pq, 77, qs, ls, 8, 2, 128, 64)
    last, pages = lens.clone(), table.clone()
    O = torch.zeros_like(Q)
    lens.copy_(last.clamp_max(1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pq.pq_kv4_attention(cache, Q, O, starts, lens, table, max(qs), max(ls))
    for n, flip in ((last.clamp_max(1), False), (last, False), (last // 3, False), (last.flip(0).minimum(last), False), (last, True)):
        lens.copy_(n)
        if flip:                                             # the first two sequences trade places
            for x in (lens, table):
                x[:2] = x[:2].flip(0)
        O.fill_(7)
        graph.replay()
        want = torch.full_like(Q, 7)
        pq.pq_kv4_attention(cache, Q, want, starts, lens, table, max(qs), max(ls))
        assert torch.equal(O, want)
        exact, tol = attention64(cache, Q, starts, lens, table, 128 ** -0.5, 0, torch.full(Q.shape, 7.0, dtype=torch.float64, device="cuda"))
        assert ((O.double() - exact).abs() <= tol).all()
    pq.pq_check_status()


def test_large_cache_offsets(pq):
    """Pages whose bytes lie beyond 2^31 (codes) of the cache's start."""
    hkv, hd, page = 8, 128, 256
    pages = (1 << 31) // (hkv * page * hd // 2) + 40
    codes = torch.zeros(pages, hkv, page, hd // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, hkv, page, device="cuda")
    cache = pq.KV4Cache(codes, scales, torch.zeros_like(codes), torch.zeros_like(scales), rotate_k=False, rotate_v=False)
    small = make_case(pq, 12, [1, 150], [900, 400], 8, 8, hd, page, rv=False, poison=False)
    shift = pages - small[0].pages
    for i in range(4):
        cache.tensors[i][shift:] = small[0].tensors[i]
    small[0].rotate_k = False
    case = (cache, small[1], small[2], small[3], small[4] + shift)
    run_and_check(pq, case, 150, 900)


# ---------------------------------------------------------------------------------- all together
@pytest.mark.parametrize("rk,rv", [(True, True), (False, False), (True, False)])
def test_a_layer_step_by_step(pq, rk, rv):
    """A prompt in two chunks and then single tokens: projections in 4 bits, append, attention, output in 8 bits; the
    attention against float64 on the values that the cache holds, and the whole against unquantised attention."""
    D, hq, hkv, hd, page, L = 512, 4, 2, 128, 16, 90
    gen = generator(77)
    x = torch.randn(L, D, generator=gen, device="cuda").to(torch.bfloat16)
    W = (torch.randn((hq + 2 * hkv) * hd, D, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    Wo = (torch.randn(D, hq * hd, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    plan = pq.Plan("hadamard", D)
    cw = torch.empty(W.shape[0], D // 2, dtype=torch.uint8, device="cuda")
    sw = torch.empty(W.shape[0], D // 128, device="cuda")
    pq.pq_pack_weights(plan, W, cw, sw)
    co, so = torch.empty(D, hq * hd, dtype=torch.int8, device="cuda"), torch.empty(D, device="cuda")
    pq.pq_quant_rows8(Wo, co, so, g=128)
    cache = pq.KV4Cache.empty(L // page + 2, hkv, page, hd, rotate_k=rk, rotate_v=rv)
    table = torch.randperm(cache.pages, generator=gen, device="cuda")[None].to(torch.int32)
    rope = rope_table(L, hd)
    outs, qkvs, done = [], [], 0
    for n in (50, 33, 1, 1, 1, 4):
        T = n
        ca, sa = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(T, D // 128, device="cuda")
        qkv = torch.empty(T, W.shape[0], dtype=torch.bfloat16, device="cuda")
        pq.pq_w4a4_linear(plan, x[done:done + T], ca, sa, cw, sw, qkv)
        pos = torch.arange(done, done + T, device="cuda", dtype=torch.int32)
        slots = table[0, (pos // page).long()].long() * page + pos % page
        q, k, v = qkv[:, :hq * hd], qkv[:, hq * hd:(hq + hkv) * hd], qkv[:, (hq + hkv) * hd:]
        q_out, O = (torch.empty(T, hq, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pq.pq_kv4_append(cache, q, k, v, q_out, pos, slots, rope=rope)
        starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        lens = torch.tensor([done + T], dtype=torch.int32, device="cuda")
        pq.pq_kv4_attention(cache, q_out, O, starts, lens, table, T, done + T)
        want, tol = attention64(cache, q_out, starts, lens, table, hd ** -0.5, 0, torch.zeros(T, hq, hd, dtype=torch.float64, device="cuda"),
                                fp16_operands=T * hq // hkv > 64)
        assert ((O.double() - want).abs() <= tol).all()
        c8, s8 = torch.empty(T, hq * hd, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        Y = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        pq.pq_w8a8_linear(O.view(T, -1), c8, s8, co, so, Y, g=128)
        outs.append((O, Y))
        qkvs.append(qkv)
        done += T
    pq.pq_check_status()
    # unquantised attention on the same projections: the cache's 4-bit rounding alone stands between (each key and value
    # is off by at most scale / 2 per rotated channel, relative to its norm about 1/7 * max/rms / sqrt(12) < 0.15)
    qkv = torch.cat(qkvs)
    parts = [heads64(z, h, hd, None, 0, r, torch.arange(done, device="cuda"), False, False)[0]
             for z, h, r in ((qkv[:, :hq * hd], hq, rope), (qkv[:, hq * hd:(hq + hkv) * hd], hkv, rope), (qkv[:, (hq + hkv) * hd:], hkv, None))]
    q, k, v = parts
    k, v = (z.repeat_interleave(hq // hkv, dim=1) for z in (k, v))
    s = torch.einsum("qhd,khd->hqk", q, k) / hd ** 0.5
    s = s.masked_fill(torch.ones(done, done, device="cuda").triu(1).bool(), float("-inf"))
    full = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v)
    O = torch.cat([o for o, _ in outs]).double()
    assert float((O - full).norm() / full.norm()) < 0.3
    Y = torch.cat([y for _, y in outs]).double()
    direct = O.reshape(done, -1) @ Wo.double().t()
    assert float((Y - direct).norm() / direct.norm()) < 0.03

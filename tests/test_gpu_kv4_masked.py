"""Attention over the 4-bit cache with sinks and trees of drafted tokens, every output within the spread of its roundings."""
import pytest
import torch

from tests.masked64 import attention, pack, random_tree, seen
from tests.test_gpu_kv4 import make_case, rope_table, spread

pytestmark = pytest.mark.gpu

FEW_ROWS = 32         # query rows a key/value head and sequence up to which pq.h promises exact codes


@pytest.fixture(scope="module")
def pq():
    from rotation_int4_w4a4_b200 import pq as _pq
    return _pq


def trees_of(qs, seed, chain=0.5):
    gen = torch.Generator().manual_seed(seed)
    return [random_tree(m, gen, chain) for m in qs]


def check(pq, case, max_q, max_len, window=0, sinks=0, trees=None, scale=None, words=None, poison=True):
    """poison: pages that nobody sees are not to be followed: their entries in the table go astray."""
    cache, Q, starts, lens, table = case
    T, hq, hd = Q.shape
    page = cache.page_size
    table = table.clone()
    if poison:
        for b, n in enumerate(lens.tolist()):
            m = int(starts[b + 1] - starts[b])
            used = seen(m, n, window, sinks, trees[b] if trees else None).any(0) if m else torch.zeros(n, dtype=torch.bool)
            first = n - m - max(0, window - 1)             # the first row's window, whatever the list holds
            for i in range(-(-n // page)):
                in_window = not window or (i + 1) * page > first
                if not bool(used[i * page:(i + 1) * page].any()) and not in_window and i * page >= sinks:
                    table[b, i] = -5
    O = torch.full((T, hq, hd), 11.0, dtype=torch.bfloat16, device="cuda")
    lists = None
    if trees is not None:
        words = words or max(1, -(-max(max(q.shape[0] for q in trees), 1) // 32))
        lists = pack(trees, words).cuda()
    pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, max_q, max_len, scale=scale, window=window, sinks=sinks, tree=lists)
    want, tol = attention(cache, Q, starts, lens, table, hd ** -0.5 if scale is None else scale, window, sinks, trees,
                          max_q * (hq // cache.heads) > FEW_ROWS)
    off = (O.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / tol).nan_to_num(1e9).max()):.3g} "
                           f"of its bound, first at {bad.nonzero()[0].tolist()}")
    pq.pq_check_status()
    return O


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page", [
    ([1], [1], 1, 1, 16), ([2], [2], 4, 2, 16), ([8], [1029], 32, 8, 64), ([3, 8, 0, 1], [700, 8, 0, 3000], 8, 2, 32),
    ([5], [5], 7, 1, 128), ([4, 2], [900, 133], 14, 2, 16), ([31], [400], 1, 1, 64),
])
def test_tree_of_few(pq, hd, qs, ls, hq, hkv, page):
    check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page), max(qs), max(ls), trees=trees_of(qs, sum(ls)))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("qs,ls,hq,hkv,page", [
    ([16], [16], 8, 2, 16), ([61, 12, 0, 33], [1500, 12, 0, 100], 32, 8, 64), ([64, 64], [64, 3001], 4, 4, 32), ([65], [700], 14, 2, 16),
    ([128], [128], 4, 2, 64), ([200, 5], [777, 900], 5, 1, 128), ([33], [160], 2, 1, 256), ([300], [4000], 8, 2, 64),
])
def test_tree_of_many(pq, hd, qs, ls, hq, hkv, page):
    check(pq, make_case(pq, sum(ls) + hd, qs, ls, hq, hkv, hd, page), max(qs), max(ls), trees=trees_of(qs, sum(ls), 0.8))


@pytest.mark.parametrize("window,sinks", [(1, 1), (2, 5), (16, 4), (100, 1), (129, 130), (511, 64), (300, 600), (5000, 7)])
@pytest.mark.parametrize("qs,ls", [([1, 1], [1000, 130]), ([1], [5000]), ([4], [777]), ([200, 30], [200, 999]), ([100, 1], [3000, 40])])
def test_sinks(pq, window, sinks, qs, ls):
    check(pq, make_case(pq, window, qs, ls, 8, 2, 128, 16), max(qs), max(ls), window=window, sinks=sinks)


@pytest.mark.parametrize("hd,hq,hkv,page,rv", [(64, 14, 2, 64, False), (128, 4, 4, 256, True), (128, 32, 8, 32, False)])
@pytest.mark.parametrize("q,n,window,sinks", [(1, 9000, 1000, 4), (7, 2999, 700, 5), (33, 2000, 128, 128), (257, 1500, 200, 17), (40, 8000, 64, 300)])
def test_sinks_of_head_layouts(pq, hd, hq, hkv, page, rv, q, n, window, sinks):
    check(pq, make_case(pq, n, [q, 1], [n, 50], hq, hkv, hd, page, rv=rv), q, n, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (20, 4), (100, 150), (512, 4), (4000, 3)])
@pytest.mark.parametrize("qs,ls", [([8], [300]), ([6, 2], [2000, 6]), ([25, 40], [2999, 700]), ([64], [64]), ([100], [9000])])
def test_trees_under_a_window(pq, window, sinks, qs, ls):
    check(pq, make_case(pq, window, qs, ls, 8, 2, 128, 16), max(qs), max(ls), window=window, sinks=sinks, trees=trees_of(qs, 7))


@pytest.mark.parametrize("qs,ls", [([4], [4]), ([4], [100]), ([70], [70]), ([70], [500]), ([40, 3], [40, 3])])
def test_lists_of_any_kind(pq, qs, ls):
    """Rows that see nothing of the new tokens (nor, without older ones, anything: 0), all of them, or later ones."""
    gen = torch.Generator().manual_seed(9)
    trees = [torch.rand(m, m, generator=gen) < 0.4 for m in qs]
    for bits in trees:
        bits[0] = False
        bits[-1] = True
        bits[len(bits) // 2] = False
    O = check(pq, make_case(pq, 5, qs, ls, 8, 2, 128, 16), max(qs), max(ls), trees=trees)
    if qs == ls:
        assert (O[0] == 0).all() and (O[qs[0] // 2] == 0).all()


@pytest.mark.parametrize("qs,ls", [([5, 1], [3, 0]), ([200], [60]), ([300, 4], [0, 4])])
def test_more_rows_than_tokens(pq, qs, ls):
    case = make_case(pq, 3, qs, ls, 4, 2, 128, 16)
    check(pq, case, max(qs), max(1, max(ls)), trees=trees_of(qs, 1, 0.9))
    check(pq, case, max(qs), max(1, max(ls)), window=2, sinks=1)


@pytest.mark.parametrize("q", [6, 40])
def test_bits_past_the_sequence_and_short_lists(pq, q):
    """Bits of tokens that the sequence does not have say nothing; new tokens behind the last word are seen by nobody."""
    case = make_case(pq, 8, [q, q], [200, 333], 8, 2, 128, 16)
    cache, Q, starts, lens, table = case
    trees = trees_of([q, q], 4)
    want = check(pq, case, q, 333, trees=trees, window=50, sinks=2, poison=False)
    lists = pack(trees, 3)
    for j in range(q, 96):
        lists[:, j // 32] |= 1 << j % 32 if j % 32 < 31 else -(1 << 31)
    O = torch.empty_like(Q)
    pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, 333, window=50, sinks=2, tree=lists.cuda())
    assert torch.equal(O, want)
    if q > 32:
        cut = [t.clone() for t in trees]
        for t in cut:
            t[:, 32:] = False
        # the lists' first word: depths come from what it holds
        check(pq, case, q, 333, trees=cut, words=1)


@pytest.mark.parametrize("q,n", [(1, 700), (8, 500), (40, 900), (200, 300)])
def test_a_line_of_drafts_is_causal(pq, q, n):
    """A tree without branches, and sinks that reach into the window, give the causal call's result within two roundings."""
    cache, Q, starts, lens, table = make_case(pq, n, [q], [n], 8, 2, 128, 16)
    a, b, c = (torch.empty_like(Q) for _ in range(3))
    pq.pq_kv4_attention(cache, Q, a, starts, lens, table, q, n)
    line = torch.tril(torch.ones(q, q, dtype=torch.bool))
    pq.pq_kv4_attention_masked(cache, Q, b, starts, lens, table, q, n, tree=pack([line], -(-q // 32)).cuda())
    pq.pq_kv4_attention_masked(cache, Q, c, starts, lens, table, q, n, window=n, sinks=3)
    _, tol = attention(cache, Q, starts, lens, table, 128 ** -0.5, 0, 0, [line], q * 4 > FEW_ROWS)
    assert bool(((a.double() - b.double()).abs() <= 2 * tol).all()) and bool(((a.double() - c.double()).abs() <= 2 * tol).all())
    d = torch.empty_like(Q)
    pq.pq_kv4_attention_masked(cache, Q, d, starts, lens, table, q, n)              # no mask: the same call
    assert torch.equal(a, d)


@pytest.mark.parametrize("q,n", [(3, 300), (30, 500), (130, 400)])
def test_hidden_tokens_may_hold_anything(pq, q, n):
    """NaN and infinite scales of what a row does not see change no bit of it: a sibling branch, and the tokens between the
    sinks and the window."""
    cache, Q, starts, lens, table = make_case(pq, 5, [q], [n], 4, 2, 128, 16, poison=False)
    bits = random_tree(q, torch.Generator().manual_seed(2))
    bits[:, q // 2] = False
    bits[q // 2, q // 2] = True
    lists = pack([bits], -(-q // 32)).cuda()
    window, sinks = 100, 20
    args = dict(window=window, sinks=sinks, tree=lists)
    O = torch.empty_like(Q)
    pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, n, **args)
    places = [n - q + q // 2, sinks, sinks + 7, n - q - window]
    for k, v in ((float("nan"), 1.0), (1.0, float("inf")), (float("inf"), float("nan")), (1.0, 1e30)):
        for t in places:
            cache.tensors[1][int(table[0, t // 16]), :, t % 16] = k
            cache.tensors[3][int(table[0, t // 16]), :, t % 16] = v
        O2 = torch.empty_like(Q)
        pq.pq_kv4_attention_masked(cache, Q, O2, starts, lens, table, q, n, **args)
        others = [i for i in range(q) if i != q // 2]
        assert torch.equal(O[others], O2[others])


@pytest.mark.parametrize("q,n,B", [(1, 5000, 2), (8, 1500, 3), (61, 900, 2)])
def test_repeats_capture_and_new_lists(pq, q, n, B):
    """The same call gives the same bits; a captured one follows new lists, lengths and pages; two graphs share nothing."""
    cache, Q, starts, lens, table = make_case(pq, 6, [q] * B, [n] * B, 8, 2, 128, 16, poison=False)
    trees = trees_of([q] * B, 3)
    lists = pack(trees, 2).cuda()
    outs = [torch.empty_like(Q) for _ in range(2)]
    call = lambda O: pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, n, window=700, sinks=10, tree=lists)  # noqa: E731
    call(outs[0])
    for _ in range(5):
        call(outs[1])
        assert torch.equal(outs[0], outs[1])
    graphs = []
    for O in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(O)
        graphs.append(g)
    lists.copy_(pack(trees_of([q] * B, 11), 2))
    lens.sub_(3)
    for O in outs:
        O.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs[0].replay()
    with torch.cuda.stream(side):
        graphs[1].replay()
    torch.cuda.synchronize()
    want = torch.empty_like(Q)
    call(want)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    pq.pq_check_status()


@pytest.mark.parametrize("q", [2, 60])
def test_bad_pages(pq, q):
    """A listed page outside the cache is 16-token pieces that nobody sees, and the status says so."""
    cache, Q, starts, lens, table = make_case(pq, 6, [q], [400], 8, 2, 128, 16, poison=False)
    O = torch.empty_like(Q)
    table[0, 0] = 1 << 20
    pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, 400, window=64, sinks=20)
    with pytest.raises(pq.PQError):
        pq.pq_check_status()
    table[0, 0] = 0
    table[0, 3] = -9                                       # between sinks and window: not looked at
    pq.pq_kv4_attention_masked(cache, Q, O, starts, lens, table, q, 400, window=64, sinks=20)
    pq.pq_check_status()


def test_rows_outside_every_sequence_stay(pq):
    cache, Q, starts, lens, table = make_case(pq, 6, [3, 5], [90, 200], 8, 2, 128, 16)
    wide = torch.cat([Q, Q.new_full((4, 8, 128), float("nan"))])
    O = torch.full_like(wide, 7.0)
    lists = torch.cat([pack(trees_of([3, 5], 1), 1), torch.full((4, 1), -1, dtype=torch.int32)]).cuda()
    pq.pq_kv4_attention_masked(cache, wide, O, starts, lens, table, 5, 200, tree=lists)
    assert (O[8:] == 7).all() and not (O[:8] == 7).all()


@pytest.mark.parametrize("hd,hq,hkv,page,window,sinks,qs,ls", [
    (128, 8, 2, 16, 300, 8, *spread(41, 70, 1, 3000, 7)), (64, 4, 4, 64, 1024, 100, *spread(7, 40, 8, 5000, 5)),
])
def test_many_sequences_in_equal_shares(pq, hd, hq, hkv, page, window, sinks, qs, ls):
    case = make_case(pq, 8, qs, ls, hq, hkv, hd, page)
    check(pq, case, max(qs), max(ls), window=window, sinks=sinks)
    check(pq, case, max(qs), max(ls), window=window, sinks=sinks, trees=trees_of(qs, 3))


@pytest.mark.parametrize("hd,hq,hkv,page,rv,window,sinks,tree,qs,ls", [
    (128, 32, 8, 64, True, 0, 0, True, [500], [8000]), (64, 14, 2, 16, False, 0, 0, True, [300, 0, 77, 640, 2], [9000, 0, 5000, 9100, 2]),
    (128, 32, 8, 32, True, 4000, 7, False, [1000], [6000]), (128, 16, 4, 64, False, 300, 130, False, [5000], [5003]),
    (64, 8, 8, 128, True, 1000, 4, False, [3000, 100, 2000, 1], [5000, 100, 4100, 3000]), (128, 24, 8, 16, True, 2500, 20, True, [300, 200, 280], [5000, 9000, 700]),
])
def test_many_tiles(pq, hd, hq, hkv, page, rv, window, sinks, tree, qs, ls):
    """Calls of many tiles, cut into parts by their lengths; the same bits each time."""
    case = make_case(pq, sum(ls), qs, ls, hq, hkv, hd, page, rv=rv)
    trees = trees_of(qs, 5, 0.9) if tree else None
    O = check(pq, case, max(qs), max(ls), window=window, sinks=sinks, trees=trees)
    lists = pack(trees, -(-max(qs) // 32)).cuda() if tree else None
    for _ in range(3):
        again = torch.empty_like(O)
        pq.pq_kv4_attention_masked(case[0], case[1], again, *case[2:], max(qs), max(ls), window=window, sinks=sinks, tree=lists)
        assert torch.equal(O, again)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_a_verification_step(pq, fmt):
    """A layer's step with drafted tokens: 4-bit projections, append at the drafts' depths, attention of the tree under a window
    with sinks; then the accepted branch appended to its own slots attends as if it had come token by token."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    D, hq, hkv, hd, page, n, m, window, sinks = 512, 8, 2, 64, 16, 150, 10, 48, 3
    width = (hq + 2 * hkv) * hd
    W = (torch.randn(width, D, generator=gen, device="cuda") * 0.05).to(torch.bfloat16)
    fw = float(W.float().abs().max()) / (6 * 448) if fmt == "nv" else 1.0
    codes_W = torch.empty(width, D // 2, dtype=torch.uint8, device="cuda")
    scales_W = torch.empty(pq.pq_fp4_scale_bytes(width, D, fmt), dtype=torch.uint8, device="cuda")
    pq.pq_quant_fp4(W, codes_W, scales_W, fmt=fmt, g=128, factor=fw)
    rope = rope_table(400, hd)
    cache = pq.KV4Cache.empty(20, hkv, page, hd)
    table = torch.randperm(20, generator=gen, device="cuda").to(torch.int32)[None, :16].contiguous()
    slot = lambda t: table[0, t // page].long() * page + t % page  # noqa: E731

    def project(x):
        T = x.shape[0]
        ca = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda")
        sa = torch.empty(pq.pq_fp4_scale_bytes(T, D, fmt), dtype=torch.uint8, device="cuda")
        out = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
        pq.pq_fp4_linear(x, ca, sa, codes_W, scales_W, out, fmt=fmt, g=128, factor_A=0.01, factor_W=fw)
        return out

    def step(x, positions, slots, length, tree=None):
        qkv = project(x)
        T = x.shape[0]
        Q = torch.empty(T, hq, hd, dtype=torch.bfloat16, device="cuda")
        pq.pq_kv4_append(cache, qkv[:, :hq * hd], qkv[:, hq * hd:(hq + hkv) * hd], qkv[:, (hq + hkv) * hd:], Q,
                         positions.to(torch.int32), slots, rope=rope)
        O = torch.empty_like(Q)
        pq.pq_kv4_attention_masked(cache, Q, O, torch.tensor([0, T], dtype=torch.int32, device="cuda"),
                                   torch.tensor([length], dtype=torch.int32, device="cuda"), table, T, length, window=window,
                                   sinks=sinks, tree=tree)
        return Q, O

    t = torch.arange(n, device="cuda")
    X = torch.randn(n, D, generator=gen, device="cuda").to(torch.bfloat16)
    step(X, t, slot(t), n)
    bits = random_tree(m, torch.Generator().manual_seed(4), 0.4)
    depth = (bits.sum(1) - 1).cuda()
    new = torch.arange(n, n + m, device="cuda")
    drafts = torch.randn(m, D, generator=gen, device="cuda").to(torch.bfloat16)
    Q, O = step(drafts, n + depth, slot(new), n + m, tree=pack([bits], 1).cuda())
    # the longest branch, token by token
    leaf = int(bits.sum(1).argmax())
    branch = bits[leaf].nonzero()[:, 0]
    assert len(branch) >= 3
    for d, i in enumerate(branch.tolist()):
        at = torch.tensor([n + d], device="cuda")
        Qi, Oi = step(drafts[i:i + 1], at, slot(at), n + d + 1)
        assert torch.equal(Qi[0], Q[i])
        # the same tokens in other places: the same sums in another order
        off = (Oi[0].double() - O[i].double()).abs()
        assert bool((off <= 2.0 ** -6 * (O[i].double().abs() + O[i].double().square().mean().sqrt())).all())
    pq.pq_check_status()

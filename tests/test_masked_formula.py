"""What the masks mean, without a GPU: the definition against hand-written cases, and mistakes that
the outputs' bound has to catch."""
import types

import torch

from tests.masked64 import attention, pack, random_tree, seen


def rows(mask):
    return ["".join("x" if v else "." for v in r) for r in mask.tolist()]


def test_sinks():
    assert rows(seen(3, 8, 2, 1, None)) == ["x...xx..", "x....xx.", "x.....xx"]
    assert rows(seen(2, 5, 0, 3, None)) == ["xxxx.", "xxxxx"]
    assert rows(seen(2, 5, 9, 3, None)) == ["xxxx.", "xxxxx"]
    assert rows(seen(3, 3, 1, 2, None)) == ["x..", "xx.", "xxx"]          # sinks are not seen before their time
    assert rows(seen(4, 2, 1, 1, None)) == ["..", "..", "x.", "xx"]       # more new rows than tokens


def test_tree():
    bits = torch.tensor([[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [0, 0, 0, 0]], dtype=torch.bool)
    assert rows(seen(4, 6, 0, 0, bits)) == ["xxx...", "xxxx..", "xxx.x.", "xx...."]
    # a window of 2: the two children lie at position 3, whatever slot they are in; what a list holds stays seen
    assert rows(seen(4, 6, 2, 1, bits)) == ["xxx...", "x.xx..", "x.x.x.", "xx...."]
    assert rows(seen(4, 6, 2, 0, bits)) == [".xx...", "..xx..", "..x.x.", ".x...."]
    assert pack([bits, bits[:1, :1]], 1).tolist() == [[1], [3], [5], [0], [1]]
    wide = torch.zeros(40, 40, dtype=torch.bool)
    wide[39, 31] = wide[39, 39] = True
    assert pack([wide], 2)[39].tolist() == [-(1 << 31), 1 << 7]


def test_the_bound_catches_mistakes():
    gen = torch.Generator().manual_seed(3)
    page, hkv, hd, m, n = 16, 2, 64, 6, 90
    codes = [torch.randint(0, 256, (6, hkv, page, hd // 2), generator=gen, dtype=torch.uint8) for _ in "kv"]
    scales = [torch.randn(6, hkv, page, generator=gen).abs() * 0.2 + 0.02 for _ in "kv"]
    cache = types.SimpleNamespace(tensors=(codes[0], scales[0], codes[1], scales[1]), head_dim=hd, heads=hkv, page_size=page, rotate_v=True)
    Q = torch.randn(m, 4, hd, generator=gen)
    starts, lens, table = torch.tensor([0, m]), torch.tensor([n]), torch.arange(6)[None]
    bits = random_tree(m, gen)
    args = (cache, Q, starts, lens, table, hd ** -0.5)
    for many in (False, True):
        want, tol = attention(*args, 40, 4, [bits], many)
        flipped = bits.clone()
        flipped[4, 1] ^= True
        wrong = [attention(*args, 40, 4, [flipped], many)[0], attention(*args, 40, 0, [bits], many)[0], attention(*args, 40, 4, None, many)[0],
                 attention(*args, 0, 0, [bits], many)[0], attention(*args, 40, 5, [bits], many)[0], attention(*args, 41, 4, [bits], many)[0]]
        for w in wrong:
            assert bool(((w - want).abs() > tol).any())
        assert bool(((want - want * 1.03).abs() > tol).any())

"""Masked attention over the 4-bit cache in float64: which tokens a row sees (sinks, trees of drafted tokens), the outputs, and
what they may be off by from the spread of the kernels' roundings (the terms that spread64.py lists and derives)."""
import math

import torch

from tests.plain64 import hadamard, unpack
from tests.spread64 import DEVIATIONS, H11


def seen(m, n, window, sinks, bits, device="cpu"):
    """bool [m][n]: the tokens that each of the last m of n sees.  bits: bool [m][m] of a tree, or None.  By the definition, a
    row at a time."""
    out = torch.zeros(m, n, dtype=torch.bool)
    t = torch.arange(n)
    for i in range(m):
        depth = (max(int(bits[i].sum()), 1) - 1) if bits is not None else i
        p = n - m + depth
        out[i] = t <= p
        if window:
            out[i] &= (t > p - window) | (t < sinks)
        if bits is not None:
            out[i, max(n - m, 0):] = bits[i, max(m - n, 0):]
    return out.to(device)


def pack(trees, words, rows=None):
    """Rows' lists as int32 [rows][words] of bool [m][m] matrices, one a sequence."""
    out = []
    for bits in trees:
        for row in bits.tolist():
            v = sum(1 << j for j, b in enumerate(row) if b)
            w = [(v >> (32 * k)) & 0xFFFFFFFF for k in range(words)]
            out.append([x - (1 << 32) if x >> 31 else x for x in w])
    return torch.tensor(out, dtype=torch.int32).reshape(-1, words)


def random_tree(m, gen, chain=0.5):
    """bool [m][m]: each token's ancestors and itself; its parent is the one before it, any before it, or none."""
    bits = torch.zeros(m, m, dtype=torch.bool)
    for i in range(m):
        u = float(torch.rand((), generator=gen))
        parent = i - 1 if u < chain else int(torch.randint(-1, i, (1,), generator=gen)) if i else -1
        if parent >= 0:
            bits[i] = bits[parent]
        bits[i, i] = True
    return bits


def attention(cache, Q, q_start, seq_lens, table, scale, window, sinks, trees, many_rows):
    """(output, bound), float64 [T][heads_q][hd]; rows of no sequence: (nan, nan)."""
    kc, ks, vc, vs = cache.tensors
    hd, hkv, page = cache.head_dim, cache.heads, cache.page_size
    T = Q.shape[0]
    q_all = Q.reshape(T, hkv, -1, hd).double()
    group = q_all.shape[2]
    want = torch.full(q_all.shape, math.nan, dtype=torch.float64, device=Q.device)
    tol = want.clone()
    H = hadamard(hd, Q.device) if cache.rotate_v else None
    starts, lens = q_start.tolist(), seq_lens.tolist()
    for b, n in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        m = last - first
        if m <= 0:
            continue
        n = max(n, 0)
        mask = seen(m, n, window, sinks, trees[b] if trees is not None else None, Q.device)
        want[first:last], tol[first:last] = 0, 0
        used = mask.any(0)
        blocks = [i for i in range(-(-n // page)) if bool(used[i * page:(i + 1) * page].any())]
        if not blocks:
            continue
        # only the pages that someone sees are looked at
        t = torch.cat([torch.arange(i * page, min(n, (i + 1) * page), device=Q.device) for i in blocks])
        pages = table[b, torch.tensor(blocks, device=Q.device)].long()
        code, _ = unpack(kc[pages], ks[pages])
        _, val = unpack(vc[pages], vs[pages])
        kcode = code.double().permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :len(t)]
        key_s = ks[pages].double().permute(1, 0, 2).reshape(hkv, -1)[:, :len(t)]
        val = val.permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :len(t)]
        mask = mask[:, t]
        live = mask.any(0)
        hide = ~mask.repeat_interleave(group, dim=0)
        for g in range(hkv):
            x = q_all[first:last, g].reshape(m * group, hd)
            k_s = torch.where(live, key_s[g], torch.zeros_like(key_s[g]))
            v = torch.where(live[:, None], val[g], torch.zeros_like(val[g]))
            s = ((x @ kcode[g].t()) * k_s * scale).masked_fill(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.where(hide, torch.zeros_like(s), torch.exp(s - torch.where(top.isfinite(), top, torch.zeros_like(top))))
            p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
            y, vr = (p @ v, v) if H is None else (p @ v @ H, v @ H)
            mag = x.abs().sum(-1, keepdim=True)
            d = abs(scale) * k_s.abs() * (mag * 24 * 8 * 2.0 ** -22 + x.abs().amax(-1, keepdim=True) * hd * 8 * 2.0 ** -35) + \
                4 * 2.0 ** -24 * torch.where(hide, torch.zeros_like(s), s.abs())
            pd = p * torch.where(hide, torch.zeros_like(d), torch.expm1(d))
            full = pd @ vr.abs() + pd.sum(-1, keepdim=True) * y.abs()
            var = (p * p) @ (vr * vr) * (H11 ** 2 / 3) * (2 if many_rows else 1)
            if many_rows:
                channel = (p * p) @ (v * v) * (H11 ** 2 / 3)
                var = var + (channel if H is None else channel.mean(-1, keepdim=True).expand_as(channel))
                sv = (x * x) @ (kcode[g] * kcode[g]).t() * (scale * k_s) ** 2 * (H11 ** 2 / 3)
                w = p * p * torch.where(hide, torch.zeros_like(sv), sv)
                var = var + ((w @ (vr * vr)) - 2 * (w @ vr) * y + w.sum(-1, keepdim=True) * y * y).clamp_min(0)
            most = (p * v.abs().amax(-1)).amax(-1, keepdim=True)
            count = (~hide).sum(-1, keepdim=True).double()
            var = var + count / 3 * (most * (2.0 ** -19 if many_rows else 2.0 ** -25)) ** 2
            rms = y.square().mean(-1, keepdim=True).sqrt()
            err = DEVIATIONS * var.sqrt() + full + (len(t) / 16 + 64) * 2.0 ** -22 * (y.abs() + rms)
            err = err + 2.0 ** -8 * (y.abs() + err)
            want[first:last, g] = y.reshape(m, group, hd)
            tol[first:last, g] = err.reshape(m, group, hd)
    return want.reshape(T, -1, hd), tol.reshape(T, -1, hd)

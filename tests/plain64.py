"""Plain float64 forms of the 8-bit product and of the 4-bit key/value cache, and the bounds their
float32 kernels are held to.  Test infrastructure: elementary torch operations, no library kernels."""
import math

import torch

U = 2.0 ** -24            # half a float32 step, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11}


def hadamard(n, device):
    i = torch.arange(n, device=device)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(n.bit_length())) % 2
    return (1 - 2 * odd).double() / math.sqrt(n)


# ------------------------------------------------------------------------------------ 8-bit rows
def rows8(X, g):
    """(y, scale, band): rotated rows, their scales, and how far from a half-integer y / scale must be for
    the float32 code to be certain.  Each of the log2(g) butterfly stages rounds once, relative to a partial
    sum of at most sum|x|; the row's maximum carries the same error, and the product with 127 / max three
    more roundings."""
    x = X.double()
    if g:
        D = x.shape[1]
        blocks = x.reshape(x.shape[0], D // g, g)
        y = (blocks @ hadamard(g, x.device)).reshape(x.shape)
        mass = (blocks.abs().sum(dim=-1, keepdim=True) / math.sqrt(g)).expand_as(blocks).reshape(x.shape)
        err = math.log2(g) * U * mass.amax(dim=1, keepdim=True)
    else:
        y, err = x, torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device)
    m = y.abs().amax(dim=1, keepdim=True)
    band = 2 * 127 * torch.where(m > 0, err / m, torch.zeros_like(m)) + 127 * 4 * U
    return y, (m / 127)[:, 0], band, (torch.where(m > 0, err / m, torch.zeros_like(m)) + 4 * U)[:, 0]


def check_codes(codes, ratio, band):
    """codes equal round(ratio) away from half-integers by more than band, and are within 1 of it elsewhere."""
    want = torch.round(ratio)
    near = ((ratio - torch.floor(ratio)) - 0.5).abs() <= band
    diff = (codes.double() - want).abs()
    assert not ((diff != 0) & ~near).any(), f"{int(((diff != 0) & ~near).sum())} codes differ away from ties"
    assert (diff <= 1).all()


# ------------------------------------------------------------------------------------ cache rows
def heads64(x, heads, hd, norm, eps, rope, positions, interleaved, rotate):
    """[T][heads][hd] in float64 and a bound of the float32 error of each element (before any factor 1/sqrt(hd)
    is lost: both are in the output's units).

    Norm: 8 roundings in the sum of squares (all terms positive), one in the mean, one with eps, halved by
    the root, one each for the root, the reciprocal and the two products: 9 at most.  Turning: two products
    and a sum: 2 more of |a| + |b|.  The log2(hd) Hadamard stages: one each of the sum of all channels'
    magnitudes; the factor one more."""
    T = x.shape[0]
    y = x.double().reshape(T, heads, hd)
    rel = 0.0
    if norm is not None:
        y = y / (y.square().mean(dim=-1, keepdim=True) + eps).sqrt() * norm.double()
        rel += 9
    size = y.abs()
    if rope is not None:
        rd = rope.shape[1]
        cs = rope[positions.long()].double()[:, None, :]
        cos, sin = cs[..., :rd // 2], cs[..., rd // 2:]
        if interleaved:
            a, b = y[..., 0:rd:2].clone(), y[..., 1:rd:2].clone()
            y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
            both = (a.abs() + b.abs()).repeat_interleave(2, dim=-1)
        else:
            a, b = y[..., :rd // 2].clone(), y[..., rd // 2:rd].clone()
            y[..., :rd // 2], y[..., rd // 2:rd] = a * cos - b * sin, b * cos + a * sin
            both = (a.abs() + b.abs()).repeat(1, 1, 2)
        size = torch.cat([both, size[..., rd:]], dim=-1)
        rel += 2
    err = rel * U * size
    if rotate:
        y = y @ hadamard(hd, y.device)
        total = size.sum(dim=-1, keepdim=True) / math.sqrt(hd)
        err = ((rel + math.log2(hd) + 1) * U * total).expand_as(y)
    return y, err


def unpack(codes, scales):
    """Cache codes [...][hd / 2] and scales [...] -> (integer codes, float64 values)."""
    u = codes.to(torch.int32)
    u = torch.stack([u & 15, u >> 4], dim=-1).flatten(-2)
    u = torch.where(u > 7, u - 16, u)
    return u, u.double() * scales.double()[..., None]


# ------------------------------------------------------------------------------------- attention
def attention64(cache, Q, q_start, seq_lens, table, scale, window, out, fp16_operands=False):
    """(output, bound) in float64: `out` (float64) with the sequences' rows replaced.

    The bound per element: each probability's fp16 rounding (2^-11 relative, and 2^-25 of the largest scale
    where it leaves fp16's normal range), the scores' float32 sums (the operands 136 + code are summed with the
    queries, so 16 * 9 magnitudes per channel; the exponent sees them twice, in the numerator and the sum),
    float32 accumulation over the tokens, and half a bf16 step of the result.

    fp16_operands (calls of many rows, where scales are multiplied into fp16 keys and values): each product of a code
    and its key scale is off by 2^-11 of it at most (one rounding; the low part of the scale adds 2^-21), or 2^-25 of
    the largest scale below fp16's normal range, and so is each query channel; each value by 2^-11 twice (its scale,
    then the product), or 2^-25 of the largest."""
    kc, ks, vc, vs = cache.tensors
    hd, hkv, page = cache.head_dim, cache.heads, cache.page_size
    T = Q.shape[0]
    q = Q.reshape(T, -1, hd).double()
    group = q.shape[1] // hkv
    want, tol = out.clone(), torch.zeros_like(out)
    starts, lens = q_start.tolist(), seq_lens.tolist()
    H = hadamard(hd, Q.device) if cache.rotate_v else None
    for b, n in enumerate(lens):
        first, last = starts[b], starts[b + 1]
        if last <= first:
            continue
        n = max(n, 0)
        if n == 0:
            want[first:last] = 0
            continue
        pages = table[b, :-(-n // page)].long()
        k_code, _ = unpack(kc[pages], ks[pages])
        _, v = unpack(vc[pages], vs[pages])
        k_code = k_code.permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n].double()
        k_s = ks[pages].permute(1, 0, 2).reshape(hkv, -1)[:, :n].double()
        v_s = vs[pages].permute(1, 0, 2).reshape(hkv, -1)[:, :n].double().abs()
        v = v.permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n]
        m = last - first
        back = torch.arange(n - m, n, device=Q.device)[:, None] - torch.arange(n, device=Q.device)[None, :]
        hidden = (back < 0) | (back >= window) if window else back < 0
        for h in range(q.shape[1]):
            kv = h // group
            x = q[first:last, h]
            s = (x @ k_code[kv].t()) * k_s[kv] * scale
            s_err = (x.abs().sum(-1, keepdim=True) * 144 * 140 * 2 * U) * k_s[kv].abs() * abs(scale) + 4 * U * s.abs()
            if fp16_operands:
                mag = k_code[kv].abs()
                small = x.abs().amax(-1, keepdim=True) * 2.0 ** -24
                s_err = s_err + abs(scale) * ((x.abs() @ mag.t()) * (2.0 ** -11 + 2.0 ** -20) * k_s[kv] +
                                              x.abs().sum(-1, keepdim=True) * 8 * 2.0 ** -24 * k_s[kv].max() + small * mag.sum(-1) * k_s[kv])
            s = s.masked_fill(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.where(hidden, torch.zeros_like(s), torch.exp(s - torch.where(top.isfinite(), top, torch.zeros_like(top))))
            total = p.sum(-1, keepdim=True)
            p = torch.where(total > 0, p / total, torch.zeros_like(p))
            vv = torch.where(hidden.all(0)[:, None], torch.zeros_like(v[kv]), v[kv])   # never seen: anything may be there
            pe = p * ((3 if fp16_operands else 1) * 2.0 ** -11 + 2 * torch.where(hidden, torch.zeros_like(s_err), s_err).amax(-1, keepdim=True) + (n + 64) * 2 * U)
            seen_vs = torch.where(hidden, torch.zeros_like(s), v_s[kv].expand_as(s)).amax(-1, keepdim=True)
            o = p @ vv
            e = pe @ vv.abs() + torch.where(total > 0, (2 if fp16_operands else 1) * 8 * n * seen_vs * 2.0 ** -25 / total.clamp_min(1e-300), torch.zeros_like(total))
            if H is not None:
                o = o @ H
                e = (e.sum(-1, keepdim=True) / math.sqrt(hd) * (1 + 10 * U)).expand_as(o) + 16 * U * o.abs().amax(-1, keepdim=True)
            want[first:last, h] = o
            tol[first:last, h] = e + HALF_STEP[torch.bfloat16] * (o.abs() + e) + 1e-30
    return want, tol

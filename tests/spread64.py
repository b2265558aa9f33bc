"""Attention over the 4-bit cache in float64 with the spread that its kernels' roundings give each output: what an output may
be off by, closely enough that a block of tokens left out, a scale a few percent off or zeros do not pass.

The roundings that matter are many and independent (one for each token, or token and channel), each at most half a step,
h = 2^-11 of an fp16 value x, so of variance (h x)^2 / 3 at most.  With p the probabilities, v the values, o the output:
  - a probability times its value's scale, to fp16: e_t p_t v_t, the same e_t for all channels of a token;
  - in calls of many rows the scale of a value, to fp16: the same form; and code times that scale: one e for each channel;
    code times key scale: the score is off by d_t = scale sum_k e_k q_k kc_k ks, of variance
    h^2 / 3 sum_k (scale q_k kc_k ks)^2, and the output by p_t d_t (v_t - o) (the sum of the probabilities moves too).
The bound is 7 of the sum's standard deviations (one in 10^11 for a normal distribution), and in full, not as deviations:
  - half a step of bf16 of the output, 2^-8;
  - float32 sums: a step of 16 (or 64) tokens loses 2^-22 of what has been summed; n / 16 steps, and 64 for scores, joins
    and the rotation;
  - queries rounded to 2^-35 of their largest channel, and score sums of 8 steps, each losing 2^-22 of the magnitudes summed
    (codes enter with an offset of 8): a score's float32 error, as e^d - 1 on its probability;
  - products below fp16's normal range: 2^-25 of the largest product a token (2^-19 in calls of many rows, where the largest
    may be taken 64 times too large).
"""
import math

import torch

from tests.plain64 import hadamard, unpack

H11 = 2.0 ** -11
DEVIATIONS = 7.0


def attention(cache, Q, q_start, seq_lens, table, scale, window, many_rows):
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
        if n <= 0:
            want[first:last] = 0
            tol[first:last] = 0
            continue
        # pages in front of what the first row sees are not looked at
        lo = max(0, n - m - window + 1) // page if window else 0
        pages = table[b, lo:-(-n // page)].long()
        lo *= page
        code, _ = unpack(kc[pages], ks[pages])
        _, val = unpack(vc[pages], vs[pages])
        kcode = code.double().permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n - lo]
        key_s = ks[pages].double().permute(1, 0, 2).reshape(hkv, -1)[:, :n - lo]
        val = val.permute(1, 0, 2, 3).reshape(hkv, -1, hd)[:, :n - lo]
        t = torch.arange(lo, n, device=Q.device)
        pos = torch.arange(n - m, n, device=Q.device)
        hidden = t[None, :] > pos[:, None]
        if window:
            hidden |= t[None, :] <= pos[:, None] - window
        for g in range(hkv):
            live = ~hidden.all(0)
            x = q_all[first:last, g].reshape(m * group, hd)
            hide = hidden.repeat_interleave(group, dim=0)
            k_s = torch.where(live, key_s[g], torch.zeros_like(key_s[g]))
            v = torch.where(live[:, None], val[g], torch.zeros_like(val[g]))
            s = (x @ kcode[g].t()) * k_s * scale
            s = s.masked_fill(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            p = torch.where(hide, torch.zeros_like(s), torch.exp(s - torch.where(top.isfinite(), top, torch.zeros_like(top))))
            total = p.sum(-1, keepdim=True)
            p = p / total.clamp_min(1e-300)
            o = p @ v
            # float32 errors of a score, in full
            mag = x.abs().sum(-1, keepdim=True)
            d = abs(scale) * k_s.abs() * (mag * 24 * 8 * 2.0 ** -22 + x.abs().amax(-1, keepdim=True) * hd * 8 * 2.0 ** -35) + \
                4 * 2.0 ** -24 * torch.where(hide, torch.zeros_like(s), s.abs())
            pd = p * torch.where(hide, torch.zeros_like(d), torch.expm1(d))
            y, vr = (o, v) if H is None else (o @ H, v @ H)
            full = pd @ vr.abs() + pd.sum(-1, keepdim=True) * y.abs()
            # independent roundings: variances
            var = (p * p) @ (vr * vr) * (H11 ** 2 / 3) * (2 if many_rows else 1)
            if many_rows:
                channel = (p * p) @ (v * v) * (H11 ** 2 / 3)
                var = var + (channel if H is None else channel.mean(-1, keepdim=True).expand_as(channel))
                sv = (x * x) @ (kcode[g] * kcode[g]).t() * (scale * k_s) ** 2 * (H11 ** 2 / 3)
                w = p * p * torch.where(hide, torch.zeros_like(sv), sv)
                # (v - o)^2 = v^2 - 2 v o + o^2
                var = var + ((w @ (vr * vr)) - 2 * (w @ vr) * y + w.sum(-1, keepdim=True) * y * y).clamp_min(0)
            # products below the normal range
            most = (p * v.abs().amax(-1)).amax(-1, keepdim=True)
            seen = (~hide).sum(-1, keepdim=True).double()
            var = var + seen / 3 * (most * (2.0 ** -19 if many_rows else 2.0 ** -25)) ** 2
            rms = y.square().mean(-1, keepdim=True).sqrt()
            err = DEVIATIONS * var.sqrt() + full + (n / 16 + 64) * 2.0 ** -22 * (y.abs() + rms)
            err = err + 2.0 ** -8 * (y.abs() + err)
            want[first:last, g] = y.reshape(m, group, hd)
            tol[first:last, g] = err.reshape(m, group, hd)
    return want.reshape(T, -1, hd), tol.reshape(T, -1, hd)

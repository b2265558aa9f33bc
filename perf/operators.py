"""Cases, plain forms and 64-bit values of the 8-bit product and the 4-bit key/value cache.

Three operators, in the order in which a layer whose linear maps run on low-bit codes calls them:

* ``w8a8``: rows of bf16 activations, rotated by a block Hadamard (or not), take one symmetric 8-bit scale a token;
  the codes are multiplied with weights that have one 8-bit scale an output channel.
* ``append``: queries and keys of each head are normalised, rotated by position and by a Hadamard matrix; keys and values
  are written into a paged cache as 4-bit codes with one scale a token and head.
* ``attention``: causal attention of new tokens over that cache, from one token a sequence to whole prompts.

``run`` computes the operators from elementary torch operations in 32 bits; where ``own`` is true it makes the calls of
``rotation_int4_w4a4_b200.pq`` instead.  ``exact`` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-5
ROPE_BASE = 500000.0


# ---------------------------------------------------------------------------------------------- cases
def _w8a8(name, T, N, D, g, out, quantised):
    """quantised: the activations' codes are in hand (the product alone); otherwise bf16 rows come in."""
    return {"name": name, "op": "w8a8", "T": T, "N": N, "D": D, "g": g, "out": out, "quantised": quantised}


def _append(name, T, hq, hkv, hd, page, norm, rope_dim, interleaved, rotate, pad):
    """pad: every pad-th token has no slot (0: all have one)."""
    return {"name": name, "op": "append", "T": T, "hq": hq, "hkv": hkv, "hd": hd, "page": page, "norm": norm,
            "rope_dim": rope_dim, "interleaved": interleaved, "rotate": rotate, "pad": pad}


def _attend(name, B, q, ctx, ragged, hq, hkv, hd, page, window, rotate):
    """B sequences of up to q new tokens over up to ctx cached ones (the new ones among them)."""
    return {"name": name, "op": "attention", "B": B, "q": q, "ctx": ctx, "ragged": ragged, "hq": hq, "hkv": hkv,
            "hd": hd, "page": page, "window": window, "rotate": rotate}


def listed():
    return [
        # One token through a 4096 x 4096 projection: generation for one user, where latency counts.
        _w8a8("8-bit linear, 1 token", 1, 4096, 4096, 128, "bf16", False),
        # A decode batch through the up projection of the LLaMA-3-8B shape.
        _w8a8("8-bit linear, 64 tokens", 64, 14336, 4096, 128, "bf16", False),
        # Odd sizes: a short prompt, a head of 1003 outputs, a reduction that fills no whole tile.
        _w8a8("8-bit product, odd sizes", 391, 1003, 4176, 0, "f32", True),
        # The down projection of the LLaMA-3-8B shape over a long prompt: the layer that 4 bits hurt most.
        _w8a8("8-bit linear, down projection", 8192, 4096, 14336, 128, "bf16", False),
        # A decode step of 32 users: new keys and values of one token each.
        _append("cache append, 32 tokens", 32, 32, 8, 128, 64, False, 128, False, True, 0),
        # A packed prompt with padding rows, heads of 64 with norms, half of each head rotated by position.
        _append("cache append, heads of 64", 777, 14, 2, 64, 16, True, 32, True, True, 9),
        # A long prompt of the LLaMA-3-8B head layout, queries and keys normalised.
        _append("cache append, 8192 tokens", 8192, 32, 8, 128, 64, True, 128, False, True, 0),
        # One user, a short context: the smallest step.
        _attend("attention, 1 token over 517", 1, 1, 517, False, 32, 8, 128, 64, 0, True),
        # One user, a long context: the cache of one sequence is split over the whole card.
        _attend("attention, 1 token over 65536", 1, 1, 65536, False, 32, 8, 128, 64, 0, True),
        # A decode batch over ragged contexts, some of them empty.
        _attend("attention, 64 users, ragged", 64, 1, 8192, True, 32, 8, 128, 64, 0, True),
        # Ragged chunks of prompts over earlier context, heads of 64 in groups of 7, a sliding window.
        _attend("attention, ragged chunks", 6, 801, 2999, True, 14, 2, 64, 16, 1024, False),
        # The second half of a prompt of 8192 tokens.
        _attend("attention, 4096 of 8192 tokens", 1, 4096, 8192, False, 32, 8, 128, 64, 0, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("w8a8", "w8a8", "append", "attention", "attention", "attention"))
    if op == "w8a8":
        g = rng.choice((0, 64, 128, 256))
        T, N = _log(rng, 1, 8192), _log(rng, 16, 14336)
        D = 256 * _log(rng, 1, 56) if g else 16 * _log(rng, 8, 896)
        c = _w8a8("", T, N, D, g, rng.choice(("bf16", "f32")), False)
        c["quantised"] = c["out"] == "f32"   # f32 outputs: the product alone, from codes in hand
        c["g"] = 0 if c["quantised"] else g
    elif op == "append":
        hd = rng.choice((64, 128))
        hkv = rng.choice((1, 2, 4, 8))
        c = _append("", _log(rng, 1, 8192), hkv * rng.choice((1, 2, 4, 5, 7, 8)) if hkv < 8 else 32, hkv, hd,
                    rng.choice((16, 32, 64, 128)), rng.random() < 0.5, rng.choice((0, hd // 2, hd)),
                    rng.random() < 0.3, rng.random() < 0.7, rng.choice((0, 0, 3, 10)))
    else:
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 4, 5, 7, 8)) if hkv < 8 else 32
        ctx = _log(rng, 1, 32768)
        q = min(ctx, rng.choice((1, 1, _log(rng, 2, 32), _log(rng, 33, 2048))))
        B = _log(rng, 1, max(1, min(64, (1 << 19) // ctx, (1 << 29) // (ctx * q * hq) if q > 1 else 64)))
        c = _attend("", B, q, ctx, rng.random() < 0.7, hq, hkv, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)),
                    rng.choice((0, 0, _log(rng, 1, 4096))), rng.random() < 0.7)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, cached tokens) of each sequence, from the case alone.  Ragged: one sequence in eight is empty
    (nothing cached, nothing asked), the others' lengths are spread evenly."""
    B, q, ctx = case["B"], case["q"], case["ctx"]
    if not case["ragged"] or B == 1:
        return [q] * B, [ctx] * B
    r = random.Random(B * 1000003 + q * 1009 + ctx)
    qs, ls = [], []
    for b in range(B):
        n = 0 if b % 8 == 5 else (ctx if b == 0 else r.randint(1, ctx))
        m = min(n, q if q == 1 else r.randint(1, q))
        qs.append(m)
        ls.append(n)
    return qs, ls


# --------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return gen


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _prepare_w8a8(case, seed):
    gen = _generator(seed)
    T, N, D = case["T"], case["N"], case["D"]
    x = _normal(gen, T, D)
    x[:, torch.randperm(D, generator=gen, device=DEV)[:8]] *= 30.0   # outlier channels, as activations have them
    st = {"X": x.to(torch.bfloat16)}
    if case["quantised"]:
        scale = st["X"].float().abs().amax(dim=1).clamp_min(1e-30) / 127
        st["codes_A"] = torch.round(st["X"].float() / scale[:, None]).to(torch.int8)
        st["scales_A"] = scale
    else:
        st["codes_A"] = torch.empty(T, D, dtype=torch.int8, device=DEV)      # written by the call
        st["scales_A"] = torch.empty(T, dtype=torch.float32, device=DEV)
    w = _normal(gen, N, D) * 0.02
    sw = w.abs().amax(dim=1) / 127
    st["codes_W"] = torch.round(w / sw[:, None]).to(torch.int8)
    st["scales_W"] = sw
    st["Y"] = torch.empty(T, N, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
    return st


def _rope_table(rows, dim):
    """cos and sin of each position and frequency, [rows][dim / 2] each, side by side: [rows][dim]."""
    inv = ROPE_BASE ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=DEV) / dim)
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _prepare_append(case, seed):
    gen = _generator(seed)
    T, hq, hkv, hd, page = case["T"], case["hq"], case["hkv"], case["hd"], case["page"]
    # one projection's output: queries, keys and values side by side in each row
    qkv = _normal(gen, T, (hq + 2 * hkv) * hd)
    qkv[:, hq * hd:(hq + hkv) * hd].view(T, hkv, hd)[:, :, :3] *= 8.0    # keys have outlier channels
    qkv = qkv.to(torch.bfloat16)
    pages = -(-T // page) + 3
    slots = torch.randperm(pages * page, generator=gen, device=DEV)[:T].to(torch.int64)
    if case["pad"]:
        slots[:: case["pad"]] = -1
    first = int(torch.randint(0, 4096, (1,), generator=gen, device=DEV))
    positions = first + torch.arange(T, device=DEV, dtype=torch.int32)
    st = {"Q": qkv[:, :hq * hd], "K": qkv[:, hq * hd:(hq + hkv) * hd], "V": qkv[:, (hq + hkv) * hd:],
          "slots": slots, "positions": positions, "Q_out": torch.empty(T, hq * hd, dtype=torch.bfloat16, device=DEV),
          "K_out": torch.empty(T, hkv * hd, dtype=torch.bfloat16, device=DEV),
          "V_out": torch.empty(T, hkv * hd, dtype=torch.bfloat16, device=DEV),
          "rope": _rope_table(first + T, case["rope_dim"]) if case["rope_dim"] else None,
          "q_norm": (1 + 0.1 * _normal(gen, hd)).to(torch.bfloat16) if case["norm"] else None,
          "k_norm": (1 + 0.1 * _normal(gen, hd)).to(torch.bfloat16) if case["norm"] else None,
          "keep": {}}
    for kv in "kv":
        st[kv + "_codes"] = torch.zeros(pages, hkv, page, hd // 2, dtype=torch.uint8, device=DEV)
        st[kv + "_scales"] = torch.zeros(pages, hkv, page, dtype=torch.float32, device=DEV)
    return st


def _prepare_attention(case, seed):
    gen = _generator(seed)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    qs, ls = _lengths(case)
    B, T = len(qs), sum(qs)
    width = max(1, max(-(-n // page) for n in ls))
    used = [-(-n // page) for n in ls]
    pages = sum(used) + 2
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    st = {"Q": _normal(gen, T, hq * hd).to(torch.bfloat16), "O": torch.empty(T, hq * hd, dtype=torch.bfloat16, device=DEV),
          "q_start": torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV),
          "seq_lens": torch.tensor(ls, dtype=torch.int32, device=DEV), "table": table,
          "max_q": max(qs), "max_len": max(ls), "keep": {}}
    for kv in "kv":
        y = _normal(gen, pages, hkv, page, hd)
        m = y.abs().amax(dim=-1)
        u = torch.round(y * (7 / m)[..., None]).to(torch.int32) & 15
        st[kv + "_codes"] = (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8)
        st[kv + "_scales"] = m / 7
    return st


def prepare(case, seed):
    st = {"w8a8": _prepare_w8a8, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, seed)
    st["case"] = dict(case)
    return st


# --------------------------------------------------------------------------------------- plain forms
def _hadamard_tree(y):
    """y H along the last axis (H_ij = (-1)^popcount(i & j), no factor) by butterflies, nearest channels first."""
    n, shape = y.shape[-1], y.shape
    h = 1
    while h < n:
        v = y.reshape(*shape[:-1], n // (2 * h), 2, h)
        a, b = v[..., 0, :], v[..., 1, :]
        y = torch.stack([a + b, a - b], dim=-2).reshape(shape)
        h *= 2
    return y


def _plain_w8a8(st):
    c = st["case"]
    if c["quantised"]:
        qa, sa = st["codes_A"].float(), st["scales_A"]
    else:
        y = st["X"].float()
        g = c["g"]
        if g:
            y = _hadamard_tree(y.reshape(c["T"], -1, g)).reshape(c["T"], c["D"]) * (1 / math.sqrt(g))
        m = y.abs().amax(dim=1)
        sa = m / 127
        qa = torch.round(y * torch.where(m > 0, 127 / m, torch.zeros_like(m))[:, None])
    y = qa @ st["codes_W"].float().t()
    return (y * sa[:, None] * st["scales_W"][None, :]).to(st["Y"].dtype)


def _pair_sum(v):
    """Sum along the last axis by adding neighbours, then neighbours' sums, and so on."""
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v


def _heads(st, name, heads, norm):
    """Rows of one of the three inputs as [T][heads][hd], normalised and rotated by position."""
    c = st["case"]
    T, hd, rd = c["T"], c["hd"], c["rope_dim"]
    x = st[name].float().reshape(T, heads, hd)
    if norm is not None:
        r = 1 / torch.sqrt(_pair_sum(x * x) * (1 / hd) + EPS)
        x = (x * r) * norm.float()
    if rd and name != "V":
        cs = st["rope"][st["positions"].long()][:, None, :]
        cos, sin = cs[..., :rd // 2], cs[..., rd // 2:]
        a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if c["interleaved"] else (x[..., :rd // 2], x[..., rd // 2:rd])
        u, v = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([u, v], dim=-1).flatten(-2) if c["interleaved"] else torch.cat([u, v], dim=-1)
        x = torch.cat([turned, x[..., rd:]], dim=-1)
    return x


def _plain_append(st):
    c = st["case"]
    T, hd = c["T"], c["hd"]
    q = _heads(st, "Q", c["hq"], st["q_norm"])
    if c["rotate"]:
        q = _hadamard_tree(q) * (1 / math.sqrt(hd))
    out = [q.to(torch.bfloat16).reshape(T, -1)]
    written = (st["slots"] >= 0)[:, None]
    for name, norm in (("K", st["k_norm"]), ("V", None)):
        y = _heads(st, name, c["hkv"], norm)
        if c["rotate"]:
            y = _hadamard_tree(y)
        m = y.abs().amax(dim=-1, keepdim=True)
        code = torch.round(y * torch.where(m > 0, 7 / m, torch.zeros_like(m)))
        scale = m * (1 / (7 * math.sqrt(hd)) if c["rotate"] else 1 / 7)
        values = (code * scale).to(torch.bfloat16).reshape(T, -1)
        out.append(torch.where(written, values, torch.zeros_like(values)))
    return out


def _cached(st, kv, b):
    """Keys or values of the cache in float32, [len(b)][hkv][table width * page][hd]."""
    codes, scales = st[kv + "_codes"], st[kv + "_scales"]
    pages = st["table"][b].long()                                    # [B][width]
    u = codes[pages].to(torch.int32)                                 # [B][width][hkv][page][hd / 2]
    u = torch.stack([u & 15, u >> 4], dim=-1).flatten(-2)
    v = torch.where(u > 7, u - 16, u).float() * scales[pages][..., None]
    return v.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(st):
    c = st["case"]
    hq, hkv, hd, q, n = c["hq"], c["hkv"], c["hd"], st["max_q"], st["max_len"]
    start, lens, T = st["q_start"].long(), st["seq_lens"].long(), st["Q"].shape[0]
    B = lens.numel()
    i = torch.arange(q, device=DEV)
    real = i[None, :] < (start[1:] - start[:-1])[:, None]            # [B][q]
    row = torch.where(real, start[:-1, None] + i, torch.full_like(i, T)[None, :])
    k, v = (_cached(st, x, slice(None))[:, :, :n] for x in "kv")      # [B][hkv][n][hd]
    qs = torch.cat([st["Q"], st["Q"].new_zeros(1, hq * hd)])[row].float().reshape(B, q, hkv, hq // hkv, hd)
    s = torch.einsum("bqhgd,bhnd->bhgqn", qs, k) * (1 / math.sqrt(hd))
    place = (lens - (start[1:] - start[:-1]))[:, None] + i           # position of each new token
    t = torch.arange(n, device=DEV)
    seen = t[None, None, :] <= place[..., None]
    if c["window"]:
        seen &= t[None, None, :] > place[..., None] - c["window"]
    s = s.masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(dim=-1, keepdim=True))
    o = torch.einsum("bhgqn,bhnd->bqhgd", p / p.sum(dim=-1, keepdim=True), v)
    if c["rotate"]:
        o = _hadamard_tree(o) * (1 / math.sqrt(hd))                  # the cached values are rotated
    out = torch.zeros(T + 1, hq * hd, dtype=torch.float32, device=DEV)
    out[row] = o.reshape(B, q, hq * hd)
    return out[:T].to(torch.bfloat16)


# ------------------------------------------------------------------------------ the framework's calls
def _own_cache(st, pq):
    """The cache handle that a user's program keeps with its buffers."""
    if "cache" not in st["keep"]:
        r = st["case"]["rotate"]
        st["keep"]["cache"] = pq.KV4Cache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"],
                                          rotate_k=r, rotate_v=r)
    return st["keep"]["cache"]


def _own_run(st):
    from rotation_int4_w4a4_b200 import pq
    c = st["case"]
    if c["op"] == "w8a8":
        if c["quantised"]:
            pq.pq_w8a8_gemm(st["codes_A"], st["scales_A"], st["codes_W"], st["scales_W"], st["Y"])
        else:
            pq.pq_w8a8_linear(st["X"], st["codes_A"], st["scales_A"], st["codes_W"], st["scales_W"], st["Y"], g=c["g"])
        return st["Y"]
    cache = _own_cache(st, pq)
    if c["op"] == "append":
        pq.pq_kv4_append(cache, st["Q"], st["K"], st["V"], st["Q_out"], st["positions"], st["slots"], rope=st["rope"],
                         q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS, interleaved=c["interleaved"])
        pq.pq_kv4_read(cache, st["slots"], st["K_out"], st["V_out"])
        return [st["Q_out"], st["K_out"], st["V_out"]]
    pq.pq_kv4_attention(cache, st["Q"], st["O"], st["q_start"], st["seq_lens"], st["table"], max_q=st["max_q"],
                        max_len=st["max_len"], scale=1 / math.sqrt(c["hd"]), window=c["window"])
    return st["O"]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_w8a8(state) if op == "w8a8" else _plain_append(state) if op == "append" else _plain_attention(state)


# ------------------------------------------------------------------------------------ work and values
def work(case):
    if case["op"] == "w8a8":
        T, N, D = case["T"], case["N"], case["D"]
        rows = T * D + 4 * T if case["quantised"] else 2 * T * D
        return {"bytes": rows + N * D + 4 * N + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * D}
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":
        T = case["T"]
        kept = T - (-(-T // case["pad"]) if case["pad"] else 0)
        # queries in and out; keys and values in, their codes and scales out and back in, their values out
        moved = 4 * T * hq * hd + 2 * hkv * (T * 2 * hd + kept * 2 * (hd // 2 + 4) + T * 2 * hd)
        tables = T * (12 + 4 * case["rope_dim"])
        levels = int(math.log2(hd)) if case["rotate"] else 0
        return {"bytes": moved + tables, "flops": T * hd * ((hq + hkv) * (10 + levels) + hkv * (6 + levels))}
    qs, ls = _lengths(case)
    pairs = kv = 0
    for q, n in zip(qs, ls):
        w = case["window"] or n
        seen = [min(n - q + i + 1, w) for i in range(q)]
        pairs += sum(seen)
        kv += min(n, w + q - 1) if q else 0
    return {"bytes": 4 * sum(qs) * hq * hd + kv * hkv * 2 * (hd // 2 + 4), "flops": 4 * pairs * hq * hd}


def _hadamard_matrix(n):
    i = torch.arange(n, device=DEV)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(n.bit_length())) % 2
    return (1 - 2 * odd).double() / math.sqrt(n)


def _exact_w8a8(st):
    c = st["case"]
    if c["quantised"]:
        qa, sa = st["codes_A"].double(), st["scales_A"].double()
    else:
        y = st["X"].double()
        if c["g"]:
            y = (y.reshape(-1, c["g"]) @ _hadamard_matrix(c["g"])).reshape(c["T"], c["D"])
        sa = y.abs().amax(dim=1) / 127
        qa = torch.round(torch.nan_to_num(y / sa[:, None]))
    return (qa @ st["codes_W"].double().t()) * sa[:, None] * st["scales_W"].double()


def _exact_append(st):
    c = st["case"]
    T, hd, rd = c["T"], c["hd"], c["rope_dim"]
    H = _hadamard_matrix(hd) if c["rotate"] else torch.eye(hd, dtype=torch.float64, device=DEV)
    out = []
    for name, heads, norm in (("Q", c["hq"], st["q_norm"]), ("K", c["hkv"], st["k_norm"]), ("V", c["hkv"], None)):
        x = st[name].double().reshape(T, heads, hd)
        if norm is not None:
            x = x / (x.square().mean(dim=-1, keepdim=True) + EPS).sqrt() * norm.double()
        if rd and name != "V":
            # the same rotation as complex numbers
            turn = torch.complex(*(t.double() for t in st["rope"][st["positions"].long()].chunk(2, dim=-1)))[:, None]
            if c["interleaved"]:
                z = torch.complex(x[..., 0:rd:2], x[..., 1:rd:2]) * turn
                head = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * turn
                head = torch.cat([z.real, z.imag], dim=-1)
            x = torch.cat([head, x[..., rd:]], dim=-1)
        y = x @ H
        if name != "Q":
            scale = y.abs().amax(dim=-1, keepdim=True) / 7
            y = torch.round(torch.nan_to_num(y / scale)) * scale
            y = y * (st["slots"] >= 0)[:, None, None]
        out.append(y.reshape(T, -1))
    return out


def _exact_attention(st):
    c = st["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    qs, ls = _lengths(c)
    H = _hadamard_matrix(hd) if c["rotate"] else torch.eye(hd, dtype=torch.float64, device=DEV)
    out, at = torch.zeros(sum(qs), hq, hd, dtype=torch.float64, device=DEV), 0
    for b, (q, n) in enumerate(zip(qs, ls)):
        if q == 0:
            continue
        k, v = (_cached(st, x, slice(b, b + 1))[0, :, :n].double() for x in "kv")
        back = torch.arange(n - q, n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        hidden = (back < 0) | (back >= (c["window"] or n + 1))
        x = st["Q"][at:at + q].double().reshape(q, hq, hd)
        for h in range(hq):
            s = (x[:, h] @ k[h * hkv // hq].t()) / math.sqrt(hd)
            out[at:at + q, h] = torch.softmax(s.masked_fill(hidden, -math.inf), dim=-1) @ v[h * hkv // hq] @ H
        at += q
    return out.reshape(sum(qs), hq * hd)


def exact(case, seed):
    st = prepare(case, seed)
    return {"w8a8": _exact_w8a8, "append": _exact_append, "attention": _exact_attention}[case["op"]](st)

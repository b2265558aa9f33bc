"""Cases, plain forms and 64-bit values of the 4-bit floating-point product and of masked attention over the 4-bit cache.

Three operators of a decoder layer that is served with drafted tokens and a bounded context:

* ``fp4``: rows of bf16 activations, rotated by a block Hadamard (or not), become E2M1 codes with one scale a block of
  channels (``mx``: 32 channels, a power of two; ``nv``: 16 channels, an E4M3 number, and one factor a tensor); the codes are
  multiplied with weights held the same way.
* ``tree``: attention of a tree of drafted tokens over the paged 4-bit cache: each new token sees the sequence so far and
  those new tokens that its mask lists (its ancestors and itself).
* ``sinks``: causal attention over the same cache through a sliding window, with a few first tokens that stay visible.

``run`` computes the operators from elementary torch operations in 32 bits; where ``own`` is true it makes the calls of
``rotation_int4_w4a4_b200.pq`` instead.  ``exact`` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False
DEV = "cuda"
BLOCK = {"mx": 32, "nv": 16}
TINY = 2.0 ** -100          # a block whose largest magnitude is below this counts as zero


# ---------------------------------------------------------------------------------------------- cases
def _fp4(name, T, N, D, g, fmt, out, quantised):
    """quantised: the activations' codes are in hand (the product alone); otherwise bf16 rows come in."""
    return {"name": name, "op": "fp4", "T": T, "N": N, "D": D, "g": g, "fmt": fmt, "out": out, "quantised": quantised}


def _attend(name, op, B, q, ctx, ragged, hq, hkv, hd, page, window, sinks, rotate):
    """B sequences of up to q new tokens over up to ctx cached ones (the new ones among them)."""
    return {"name": name, "op": op, "B": B, "q": q, "ctx": ctx, "ragged": ragged, "hq": hq, "hkv": hkv, "hd": hd,
            "page": page, "window": window, "sinks": sinks, "rotate": rotate}


def listed():
    return [
        # One token through a 4096 x 4096 projection: generation for one user, where latency counts.
        _fp4("fp4 linear 1 token", 1, 4096, 4096, 128, "nv", "bf16", False),
        # A decode batch through the up projection of the LLaMA-3-8B shape.
        _fp4("fp4 linear 64 tokens", 64, 14336, 4096, 128, "mx", "bf16", False),
        # Odd sizes: a short prompt, a head of 1003 outputs, a reduction that fills no whole tile.
        _fp4("fp4 product odd sizes", 391, 1003, 4192, 0, "nv", "f32", True),
        # A prompt of 2048 tokens through the query projection of the LLaMA-3-8B shape.
        _fp4("fp4 linear 2048 tokens", 2048, 4096, 4096, 64, "mx", "bf16", False),
        # The down projection of the LLaMA-3-8B shape over a long prompt.
        _fp4("fp4 linear down projection", 8192, 4096, 14336, 128, "nv", "bf16", False),
        # One user, a short context, a tree of 8 drafted tokens: the smallest verification step.
        _attend("tree 8 drafts over 1029", "tree", 1, 8, 1029, False, 32, 8, 128, 64, 0, 0, True),
        # A verification step of 16 users over ragged contexts, some of them empty, with trees of up to 61 drafts.
        _attend("tree 16 users 61 drafts", "tree", 16, 61, 8192, True, 32, 8, 128, 64, 0, 0, True),
        # Heads of 64 in groups of 7, trees under a window with sinks.
        _attend("tree window and sinks", "tree", 5, 25, 2999, True, 14, 2, 64, 16, 512, 4, False),
        # One user, a long conversation through a window with sinks: the smallest step of that kind.
        _attend("sinks 1 token over 65536", "sinks", 1, 1, 65536, False, 32, 8, 128, 64, 4096, 4, True),
        # A decode batch over ragged contexts, some of them empty.
        _attend("sinks 64 users ragged", "sinks", 64, 1, 8192, True, 32, 8, 128, 64, 1024, 100, True),
        # Ragged chunks of prompts over earlier context, heads of 64 in groups of 7.
        _attend("sinks ragged chunks", "sinks", 6, 801, 2999, True, 14, 2, 64, 16, 700, 5, False),
        # The second half of a prompt of 8192 tokens.
        _attend("sinks 4096 of 8192 tokens", "sinks", 1, 4096, 8192, False, 32, 8, 128, 64, 2048, 16, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("fp4", "fp4", "tree", "tree", "sinks", "sinks"))
    if op == "fp4":
        g = rng.choice((0, 64, 128, 256))
        T, N = _log(rng, 1, 8192), _log(rng, 16, 14336)
        D = 256 * _log(rng, 1, 56) if g else 32 * _log(rng, 4, 448)
        c = _fp4("", T, N, D, g, rng.choice(("mx", "nv")), rng.choice(("bf16", "f32")), False)
        c["quantised"] = c["out"] == "f32"   # f32 outputs: the product alone, from codes in hand
        c["g"] = 0 if c["quantised"] else g
    else:
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 4, 5, 7, 8)) if hkv < 8 else 32
        ctx = _log(rng, 1, 32768)
        if op == "tree":
            q = min(ctx, _log(rng, 2, 128))
            window, sinks = rng.choice(((0, 0), (0, 0), (_log(rng, 128, 8192), _log(rng, 1, 128))))
        else:
            q = min(ctx, rng.choice((1, 1, _log(rng, 2, 32), _log(rng, 33, 2048))))
            window, sinks = _log(rng, 1, 8192), _log(rng, 1, 256)
        B = _log(rng, 1, max(1, min(64, (1 << 19) // ctx, (1 << 29) // (ctx * q * hq) if q > 1 else 64)))
        c = _attend("", op, B, q, ctx, rng.random() < 0.7, hq, hkv, rng.choice((64, 128)), rng.choice((16, 32, 64, 128)),
                    window, sinks, rng.random() < 0.7)
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
        qs.append(min(n, q if q == 1 else r.randint(1, q)))
        ls.append(n)
    return qs, ls


def _trees(case):
    """Of each sequence's new tokens, the tokens each sees (bit j: new token j) as numbers, from the case alone: a token's
    parent is any one before it (most often a near one), or the sequence itself."""
    r = random.Random(case["B"] * 7919 + case["q"] * 104729 + case["ctx"])
    trees = []
    for q in _lengths(case)[0]:
        seen = []
        for i in range(q):
            parent = max(-1, i - 1 - int(r.expovariate(0.3)))
            seen.append((1 << i) | (seen[parent] if parent >= 0 else 0))
        trees.append(seen)
    return trees


# --------------------------------------------------------------------------------------------- inputs
def _generator(seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return gen


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32)


def _place_scales(s):
    """Scale bytes [rows][blocks] in the order in which the product takes them: pieces of 128 rows and 4 blocks, in each
    the rows 32 apart side by side."""
    rows, blocks = s.shape
    R, C = -(-rows // 128), -(-blocks // 4)
    out = torch.zeros(R * 128, C * 4, dtype=torch.uint8, device=s.device)
    out[:rows, :blocks] = s
    return out.reshape(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _scale_bytes(rows, blocks):
    return -(-rows // 128) * -(-blocks // 4) * 512


def _prepare_fp4(case, seed):
    gen = _generator(seed)
    T, N, D, fmt = case["T"], case["N"], case["D"], case["fmt"]
    x = _normal(gen, T, D)
    x[:, torch.randperm(D, generator=gen, device=DEV)[:8]] *= 30.0   # outlier channels, as activations have them
    st = {"X": x.to(torch.bfloat16), "factor_A": 1.0, "factor_W": 1.0}
    w = _normal(gen, N, D) * 0.02
    if fmt == "nv":                                  # factors of the tensors, as a calibration leaves them
        st["factor_A"] = float(torch.tensor(128.0 / (6 * 448), dtype=torch.float32))
        st["factor_W"] = float(torch.tensor(0.12 / (6 * 448), dtype=torch.float32))
    if case["quantised"]:
        st["codes_A"], s = _quantise(st["X"].float(), fmt, 1.0, st["factor_A"])
        st["scales_A"] = _place_scales(s)
    else:                                            # written by the call
        st["codes_A"] = torch.empty(T, D // 2, dtype=torch.uint8, device=DEV)
        st["scales_A"] = torch.empty(_scale_bytes(T, D // BLOCK[fmt]), dtype=torch.uint8, device=DEV)
    st["codes_W"], s = _quantise(w, fmt, 1.0, st["factor_W"])
    st["scales_W"] = _place_scales(s)
    st["Y"] = torch.empty(T, N, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=DEV)
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
          "max_q": max(qs), "max_len": max(ls), "tree": None, "keep": {}}
    if case["op"] == "tree":
        words = -(-max(qs) // 32)
        bits = [[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for seen in _trees(case) for m in seen]
        st["tree"] = torch.tensor([[b - (1 << 32) if b >> 31 else b for b in row] for row in bits], dtype=torch.int32, device=DEV)
    for kv in "kv":
        y = _normal(gen, pages, hkv, page, hd)
        m = y.abs().amax(dim=-1)
        u = torch.round(y * (7 / m)[..., None]).to(torch.int32) & 15
        st[kv + "_codes"] = (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8)
        st[kv + "_scales"] = m / 7
    return st


def prepare(case, seed):
    st = (_prepare_fp4 if case["op"] == "fp4" else _prepare_attention)(case, seed)
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


def _quantise(y, fmt, unit, factor):
    """Codes (two a byte) and scale bytes [rows][blocks] of rows y * unit / factor, in float32."""
    T, D = y.shape
    v = y.reshape(T, -1, BLOCK[fmt])
    m = v.abs().amax(dim=-1)
    u = torch.tensor(unit, dtype=torch.float32, device=y.device)
    if fmt == "mx":                                  # 2^(floor(log2 largest) - 2): the largest lies in 4..8, and 6 is the top
        m = m * u
        e = (torch.frexp(m).exponent - 3).clamp(-127, 127)
        live = m >= TINY
        scale = torch.where(live, e + 127, torch.zeros_like(e)).to(torch.uint8)
        f = torch.where(live, u * torch.exp2(-e.float()), torch.zeros_like(m))
    else:
        r = m * torch.tensor(unit / (6 * factor), dtype=torch.float32, device=y.device)
        e4m3 = r.clamp(max=448).to(torch.float8_e4m3fn)
        scale, s = e4m3.view(torch.uint8), e4m3.float()
        f = torch.where(s > 0, torch.tensor(unit / factor, dtype=torch.float32, device=y.device) / s, torch.zeros_like(s))
    v = v * f[..., None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.int32) | torch.where(v < 0, 8, 0)
    code = code.reshape(T, D)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), scale


def _values(codes, scales, fmt, T, D, dtype):
    """The numbers that codes and placed scales stand for (without the tensor's factor)."""
    blocks = D // BLOCK[fmt]
    R, C = -(-T // 128), -(-blocks // 4)
    s = scales[:R * C * 512].reshape(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)[:T, :blocks]
    s = torch.exp2(s.to(dtype) - 127) if fmt == "mx" else s.contiguous().view(torch.float8_e4m3fn).to(dtype)
    c = codes.to(torch.int32)
    c = torch.stack([c & 15, c >> 4], dim=-1).reshape(T, D)
    k = (c & 7).to(dtype)
    a = torch.where(k < 4, k / 2, torch.where(k < 6, k - 2, 2 * k - 8))
    return (torch.where(c > 7, -a, a).reshape(T, blocks, -1) * s[..., None]).reshape(T, D)


def _plain_fp4(st):
    c = st["case"]
    T, N, D, fmt, g = c["T"], c["N"], c["D"], c["fmt"], c["g"]
    if c["quantised"]:
        a = _values(st["codes_A"], st["scales_A"], fmt, T, D, torch.float32)
    else:
        y = st["X"].float()
        if g:
            y = _hadamard_tree(y.reshape(T, -1, g)).reshape(T, D)
        codes, s = _quantise(y, fmt, 1 / math.sqrt(g) if g else 1.0, st["factor_A"])
        a = _values(codes, _place_scales(s), fmt, T, D, torch.float32)
    w = _values(st["codes_W"], st["scales_W"], fmt, N, D, torch.float32)
    return ((a @ w.t()) * (st["factor_A"] * st["factor_W"])).to(st["Y"].dtype)


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
    before = lens - (start[1:] - start[:-1])                         # tokens cached before the new ones
    t = torch.arange(n, device=DEV)
    if st["tree"] is None:
        place = before[:, None] + i                                  # position of each new token
        seen = t[None, None, :] <= place[..., None]
        if c["window"]:
            seen &= (t[None, None, :] > place[..., None] - c["window"]) | (t < c["sinks"])
    else:
        bits = torch.cat([st["tree"], torch.zeros_like(st["tree"][:1])])[row]          # [B][q][words]
        bits = ((bits[..., None] >> torch.arange(32, device=DEV)) & 1).flatten(-2)      # [B][q][32 words]
        place = before[:, None] + bits.sum(dim=-1) - 1               # a drafted token lies behind its ancestors
        old = t[None, None, :] < before[:, None, None]
        if c["window"]:
            old = old & ((t[None, None, :] > place[..., None] - c["window"]) | (t < c["sinks"]))
        j = t[None, :] - before[:, None]                             # [B][n], new token
        new = torch.gather(bits, 2, j.clamp(0, bits.shape[-1] - 1)[:, None, :].expand(B, q, n)) > 0
        seen = old | (new & ((j >= 0) & (t < lens[:, None]))[:, None, :])
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
    if c["op"] == "fp4":
        if c["quantised"]:
            pq.pq_fp4_gemm(st["codes_A"], st["scales_A"], st["codes_W"], st["scales_W"], st["Y"], fmt=c["fmt"],
                           alpha=st["factor_A"] * st["factor_W"])
        else:
            pq.pq_fp4_linear(st["X"], st["codes_A"], st["scales_A"], st["codes_W"], st["scales_W"], st["Y"], fmt=c["fmt"],
                             g=c["g"], factor_A=st["factor_A"], factor_W=st["factor_W"])
        return st["Y"]
    pq.pq_kv4_attention_masked(_own_cache(st, pq), st["Q"], st["O"], st["q_start"], st["seq_lens"], st["table"],
                               max_q=st["max_q"], max_len=st["max_len"], scale=1 / math.sqrt(c["hd"]), window=c["window"],
                               sinks=c["sinks"], tree=st["tree"])
    return st["O"]


def run(state):
    if own:
        return _own_run(state)
    return _plain_fp4(state) if state["case"]["op"] == "fp4" else _plain_attention(state)


# ------------------------------------------------------------------------------------ work and values
def work(case):
    if case["op"] == "fp4":
        T, N, D, b = case["T"], case["N"], case["D"], BLOCK[case["fmt"]]
        rows = T * (D // 2 + D // b) if case["quantised"] else 2 * T * D
        return {"bytes": rows + N * (D // 2 + D // b) + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * D}
    hq, hkv, hd, W, S = case["hq"], case["hkv"], case["hd"], case["window"], case["sinks"]
    qs, ls = _lengths(case)
    trees = _trees(case) if case["op"] == "tree" else [None] * len(qs)
    pairs = kv = 0
    for q, n, tree in zip(qs, ls, trees):
        far = n                                                      # the first token inside any row's window
        for i in range(q):
            new = bin(tree[i]).count("1") if tree else i + 1
            lo = max(0, n - q + new - W) if W else 0                 # a row's window begins here
            far = min(far, lo)
            pairs += max(0, n - q - lo) + min(new, W or new) if tree is None else max(0, n - q - lo) + new
            pairs += min(S, lo, n - q + (new if tree is None else 0))
        kv += n - far + min(S, far) if q else 0
    return {"bytes": 4 * sum(qs) * hq * hd + kv * hkv * 2 * (hd // 2 + 4), "flops": 4 * pairs * hq * hd}


def _hadamard_matrix(n):
    i = torch.arange(n, device=DEV)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> k) & 1 for k in range(n.bit_length())) % 2
    return (1 - 2 * odd).double() / math.sqrt(n)


def _exact_rows(x, fmt, factor):
    """What rows x / factor are rounded to: of each block, the scale and then every channel, in 64 bits."""
    v = x.reshape(x.shape[0], -1, BLOCK[fmt]) / factor
    m = v.abs().amax(dim=-1, keepdim=True)
    if fmt == "mx":
        s = torch.exp2(torch.floor(torch.log2(m)) - 2)
    else:                                            # E4M3: 3 bits behind the leading one, down to 2^-9, up to 448
        r = m / 6
        unit = torch.exp2(torch.floor(torch.log2(r)).clamp(min=-6) - 3)
        s = (torch.round(r / unit) * unit).clamp(max=448)
    z = torch.nan_to_num(v / s, nan=0.0, posinf=0.0, neginf=0.0)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    i = torch.bucketize(z.abs().contiguous(), (grid[:-1] + grid[1:]) / 2)             # a border goes to the lower neighbour
    half = torch.cat([(grid[:-1] + grid[1:]) / 2, grid.new_full((1,), math.inf)])
    i = i + ((z.abs() == half[i]) & (i % 2 == 1)).long()                              # .. and to the even one
    return (torch.sign(z) * grid[i] * s).reshape(x.shape)


def _exact_fp4(st):
    c = st["case"]
    T, N, D, fmt = c["T"], c["N"], c["D"], c["fmt"]
    if c["quantised"]:
        a = _values(st["codes_A"], st["scales_A"], fmt, T, D, torch.float64)
    else:
        a = st["X"].double()
        if c["g"]:
            a = (a.reshape(-1, c["g"]) @ _hadamard_matrix(c["g"])).reshape(T, D)
        a = _exact_rows(a, fmt, st["factor_A"])
    w = _values(st["codes_W"], st["scales_W"], fmt, N, D, torch.float64)
    return (a @ w.t()) * (st["factor_A"] * st["factor_W"])


def _exact_attention(st):
    c = st["case"]
    hq, hkv, hd, W = c["hq"], c["hkv"], c["hd"], c["window"]
    qs, ls = _lengths(c)
    trees = _trees(c) if c["op"] == "tree" else [None] * len(qs)
    H = _hadamard_matrix(hd) if c["rotate"] else torch.eye(hd, dtype=torch.float64, device=DEV)
    out, at = torch.zeros(sum(qs), hq, hd, dtype=torch.float64, device=DEV), 0
    for b, (q, n, tree) in enumerate(zip(qs, ls, trees)):
        if q == 0:
            continue
        k, v = (_cached(st, x, slice(b, b + 1))[0, :, :n].double() for x in "kv")
        t = torch.arange(n, device=DEV)[None, :]
        if tree:
            among = torch.tensor([[(m >> j) & 1 for j in range(q)] for m in tree], dtype=torch.bool, device=DEV)
            depth = among.sum(dim=1)[:, None]
            hidden = t > n - q - 1
            if W:
                hidden = hidden | ((t >= c["sinks"]) & (n - q + depth - 1 - t >= W))
            hidden = hidden.expand(q, n).clone()
            hidden[:, n - q:] = ~among
        else:
            back = torch.arange(n - q, n, device=DEV)[:, None] - t
            hidden = (back < 0) | ((back >= (W or n + 1)) & (t >= c["sinks"]))
        x = st["Q"][at:at + q].double().reshape(q, hq, hd)
        for h in range(hq):
            s = (x[:, h] @ k[h * hkv // hq].t()) / math.sqrt(hd)
            out[at:at + q, h] = torch.softmax(s.masked_fill(hidden, -math.inf), dim=-1) @ v[h * hkv // hq] @ H
        at += q
    return out.reshape(sum(qs), hq * hd)


def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_fp4 if case["op"] == "fp4" else _exact_attention)(st)

"""Cases that measure alpha-entmax attention with a sliding window, and the 4-bit key/value cache with
the attention that reads it.

Three kinds of case:
  window   training attention in which query i sees key j when j <= i and (i - j < window or j < sinks):
           O = P V, P the alpha-entmax of the visible scores, and dQ, dK, dV for a given dO;
  append   new keys and values quantised to 4 bits into a paged cache, and the rows just written read back;
  read     a stretch of every sequence of the cache read back as values;
  decode   queries of the newest tokens against the cache, with the same window and sinks.

With ``own`` false `run` computes them from elementary operations, with ``own`` true by the package's calls.

The cache holds, for each token and key/value head, d/2 bytes of codes and d/32 pairs (scale, zero) of
bfloat16, one pair for each 32 consecutive dimensions:
    zero  = bf16(min x),   scale = bf16((max x - zero) / 15)  (0 where max x <= zero),
    code  = round_half_even((x - zero) / scale) clamped to [0, 15]  (0 where scale = 0),
    value = zero + scale * code.
The 4-byte word (c, w) of a token's codes, at index c * (d/32) + w for c = 0..3, holds the dimensions
32 w + 8 c + i in its bits 4 i .. 4 i + 3.  Arrays are [page][head][token of the page][...].
"""
import math

import numpy as np
import torch

own = False

GROUP = 32


# ------------------------------------------------------------------ cases
def _window(name, B, H, N, d, dtype, alpha, window, sinks, beta):
    return dict(kind="window", name=name, B=B, H=H, N=N, d=d, dtype=dtype, alpha=alpha, window=window,
                sinks=sinks, beta=beta)


def _cache(kind, name, B, Hkv, d, page, longest, n, dtype):
    return dict(kind=kind, name=name, B=B, Hkv=Hkv, d=d, page=page, longest=longest, n=n, dtype=dtype)


def _decode(name, B, Hq, Hkv, d, page, longest, L, dtype, alpha, window, sinks, beta):
    return dict(kind="decode", name=name, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, longest=longest, L=L,
                dtype=dtype, alpha=alpha, window=window, sinks=sinks, beta=beta)


def listed():
    return [
        # one float32 head pair of odd length: a unit-sized training step
        _window("window f32 257", 1, 2, 257, 64, "f32", 1.5, 64, 4, 1.0),
        # the language-model step of the benchmark, with a window of a quarter of the sequence
        _window("window lm 2048", 8, 12, 2048, 64, "bf16", 1.5, 512, 4, 1.0),
        # a long document under a window, wide heads
        _window("window long 8192", 1, 16, 8192, 128, "bf16", 1.5, 1024, 16, 2.0),
        # an odd length and a window that is no multiple of a tile, no sinks, denser weights
        _window("window ragged 1000", 2, 12, 1000, 128, "bf16", 1.25, 200, 0, 4.0),
        # a serving step's writes: one new token for each of 32 sequences
        _cache("append", "append one token", 32, 8, 128, 64, 4096, 1, "bf16"),
        # prompts of unequal length, written at once
        _cache("append", "append prompts", 4, 8, 128, 64, 4096, 4096, "bf16"),
        # a shared prefix looked at in float32
        _cache("read", "read short f32", 2, 4, 64, 16, 700, 333, "f32"),
        # whole sequences taken back to bf16, as before a recomputation
        _cache("read", "read whole", 8, 8, 128, 64, 8192, 8192, "bf16"),
        # one short sequence, as many key heads as query heads: latency
        _decode("decode one short", 1, 12, 12, 64, 16, 200, 1, "bf16", 1.5, 0, 0, 1.0),
        # a batch of ordinary length, grouped heads
        _decode("decode batch 4096", 16, 32, 8, 128, 64, 4096, 1, "bf16", 1.5, 0, 0, 2.0),
        # a few tokens at once (a draft to be checked), float32, window and sinks, sparsemax
        _decode("decode draft window", 4, 16, 2, 64, 32, 6000, 5, "f32", 2.0, 1000, 4, 1.0),
        # the largest: a full batch of long sequences
        _decode("decode batch 32768", 16, 32, 8, 128, 64, 32768, 1, "bf16", 1.5, 0, 0, 1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["window", "append", "read", "decode", "decode"])
    d = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "window":
        # the float32 path is for small models: a tenth of the largest case's work
        N = _log_int(rng, 16, 8192 if dtype == "bf16" else 2048)
        heads = max(1, min(96, (1 << 30) // (N * N) if dtype == "bf16" else (1 << 24) // (N * N)))
        B = _log_int(rng, 1, min(8, heads))
        H = _log_int(rng, 1, max(1, min(16, heads // B)))
        return dict(kind=kind, B=B, H=H, N=N, d=d, dtype=dtype, alpha=rng.choice([1.25, 1.5]),
                    window=_log_int(rng, 1, N if N < 2048 else 1024), sinks=rng.choice([0, 1, 4, 16, 130]),
                    beta=rng.choice([1.0, 2.0, 4.0]))
    Hkv = rng.choice([1, 2, 4, 8, 12])
    page = rng.choice([16, 32, 64, 128])
    B = _log_int(rng, 1, 32)
    # at most as many cached values as the largest listed case
    top = max(64, (16 * 8 * 128 * 32768) // (B * Hkv * d * (8 if kind != "decode" else 1)))
    longest = _log_int(rng, 20, min(100000, top))
    if kind in ("append", "read"):
        n = rng.choice([1, _log_int(rng, 1, longest), _log_int(rng, 1, longest)])
        return dict(kind=kind, B=B, Hkv=Hkv, d=d, page=page, longest=longest, n=n, dtype=dtype)
    L = rng.choice([1, 1, 2, 3, 5, 8])
    window = rng.choice([0, 0, _log_int(rng, 1, longest)])
    return dict(kind=kind, B=B, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, d=d, page=page, longest=longest, L=L,
                dtype=dtype, alpha=rng.choice([1.25, 1.5, 2.0]), window=window,
                sinks=rng.choice([0, 1, 4, 16]) if window else 0, beta=rng.choice([1.0, 2.0]))


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _quantise(x):
    """x [..., d] to (codes uint8 [..., d/2], meta bf16 [..., d/32, 2]) by the rule above, in 64 bits."""
    g = x.double().unflatten(-1, (-1, GROUP))
    zero = g.amin(-1).float().to(torch.bfloat16)
    z = zero.double()
    top = g.amax(-1)
    scale = torch.where(top > z, (top - z) / 15, torch.zeros_like(z)).float().to(torch.bfloat16)
    s = scale.double()
    q = torch.where(s[..., None] > 0, (g - z[..., None]) / s[..., None], torch.zeros_like(g))
    code = q.round().clamp(0, 15).to(torch.uint8)                      # [..., w, 32]
    code = code.unflatten(-1, (4, 4, 2)).transpose(-4, -3)             # [..., c, w, byte, nibble]
    return (code[..., 0] | code[..., 1] << 4).flatten(-3), torch.stack((scale, zero), -1)


def _values(codes, meta):
    """The float32 values that codes and meta stand for."""
    w = meta.shape[-2]
    both = torch.stack((codes & 15, codes >> 4), -1).float()           # [..., d/2, 2]
    both = both.flatten(-2).unflatten(-1, (4, w, 8)).transpose(-3, -2).flatten(-2)   # [..., w, 32]
    m = meta.float()
    return (m[..., 1:] + m[..., :1] * both).flatten(-2)


def _kv(gen, shape, H):
    """Keys or values: normal, with channels of unequal spread and a mean of their own, as projections give."""
    d = shape[-1]
    spread = torch.exp(0.3 * torch.randn(H, 1, d, generator=gen, device="cuda"))
    mean = 0.3 * torch.randn(H, 1, d, generator=gen, device="cuda")
    x = torch.randn(shape, generator=gen, device="cuda")
    return x * (spread / spread.square().mean(-1, keepdim=True).sqrt()) + mean


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _dtype(case)
    if case["kind"] == "window":
        shape = (case["B"], case["H"], case["N"], case["d"])
        q, k, v, do = (torch.randn(shape, generator=gen, device="cuda") for _ in range(4))
        q, k, v = (x.to(t).requires_grad_() for x in (q * case["beta"], k, v))
        return dict(case=case, q=q, k=k, v=v, do=do.to(t))
    B, Hkv, d, page, longest = (case[n] for n in ("B", "Hkv", "d", "page", "longest"))
    L = case["n"] if case["kind"] != "decode" else case["L"]
    # sequences of unequal length, the first of them the longest; new_lens rows of each are real
    whole = torch.randint(max(1, longest // 2), longest + 1, (B,), generator=gen, device="cuda")
    whole[0] = longest
    new_lens = torch.randint(max(1, L // 2), L + 1, (B,), generator=gen, device="cuda")
    new_lens[0] = L
    new_lens = torch.minimum(new_lens, whole)
    if case["kind"] == "read":
        start = (torch.rand(B, generator=gen, device="cuda") * (whole - new_lens + 1)).long()
    else:
        start = whole - new_lens
    pages = -(-longest // page)
    order = torch.randperm(B * pages + 3, generator=gen, device="cuda")[:B * pages]
    block_table = order.view(B, pages).to(torch.int32)
    state = dict(case=case, start=start.to(torch.int32), new_lens=new_lens.to(torch.int32), block_table=block_table)
    # the cache as earlier steps left it (for an append: other values, to be written over)
    buffers = []
    for _ in "kv":
        x = _kv(gen, (B * pages + 3, Hkv, page, d), Hkv)
        chunks = [_quantise(c) for c in x.split(max(1, (1 << 25) // (Hkv * page * d)))]
        buffers += [torch.cat([c[0] for c in chunks]), torch.cat([c[1] for c in chunks])]
        del x, chunks
    state["cache"] = tuple(buffers)                                     # k_codes, k_meta, v_codes, v_meta
    if case["kind"] == "append":
        state["k"], state["v"] = (_kv(gen, (B, Hkv, L, d), Hkv).to(t) for _ in "kv")
    if case["kind"] == "decode":
        state["q"] = (case["beta"] * torch.randn(B, case["Hq"], L, d, generator=gen, device="cuda")).to(t)
    return state


# ------------------------------------------------------------------ the plain form
def _entmax(x, gamma):
    """(p, u) of p = u^gamma, u = (x - tau)_+, with sum p = 1 over the last axis (nothing where every x is -inf).

    Newton's steps from max - 1, where the sum is at least one: it is convex and falls with tau, so every step
    stays below the root; 24 take the slowest case (gamma 4, 1e5 equal scores) to the last bit."""
    x = x - x.amax(-1, keepdim=True)
    x = torch.where(x.isnan(), -math.inf, x)
    tau = torch.full_like(x[..., :1], -1.0)
    for _ in range(24):
        u = (x - tau).clamp_min(0)
        g = u.pow(gamma - 1) if gamma != 1 else (u > 0).float()
        f = (g * u).sum(-1, keepdim=True) - 1
        tau = tau + f / (gamma * g.sum(-1, keepdim=True)).clamp_min(1e-30)
        tau = tau.clamp(-1, 0)
    u = (x - tau).clamp_min(0)
    u = torch.where(x > -math.inf, u, 0)
    return u.pow(gamma), u


def _plain_window(s):
    c = s["case"]
    q, k, v, do = (s[n].detach().float() for n in ("q", "k", "v", "do"))
    i = torch.arange(c["N"], device=q.device)
    back = i[:, None] - i[None, :]
    seen = (back >= 0) & ((back < c["window"]) | (i[None, :] < c["sinks"]))
    scale, gamma = 1 / math.sqrt(c["d"]), 1 / (c["alpha"] - 1)
    x = (q @ k.transpose(-1, -2)) * ((c["alpha"] - 1) * scale)
    p, u = _entmax(x.masked_fill_(~seen, -math.inf), gamma)
    del x
    o = p @ v
    dv = p.transpose(-1, -2) @ do
    del p
    g = u.pow_(gamma - 1)
    dp = do @ v.transpose(-1, -2)
    dp -= (g * dp).sum(-1, keepdim=True) / g.sum(-1, keepdim=True)
    ds = g.mul_(dp)
    dq, dk = ds @ k * scale, ds.transpose(-1, -2) @ q * scale
    return [y.to(_dtype(c)) for y in (o, dq, dk, dv)]


def _rows(s, n):
    """(page, row in the page, whether it is there) of positions start .. start + n - 1 of every sequence."""
    off = torch.arange(n, device=s["start"].device)
    at = s["start"].long()[:, None] + off
    there = off < s["new_lens"][:, None]
    page = s["case"]["page"]
    at = torch.where(there, at, 0)
    return s["block_table"].long().gather(1, at // page), at % page, there


def _plain_read(s, n, dtype):
    pages, rows, there = _rows(s, n)
    out = []
    for codes, meta in (s["cache"][:2], s["cache"][2:]):
        x = _values(codes[pages, :, rows], meta[pages, :, rows])        # [B, n, H, d]
        out.append(torch.where(there[..., None, None], x, 0).transpose(1, 2).to(dtype))
    return out


def _plain_append(s):
    pages, rows, there = _rows(s, s["case"]["n"])
    for x, codes, meta in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
        c, m = _quantise(x.transpose(1, 2)[there])
        codes[pages[there], :, rows[there]] = c
        meta[pages[there], :, rows[there]] = m
    return _plain_read(s, s["case"]["n"], torch.float32)


def _plain_decode(s):
    c = s["case"]
    B, Hq, L, d = s["q"].shape
    group = Hq // c["Hkv"]
    table = s["block_table"].long()
    k, v = (_values(codes[table], meta[table]).transpose(1, 2).flatten(2, 3)
            for codes, meta in (s["cache"][:2], s["cache"][2:]))        # [B, Hkv, n, d]
    j = torch.arange(k.shape[2], device=k.device)
    row = torch.arange(L, device=k.device)
    pos = s["start"].long()[:, None] + row
    back = pos[:, :, None] - j                                          # [B, L, n]
    seen = (back >= 0) & (row < s["new_lens"][:, None])[:, :, None]
    if c["window"]:
        seen &= (back < c["window"]) | (j < c["sinks"])
    q = s["q"].float().view(B, c["Hkv"], group, L, d).flatten(2, 3)
    x = (q @ k.transpose(-1, -2)) * ((c["alpha"] - 1) / math.sqrt(d))
    x = x.view(B, c["Hkv"], group, L, -1).masked_fill_(~seen[:, None, None], -math.inf)
    p, _ = _entmax(x, 1 / (c["alpha"] - 1))
    return (p.flatten(2, 3) @ v).view(B, Hq, L, d).to(_dtype(c))


def run(state):
    c = state["case"]
    kind = c["kind"]
    if own:
        import adaptive_sparse_flash_entmax_b200 as ent
        if kind == "window":
            q, k, v = state["q"], state["k"], state["v"]
            o = ent.entmax_attention(q, k, v, c["alpha"], True, window=c["window"], sinks=c["sinks"])
            return [o.detach(), *torch.autograd.grad(o, (q, k, v), state["do"])]
        cache, table, start, new_lens = (state[n] for n in ("cache", "block_table", "start", "new_lens"))
        if kind == "append":
            ent.kv4_write(cache, state["k"], state["v"], table, start, new_lens)
            return list(ent.kv4_read(cache, table, start, c["n"], new_lens, dtype=torch.float32))
        if kind == "read":
            return list(ent.kv4_read(cache, table, start, c["n"], new_lens, dtype=_dtype(c)))
        return ent.entmax_attn_kv4(state["q"], cache, table, start, c["alpha"], new_lens=new_lens,
                                   window=c["window"] or None, sinks=c["sinks"])
    if kind == "window":
        return _plain_window(state)
    if kind == "append":
        return _plain_append(state)
    if kind == "read":
        return _plain_read(state, c["n"], _dtype(c))
    return _plain_decode(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _support(n, alpha, spread):
    """Keys with a weight among n whose scores are normal with that spread (a bisection on the mean of u^gamma)."""
    gamma = 1 / (alpha - 1)
    step = 0.02
    z = [i * step for i in range(-300, 301)]
    pdf = [math.exp(-t * t / 2) / math.sqrt(2 * math.pi) * step for t in z]
    sd = (alpha - 1) * spread
    lo, hi = -6.0, 6.0
    for _ in range(30):
        mid = (lo + hi) / 2
        total = n * sum(w * (sd * (t - mid)) ** gamma for t, w in zip(z, pdf) if t > mid)
        lo, hi = (mid, hi) if total > 1 else (lo, mid)
    return max(1.0, min(n, n * 0.5 * math.erfc(lo / math.sqrt(2))))


def work(case):
    d = case["d"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["kind"] == "window":
        heads, N, W, S = case["B"] * case["H"], case["N"], min(case["window"], case["N"]), min(case["sinks"], case["N"])
        pairs = W * N - W * (W - 1) // 2                                # the window's
        pairs += sum(max(0, min(S, i + 1 - W)) for i in range(N))      # sinks that lie before it
        # q, k, v, dO in, O, dQ, dK, dV out; six products of every visible pair: S, P V, dP, dQ, dK, dV
        return {"bytes": heads * N * d * 8 * size, "flops": heads * pairs * d * 12}
    B, Hkv = case["B"], case["Hkv"]
    row = d // 2 + d // GROUP * 4                                       # one token's codes and pairs, keys or values
    mean = 0.75 * case["longest"]                                       # lengths lie between half and whole
    if case["kind"] in ("append", "read"):
        rows = B * Hkv * case["n"] * (0.75 if case["n"] > 1 else 1)
        if case["kind"] == "append":
            return {"bytes": 2 * rows * (d * size + row + d * 4), "flops": 2 * rows * d * 6}
        return {"bytes": 2 * rows * (row + d * size), "flops": 2 * rows * d * 2}
    L, group = case["L"], case["Hq"] // Hkv
    n = min(mean, case["window"] + case["sinks"] + L - 1) if case["window"] else mean
    sup = _support(max(1, int(n)), case["alpha"], case["beta"])
    # every visible key; of the values only the rows that some query of the group weighs
    read = B * Hkv * (n + min(n, sup * group * L)) * row
    return {"bytes": read + 2 * B * case["Hq"] * L * d * size, "flops": 2 * B * case["Hq"] * L * d * (n + sup)}


# ------------------------------------------------------------------ the definition in 64 bits
def _bisect(x, gamma):
    """u = (x - tau)_+ with sum u^gamma = 1, for every row of x, by halving [max - 1, max]."""
    m = x.max(-1, keepdim=True).values
    some = m > -math.inf
    hi = torch.where(some, m, torch.zeros_like(m))
    lo = hi - 1
    for _ in range(54):
        mid = (lo + hi) / 2
        over = torch.relu(x - mid).pow(gamma).sum(-1, keepdim=True) > 1
        lo, hi = torch.where(over, mid, lo), torch.where(over, hi, mid)
    return torch.relu(x - (lo + hi) / 2) * some


def _exact_window(case, s):
    N, W, S, alpha, d = (case[n] for n in ("N", "window", "sinks", "alpha", "d"))
    gamma = 1 / (alpha - 1)
    i = torch.arange(N, device="cuda").view(-1, 1)
    j = i.view(1, -1)
    hidden = (j > i) | ((j <= i - W) & (j >= S))
    outs = [torch.empty(s["q"].shape, dtype=torch.float64, device="cuda") for _ in range(4)]
    for b in range(case["B"]):
        for h in range(case["H"]):
            q, k, v, do = (s[n][b, h].detach().double() for n in ("q", "k", "v", "do"))
            x = torch.einsum("id,jd->ij", q, k) * (alpha - 1) / d ** 0.5
            u = _bisect(x.masked_fill(hidden, -math.inf), gamma)
            p, g = u ** gamma, torch.where(u > 0, u ** (gamma - 1), 0)
            dp = torch.einsum("id,jd->ij", do, v)
            ds = g * (dp - (g * dp).sum(1, keepdim=True) / g.sum(1, keepdim=True)) / d ** 0.5
            for o, a in zip(outs, (p @ v, ds @ k, ds.T @ q, p.T @ do)):
                o[b, h] = a
    return outs


def _bf16(x):
    """float64 array to the nearest bfloat16 by way of float32, as float64 (ties to even bits)."""
    bits = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def _exact_cache(case, s):
    """What a read gives: of rows just written the quantised inputs, else the stored values."""
    B, H, d, n, page = (case[k] for k in ("B", "Hkv", "d", "n", "page"))
    start, lens, table = (s[k].cpu().numpy() for k in ("start", "new_lens", "block_table"))
    outs = []
    for which, x in enumerate((s.get("k"), s.get("v"))):
        out = np.zeros((B, H, n, d))
        if case["kind"] == "append":
            x = x.double().cpu().numpy().reshape(B, H, n, d // GROUP, GROUP)
            z = _bf16(x.min(-1, keepdims=True))
            step = _bf16(np.maximum(x.max(-1, keepdims=True) - z, 0) / 15)
            c = np.clip(np.rint((x - z) / np.where(step > 0, step, 1)), 0, 15) * (step > 0)
            full = (z + step * c).reshape(B, H, n, d)
            for b in range(B):
                out[b, :, :lens[b]] = full[b, :, :lens[b]]
        else:
            codes, meta = s["cache"][2 * which].cpu().numpy(), s["cache"][2 * which + 1].double().cpu().numpy()
            for b in range(B):
                at = start[b] + np.arange(lens[b])
                out[b, :, :lens[b]] = _unpack(codes, meta, table[b, at // page], at % page)
        outs.append(torch.from_numpy(out))
    return outs


def _unpack(codes, meta, pages, rows):
    """[heads, len(rows), d] values of those rows, dimension by dimension."""
    c, m = codes[pages, :, rows], meta[pages, :, rows]                  # [rows, H, d/2], [rows, H, w, 2]
    w = m.shape[2]
    out = np.empty((c.shape[1], c.shape[0], w * GROUP))
    for dim in range(w * GROUP):
        g, r = divmod(dim, GROUP)
        quarter, i = divmod(r, 8)
        byte = c[:, :, 4 * (quarter * w + g) + i // 2]
        out[:, :, dim] = (m[:, :, g, 1] + m[:, :, g, 0] * ((byte >> (4 * (i % 2))) & 15)).T
    return out


def _exact_decode(case, s):
    Hq, Hkv, L, d, page, alpha = (case[k] for k in ("Hq", "Hkv", "L", "d", "page", "alpha"))
    gamma, group = 1 / (alpha - 1), Hq // Hkv
    k_codes, k_meta, v_codes, v_meta = s["cache"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    w = d // GROUP
    # where dimension dim of a token lies: byte, and shift in it
    dim = torch.arange(d, device="cuda")
    byte = 4 * ((dim % GROUP) // 8 * w + dim // GROUP) + dim % 8 // 2
    shift = (4 * (dim % 2)).to(torch.uint8)

    def take(codes, meta, pages, rows):                                 # [n, Hkv, d]
        c = (codes[pages, :, rows][..., byte] >> shift) & 15
        m = meta[pages, :, rows][:, :, dim // GROUP].double()
        return m[..., 1] + m[..., 0] * c.double()
    for b in range(case["B"]):
        for r in range(int(s["new_lens"][b])):
            pos = int(s["start"][b]) + r
            at = torch.arange(pos + 1, device="cuda")
            if case["window"]:
                at = at[(at > pos - case["window"]) | (at < case["sinks"])]
            pages, rows = s["block_table"][b].long()[at // page], at % page
            k, v = take(k_codes, k_meta, pages, rows), take(v_codes, v_meta, pages, rows)
            q = s["q"][b, :, r].double().view(Hkv, group, d)
            x = torch.einsum("hgd,nhd->hgn", q, k) * (alpha - 1) / d ** 0.5
            o[b, :, r] = torch.einsum("hgn,nhd->hgd", _bisect(x, gamma) ** gamma, v).reshape(Hq, d)
    return o


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "window":
        return _exact_window(case, s)
    return _exact_decode(case, s) if case["kind"] == "decode" else _exact_cache(case, s)

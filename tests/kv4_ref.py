"""64-bit restatement of the 4-bit cache and its attention (test infrastructure).

The error bound of the attention, from the kernel's arithmetic (float sums, exact codes):
scores.  A score is off by at most delta = cx * (d/16 + 24) * 2^-23 * sum_c |q_c| (|zero| + 16 scale): the
    product's partial sums are of that size at most and each addition rounds by at most 2^-23 of them
    (one per 16 dimensions in the tensor cores, six per group after them); a float32 q is held as two
    halves, within 2^-22 of it.
tau.  It moves by at most the largest score error (tau is monotone and shifts with the scores), so
    u_j moves by at most 2 delta and sum_j |dp_j| <= 2 delta gamma sum_j (u_j + 2 delta)^(gamma-1) over the
    keys with u_j > -2 delta.  The solver stops at |f| <= 2e-7 or a step of 6e-8 (f moves by gamma F1 times
    that) and sees f within its own rounding, (n/128 + 16) 2^-24 for a sum of n terms that totals one.
O.  The p above times |v|, plus the rounding of the sum over the support (n + 16) 2^-24 sum p |v|, plus
    half a step of the output's type.
"""
import math

import numpy as np
import torch

GROUP = 32


def bf16_rne(x):
    return torch.as_tensor(x).float().to(torch.bfloat16)


def quantise(x):
    """x [..., d] (any float dtype) to integer codes [..., d], scale and zero bf16 [..., d/32]."""
    g = x.double().unflatten(-1, (-1, GROUP))
    fine = torch.isfinite(g).all(-1)
    safe = torch.where(fine[..., None], g, torch.zeros_like(g))
    zero = bf16_rne(safe.amin(-1))
    fine = fine & torch.isfinite(zero.double())
    z = torch.where(fine, zero.double(), torch.zeros_like(zero.double()))
    safe = torch.where(fine[..., None], safe, torch.zeros_like(g))
    rng = safe.amax(-1) - z
    scale = bf16_rne(torch.where(rng > 0, rng / 15, torch.zeros_like(rng)))
    s = scale.double()[..., None]
    q = torch.where(s > 0, (safe - z[..., None]) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    codes = q.round().clamp(0, 15).to(torch.uint8)
    scale = torch.where(fine, scale, torch.zeros_like(scale))
    zero = torch.where(fine, zero, torch.full_like(zero, math.nan))
    return codes.flatten(-2), scale, zero


def unpack(codes):
    """Stored bytes [..., d/2] to integer codes [..., d], dimension by dimension as documented."""
    c = codes.cpu().numpy()
    d = 2 * c.shape[-1]
    w = d // GROUP
    out = np.empty(c.shape[:-1] + (d,), np.uint8)
    for dim in range(d):
        g, r = divmod(dim, GROUP)
        quarter, i = divmod(r, 8)
        out[..., dim] = (c[..., 4 * (quarter * w + g) + i // 2] >> (4 * (i % 2))) & 15
    return torch.from_numpy(out)


def values(codes, meta):
    """float64 values of stored codes [..., d/2] and meta [..., d/32, 2]."""
    m = meta.cpu().double()
    c = unpack(codes).double().unflatten(-1, (-1, GROUP))
    return (m[..., 1:] + m[..., :1] * c).flatten(-2)


def sequence(codes, meta, table, n, page):
    """float64 values [n, heads, d] of a sequence's first n tokens; a row of a missing page is None's NaN."""
    pages = codes.shape[0]
    heads, d = codes.shape[1], 2 * codes.shape[3]
    out = torch.full((n, heads, d), math.nan, dtype=torch.float64)
    there = torch.zeros(n, dtype=torch.bool)
    for p in range(-(-n // page)):
        t = int(table[p])
        if not 0 <= t < pages:
            continue
        rows = min(page, n - p * page)
        out[p * page:p * page + rows] = values(codes[t, :, :rows], meta[t, :, :rows]).transpose(0, 1)
        there[p * page:p * page + rows] = True
    return out, there


def solve(x, gamma):
    """u = (x - tau)_+ of one row (float64, finite), sum u^gamma = 1."""
    hi = float(x.max())
    lo = hi - 1
    for _ in range(60):
        mid = (lo + hi) / 2
        if float(torch.relu(x - mid).pow(gamma).sum()) > 1:
            lo = mid
        else:
            hi = mid
    return (lo + hi) / 2


def attend(q, cache, table, start, new_lens, alpha, window, sinks, page, half_step, q_parts=1):
    """(o, tau, bound) float64 [B, Hq, L, d], [B, Hq, L] and the largest admissible |error| of o, tau's."""
    kc, km, vc, vm = (t.cpu() for t in cache)
    q = q.cpu().double()
    B, Hq, L, d = q.shape
    Hkv = kc.shape[1]
    gamma = 1 / (float(np.float32(alpha)) - 1)
    cx = (float(np.float32(alpha)) - 1) / math.sqrt(d)
    o, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    tau, tau_bound = torch.zeros((B, Hq, L), dtype=torch.float64), torch.zeros((B, Hq, L), dtype=torch.float64)
    for b in range(B):
        for l in range(int(new_lens[b])):
            pos = int(start[b]) + l
            k, there = sequence(kc, km, table[b], pos + 1, page)
            v, _ = sequence(vc, vm, table[b], pos + 1, page)
            j = torch.arange(pos + 1)
            seen = there & ((j > pos - window) | (j < sinks) if window else torch.ones(pos + 1, dtype=torch.bool))
            if not bool(seen.any()):
                continue
            k, v, n = k[seen], v[seen], int(seen.sum())
            size = torch.zeros_like(k)   # |zero| + 16 scale of each value's group, from the values' own pairs
            idx = j[seen]
            for p in range(int(idx.max()) // page + 1):
                on = idx // page == p
                if bool(on.any()):
                    m = km[int(table[b][p])][:, (idx[on] % page)].double().transpose(0, 1)
                    size[on] = (m[..., 1].abs() + 16 * m[..., 0]).repeat_interleave(GROUP, -1)
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                row = q[b, h, l]
                x = cx * (k[:, hk] @ row)
                t = solve(x, gamma)
                u = torch.relu(x - t)
                p = u ** gamma
                o[b, h, l] = p @ v[:, hk]
                tau[b, h, l] = t
                delta = float(cx * (d / 16 + 24 + (4 if q_parts > 1 else 0)) * 2.0 ** -23
                              * (size[:, hk] @ row.abs()).max())
                near = x - t > -2 * delta
                f1 = float((torch.relu(x - t) + 2 * delta)[near].pow(gamma - 1).sum())
                dp = 2 * delta * gamma * f1 + 2e-7 + 6e-8 * gamma * f1 + (n / 128 + 16) * 2.0 ** -24
                vmax = v[:, hk][near].abs().amax(0)
                vsum = p @ v[:, hk].abs()
                bound[b, h, l] = dp * vmax + ((int((p > 0).sum()) + 16) * 2.0 ** -24) * vsum
                bound[b, h, l] += half_step * (o[b, h, l].abs() + bound[b, h, l])
                tau_bound[b, h, l] = delta + dp / max(gamma * float((u ** (gamma - 1) * (u > 0)).sum()), 1e-30) \
                    + 2.0 ** -23 * (abs(t) + 1)
    return o, tau, bound, tau_bound

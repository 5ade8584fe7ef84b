"""Windowed attention with sinks on the GPU against the definition in 64 bits.

Tolerances.  float32: those of the float32 path (1e-4 on O); its gradients are float sums of terms with tau off by
at most 1e-6: 1e-4 relative (2-norm).  bfloat16: on each element of O, P rounded once (2^-8 of sum p |v|), the
forward's own bound |sum p - 1| <= 1e-4 (times max |v|), and the output's rounding (2^-8 |o|); on gradients, two
roundings of 2^-8 at most on each term (the operand P or dS, and the output) and 2e-3 for tau and delta: 1e-2
relative (2-norm)."""
import pytest
import torch

from adaptive_sparse_flash_entmax_b200 import attention as A
from adaptive_sparse_flash_entmax_b200 import entmax_attention

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GRAD = {"f32": 1e-4, "bf16": 1e-2}


def visible(N, window, sinks):
    i = torch.arange(N, device="cuda")
    back = i[:, None] - i[None, :]
    return (back >= 0) & ((back < window) | (i[None, :] < sinks))


def forward64(q, k, v, alpha, window, sinks):
    """(o, p, u) in float64."""
    gamma = 1 / (alpha - 1)
    x = (alpha - 1) * (q @ k.transpose(-1, -2)) / q.shape[-1] ** 0.5
    x = x.masked_fill(~visible(q.shape[-2], window, sinks), float("-inf"))
    hi = x.amax(-1, keepdim=True)
    lo = hi - 1
    for _ in range(56):
        mid = (lo + hi) / 2
        up = torch.relu(x - mid).pow(gamma).sum(-1, keepdim=True) > 1
        lo, hi = torch.where(up, mid, lo), torch.where(up, hi, mid)
    u = torch.relu(x - (lo + hi) / 2)
    p = u ** gamma
    return p @ v, p, u


def reference(q, k, v, do, alpha, window, sinks):
    q, k, v, do = (t.double() for t in (q, k, v, do))
    gamma, scale = 1 / (alpha - 1), q.shape[-1] ** -0.5
    o, p, u = forward64(q, k, v, alpha, window, sinks)
    g = torch.where(u > 0, u ** (gamma - 1), torch.zeros_like(u))
    dp = do @ v.transpose(-1, -2)
    ds = g * (dp - (g * dp).sum(-1, keepdim=True) / g.sum(-1, keepdim=True))
    return o, ds @ k * scale, ds.transpose(-1, -2) @ q * scale, p.transpose(-1, -2) @ do, p @ v.abs()


def make(B, H, N, d, dtype, seed, beta=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(B, H, N, d, generator=g, device="cuda") for _ in range(4))
    return [t.to(DT[dtype]) for t in (beta * q, k, v, do)]


def check(got, want, dtype, v, grads=("dq", "dk", "dv")):
    o, pv = want[0], want[4]
    err = (got[0].double() - o).abs()
    if dtype == "f32":
        tol = torch.full_like(o, 1e-4)
    else:
        tol = 2.0 ** -8 * pv + 1e-4 * v.double().abs().amax() + 1e-5
        tol = tol + 2.0 ** -8 * (o.abs() + tol)
    assert bool((err <= tol).all()), f"o off by {float((err - tol).max()):.3g} too much"
    for name, a, b in zip(("dq", "dk", "dv"), got[1:], want[1:4]):
        if name not in grads:
            continue
        norm = float(b.norm())
        rel = float((a.double() - b).norm()) / norm if norm else float(a.double().norm())
        assert rel <= GRAD[dtype], f"{name} off by {rel:.3g}"


def grads_of(q, k, v, do, alpha, window, sinks, delta):
    q, k, v = (t.clone().requires_grad_() for t in (q, k, v))
    o = entmax_attention(q, k, v, alpha, True, delta, window, sinks)
    return [o.detach(), *torch.autograd.grad(o, (q, k, v), do)]


SHAPES = [  # B, H, N, d, window, sinks
    (1, 1, 1, 64, 1, 0),
    (2, 1, 5, 32, 2, 1),
    (1, 2, 127, 64, 64, 0),
    (1, 2, 128, 128, 127, 4),
    (2, 2, 129, 64, 128, 1),
    (1, 3, 300, 128, 129, 16),
    (1, 2, 515, 64, 1, 0),
    (1, 2, 515, 64, 3, 130),
    (1, 2, 515, 32, 200, 300),
    (1, 1, 700, 128, 1, 700),
    (1, 2, 900, 64, 256, 4),
    (1, 1, 900, 128, 5000, 3),
    (1, 1, 1500, 64, 1400, 200),   # a float32 window near the largest that shared memory takes, and one past it
    (1, 1, 1700, 128, 1500, 64),
]


@pytest.mark.parametrize("delta", ["otilde", "recompute"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,N,d,window,sinks", SHAPES)
def test_forward_and_gradients(B, H, N, d, window, sinks, dtype, delta):
    q, k, v, do = make(B, H, N, d, dtype, N + window)
    got = grads_of(q, k, v, do, 1.5, window, sinks, delta)
    # a row that sees one key has a constant output: dq is rounding there (dS = 0 for every row when window 1, no sinks)
    check(got, reference(q, k, v, do, 1.5, window, sinks), dtype, v,
          ("dv",) if window == 1 and sinks == 0 else ("dq", "dk", "dv"))
    if window == 1 and sinks == 0:
        # o = p v with the one p: in bfloat16 it is 1 (|p - 1| <= 1e-4 rounds to 1); in float32 it stops at
        # |p - 1| <= 1e-6 or a step of 4e-7 max(1, |tau|), twice that in p, plus 2^-23 |tau| for u = x - tau, |tau| < 6
        off = 0 if dtype == "bf16" else 6 * (2 * 4e-7 + 2.0 ** -22)
        assert bool(((got[0].double() - v.double()).abs() <= off * v.double().abs()).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("alpha", [1.25, 4 / 3, 1.7, 2.0])
def test_alphas(alpha, dtype):
    q, k, v, do = make(1, 2, 400, 64, dtype, 3)
    got = grads_of(q, k, v, do, alpha, 150, 8, "otilde")
    # from gamma = 1/(alpha-1) < 1.5 on, g = u^(gamma-1) jumps or is steep at the border of the support, where the
    # rounding of a score decides it: dq and dk are held to the formula for the others
    check(got, reference(q, k, v, do, alpha, 150, 8), dtype, v, ("dv",) if alpha > 1.6 else ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype,N", [("f32", 450), ("f32", 1700), ("bf16", 450)])
def test_a_window_over_everything_is_causal_attention(dtype, N, monkeypatch):
    """Bit for bit where the kernels are the same (bfloat16 from the same start of the solver, and float32 windows
    beyond shared memory); a short float32 window has kernels of its own, and each route is within the path's
    bounds of the definition."""
    monkeypatch.setenv("ENTATTN_CALIB", "0")
    q, k, v, do = make(1, 2, N, 64, dtype, 4)
    o, tau, mask, _ = A.entmax_attn_fwd(q, k, v, 1.5, True)
    ow, tw, mw, _ = A.entmax_attn_fwd(q, k, v, 1.5, True, window=10 ** 12, sinks=7)
    grads = A.entmax_attn_bwd(q, k, v, o, do, tau, mask, 1.5, True)
    gradw = A.entmax_attn_bwd(q, k, v, None, do, tw, mw, 1.5, True, window=N, sinks=7)
    if (dtype, N) == ("f32", 450):
        assert float((o - ow).abs().max()) <= 2e-4 and float((tau - tw).abs().max()) <= 2e-4
        assert all(float((a - b).norm()) <= 2 * GRAD["f32"] * float(a.norm()) for a, b in zip(grads, gradw))
    else:
        assert torch.equal(o, ow) and torch.equal(tau, tw) and torch.equal(mask, mw)
        assert all(torch.equal(a, b) for a, b in zip(grads, gradw))


def test_block_mask_and_work_stay_inside():
    """No block outside the window or the sinks is live or visited."""
    N, W, S = 2000, 256, 3
    q, k, v, _ = make(1, 2, N, 64, "bf16", 5)
    ws = A.workspace(1 << 24, q.device)
    _, _, mask, _ = A.entmax_attn_fwd(q, k, v, 1.5, True, window=W, sinks=S, ws=ws)
    T = mask.shape[-1]
    seen = torch.nn.functional.pad(visible(N, W, S), (0, T * 128 - N, 0, T * 128 - N)).view(T, 128, T, 128).any(3).any(1)
    assert not bool(mask[:, :, ~seen].any())
    assert bool(mask[:, :, torch.arange(T), torch.arange(T)].all())
    visited, passes = A.read_status(ws)[0], A.read_status(ws)[2]
    assert visited <= int(seen.sum()) * 2 * 26 and passes >= 2 * T


def test_against_differences():
    """The gradients against central differences of the 64-bit forward (its error is eps^2 and 1e-16 / eps)."""
    q, k, v, do = make(1, 1, 140, 32, "f32", 6, beta=1.0)
    got = grads_of(q, k, v, do, 1.5, 20, 2, "recompute")
    base = [t.double() for t in (q, k, v)]
    g = torch.Generator(device="cuda").manual_seed(7)
    for n in range(3):
        for _ in range(4):
            step = torch.randn(base[n].shape, generator=g, device="cuda", dtype=torch.float64)
            eps = 1e-5
            ends = []
            for s in (eps, -eps):
                moved = list(base)
                moved[n] = base[n] + s * step
                ends.append(float((forward64(*moved, 1.5, 20, 2)[0] * do.double()).sum()))
            want = (ends[0] - ends[1]) / (2 * eps)
            have = float((got[1 + n].double() * step).sum())
            # f's second derivative jumps where a key enters the support (eps of them in reach): 1e-4 of the terms
            assert abs(have - want) <= 2e-4 * float((got[1 + n].double() * step).norm()) * 10


def test_graph_stream_and_repeats():
    q, k, v, do = make(1, 2, 600, 64, "bf16", 8)
    first = grads_of(q, k, v, do, 1.5, 200, 4, "otilde")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = grads_of(q, k, v, do, 1.5, 200, 4, "otilde")
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    ot = torch.empty(q.shape, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, tau, mask, _ = A.entmax_attn_fwd(q, k, v, 1.5, True, otilde=ot, window=200, sinks=4)
        outs = [o, *A.entmax_attn_bwd(q, k, v, None, do, tau, mask, 1.5, True, otilde=ot, window=200, sinks=4)]
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    new = make(1, 2, 600, 64, "bf16", 9)
    for t, n in zip((q, k, v, do), new):
        t.copy_(n)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(grads_of(*new, 1.5, 200, 4, "otilde"), outs))


def test_long_window():
    """Over 64 tiles, where full attention would calibrate its start and bound its blocks: sampled rows."""
    N, W, S = 9001, 700, 5
    q, k, v, _ = make(1, 1, N, 64, "bf16", 10)
    o = entmax_attention(q, k, v, 1.5, True, window=W, sinks=S)[0, 0]
    seen = visible(N, W, S)
    for i in (0, 1, 699, 700, 705, 4500, 8192, 9000):
        kk, vv = k[0, 0][seen[i]].double(), v[0, 0][seen[i]].double()
        x = 0.5 * (kk @ q[0, 0, i].double()) / 8
        hi = x.max()
        lo = hi - 1
        for _ in range(56):
            mid = (lo + hi) / 2
            lo, hi = (mid, hi) if float(torch.relu(x - mid).square().sum()) > 1 else (lo, mid)
        p = torch.relu(x - lo).square()
        want = p @ vv
        tol = 2.0 ** -8 * (p @ vv.abs()) + 1e-4 * vv.abs().max() + 1e-5
        assert bool(((o[i].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


@pytest.mark.parametrize("alpha,beta", [(1.5, 1.0), (1.5, 4.0)])
def test_a_bfloat16_window_over_everything_has_all_that_causal_attention_has(alpha, beta):
    """Over 64 tiles, where the bound pass skips blocks and the start is calibrated: the same bits and the same work,
    forward and backward; one key less is a window."""
    N = 8400
    q, k, v, do = make(1, 1, N, 64, "bf16", 11, beta)
    ws = A.workspace(1 << 26, q.device)
    runs = []
    for kw in ({}, dict(window=N, sinks=3), dict(window=10 ** 12), dict(window=N - 1)):
        o, tau, mask, _ = A.entmax_attn_fwd(q, k, v, alpha, True, ws=ws, **kw)
        work = A.read_status(ws)
        runs.append((work[0], o, tau, mask, *A.entmax_attn_bwd(q, k, v, o, do, tau, mask, alpha, True, **kw)))
    for other in runs[1:3]:
        assert other[0] == runs[0][0] and all(torch.equal(a, b) for a, b in zip(other[1:], runs[0][1:]))
    assert runs[3][0] != runs[0][0]


@pytest.mark.parametrize("kw", [{}, dict(window=64, sinks=2), dict(window=1700, sinks=3)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_query_that_is_no_number(bad, dtype, kw):
    """It has no weights: zeros in O and dQ, tau not finite, by every kernel and with either delta; the other rows'
    O and dQ keep their bits."""
    N, r = 1750, 900
    q, k, v, do = make(1, 2, N, 64, dtype, 12)
    ot = torch.empty(q.shape, device="cuda")

    def both(q):
        o, tau, mask, _ = A.entmax_attn_fwd(q, k, v, 1.5, True, otilde=ot, **kw)
        dq = A.entmax_attn_bwd(q, k, v, None, do, tau, mask, 1.5, True, otilde=ot, **kw)[0]
        return o, dq, A.entmax_attn_bwd(q, k, v, o, do, tau, mask, 1.5, True, **kw)[0], tau

    clean = both(q)
    spoilt = q.clone()
    spoilt[0, 1, r, 7] = bad
    got = both(spoilt)
    assert not bool(torch.isfinite(got[3][0, 1, r]))
    for a, b in zip(got[:3], clean[:3]):
        assert not bool(a[0, 1, r].any())      # (a NaN is true)
        a[0, 1, r] = b[0, 1, r]
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,most", [(32, 1584), (64, 1392), (128, 1072)])
@pytest.mark.parametrize("sinks", [0, 130])
def test_both_sides_of_the_shared_memory_border(d, most, sinks):
    """The largest float32 window whose scores fit in shared memory and the next one; the counters tell the routes
    apart (the general kernels visit their blocks again in every pass)."""
    N = most + 270
    q, k, v, do = make(1, 1, N, d, "f32", 13)
    for window, general in ((most - sinks, False), (most + 1 - sinks, True)):
        ws = A.workspace(1 << 22, q.device)
        A.entmax_attn_fwd(q, k, v, 1.5, True, window=window, sinks=sinks, ws=ws)
        visited, weighed, passes, _ = A.read_status(ws)[:4]
        assert passes > 0 and (visited > weighed) == general
        want = reference(q, k, v, do, 1.5, window, sinks)
        for delta in ("otilde", "recompute"):
            check(grads_of(q, k, v, do, 1.5, window, sinks, delta), want, "f32", v)


@pytest.mark.parametrize("dtype,window,sinks", [("f32", 600, 130), ("f32", 1500, 4), ("bf16", 600, 130),
                                                ("bf16", 1500, 4), ("bf16", 4299, 0)])
def test_gradients_over_many_tiles(dtype, window, sinks):
    """34 query tiles: more than dkv looks at in one step."""
    q, k, v, do = make(1, 1, 4300, 64, dtype, 14)
    want = reference(q, k, v, do, 1.5, window, sinks)
    for delta in ("otilde", "recompute"):
        check(grads_of(q, k, v, do, 1.5, window, sinks, delta), want, dtype, v)


@pytest.mark.parametrize("delta", ["otilde", "recompute"])
@pytest.mark.parametrize("dtype,N,window,sinks", [("f32", 400, 150, 8), ("f32", 1700, 1500, 4), ("bf16", 400, 150, 8),
                                                  ("bf16", 900, 257, 130)])
@pytest.mark.parametrize("alpha", [1.7, 2.0])
def test_gradients_where_g_is_steep(alpha, dtype, N, window, sinks, delta):
    """alpha above 1.6: g = u^(gamma-1) jumps or is steep at the border of the support, so a key whose score lies
    within its rounding of tau may be in or out.  The formula is taken at the kernel's own tau, and rows with such a
    key get dO = 0, which leaves dS = 0 whatever g is: the others are held to the bounds of the smooth case.  A
    score's rounding: sums of d products in float, 2^-24 of sum |q k| for each (the tensor core's truncation twice
    that), and a rounding of x and of tau."""
    B, H, d = 1, 2, 64
    q, k, v, do = make(B, H, N, d, dtype, 15)
    ot = torch.empty(q.shape, device="cuda") if delta == "otilde" else None
    o, tau, mask, _ = A.entmax_attn_fwd(q, k, v, alpha, True, otilde=ot, window=window, sinks=sinks)
    q6, k6, v6 = (t.double() for t in (q, k, v))
    gamma, scale, seen = 1 / (alpha - 1), d ** -0.5, visible(N, window, sinks)
    x = (alpha - 1) * scale * (q6 @ k6.transpose(-1, -2))
    u = x - tau.double()[..., None]
    off = 2 * d * 2.0 ** -24 * (alpha - 1) * scale * (q6.abs() @ k6.abs().transpose(-1, -2))
    off = off + 2.0 ** -23 * (x.abs() + tau.double().abs()[..., None])
    unsure = ((u.abs() <= off) & seen).any(-1)
    assert float(unsure.double().mean()) < 0.1
    do = do.masked_fill(unsure[..., None], 0)
    u = torch.where(seen, u, -1.0).clamp_min(0)
    g = torch.where(u > 0, u ** (gamma - 1), 0.0)
    dp = do.double() @ v6.transpose(-1, -2)
    ds = g * (dp - (g * dp).sum(-1, keepdim=True) / g.sum(-1, keepdim=True)) * scale
    got = A.entmax_attn_bwd(q, k, v, None if delta == "otilde" else o, do, tau, mask, alpha, True, otilde=ot,
                            window=window, sinks=sinks)
    want = (ds @ k6, ds.transpose(-1, -2) @ q6, (u ** gamma).transpose(-1, -2) @ do.double())
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= GRAD[dtype], f"{name} off by {rel:.3g}"


@pytest.mark.parametrize("delta", ["otilde", "recompute"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_visible_key_has_no_gradient_of_scores(dtype, delta):
    """window 1: dS = g (dP - delta) with dP = delta but for rounding, d products of 2^-22 of sum |dO v| at most
    (g = 1 within 1e-4), and dQ and dK are that times one key or query."""
    q, k, v, do = make(1, 2, 515, 64, dtype, 16)
    got = grads_of(q, k, v, do, 1.5, 1, 0, delta)
    ds = 64 * 2.0 ** -22 * (do.double().abs() * v.double().abs()).sum(-1, keepdim=True) * 64 ** -0.5 * 1.01
    assert bool((got[1].double().abs() <= ds * k.double().abs()).all())
    assert bool((got[2].double().abs() <= ds * q.double().abs()).all())


@pytest.mark.parametrize("d", [64, 128])
def test_work_grows_with_the_window_not_with_the_sequence(d):
    """A pass of a tile visits its visible blocks and at most the two of a job that was started early."""
    N, W, S = 4000, 256, 3
    q, k, v, _ = make(1, 2, N, d, "bf16", 17)
    ws = A.workspace(1 << 24, q.device)
    A.entmax_attn_fwd(q, k, v, 1.5, True, window=W, sinks=S, ws=ws)
    visited, _, passes, tiles = A.read_status(ws)[:4]
    assert tiles == 2 * 32 and visited <= (passes + tiles) * (4 + 2)
    A.entmax_attn_fwd(q, k, v, 1.5, True, ws=ws)
    assert A.read_status(ws)[0] > 2 * visited


@pytest.mark.parametrize("N,d,window,sinks,alpha", [(2000, 64, 512, 4, 1.5), (1500, 128, 300, 130, 1.25),
                                                    (9000, 64, 700, 0, 1.5)])
@pytest.mark.parametrize("otilde", [False, True])
def test_tiles_solved_again(N, d, window, sinks, alpha, otilde, monkeypatch):
    """With a tolerance that every unevaluated stop misses, tiles are solved again by whichever CTA is free: the bits
    of evaluated stops."""
    q, k, v, _ = make(1, 3, N, d, "bf16", 18)
    runs = []
    for name, value in (("ENTATTN_VERIFY_TOL", "-1"), ("ENTATTN_ACCEPT", "0")):
        with monkeypatch.context() as m:
            m.setenv(name, value)
            ws = A.workspace(1 << 26, q.device)
            ot = torch.empty(q.shape, device="cuda") if otilde else None
            out = A.entmax_attn_fwd(q, k, v, alpha, True, with_iters=True, otilde=ot, window=window, sinks=sinks, ws=ws)
            runs.append((A.read_status(ws)[3], *out, *([ot] if otilde else [])))
    assert runs[0][0] > runs[1][0] == 3 * -(-N // 128)
    assert all(torch.equal(a, b) for a, b in zip(runs[0][1:], runs[1][1:]))


@pytest.mark.parametrize("delta", ["otilde", "recompute"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("alpha,N,d", [(1.25, 24, 32), (1.5, 515, 64), (2.0, 300, 128)])
def test_one_visible_key_exactly(alpha, N, d, dtype, delta):
    """window 1 without sinks: dQ and dK are zeros, dV is dO but for p's own error (test_forward_and_gradients)."""
    q, k, v, do = make(2, 3, N, d, dtype, 19, beta=4.0)
    _, dq, dk, dv = grads_of(q, k, v, do, alpha, 1, 0, delta)
    assert not bool(dq.any()) and not bool(dk.any())
    assert float((dv.double() - do.double()).norm()) <= GRAD[dtype] * float(do.double().norm())


@pytest.mark.parametrize("B,H,N,d,window,sinks,alpha,beta", [(1, 8, 24, 128, 10, 0, 1.5, 4.0), (2, 8, 30, 64, 12, 2, 1.5, 4.0),
                                                             (1, 8, 257, 64, 64, 4, 1.5, 1.0), (1, 8, 300, 32, 90, 4, 1.25, 2.0)])
def test_float32_is_as_near_as_float_scores(B, H, N, d, window, sinks, alpha, beta):
    """O's error (2-norm) is that of the exact entmax of float32 scores and at most 5e-7 beside it: |sum p - 1| <= 4e-7,
    a factor of a row's p, and two roundings of 2^-24 (p and the sum)."""
    q, k, v, _ = make(B, H, N, d, "f32", 20, beta)
    o = entmax_attention(q, k, v, alpha, True, window=window, sinks=sinks).double()
    want = forward64(q.double(), k.double(), v.double(), alpha, window, sinks)[0]
    assert not torch.backends.cuda.matmul.allow_tf32
    x = ((q @ k.transpose(-1, -2)) * ((alpha - 1) / d ** 0.5)).double().masked_fill(~visible(N, window, sinks), float("-inf"))
    hi = x.amax(-1, keepdim=True)
    lo = hi - 1
    for _ in range(56):
        mid = (lo + hi) / 2
        up = torch.relu(x - mid).pow(1 / (alpha - 1)).sum(-1, keepdim=True) > 1
        lo, hi = torch.where(up, mid, lo), torch.where(up, hi, mid)
    plain = torch.relu(x - (lo + hi) / 2).pow(1 / (alpha - 1)) @ v.double()
    assert float((o - want).norm()) <= float((plain - want).norm()) + 5e-7 * float(want.norm())

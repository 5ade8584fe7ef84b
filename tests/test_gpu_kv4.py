"""The 4-bit key/value cache and the attention over it on the GPU, against a 64-bit restatement
(tests/kv4_ref.py, which derives the tolerances)."""
import math

import pytest
import torch

import kv4_ref
from adaptive_sparse_flash_entmax_b200 import (capi, entmax_attn_fwd, entmax_attn_kv4, kv4_alloc, kv4_read,
                                               kv4_workspace, kv4_write)

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step, relative


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(pages, heads, page, d, gen, dtype=torch.float32):
    """A cache filled through the restated quantiser (not by the kernel under test)."""
    cache = kv4_alloc(pages, heads, page, d, "cuda")
    for codes, meta in (cache[:2], cache[2:]):
        x = torch.randn(pages, heads, page, d, generator=gen) * (1 + torch.rand(heads, 1, d, generator=gen)) \
            + torch.randn(heads, 1, d, generator=gen)
        c, s, z = kv4_ref.quantise(x)
        w = d // 32
        c = c.unflatten(-1, (w, 4, 4, 2)).transpose(-4, -3)
        codes.copy_((c[..., 0] | c[..., 1] << 4).flatten(-3))
        meta.copy_(torch.stack((s, z), -1))
    return cache


def tables(B, max_pages, pages, gen):
    return torch.randperm(pages, generator=gen)[:B * max_pages].view(B, max_pages).to(torch.int32)


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,page,B,H,L,start,lens", [
    (128, 64, 3, 2, 5, [0, 61, 100], [5, 4, 0]),
    (64, 16, 2, 3, 40, [0, 9], [40, 33]),
    (32, 32, 4, 1, 1, [0, 31, 32, 63], None),
    (128, 16, 1, 1, 1, [79], [1]),
])
def test_write_matches_the_rule_exactly(dtype, d, page, B, H, L, start, lens):
    gen = torch.Generator().manual_seed(d + page)
    max_pages = 5
    pages = B * max_pages + 2
    k, v = (torch.randn(B, H, L, d, generator=gen) * torch.exp(torch.randn(B, H, L, 1, generator=gen)) for _ in "kv")
    k[:, :, 0, :32] = torch.randint(-8, 8, (32,), generator=gen).float()   # many exact ties
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    table = tables(B, max_pages, pages, gen)
    cache = pool(pages, H, page, d, gen)
    before = [t.clone() for t in cache]
    bad = i32([0])
    kv4_write(cache, k.cuda(), v.cuda(), table.cuda(), i32(start), None if lens is None else i32(lens), bad=bad)
    torch.cuda.synchronize()
    assert int(bad) == 0
    lens = [L] * B if lens is None else lens
    for x, codes, meta, old_c, old_m in ((k, cache[0], cache[1], before[0], before[1]),
                                         (v, cache[2], cache[3], before[2], before[3])):
        want_c, want_s, want_z = kv4_ref.quantise(x)
        written = torch.zeros(pages, page, dtype=torch.bool)
        for b in range(B):
            for l in range(lens[b]):
                pos = start[b] + l
                p, r = int(table[b, pos // page]), pos % page
                written[p, r] = True
                assert torch.equal(kv4_ref.unpack(codes[p, :, r]), want_c[b, :, l])
                assert torch.equal(meta[p, :, r, :, 0].cpu(), want_s[b, :, l])
                assert torch.equal(meta[p, :, r, :, 1].cpu(), want_z[b, :, l])
        rest = (~written).cuda()
        assert torch.equal(codes.transpose(1, 2)[rest], old_c.transpose(1, 2)[rest])
        assert torch.equal(meta.transpose(1, 2)[rest], old_m.transpose(1, 2)[rest])


def test_write_extreme_values():
    """Constant groups, subnormals, huge ranges, infinities and NaN."""
    gen = torch.Generator().manual_seed(5)
    d, page = 128, 16
    rows = torch.randn(1, 1, 12, d, generator=gen)
    rows[0, 0, 0] = 1.7
    rows[0, 0, 1] = 0
    rows[0, 0, 2] *= 1e-42
    rows[0, 0, 3] *= 1e-37
    rows[0, 0, 4] *= 5e37
    rows[0, 0, 5, ::2] = 3e38
    rows[0, 0, 5, 1::2] = -3e38
    rows[0, 0, 6, 3] = math.inf
    rows[0, 0, 7, 40] = math.nan
    rows[0, 0, 8, 100] = -math.inf
    rows[0, 0, 9, 0] = -3.4028234e38      # rounds to -inf in bf16
    rows[0, 0, 10] = 100 + 1e-3 * rows[0, 0, 10]
    rows[0, 0, 11] = -rows[0, 0, 11].abs()
    cache = kv4_alloc(1, 1, page, d, "cuda")
    zero = i32([0])
    kv4_write(cache, rows.cuda(), rows.cuda(), i32([[0]]), zero)
    k, v = kv4_read(cache, i32([[0]]), zero, 12, dtype=torch.float32)
    c, s, z = kv4_ref.quantise(rows)
    assert torch.equal(kv4_ref.unpack(cache[0][0, 0, :12]), c[0, 0])
    assert torch.equal(cache[1][0, 0, :12, :, 0].cpu().view(torch.int16), s[0, 0].view(torch.int16))
    assert torch.equal(torch.nan_to_num(cache[1][0, 0, :12, :, 1].cpu().float(), nan=9e9),
                       torch.nan_to_num(z[0, 0].float(), nan=9e9))
    assert torch.equal(torch.nan_to_num(k, nan=9e9), torch.nan_to_num(v, nan=9e9))
    nan = torch.isnan(k[0, 0].cpu()).unflatten(-1, (4, 32))
    want = torch.zeros(12, 4, dtype=torch.bool)
    want[6, 0] = want[7, 1] = want[8, 3] = want[9, 0] = True
    assert torch.equal(nan.all(-1), want) and torch.equal(nan.any(-1), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,page,B,H,n,start,lens", [
    (128, 64, 2, 3, 70, [0, 100], [70, 20]),
    (64, 16, 3, 1, 1, [0, 15, 79], None),
    (32, 128, 1, 2, 33, [95], [0]),
])
def test_read(dtype, d, page, B, H, n, start, lens):
    gen = torch.Generator().manual_seed(n)
    max_pages = 5
    cache = pool(B * max_pages + 1, H, page, d, gen)
    table = tables(B, max_pages, B * max_pages + 1, gen)
    got = kv4_read(cache, table.cuda(), i32(start), n, None if lens is None else i32(lens), dtype=DT[dtype])
    lens = [n] * B if lens is None else lens
    for out, codes, meta in zip(got, cache[::2], cache[1::2]):
        out = out.cpu().double()
        for b in range(B):
            want, _ = kv4_ref.sequence(codes.cpu(), meta.cpu(), table[b], start[b] + lens[b], page)
            want = want[start[b]:].transpose(0, 1)
            # one fused multiply-add in float, then the rounding to the output type
            tol = (2.0 ** -24 + (HALF[dtype] if dtype == "bf16" else 0)) * 1.01
            assert bool(((out[b, :, :lens[b]] - want).abs() <= tol * want.abs()).all())
            assert not bool(out[b, :, lens[b]:].any())


# ------------------------------------------------------------------ attention
def check(q, cache, table, start, lens, alpha, window, sinks, page, dtype, **kw):
    B, Hq, L, d = q.shape
    tau = torch.full((B, Hq, L), 7.0, device="cuda")
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got = entmax_attn_kv4(q, cache, table.cuda(), i32(start), alpha, new_lens=None if lens is None else i32(lens),
                          window=window or None, sinks=sinks, out=o, tau=tau, **kw)
    assert got is o
    torch.cuda.synchronize()
    lens = [L] * B if lens is None else lens
    want, want_tau, bound, tau_bound = kv4_ref.attend(q, cache, table, start, lens, alpha, window, sinks, page,
                                                      HALF[dtype], 2 if dtype == "f32" else 1)
    err = (o.cpu().double() - want).abs()
    assert bool((err <= bound).all()), f"o off by {float((err - bound).max()):.3g} more than {float(bound.max()):.3g}"
    terr = (tau.cpu().double() - want_tau).abs()
    assert bool((terr <= tau_bound).all()), f"tau off by {float(terr.max()):.3g}"
    return o


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("alpha", [1.5, 1.25, 2.0, 4 / 3, 1.7])
def test_attention_alphas(dtype, alpha):
    gen = torch.Generator().manual_seed(3)
    cache = pool(12, 2, 32, 64, gen)
    q = (2 * torch.randn(2, 4, 1, 64, generator=gen)).to(DT[dtype]).cuda()
    check(q, cache, tables(2, 5, 12, gen), [149, 70], None, alpha, 0, 0, 32, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,B,Hq,Hkv,L,start,lens,window,sinks", [
    (128, 16, 3, 2, 2, 1, [0, 1, 15], None, 0, 0),               # one, two, sixteen keys
    (128, 64, 2, 8, 1, 1, [511, 512], None, 0, 0),               # a chunk's end, and one past it
    (64, 32, 2, 10, 2, 3, [600, 37], [3, 2], 0, 0),              # 15 rows of a key head
    (128, 16, 2, 4, 1, 5, [300, 0], [5, 5], 0, 0),               # 20 rows, a prompt of five
    (32, 64, 2, 12, 4, 9, [255, 256], [9, 1], 0, 0),             # 27 rows, a ragged block
    (64, 16, 1, 16, 1, 6, [250], None, 0, 0),                    # 96 rows: several row blocks
    (64, 16, 3, 2, 1, 2, [0, 40, 90], [0, 1, 2], 0, 0),          # no new token at all
    (128, 32, 2, 4, 2, 1, [700, 90], None, 100, 0),              # a window
    (128, 32, 2, 4, 2, 4, [700, 3], [4, 2], 100, 5),             # and sinks, overlapping it at the start
    (64, 16, 2, 2, 2, 3, [130, 14], None, 1, 0),                 # each row sees itself alone
    (64, 16, 2, 2, 2, 3, [130, 14], None, 1, 20),                # itself and the sinks
    (32, 16, 2, 6, 2, 2, [200, 30], None, 1000, 3),              # a window wider than the sequence
    (64, 64, 2, 2, 1, 2, [620, 8], None, 16, 600),               # sinks over a chunk, one sequence short of them
])
def test_attention_shapes(dtype, d, page, B, Hq, Hkv, L, start, lens, window, sinks):
    gen = torch.Generator().manual_seed(d + L + B)
    max_pages = -(-(max(start) + L) // page)
    pages = B * max_pages + 1
    cache = pool(pages, Hkv, page, d, gen)
    q = torch.randn(B, Hq, L, d, generator=gen).to(DT[dtype]).cuda()
    check(q, cache, tables(B, max_pages, pages, gen), start, lens, 1.5, window, sinks, page, dtype)


@pytest.mark.parametrize("alpha", [1.25, 2.0])
def test_attention_more_candidates_than_shared_memory(alpha):
    """Nearly equal scores: every key of 5000 has a weight, more than the solver keeps on chip."""
    gen = torch.Generator().manual_seed(9)
    d, page, n = 64, 64, 5000
    max_pages = -(-n // page)
    cache = pool(max_pages, 1, page, d, gen)
    q = (1e-4 * torch.randn(1, 3, 2, d, generator=gen)).cuda()
    check(q, cache, tables(1, max_pages, max_pages, gen), [n - 2], None, alpha, 0, 0, page, "f32")


@pytest.mark.parametrize("alpha,spread", [(1.25, 1.0), (1.25, 1e-4), (2.0, 0.05)])
def test_attention_many_candidates(alpha, spread):
    """40000 keys, most of them within 1 of the maximum: the solver bounds tau by fewer keys first; with nearly
    equal scores nothing fits all the same.  The same result every time."""
    gen = torch.Generator().manual_seed(17)
    d, page, n = 32, 128, 40000
    max_pages = -(-n // page)
    cache = pool(max_pages, 1, page, d, gen)
    table = tables(1, max_pages, max_pages, gen)
    q = (spread * torch.randn(1, 2, 1, d, generator=gen)).cuda()
    o = check(q, cache, table, [n - 1], None, alpha, 0, 0, page, "f32")
    for _ in range(3):
        assert torch.equal(entmax_attn_kv4(q, cache, table.cuda(), i32([n - 1]), alpha), o)


def test_attention_large_scores():
    """Scores far beyond 2^24 apart and from zero: the largest takes all."""
    gen = torch.Generator().manual_seed(10)
    cache = pool(4, 1, 16, 32, gen)
    q = (1e9 * torch.randn(1, 2, 1, 32, generator=gen)).cuda()
    table = tables(1, 4, 4, gen)
    o = entmax_attn_kv4(q, cache, table.cuda(), i32([60]), 1.5).cpu().double()
    k, _ = kv4_ref.sequence(cache[0].cpu(), cache[1].cpu(), table[0], 61, 16)
    v, _ = kv4_ref.sequence(cache[2].cpu(), cache[3].cpu(), table[0], 61, 16)
    best = (k[:, 0] @ q[0, :, 0].cpu().double().T).argmax(0)
    assert bool(((o[0, :, 0] - v[best, 0]).abs() <= 2.0 ** -22 * (v[best, 0].abs() + 1)).all())


def test_attention_nan_and_infinity():
    gen = torch.Generator().manual_seed(11)
    d, page = 64, 16
    cache = pool(5, 2, page, d, gen)
    table = i32([[0, 1, 2, 3, 4]])
    q = torch.randn(1, 4, 2, d, generator=gen).cuda()
    clean = entmax_attn_kv4(q, cache, table, i32([70]), 1.5, window=20)
    # past the end and outside the window: no effect
    for codes, meta in (cache[:2], cache[2:]):
        meta[4, :, 8:] = math.nan
        meta[0, :, :] = math.inf
        meta[1] = math.nan
    assert torch.equal(entmax_attn_kv4(q, cache, table, i32([70]), 1.5, window=20), clean)
    # a query with a NaN or an infinity: its row alone
    for x in (math.nan, math.inf, -math.inf):
        q2 = q.clone()
        q2[0, 1, 0, 5] = x
        o = entmax_attn_kv4(q2, cache, table, i32([70]), 1.5, window=20)
        assert bool(torch.isnan(o[0, 1, 0]).all())
        o[0, 1, 0] = clean[0, 1, 0]
        assert torch.equal(o, clean)
    # a visible key with NaN: every row that sees it
    cache[1][4, 0, 7, 0, 1] = math.nan   # position 71, key head 0: the second token's rows of heads 0, 1
    o = entmax_attn_kv4(q, cache, table, i32([70]), 1.5, window=20)
    assert bool(torch.isnan(o[0, :2, 1]).all())
    o[0, :2, 1] = clean[0, :2, 1]
    assert torch.equal(o, clean)


def test_bad_pages_and_lengths():
    """Page numbers outside the pool and lengths outside the table do what the header says, in bounds."""
    gen = torch.Generator().manual_seed(12)
    d, page, H = 64, 16, 2
    cache = pool(6, H, page, d, gen)
    table = torch.tensor([[0, -1, 2], [3, 6, 5], [1, 4, 2 ** 31 - 1]], dtype=torch.int32)
    q = torch.randn(3, H, 1, d, generator=gen).cuda()
    bad = i32([0])
    check(q, cache, table, [40, 40, 40], None, 1.5, 0, 0, page, "f32", bad=bad)
    assert int(bad) == 1
    # every page missing: no key, zeros
    o = entmax_attn_kv4(q, cache, torch.full((3, 3), -7, dtype=torch.int32, device="cuda"), i32([40, 0, 5]), 1.5)
    assert not bool(o.any())
    for start, lens, rows in (([-1, 47, 48], [1, 1, 1], [0, 1, 0]), ([0, 10, 2 ** 31 - 1], [-1, 2, 1], [0, 1, 0])):
        bad.zero_()
        o = entmax_attn_kv4(q, cache, i32([[0, 1, 2]] * 3), i32(start), 1.5, new_lens=i32(lens), bad=bad)
        assert int(bad) == 2
        assert [int(bool(o[b].any())) for b in range(3)] == rows
    before = [t.clone() for t in cache]
    x = torch.randn(3, H, 4, d, generator=gen).cuda()
    bad.zero_()
    kv4_write(cache, x, x, i32([[9, 9, 9], [-1, -1, -1], [6, 6, 6]]), i32([0, 3, 47]), bad=bad)
    assert int(bad) == 3
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    bad.zero_()
    k, v = kv4_read(cache, i32([[0, 99, 1]]), i32([10]), 20, dtype=torch.float32, bad=bad)
    assert int(bad) == 1 and bool(k[:, :, :6].all()) and not bool(k[:, :, 6:].any()) and not bool(v[:, :, 6:].any())


def test_cover_arguments():
    """A window or sinks beyond 31 bits are the sequence; a cover beyond the table is refused."""
    gen = torch.Generator().manual_seed(18)
    cache = pool(4, 1, 16, 64, gen)
    table, q = i32([[0, 1, 2, 3]]), torch.randn(1, 2, 1, 64, generator=gen).cuda()
    want = entmax_attn_kv4(q, cache, table, i32([50]), 1.5)
    assert torch.equal(entmax_attn_kv4(q, cache, table, i32([50]), 1.5, window=2 ** 40, sinks=2 ** 33), want)
    assert torch.equal(entmax_attn_kv4(q, cache, table, i32([50]), 1.5, max_len=51), want)
    for kw in (dict(max_len=65), dict(max_len=-1), dict(window=0), dict(sinks=1), dict(window=3, sinks=-1)):
        with pytest.raises(ValueError):
            entmax_attn_kv4(q, cache, table, i32([50]), 1.5, **kw)
        with pytest.raises(ValueError):
            kv4_workspace(q, cache, table, **kw)
    with pytest.raises(ValueError):
        kv4_read(cache, table, i32([0]), 4, out=(torch.empty(1, 1, 4, 64), torch.empty(1, 1, 4, 64)))


def test_no_cover():
    """max_len 0 and an empty table: every row is padding."""
    cache = kv4_alloc(1, 1, 16, 32, "cuda")
    q = torch.randn(2, 1, 1, 32, device="cuda")
    o = entmax_attn_kv4(q, cache, i32([[0], [0]]), i32([0, 0]), 1.5, max_len=0)
    assert not bool(o.any())
    o = entmax_attn_kv4(q, cache, torch.empty((2, 0), dtype=torch.int32, device="cuda"), i32([0, 0]), 1.5)
    assert not bool(o.any())


def test_offsets_past_32_bits():
    """Pages whose arrays begin beyond 4 GB."""
    gen = torch.Generator().manual_seed(13)
    page, H, d = 128, 8, 128
    pages = (1 << 32) // (page * H * d // 2) + 40
    cache = kv4_alloc(pages, H, page, d, "cuda")
    assert cache[0].numel() > 1 << 32
    x = torch.randn(1, H, 200, d, generator=gen)
    table = torch.tensor([[pages - 1, pages - 30]], dtype=torch.int32)
    kv4_write(cache, x.cuda(), (x + 1).cuda(), table.cuda(), i32([0]))
    k, v = kv4_read(cache, table.cuda(), i32([0]), 200, dtype=torch.float32)
    for got, rows in ((k, x), (v, x + 1)):
        c, s, z = kv4_ref.quantise(rows)
        want = z.double().repeat_interleave(32, -1) + s.double().repeat_interleave(32, -1) * c.double()
        assert bool(((got.cpu().double() - want).abs() <= 2.0 ** -24 * 1.01 * want.abs()).all())
    small = kv4_alloc(2, H, page, d, "cuda")
    for a, b in zip(small, cache):
        a[0], a[1] = b[pages - 1], b[pages - 30]
    q = torch.randn(1, 16, 1, d, generator=gen).cuda()
    assert torch.equal(entmax_attn_kv4(q, cache, table.cuda(), i32([199]), 1.5),
                       entmax_attn_kv4(q, small, i32([[0, 1]]), i32([199]), 1.5))


# ------------------------------------------------------------------ as they are used
def test_streams_graphs_and_repeats():
    """Another stream than the default one, a captured step replayed on new inputs, and the same result
    every time; two captured calls with a workspace each."""
    gen = torch.Generator().manual_seed(14)
    d, page, B, H = 64, 16, 2, 2
    cache = pool(20, H, page, d, gen)
    table = tables(B, 10, 20, gen).cuda()
    start, lens = i32([30, 140]), i32([1, 1])
    k, v = (torch.randn(B, H, 1, d, generator=gen).cuda() for _ in "kv")
    q, q2 = (torch.randn(B, 4, 1, d, generator=gen).cuda() for _ in range(2))

    def step(ws):
        kv4_write(cache, k, v, table, start, lens)
        return (entmax_attn_kv4(q, cache, table, start, 1.5, new_lens=lens, ws=ws),
                entmax_attn_kv4(q2, cache, table, start, 1.25, new_lens=lens, window=50, sinks=2))

    ws = kv4_workspace(q, cache, table)
    want = [t.clone() for t in step(ws)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(step(ws), want))
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(ws)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # other inputs in the same tensors, further on in the sequences
    for t in (k, v, q, q2):
        t.copy_(torch.randn(t.shape, generator=gen))
    start.add_(1)
    graph.replay()
    got = [t.clone() for t in outs]
    assert all(torch.equal(a, b) for a, b in zip(step(ws), got))
    assert not torch.equal(got[0], want[0])


def test_two_calls_at_once():
    """Two streams, a workspace each: neither disturbs the other."""
    gen = torch.Generator().manual_seed(15)
    cache = pool(80, 2, 64, 128, gen)
    table = tables(2, 40, 80, gen).cuda()
    start = i32([2000, 2500])
    qs = [torch.randn(2, 8, 1, 128, generator=gen).cuda() for _ in range(2)]
    want = [entmax_attn_kv4(q, cache, table, start, 1.5).clone() for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    ws = [kv4_workspace(q, cache, table) for q in qs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for s, q, w, o in zip(streams, qs, ws, outs):
            with torch.cuda.stream(s):
                o.append(entmax_attn_kv4(q, cache, table, start, 1.5, ws=w))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for o, w in zip(outs, want) for x in o)


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_prompt_then_tokens(window, sinks):
    """A padded batch of prompts written at once, then tokens one by one; every step against the
    restatement, and the whole against the training attention on the values read back."""
    gen = torch.Generator().manual_seed(16)
    B, Hq, Hkv, d, page, L = 3, 4, 2, 64, 16, 37
    prompt, steps = [37, 20, 1], 3
    total = [p + steps for p in prompt]
    k, v = (torch.randn(B, Hkv, L + steps, d, generator=gen).bfloat16().cuda() for _ in "kv")
    q = torch.randn(B, Hq, L + steps, d, generator=gen).bfloat16().cuda()
    cache = kv4_alloc(B * 3, Hkv, page, d, "cuda")
    table = tables(B, 3, B * 3, gen)
    zero = i32([0] * B)
    kv4_write(cache, k[:, :, :L].contiguous(), v[:, :, :L].contiguous(), table.cuda(), zero, i32(prompt))
    first = check(q[:, :, :L].contiguous(), cache, table, [0] * B, prompt, 1.5, window, sinks, page, "bf16")
    rows = [[first[b, :, :prompt[b]]] for b in range(B)]
    for s in range(steps):
        at = [p + s for p in prompt]
        one = [torch.stack([t[b, :, at[b]] for b in range(B)])[:, :, None].contiguous() for t in (q, k, v)]
        kv4_write(cache, one[1], one[2], table.cuda(), i32(at))
        o = check(one[0], cache, table, at, None, 1.5, window, sinks, page, "bf16")
        for b in range(B):
            rows[b].append(o[b])
    for b in range(B):
        kk, vv = kv4_read(cache, table[b:b + 1].cuda(), zero[:1], total[b], dtype=torch.float32)
        rep = [t.repeat_interleave(Hq // Hkv, 1).contiguous() for t in (kk, vv)]
        if window:
            continue   # the windowed training attention has its own comparison
        want = entmax_attn_fwd(q[b:b + 1, :, :total[b]].float().contiguous(), *rep, 1.5, True)[0]
        got = torch.cat(rows[b], 1).float()
        # two routes in float (1e-4 is the float32 forward's own bound) and a rounding to bf16
        assert bool(((got - want[0]).abs() <= 1e-4 + 2.0 ** -8 * want[0].abs() * 1.01).all())


def test_wrapper_refusals_on_the_device():
    """Wrong shapes, types, places and layouts of the cache and of the sequences' tensors."""
    cache = kv4_alloc(3, 2, 16, 64, "cuda")
    x = torch.zeros(2, 2, 1, 64, device="cuda")
    table, start = i32([[0, 1], [2, 0]]), i32([0, 0])
    kv4_write(cache, x, x, table, start)
    bad_caches = [cache[:1] + (cache[1].float(),) + cache[2:], (cache[0][:2],) + cache[1:],
                  tuple(t.cpu() for t in cache), (cache[0].transpose(1, 2).contiguous().transpose(1, 2),) + cache[1:],
                  (cache[0][0],) + cache[1:]]
    for c in bad_caches:
        for call in (lambda: kv4_write(c, x, x, table, start), lambda: entmax_attn_kv4(x, c, table, start),
                     lambda: kv4_read(c, table, start, 1)):
            with pytest.raises(ValueError):
                call()
    for t, s, n, b in ((table.long(), start, None, None), (table[:1], start, None, None), (table.cpu(), start, None, None),
                       (table.t(), start, None, None), (table, start.long(), None, None), (table, start[:1], None, None),
                       (table, start.cpu(), None, None), (table, start, i32([1]), None), (table, start, None, i32([0, 0])),
                       (table, None, None, None)):
        for call in (lambda: kv4_write(cache, x, x, t, s, n, bad=b),
                     lambda: entmax_attn_kv4(x, cache, t, s, new_lens=n, bad=b)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        kv4_write(cache, x[..., :32].contiguous(), x[..., :32].contiguous(), table, start)
    with pytest.raises(ValueError):
        entmax_attn_kv4(torch.zeros(2, 3, 1, 64, device="cuda"), cache, table, start)
    with pytest.raises(ValueError):
        entmax_attn_kv4(x.transpose(0, 1), cache, table, start)


@pytest.mark.parametrize("alpha,group,B", [(1.25, 8, 16), (1.5, 4, 32), (1.5, 1, 64), (2.0, 4, 32)])
def test_attention_repeats_whatever_the_timing(alpha, group, B):
    """Rows with 200 to 2000 keys above their maximum - 1, where how many more candidates the scores kernel
    lists varies by hundreds from call to call: the same bits every time, with other work beside the calls."""
    gen = torch.Generator().manual_seed(19)
    n, d, page = 32768, 32, 128
    cache = pool(n // page, 1, page, d, gen)
    one = tables(1, n // page, n // page, gen).cuda()
    k, _ = kv4_read(cache, one, i32([0]), n, dtype=torch.float32)
    u = torch.randn(d, generator=gen).double().cuda()
    x = (k[0, 0].double() @ u).sort(descending=True).values
    # queries along u whose scores put key rank_r just at the maximum - 1
    rank = torch.linspace(200, 2000, 4 * B * group).long()
    beta = math.sqrt(d) / (alpha - 1) / (x[0] - x[rank.cuda()])
    table, start = one.expand(B, -1).contiguous(), i32([n - 1] * B)
    side, junk = torch.cuda.Stream(), torch.randn(1 << 20, device="cuda")
    for part in beta.split(B * group):
        q = (part[:, None] * u).float().view(B, group, 1, d).contiguous()
        tau = torch.empty(B, group, 1, device="cuda")
        o = entmax_attn_kv4(q, cache, table, start, alpha, tau=tau).clone()
        first, differ = tau.clone(), torch.zeros((), dtype=torch.int64, device="cuda")
        for i in range(60):   # (no wait between calls: it would even the timing out)
            with torch.cuda.stream(side):
                junk[:1 << (8 + i % 13)].sin_()
            again = entmax_attn_kv4(q, cache, table, start, alpha, tau=tau)
            differ += (again != o).sum() + (tau != first).sum()
        assert int(differ) == 0


def test_no_cover_is_reported():
    """max_len 0 or an empty table: a row that is there lies outside the cover, no row is fine."""
    cache = kv4_alloc(1, 2, 16, 32, "cuda")
    q = torch.randn(2, 4, 3, 32, device="cuda")
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    for start, lens, want in (([0, 0], [1, 0], 2), ([0, 0], [0, 3], 2), ([0, 0], [0, 0], 0), ([1, 0], [0, 0], 2),
                              ([0, -1], [0, 0], 2), ([0, 0], None, 2)):
        for table, kw in ((i32([[0], [0]]), dict(max_len=0)), (none, {})):
            bad = i32([0])
            o = entmax_attn_kv4(q, cache, table, i32(start), 1.5, new_lens=None if lens is None else i32(lens),
                                bad=bad, **kw)
            assert int(bad) == want and not bool(o.any())


def test_a_row_of_nan_lists_no_keys():
    """Of a row that has met a NaN the call keeps its runs' maxima and counts, no candidates: of 64 keys (one run)
    two words a row are written to the workspace."""
    gen = torch.Generator().manual_seed(20)
    cache = pool(4, 1, 16, 32, gen)
    cache[1][0, 0, 3] = math.nan
    table, q = i32([[0, 1, 2, 3]]), torch.randn(1, 8, 1, 32, generator=gen).cuda()
    ws = kv4_workspace(q, cache, table).fill_(0x5A)
    o = entmax_attn_kv4(q, cache, table, i32([63]), 1.5, ws=ws)
    assert bool(torch.isnan(o).all())
    assert int((ws.view(torch.int32) != 0x5A5A5A5A).sum()) <= 2 * 8


@pytest.mark.parametrize("d,n,Hq,L,alpha,beta", [(128, 2048, 4, 1, 1.5, 1.0), (128, 1500, 4, 4, 1.5, 2.0),
                                                 (64, 3000, 4, 5, 2.0, 1.0), (64, 1000, 1, 1, 1.5, 1.0),
                                                 (32, 1500, 4, 2, 1.25, 1.0), (32, 900, 2, 6, 1.5, 4.0)])
def test_float32_is_as_near_as_float_products(d, n, Hq, L, alpha, beta):
    """float32 rows: the error (2-norm) is no more than that of the exact entmax of float32 scores.  Those come from
    sums of d terms, each rounded; the kernel's sums over a group of 32 are exact in the query's leading 11 bits and
    it rounds four times a group (2^-24 of the partial sum each), a query's value to 2^-23 of its row's largest.
    Beside the scores: |sum p - 1| <= 2e-7 where the solver stops and 2^-24 for each of p and o: 3e-7."""
    gen = torch.Generator().manual_seed(21)
    page, B = 16, 8
    used = -(-n // page)
    cache = pool(used, 1, page, d, gen)
    one = tables(1, used, used, gen).cuda()
    q = (beta * torch.randn(B, Hq, L, d, generator=gen)).cuda()
    o = entmax_attn_kv4(q, cache, one.expand(B, -1).contiguous(), i32([n - L] * B), alpha)
    k, v = (t[0, 0] for t in kv4_read(cache, one, i32([0]), n, dtype=torch.float32))
    seen = torch.arange(n, device="cuda")[None] <= (n - L + torch.arange(L, device="cuda"))[:, None]

    def exact(x):   # of the given scores, by halving
        x = x.double().masked_fill(~seen, -math.inf)
        hi = x.amax(-1, keepdim=True)
        lo = hi - 1
        for _ in range(56):
            mid = (lo + hi) / 2
            up = torch.relu(x - mid).pow(1 / (alpha - 1)).sum(-1, keepdim=True) > 1
            lo, hi = torch.where(up, mid, lo), torch.where(up, hi, mid)
        return torch.relu(x - (lo + hi) / 2).pow(1 / (alpha - 1)) @ v.double()

    assert not torch.backends.cuda.matmul.allow_tf32
    want = exact(q.double() @ k.double().T * ((alpha - 1) / math.sqrt(d)))
    plain = exact(q @ k.T * ((alpha - 1) / math.sqrt(d)))
    assert float((o.double() - want).norm()) <= float((plain - want).norm()) + 3e-7 * float(want.norm())

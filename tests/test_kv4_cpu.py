"""The 4-bit cache on a machine without a GPU: its index arithmetic by brute force, the
refusals of the C ABI and of the PyTorch wrappers, and the restated quantiser's own error."""
import os
import shutil
import subprocess

import pytest
import torch

import kv4_ref
from adaptive_sparse_flash_entmax_b200 import build, capi, kv4_alloc, kv4_read, kv4_write, entmax_attn_kv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20   # 16-byte aligned, never dereferenced on argument errors


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def test_index_arithmetic(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = tmp_path / "kv4_index_check"
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-I",
                    os.path.join(ROOT, "adaptive_sparse_flash_entmax_b200", "csrc"),
                    os.path.join(ROOT, "tests", "c", "kv4_index_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


POOL = dict(k_codes=FAKE, k_meta=FAKE, v_codes=FAKE, v_meta=FAKE, pages=4, page=16)
SEQ = dict(block_table=FAKE, max_pages=4, start=FAKE, new_lens=None, bad=None, stream=None)
ROWS = dict(B=2, Hkv=2, L=3, d=64, dtype=capi.ENT_BF16)

COMMON = [
    (dict(d=96), capi.ENT_EUNSUPPORTED),
    (dict(dtype=5), capi.ENT_EINVAL),
    (dict(B=-1), capi.ENT_EINVAL),
    (dict(Hkv=0), capi.ENT_EINVAL),
    (dict(L=-1), capi.ENT_EINVAL),
    (dict(B=70000), capi.ENT_EUNSUPPORTED),
    (dict(page=24), capi.ENT_EINVAL),
    (dict(page=8), capi.ENT_EINVAL),
    (dict(page=0), capi.ENT_EINVAL),
    (dict(pages=-1), capi.ENT_EINVAL),
    (dict(pages=0), capi.ENT_EINVAL),
    (dict(max_pages=-1), capi.ENT_EINVAL),
    (dict(max_pages=1 << 27), capi.ENT_EUNSUPPORTED),
    (dict(block_table=None), capi.ENT_EINVAL),
    (dict(start=None), capi.ENT_EINVAL),
    (dict(k_codes=None), capi.ENT_EINVAL),
    (dict(v_meta=None), capi.ENT_EINVAL),
    (dict(k_meta=FAKE + 4), capi.ENT_EINVAL),
]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(k=None), capi.ENT_EINVAL), (dict(v=FAKE + 8), capi.ENT_EINVAL)])
@pytest.mark.parametrize("fn", ["ent_attn_kv4_write", "ent_attn_kv4_read"])
def test_write_and_read_refusals(lib, fn, kw, code):
    args = dict(POOL, **SEQ, **ROWS, k=FAKE, v=FAKE)
    args.update(kw)
    assert getattr(capi, fn)(**args) == code
    assert capi.ent_attn_last_error()


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(q=None), capi.ENT_EINVAL),
    (dict(o=None), capi.ENT_EINVAL),
    (dict(o=FAKE + 4), capi.ENT_EINVAL),
    (dict(Hq=3), capi.ENT_EINVAL),
    (dict(Hq=0), capi.ENT_EINVAL),
    (dict(alpha=1.0), capi.ENT_EINVAL),
    (dict(alpha=2.1), capi.ENT_EINVAL),
    (dict(alpha=float("nan")), capi.ENT_EINVAL),
    (dict(window=-1), capi.ENT_EINVAL),
    (dict(sinks=-1), capi.ENT_EINVAL),
    (dict(window=0, sinks=4), capi.ENT_EINVAL),
    (dict(max_len=65), capi.ENT_EINVAL),
    (dict(max_len=-1), capi.ENT_EINVAL),
    (dict(ws=None), capi.ENT_EINVAL),
    (dict(ws_bytes=8), capi.ENT_EINVAL),
    (dict(ws=FAKE + 8), capi.ENT_EINVAL),
])
def test_attention_refusals(lib, kw, code):
    args = dict(POOL, **SEQ, **ROWS, Hq=4, q=FAKE, o=FAKE, tau=None, alpha=1.5, window=0, sinks=0, max_len=64,
                ws=FAKE, ws_bytes=1 << 30)
    args.update(kw)
    assert capi.ent_attn_kv4_fwd(**args) == code
    assert capi.ent_attn_last_error()


def test_nothing_to_do(lib):
    for kw in (dict(B=0), dict(L=0)):
        assert capi.ent_attn_kv4_write(**dict(POOL, **SEQ, **dict(ROWS, **kw), k=None, v=None)) == capi.ENT_OK
        assert capi.ent_attn_kv4_read(**dict(POOL, **SEQ, **dict(ROWS, **kw), k=None, v=None)) == capi.ENT_OK
        assert capi.ent_attn_kv4_fwd(**dict(POOL, **SEQ, **dict(ROWS, **kw), Hq=4, q=None, o=None, tau=None,
                                            alpha=1.5, window=0, sinks=0, max_len=64, ws=None,
                                            ws_bytes=0)) == capi.ENT_OK


def test_workspace_sizes(lib):
    size = capi.ent_attn_kv4_workspace_size
    bf = capi.ENT_BF16
    full = size(4, 8, 2, 1, 128, bf, 8192, 0, 0)
    assert full >= 4 * 8 * 8192 * 6
    # a window bounds it, whatever the sequences' length
    assert size(4, 8, 2, 1, 128, bf, 1 << 20, 256, 4) < full
    assert size(0, 8, 2, 1, 128, bf, 8192, 0, 0) == 0
    for bad in ((-1, 8, 2, 1, 128, bf, 64, 0, 0), (1, 3, 2, 1, 128, bf, 64, 0, 0), (1, 8, 2, 1, 128, bf, -1, 0, 0),
                (1, 8, 2, 1, 128, bf, 64, -1, 0), (1, 8, 2, 1, 128, bf, 64, 0, 1)):
        assert size(*bad) == 0


def test_wrapper_refusals():
    """Shapes, types and devices are refused before the library is called (CPU tensors get that far)."""
    with pytest.raises(ValueError):
        kv4_alloc(2, 2, 24, 64, "cpu")
    with pytest.raises(ValueError):
        kv4_alloc(2, 2, 16, 48, "cpu")
    cache = kv4_alloc(3, 2, 16, 64, "cpu")
    assert [tuple(t.shape) for t in cache] == [(3, 2, 16, 32), (3, 2, 16, 2, 2)] * 2
    table, start = torch.zeros((1, 3), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kv4_write(cache, x, x, table, start)
    with pytest.raises(ValueError, match="dtype"):
        kv4_write(cache, x.half(), x.half(), table, start)
    with pytest.raises(ValueError, match="share"):
        kv4_write(cache, x, x[:, :1], table, start)
    with pytest.raises(ValueError, match="dtype"):
        kv4_read(cache, table, start, 4, dtype=torch.float16)
    with pytest.raises(ValueError, match="out must be"):
        kv4_read(cache, table, start, 4, out=(x[:, :, :2], x[:, :, :2]))
    with pytest.raises(ValueError, match="B, H, L, d"):
        entmax_attn_kv4(x[0], cache, table, start)
    with pytest.raises(ValueError, match="CUDA"):
        entmax_attn_kv4(x, cache, table, start)


def test_restated_quantiser_bounds():
    """Each value is within half a step of what it stands for, plus what the pair's rounding adds:
    zero is off by at most 2^-9 |min| (it may exceed the minimum), scale by 2^-9 of itself, which moves
    the top code's value by at most 15 scale 2^-9."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 128, generator=g) * torch.exp(2 * torch.randn(64, 1, generator=g)) + 3
    codes, scale, zero = kv4_ref.quantise(x)
    s, z = scale.double().repeat_interleave(32, -1), zero.double().repeat_interleave(32, -1)
    lo = x.double().unflatten(-1, (-1, 32)).amin(-1).repeat_interleave(32, -1)
    err = (z + s * codes.double() - x.double()).abs()
    assert bool((err <= s / 2 + 15 * s * 2.0 ** -8 + 2.0 ** -8 * lo.abs() + 1e-12).all())
    # constant groups are held to bf16 rounding
    codes, scale, zero = kv4_ref.quantise(torch.full((1, 32), 1.7))
    assert float(zero) == float(torch.tensor(1.7).bfloat16()) and int(codes.max()) <= 15


def test_no_workspace_for_what_the_call_refuses(lib):
    """The size is 0 for every size that the call itself refuses, the limits among them."""
    ok = dict(B=2, Hq=4, Hkv=2, L=3, d=64, dtype=capi.ENT_BF16, max_len=64, window=0, sinks=0)
    assert capi.ent_attn_kv4_workspace_size(**ok) > 0
    for kw in (dict(d=96), dict(d=0), dict(dtype=5), dict(B=70000), dict(max_len=(1 << 30) + 1), dict(L=1 << 30),
               dict(B=-1), dict(Hkv=0), dict(Hq=0), dict(Hq=3), dict(L=-1), dict(max_len=-1), dict(window=-1),
               dict(sinks=-1, window=4), dict(sinks=1)):
        args = dict(ok, **kw)
        assert capi.ent_attn_kv4_workspace_size(**args) == 0, kw
        covered = max(args.pop("max_len"), 0)
        st = capi.ent_attn_kv4_fwd(q=FAKE, o=FAKE, tau=None, alpha=1.5, **POOL, block_table=FAKE, start=FAKE,
                                   max_pages=-(-covered // POOL["page"]), new_lens=None, bad=None,
                                   max_len=dict(ok, **kw)["max_len"], ws=FAKE, ws_bytes=0, stream=None, **args)
        assert st in (capi.ENT_EINVAL, capi.ENT_EUNSUPPORTED), kw

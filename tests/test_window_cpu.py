"""Windowed attention on a machine without a GPU: refusals, and which blocks a query tile visits."""
import os
import shutil
import subprocess

import pytest
import torch

from adaptive_sparse_flash_entmax_b200 import attention as A
from adaptive_sparse_flash_entmax_b200 import build, capi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


CASES = [
    (dict(window=0), capi.ENT_EINVAL),
    (dict(window=-5), capi.ENT_EINVAL),
    (dict(sinks=-1), capi.ENT_EINVAL),
    (dict(alpha=1.0), capi.ENT_EINVAL),
    (dict(d=96), capi.ENT_EUNSUPPORTED),
    (dict(dtype=7), capi.ENT_EINVAL),
    (dict(N=-1), capi.ENT_EINVAL),
    (dict(N=200000), capi.ENT_EUNSUPPORTED),
    (dict(q=None), capi.ENT_EINVAL),
    (dict(otilde=FAKE + 4), capi.ENT_EINVAL),
    (dict(ws=None), capi.ENT_EINVAL),
    (dict(ws_bytes=16), capi.ENT_EINVAL),
]


@pytest.mark.parametrize("kw,code", CASES + [(dict(o=FAKE + 4), capi.ENT_EINVAL)])
def test_forward_refusals(lib, kw, code):
    args = dict(q=FAKE, k=FAKE, v=FAKE, B=1, H=1, N=128, d=64, dtype=capi.ENT_BF16, alpha=1.5, window=8, sinks=2,
                o=FAKE, tau=FAKE, block_mask=FAKE, iters=None, otilde=None, ws=FAKE, ws_bytes=1 << 30, stream=None)
    args.update(kw)
    assert capi.ent_attn_fwd_window(**args) == code
    assert capi.ent_attn_last_error()


@pytest.mark.parametrize("kw,code", CASES + [(dict(dq=FAKE + 8), capi.ENT_EINVAL), (dict(tau=None), capi.ENT_EINVAL)])
def test_backward_refusals(lib, kw, code):
    args = dict(q=FAKE, k=FAKE, v=FAKE, otilde=None, dout=FAKE, tau=FAKE, block_mask=FAKE, B=1, H=1, N=128, d=64,
                dtype=capi.ENT_BF16, alpha=1.5, window=8, sinks=2, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE,
                ws_bytes=1 << 30, stream=None)
    args.update(kw)
    assert capi.ent_attn_bwd_window(**args) == code
    assert capi.ent_attn_last_error()


def test_wrapper_refusals():
    x = torch.zeros(1, 1, 8, 64)
    for kw, what in ((dict(causal=False, window=4), "causal"), (dict(causal=True, sinks=2), "sinks"),
                     (dict(causal=True, window=0), "at least"), (dict(causal=True, window=4, sinks=-1), "at least"),
                     (dict(causal=True, window=4, delta="lists"), "lists")):
        with pytest.raises(ValueError, match=what):
            A.entmax_attention(x, x, x, 1.5, **kw)


def test_visited_blocks(tmp_path):
    """Brute force over windows, sinks and tiles: the listed blocks are in order, without repeats, and
    exactly those that hold a visible pair; the count of a row's visible keys is exact."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    text = open(os.path.join(ROOT, "adaptive_sparse_flash_entmax_b200", "csrc", "common.cuh")).read()
    part = text[text.index("struct WinBlocks"):text.index("__device__ __forceinline__ float load_f")]
    src = tmp_path / "win.cpp"
    src.write_text("""
#include <cstdio>
#include <initializer_list>
#define __host__
#define __device__
#define __forceinline__ inline
constexpr int kBlk = 128;
""" + part + """
int main() {
    for (int w : {1, 2, 100, 127, 128, 129, 255, 256, 257, 1000})
        for (int s : {0, 1, 127, 128, 129, 300, 1000})
            for (int t = 0; t < 8; ++t) {
                const WinBlocks wb(w, s, t);
                int n = 0, last = -1;
                for (int b = 0; b <= t; ++b) {
                    bool any = false;
                    for (int i = t * 128; i < t * 128 + 128 && !any; ++i)
                        for (int j = b * 128; j < b * 128 + 128 && j <= i; ++j)
                            if (i - j < w || j < s) { any = true; break; }
                    if (any != wb.has(b)) { std::printf("has %d %d %d %d\\n", w, s, t, b); return 1; }
                    if (any) { if (wb.block(n) != b || b <= last) { std::printf("block %d %d %d\\n", w, s, t); return 1; } last = b; ++n; }
                }
                if (n != wb.count(t)) { std::printf("count %d %d %d\\n", w, s, t); return 1; }
                for (int i = t * 128; i < t * 128 + 128; i += 9) {
                    int k = 0;
                    for (int j = 0; j <= i; ++j) k += i - j < w || j < s;
                    if (k != win_keys(w, s, i)) { std::printf("keys %d %d %d\\n", w, s, i); return 1; }
                }
            }
    return 0;
}
""")
    exe = tmp_path / "win"
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", str(src), "-o", str(exe)], check=True, capture_output=True,
                   text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

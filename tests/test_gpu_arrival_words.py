"""Arrival words (the last workgroup of a split result joins the others' partial
sums) in workspaces that hold anything: a word counts only if it carries the
launch's own 52-bit tag, so neither numbers near a launch's, nor tags of other
launches with any count, nor a launch's number in 32 bits start a count.

The launches are numbered from the start of the process, so the cases run in a
process of their own, whose first launches meet the patterns made for them."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CHILD = r"""
import torch
from mixed_precision_bf16_amd import fp4gemm as F

MASK = (1 << 64) - 1


def leftovers(n):
    # 64-bit words that may lie in the workspace of launch n
    spread = n * 2654435761 % (1 << 32)
    tag = lambda i: i * 0x9E3779B97F4A7 << 12 & MASK
    words = [x << 32 | c for x in (n, spread) for c in (0, 1, 2, 0xFFFFFFFF)]
    words += [tag(i) | c for i in (n - 1, n + 1, n + 2) for c in (0, 1, 2, 0xFFF)]
    words += [n, n << 12, n << 12 | 1, 1 << 12, MASK, 0x3F8000003F800000, 0x7FC000007FC00000]
    words += [tag(n) ^ 1 << bit | 1 for bit in (12, 31, 32, 63)]
    return words


def filled(nbytes, word):
    signed = word - (1 << 64) if word >> 63 else word
    return torch.full(((nbytes + 7) // 8,), signed, dtype=torch.int64, device="cuda")


def check(what, size, run):
    # zeros first, then every kind of leftover in the launch that it is made for
    want = None
    for kind in range(-1, len(leftovers(2))):
        check.launches += 1
        word = leftovers(check.launches)[kind] if kind >= 0 else 0
        got = run(filled(size, word))
        torch.cuda.synchronize()
        want = want or got
        for a, b in zip(got, want):
            assert torch.equal(a, b), (what, check.launches, hex(word))
    print("ok", what, check.launches, flush=True)


check.launches = 0
gen = torch.Generator("cuda").manual_seed(1)
heads, D, page = 2, 128, 64
cache = F.new_kv_cache(64, page, heads, D, 0)
kv = torch.randn((64 * page, 2 * heads, D), device="cuda", generator=gen).bfloat16()
F.kv_append(cache, kv[:, :heads], kv[:, heads:], torch.arange(64 * page, device="cuda"))
table = torch.arange(64, dtype=torch.int32, device="cuda").reshape(1, 64)
for rows in (1, 70):                                   # streaming kernel, tiled kernel
    lens = torch.tensor([4000], dtype=torch.int32, device="cuda")
    q = torch.randn((rows, heads * 8, D), device="cuda", generator=gen).bfloat16()
    size = F.attention_workspace_size(q, cache, table, lens)
    assert size > 0
    def attend(ws):
        out, lse = torch.full_like(q, 9.0), torch.full((rows, heads * 8), 9.0, device="cuda")
        F.attention(q, cache, table, lens, out=out, lse=lse, workspace=ws)
        return out, lse
    check(f"attention, {rows} query tokens", size, attend)

N, K, m = 1024, 8192, 16                               # split-K
codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen).cpu().numpy()
scales = torch.randint(40, 60, (N, K // 16), dtype=torch.uint8, device="cuda", generator=gen).cpu().numpy()
wq, sq = F.upload(*F.repack(codes, scales, N, K, 0))
A = torch.randn((m, K), device="cuda", generator=gen).bfloat16()
size = F.workspace_size(m, N, K, 0)
assert size > 0
def product(ws):
    out = torch.full((m, N), 9.0, dtype=torch.bfloat16, device="cuda")
    F.gemm(A, wq, sq, N, K, 0, out=out, workspace=ws)
    return (out,)
check("product split over K", size, product)
"""


def test_leftovers_in_the_workspace_are_no_arrivals():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    name = torch.cuda.get_device_properties(0).gcnArchName
    if not name.startswith("gfx950"):
        pytest.skip(f"needs gfx950, found {name}")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-u", "-c", CHILD], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=100)
    print(r.stdout, r.stderr, flush=True)
    assert r.returncode == 0 and r.stdout.count("ok ") == 3, r.stderr

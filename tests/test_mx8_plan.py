"""The choice of kernel for products of 8-bit activations (csrc/mx8_plan.h, compiled here), and
what the exact cases of tests/mx8_cases.py can show."""

import os
import shutil
import subprocess

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import build, fp4gemm as F
from mx8_cases import EVERY, sums_fit, whole_rows, whole_weights

torch = pytest.importorskip("torch")

ASK = r"""
#include <stdio.h>
#include "mx8_plan.h"
int main() {
    long long m, N, K;
    int out, gate;
    while (scanf("%lld %lld %lld %d %d", &m, &N, &K, &out, &gate) == 5) {
        const fp4::Mx8Plan p = fp4::mx8_plan(m, N, K, out, gate);
        printf("%d %d %zu\n", p.shape, p.S, p.workspace);
    }
    printf("%d %d\n", fp4::kDecodes, fp4::kTiles);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """m, N, K, out type, gate [n][5] -> kernel, split, workspace [n][3]."""
    at = tmp_path_factory.mktemp("plan")
    (at / "ask.cpp").write_text(ASK)
    cxx = shutil.which("g++") or build.HIPCC
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", build.CSRC, str(at / "ask.cpp"), "-o", str(at / "ask")], check=True)

    def ask(calls):
        text = "\n".join(" ".join(map(str, c)) for c in np.asarray(calls).tolist())
        out = subprocess.run([str(at / "ask")], input=text, capture_output=True, text=True, check=True).stdout
        got = np.array([line.split() for line in out.splitlines()[:-1]], dtype=np.int64)
        assert len(got) == len(calls)
        return got

    return ask


def _draw(n, seed):
    """Calls that the entry allows, spread over the logarithms of their sizes."""
    rng = np.random.default_rng(seed)
    log = lambda lo, hi: np.exp(rng.uniform(np.log(lo), np.log(hi), n)).round().astype(np.int64)  # noqa: E731
    m = np.where(rng.random(n) < 0.75, log(1, 4096), log(1, 1 << 20))
    N = np.where(rng.random(n) < 0.5, log(1, 65536), log(1, 1 << 24))
    K = 32 * np.where(rng.random(n) < 0.7, log(1, 2048), log(1, 32768))
    gate, out = rng.integers(0, 2, n), rng.integers(0, 2, n) * 2
    step = np.where(gate & (out == 2), 64, np.where(gate | (out == 2), 32, 1))
    N = -(-N // step) * step
    cols, rows, Kp = np.where(gate, N // 2, N), -(-m // 256) * 256, -(-K // 128) * 128
    ok = (rows * Kp < 2 ** 31) & (rows * cols * np.where(out == 2, 1, 2) < 2 ** 31) & (N <= 1 << 24)
    return np.stack([m, N, K, out, gate], 1)[ok]


def test_the_exact_cases_cover_every_kernel(plan):
    """Whatever kernel, split and form 400000 calls take is among those that the cases take."""
    calls = _draw(600000, 1)
    assert len(calls) > 400000
    reached = {(s, S, g, o) for (s, S, _), (_, _, _, o, g) in zip(plan(calls).tolist(), calls.tolist())}
    cases = [(m, N, K, 2 * eight, gate) for m, N, K, gate, eight in EVERY]
    taken = {(s, S, g, o) for (s, S, _), (_, _, _, o, g) in zip(plan(cases).tolist(), cases)}
    assert reached <= taken, sorted(reached - taken)
    assert len(taken) == len(EVERY)                                        # each once


def test_the_library_takes_this_choice(plan):
    """The workspace that the library asks for is the plan's."""
    calls = _draw(3000, 2)
    for (m, N, K, out, gate), (_, _, need) in zip(calls.tolist(), plan(calls).tolist()):
        assert F.gemm_mx8_workspace_size(m, N, K, out, gate) == need


@pytest.mark.parametrize("m,K", [(3, 1056), (24, 8224), (20, 32832), (2, 1 << 20)])
def test_exact_cases_show_what_goes_missing(m, K):
    """Mistakes planted in the oracle: nearly every output differs, in either type, for a lost
    128 k, a lost eighth of K, a row's scales taken from the block or the 512 k before, and two
    neighbouring blocks exchanged."""
    N = 16
    a, s = whole_rows(m, K, m)
    w = whole_weights(N, K, K)
    y, total = oracle.gemm_mx8_reference(a, s, *w, K)
    assert sums_fit(total) and np.array_equal(oracle.gemm_mx8_cut_reference(a[:2], s[:2], *w, K), y[:2])
    scale = 2.0 ** np.floor(np.log2(60000 / np.abs(y).max()))
    values = oracle.dequant_weights(*w, K, 1).T
    rng = np.random.default_rng(K)

    def differ(codes, scales):
        z = oracle.mx8_value(codes, scales, K) @ values
        return [(torch.from_numpy(y * f).to(t) != torch.from_numpy(z * f).to(t)).double().mean().item()
                for t, f in ((torch.bfloat16, 1.0), (torch.float16, scale))]

    for at in (0, K // 128 - 1, *rng.integers(0, K // 128, 2)):
        lost = a.copy()
        lost[:, 128 * at:128 * at + 128] = 0
        assert min(differ(lost, s)) > 0.5
    lost = a.copy()
    lost[:, (K // 512 * 7 // 8) * 512:] = 0
    assert min(differ(lost, s)) > 0.9
    for back in (1, 4, 16):
        stale = s.copy()
        stale[:, back:K // 32] = s[:, :K // 32 - back]
        assert min(differ(a, stale)) > 0.9
    turned = a.copy()
    b = int(rng.integers(0, K // 32 - 1)) * 32
    turned[:, b:b + 32], turned[:, b + 32:b + 64] = a[:, b + 32:b + 64], a[:, b:b + 32]
    assert min(differ(turned, s)) > (0.5 if K < 1 << 20 else 0.3)

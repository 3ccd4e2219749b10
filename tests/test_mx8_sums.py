"""The sums of the 8-bit matrix cores as the oracle has them: pinned on hand cases, by
bounds, and against the plain sums."""

import numpy as np
import pytest

import oracle

pytest.importorskip("torch")


def _row(**at):
    a = np.zeros(32)
    for k, v in at.items():
        a[int(k[1:])] = v
    return a


def test_groups_of_eight_lose_what_lies_below_their_largest():
    one = np.ones((1, 32))
    # 256 - 256 leave what the group keeps of the third product: 2^-5 and above
    for e in range(-9, 8):
        got = oracle.mx8_group_sums(_row(k0=256, k1=-256, k2=2.0 ** e)[None], one)[0, 0]
        assert got[0] == (2.0 ** e if e >= -5 else 0.0) and not got[1:].any()
        got = oracle.mx8_group_sums(_row(k0=256, k1=-256, k8=2.0 ** e)[None], one)[0, 0]
        assert got[0] == 0.0 and got[1] == 2.0 ** e                            # another eight: all of it
    # toward zero, product by product
    assert oracle.mx8_group_sums(_row(k0=256, k1=-256, k2=3 * 2.0 ** -6)[None], one)[0, 0, 0] == 2.0 ** -5
    assert oracle.mx8_group_sums(_row(k0=256, k1=-256, k2=-3 * 2.0 ** -6)[None], one)[0, 0, 0] == -2.0 ** -5
    assert oracle.mx8_group_sums(_row(k0=256, k1=-256, k2=2.0 ** -6, k3=2.0 ** -6)[None], one)[0, 0, 0] == 0.0
    # the exponent is that of the factors (1.875 * 2^7 by 1.5 counts as 2^7), and of nonzero products alone
    w = one.copy()
    w[0, :2] = 1.5
    assert oracle.mx8_group_sums(_row(k0=240, k1=-240, k2=2.0 ** -6)[None], w)[0, 0, 0] == 2.0 ** -6
    w[0, :2] = 0
    assert oracle.mx8_group_sums(_row(k0=448, k1=448, k2=2.0 ** -9)[None], w)[0, 0, 0] == 2.0 ** -9


def _problem(m, N, K, seed):
    rng = np.random.default_rng(seed)
    a = oracle.mx8_quantize_reference((rng.standard_normal((m, K)) * (1 + 9 * (rng.random(K) < 0.02))).astype(np.float32))
    c = rng.integers(0, 16, (N, K)).astype(np.uint8)
    return a, ((c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8), rng.integers(120, 130, (N, K // 32)).astype(np.uint8))


@pytest.mark.parametrize("m,N,K", [(3, 5, 32), (4, 7, 160), (2, 3, 2880)])
def test_cut_sums_lie_within_their_bound(m, N, K):
    """Seven products of eight lose less than 2^-13 of the eighth."""
    a, w = _problem(m, N, K, K)
    y, total = oracle.gemm_mx8_reference(*a, *w, K)
    z = oracle.gemm_mx8_cut_reference(*a, *w, K)
    assert (np.abs(z - y) < 7 * 2.0 ** -13 * total).all() and (np.abs(z - y) < 2.0 ** -10 * total).all()
    assert K < 1000 or (z != y).any()


def test_size_of_the_cut():
    """Gaussian rows of 8192: 4.4e-6 of the result's size."""
    rng = np.random.default_rng(0)
    m, N, K = 16, 16, 8192
    a = oracle.mx8_quantize_reference(rng.standard_normal((m, K)).astype(np.float32))
    w = rng.standard_normal((N, K))
    e = np.floor(np.log2(np.abs(w).reshape(N, -1, 32).max(-1))) - 2
    q = np.abs(w) / np.exp2(e).repeat(32, -1)
    c = np.abs(q[..., None] - np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])).argmin(-1).astype(np.uint8) | (w < 0).astype(np.uint8) * 8
    w = (c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8), (e + 127).astype(np.uint8)
    y, total = oracle.gemm_mx8_reference(*a, *w, K)
    off = oracle.gemm_mx8_cut_reference(*a, *w, K) - y
    size = np.sqrt((y * y).mean())
    assert 3e-6 < np.sqrt((off * off).mean()) / size < 6e-6
    assert 4e-8 < (np.abs(off) / total).mean() < 9e-8


def test_the_largest_elements_are_rounded_to_two_to_128():
    """E4M3 has steps of 16 in 128 .. 256: from 248 scales on, 256 scales."""
    x = np.zeros((2, 32))
    x[0, 3], x[1, 3] = 248.0 * 2.0 ** 120, 247.0 * 2.0 ** 120
    v = oracle.mx8_value(*oracle.mx8_quantize_reference(x), 32)
    assert v[0, 3] == 2.0 ** 128 and v[1, 3] == 240.0 * 2.0 ** 120
    largest = np.array([[np.finfo(np.float32).max] + [0.0] * 31])
    assert oracle.mx8_value(*oracle.mx8_quantize_reference(largest), 32)[0, 0] == 2.0 ** 128

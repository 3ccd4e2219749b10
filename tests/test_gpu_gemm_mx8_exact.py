"""fp4_gemm_mx8 on rows and weights whose products and sums FP32 holds (tests/mx8_cases.py), so
that every kernel, split of K and form gives the exact sums.

Bars.  Plain: the same bits, in 16 bits and in 8.  Gated: the sums are exact, the function is
evaluated in FP32: its exponential's argument, at most 88 where it matters, has six roundings
of 2^-24 (6 * 88 * 2^-24 < 2^-14), and half a step of the output's type comes on top.  Where
e^-z passes FP32 (2^128 and more), g / (1 + e^-z) u is zero instead of |g u| 2^-128 at most."""

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F
from mx8_cases import EVERY, sums_fit, whole_rows, whole_weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, FP16 = torch.bfloat16, torch.float16
FUNCTION = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def gfx950():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    name = torch.cuda.get_device_properties(0).gcnArchName
    if not name.startswith("gfx950"):
        pytest.skip(f"needs gfx950, found {name}")
    F.lib()
    yield


def _mx8(codes, scales, K):
    return F.MX8(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn),
                 torch.from_numpy(scales).cuda().view(torch.float8_e8m0fnu), K)


def _packed(N, K, seed):
    """whole_weights' distribution in the packed layout, made on the device, zero behind K."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nw, ns = F.native_repack_size(N, K)
    Np, Kp = -(-N // 16) * 16, -(-K // 512) * 512
    wq = torch.randint(0, 256, (nw,), dtype=torch.uint8, device="cuda", generator=gen)
    sq = torch.randint(126, 129, (ns,), dtype=torch.uint8, device="cuda", generator=gen)
    block = torch.arange(Kp // 128, device="cuda")[:, None] * 4 + torch.arange(4, device="cuda")
    if Kp != K:
        wq.view(Np // 16, Kp // 128, 4, 256)[:, K // 128:] *= (block[K // 128:] * 32 < K)[None, :, :, None].to(torch.uint8)
    return wq, sq


def _tiles(wq, sq, K, tiles):
    """Canonical codes and scales of the given weight tiles."""
    KB = -(-K // 512) * 4
    parts = [F.native_unpack(wq[t * KB * 1024:(t + 1) * KB * 1024].cpu(), sq[t * KB * 64:(t + 1) * KB * 64].cpu(), 16, K)
             for t in tiles]
    return [np.concatenate(x) for x in zip(*parts)]


def _power(top, size):
    return float(2.0 ** np.floor(np.log2(top / size)))


def _check8(got, want, cols, at, off):
    """8-bit rows on the columns `at` (whole blocks of 32): want's bits (off None), or off * |want| from it."""
    codes, scales = got.codes.view(torch.uint8), got.scales.view(torch.uint8)
    assert not codes[:, cols:].any() and not scales[:, cols // 32:].any()
    blocks = at[::32] // 32
    c = codes[:, torch.from_numpy(at).cuda()].cpu().numpy()
    s = scales[:, torch.from_numpy(blocks).cuda()].cpu().numpy()
    if off is None:
        wc, ws = oracle.mx8_quantize_reference(want)
        assert np.array_equal(s, ws[:, :len(blocks)]) and np.array_equal(c, wc[:, :len(at)])
        return
    step = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1)
    values = np.concatenate([oracle.layer_oracle.E4M3, [np.nan], -oracle.layer_oracle.E4M3, [np.nan]])
    far = np.abs(values[c] * step - want) - (off * np.abs(want) * (1 + 2.0 ** -4) + np.abs(want) * 2.0 ** -4 + 2.0 ** -10 * step)
    assert far.max() <= 0, (far.max(), np.argwhere(far > 0)[:4])
    top = np.abs(want).reshape(len(want), -1, 32).max(-1)
    assert (top * (1 - off) <= 448 * step[:, ::32]).all() and ((top * (1 + off) > 224 * step[:, ::32]) | (s == 0)).all()


def _check(m, N, K, gate, eight, wq, sq, a, tiles):
    A, cols = _mx8(*a, K), N // 2 if gate else N
    if eight:
        tiles = sorted({t // 2 * 2 + i for t in tiles for i in (0, 1)})
    at = np.concatenate([np.arange(16 * t, min(16 * t + 16, cols)) for t in tiles])
    w = _tiles(wq, sq, K, tiles + ([t + cols // 16 for t in tiles] if gate else []))
    y, total = oracle.gemm_mx8_reference(*a, *w, K)
    assert sums_fit(total)
    here = torch.from_numpy(at).cuda()
    if not gate:
        y = y[:, :len(at)]                                                  # the last tile may be part of one
        if eight:
            _check8(F.gemm_mx8(A, wq, sq, N, mx8=True), y, cols, at, None)
            return
        for dtype, alpha in ((BF16, 1.0), (FP16, _power(60000, max(np.abs(y).max(), 1.0)))):
            got = F.gemm_mx8(A, wq, sq, N, dtype=dtype, alpha=alpha)[:, here]
            assert got.cpu().equal(torch.from_numpy(y * alpha).to(dtype)), dtype
        return
    n = len(at)
    alpha = _power(30, max(np.abs(y[:, :n]).max(), 1.0))
    want = oracle.gate_reference(y[:, :n] * alpha, y[:, n:] * alpha, gate)
    small = np.abs(y[:, :n] * y[:, n:]) * alpha ** 2 * 2.0 ** -128
    if eight:
        _check8(F.gemm_mx8(A, wq, sq, N, gate=gate, alpha=alpha, mx8=True), want, cols, at, FUNCTION)
        return
    for dtype in (BF16, FP16):
        got = F.gemm_mx8(A, wq, sq, N, gate=gate, alpha=alpha, dtype=dtype)[:, here].double().cpu().numpy()
        half = torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + FUNCTION) + (2.0 ** -25 if dtype == FP16 else 2.0 ** -133)
        far = np.abs(got - want) - (FUNCTION * np.abs(want) + small + half)
        assert far.max() <= 0, (dtype, far.max(), np.argwhere(far > 0)[:4])


@pytest.mark.parametrize("m,N,K,gated,eight", EVERY)
def test_every_kernel(m, N, K, gated, eight):
    last = -(-(N // 2 if gated else N) // 16) - 1
    gate = None if not gated else "gelu" if (N // 32) % 4 == 3 else "silu"
    _check(m, N, K, gate, bool(eight), *_packed(N, K, m + K), whole_rows(m, K, m + N),
           sorted({0, min(1, last), last // 2, max(last - 1, 0), last}))


@pytest.mark.parametrize("eight", [False, True])
def test_many_rows_gated(eight):
    """The largest tile, unsplit, over several rounds of workgroups."""
    m, N, K = 2048, 57344, 8192
    _check(m, N, K, "silu", eight, *_packed(N, K, 1), whole_rows(m, K, 2), [0, 7, 1000, 1790, 1791])


@pytest.mark.parametrize("gate,eight", [(None, False), (None, True), ("silu", False)])
@pytest.mark.parametrize("m", [3, 24, 70])
def test_longest_rows(m, gate, eight):
    """2^20 elements, in eight shares of K from 17 rows on."""
    N, K = 64, 1 << 20
    codes, scales = whole_weights(N, K, 5)
    _check(m, N, K, gate, eight, *(t.cuda() for t in F.native_repack(codes, scales, N, K)), whole_rows(m, K, m), [0, 1] if gate else [0, 1, 2, 3])


@pytest.mark.parametrize("m", [5, 24, 40, 70, 300])
def test_the_last_k_of_the_longest_rows(m):
    """One code at a time: at the ends of the groups of 512 and of the shares of K, and at the last k."""
    N, K = 16, 1 << 20
    at = np.unique(np.concatenate([[0, 127, 128, 511, 512, K - 513, K - 512, K - 129, K - 128, K - 1],
                                   np.arange(1, 8) * (K // 8), np.arange(1, 8) * (K // 8) - 1]))
    codes, scales = whole_weights(N, K, 6)
    a, s = np.zeros((m, K), np.uint8), np.full((m, K // 32), 127, np.uint8)
    k = at[np.arange(m) % len(at)]
    a[np.arange(m), k] = 0x38
    w = oracle.dequant_weights(codes, scales, K, 1)[:, k].T
    got = F.gemm_mx8(_mx8(a, s, K), *(t.cuda() for t in F.native_repack(codes, scales, N, K)), N)
    assert np.array_equal(got.double().cpu().numpy(), w)

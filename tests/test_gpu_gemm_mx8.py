"""GPU parity of fp4_gemm_mx8 against the CPU oracle.

Bars.  Sums: the matrix core aligns the products of 16 k to the largest and keeps
13 bits below it (checked on the device), so the sum of a group is within 16 * 2^-13
= 2^-9 of its largest product, and the whole within 2^-9 sum |a w|; FP32
accumulation adds K / 16 * 2^-24 sum |a w|.  Where all products of a group lie within
12 bits and the sums fit FP32, the result is exact.  Gated: with |act'| <= 1.13, an
error dg, du of the products gives 1.13 |u| dg + |act(g)| du + 1.13 dg du; the
function's own FP32 evaluation is within 2^-16 relative (the exponential's argument,
at most 88 where it matters, is rounded to 2^-24 of itself).  Outputs: half a step of
their type."""

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F
from mixed_precision_bf16_amd import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, FP16 = torch.bfloat16, torch.float16


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
    return F.MX8(torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn),
                 torch.from_numpy(np.ascontiguousarray(scales)).cuda().view(torch.float8_e8m0fnu), K)


def _activations(m, K, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.standard_normal((m, K)) * np.exp2(rng.integers(-3, 4, (m, 1))) * (1 + 9 * (rng.random(K) < 0.02))
    return oracle.mx8_quantize_reference(x.astype(np.float32))


def _weights(N, K, seed):
    p = synth.make_random(1, N, K, 1, seed=seed)
    return p.codes, p.scales


def _upload(codes, scales, N, K):
    wq, sq = F.native_repack(codes, scales, N, K)
    return wq.cuda(), sq.cuda()


def _expected(a, w, K, gate=None, alpha=1.0):
    """(values, bound of the FP32 result's error), float64."""
    y, total = oracle.gemm_mx8_reference(*a, *w, K, alpha)
    group = 2.0 ** -9 + K / 16 * 2.0 ** -24
    err = total * (min(group, K * 2.0 ** -24) if len(y) <= 16 else group) + np.abs(y) * 2.0 ** -23
    if gate is None:
        return y, err
    n = y.shape[1] // 2
    g, u, dg, du = y[:, :n], y[:, n:], err[:, :n], err[:, n:]
    v = oracle.gate_reference(g, u, gate)
    act = np.abs(oracle.gate_reference(g, np.ones_like(g), gate))
    return v, 1.13 * np.abs(u) * dg + act * du + 1.13 * dg * du + 2.0 ** -16 * np.abs(v)


def _check16(got, want, err):
    assert got.shape == want.shape
    eps = torch.finfo(got.dtype).eps
    y = got.double().cpu().numpy()
    tiny = 2.0 ** -25 if got.dtype == FP16 else 0.0                       # half a step of FP16's subnormals
    # FP16: from 65504 and half a step (16) on, a value rounds to infinity
    over = np.isinf(y) & (np.sign(y) == np.sign(want)) & (np.abs(want) + err >= 65520.0) & (got.dtype == FP16)
    far = np.where(over, 0.0, np.abs(y - want) - (err + eps / 2 * (np.abs(want) + err) + tiny))
    assert (np.isfinite(y) | over).all() and far.max() <= 0, (far.max(), np.argwhere(far > 0)[:4])


def _check8(got, want, err):
    m, n = want.shape
    codes, scales = got.codes.view(torch.uint8).cpu().numpy(), got.scales.view(torch.uint8).cpu().numpy()
    Kp = oracle.mx8_padded(n)
    assert codes.shape == (m, Kp) and scales.shape == (m, Kp // 32)
    assert not codes[:, n:].any() and not scales[:, n // 32:].any()
    value = oracle.mx8_value(codes, scales, n)
    step = np.repeat(np.exp2(scales[:, :n // 32].astype(np.float64) - 127), 32, axis=1)
    far = np.abs(value - want) - (err + (np.abs(want) + err) * 2.0 ** -4 + 2.0 ** -10 * step)
    assert far.max() <= 0, (far.max(), np.argwhere(far > 0)[:4])
    blocks = lambda x: x.reshape(m, -1, 32)  # noqa: E731
    low, high = blocks(np.abs(want) - err).max(-1), blocks(np.abs(want) + err).max(-1)
    s = np.exp2(scales[:, :n // 32].astype(np.float64) - 127)
    assert (low <= 448 * s).all() and ((high > 224 * s) | (scales[:, :n // 32] == 0)).all()


def _run_all(m, N, K, gates, seed, alpha=1.0):
    a, w = _activations(m, K, seed), _weights(N, K, seed + 1)
    A, W = _mx8(*a, K), _upload(*w, N, K)
    for gate in gates:
        if gate and N % 32:
            continue
        want, err = _expected(a, w, K, gate, alpha)
        for dtype in (BF16, FP16):
            big = torch.full((m + 3, want.shape[1]), 7.0, dtype=dtype, device="cuda")
            got = F.gemm_mx8(A, *W, N, gate=gate, alpha=alpha, out=big[:m])
            _check16(got, want, err)
            assert big[m:].eq(7.0).all()
            assert F.gemm_mx8(A, *W, N, gate=gate, alpha=alpha, dtype=dtype).equal(got)     # the same bits again
        if want.shape[1] % 32 == 0:
            _check8(F.gemm_mx8(A, *W, N, gate=gate, alpha=alpha, mx8=True), want, err)


SIZES = [(1, 16, 32), (1, 1, 64), (2, 33, 96), (3, 32, 128), (5, 100, 544), (16, 64, 512), (17, 96, 2880), (31, 128, 160),
         (33, 1000, 640), (48, 320, 1024), (64, 160, 1056), (65, 64, 256), (100, 260, 1024), (129, 512, 2880),
         (256, 768, 512), (300, 96, 640), (513, 288, 384), (1, 2048, 28672), (16, 5000, 2880), (200, 2048, 4096)]


@pytest.mark.parametrize("m,N,K", SIZES)
def test_against_the_oracle(m, N, K):
    _run_all(m, N, K, (None, "silu", "gelu"), m * 31 + N + K)


# more than 16 rows and at most 512 k: a workgroup's first group is its last, so the first
# wait for a chunk meets the fewest loads behind it
@pytest.mark.parametrize("m,N,K", [(130, 4096, 512), (300, 2048, 384), (1000, 1024, 256), (520, 1056, 480), (2000, 2048, 160)])
def test_one_group_of_k(m, N, K):
    _run_all(m, N, K, (None, "silu"), m + N + K)


# the narrow tile's loop takes groups of 512 k two by two: one to five of them, the last
# one whole or of one to four steps of 128
@pytest.mark.parametrize("K", [544, 896, 1024, 1056, 1152, 1312, 1536, 1568, 1760, 2048, 2080, 2560])
def test_groups_of_k(K):
    _run_all(70, 160, K, (None, "silu"), K)


def test_alpha():
    _run_all(20, 192, 512, (None, "silu", "gelu"), 4, alpha=0.037)
    _run_all(3, 64, 256, (None, "silu"), 5, alpha=-8.0)


@pytest.mark.parametrize("m", [16, 48, 160])
def test_every_weight_by_one_hot_rows(m):
    """Row i holds one 1 at k: the column of weights at k, exactly."""
    N, K = 48, 2880
    codes, scales = _weights(N, K, 77)
    W = _upload(codes, scales, N, K)
    want = oracle.dequant_weights(codes, scales, K, 1)                     # [N][K]
    for first in range(0, K, m):
        ac = np.zeros((m, oracle.mx8_padded(K)), np.uint8)
        asc = np.full((m, oracle.mx8_padded(K) // 32), 127, np.uint8)
        i = np.arange(m)
        k = (first + i) % K
        ac[i, k] = 0x38
        got = F.gemm_mx8(_mx8(ac, asc, K), *W, N).double().cpu().numpy()
        assert np.array_equal(got, want[:, k].T)


@pytest.mark.parametrize("m", [7, 64, 257])
def test_whole_numbers_are_exact(m):
    rng = np.random.Generator(np.random.PCG64(m))
    N, K = 208, 1408
    ac = rng.choice(np.array([0, 0x38, 0xB8, 0x40, 0xC0], np.uint8), (m, K))           # 0, +-1, +-2
    wc = rng.choice(np.array([0, 2, 10, 4, 12], np.uint8), (N, K))
    a_s, w_s = np.full((m, K // 32), 127, np.uint8), rng.integers(127, 129, (N, K // 32)).astype(np.uint8)
    w = (wc[:, 0::2] | wc[:, 1::2] << 4).astype(np.uint8)
    y, _ = oracle.gemm_mx8_reference(ac, a_s, w, w_s, K)
    for dtype in (BF16, FP16):
        got = F.gemm_mx8(_mx8(ac, a_s, K), *_upload(w, w_s, N, K), N, dtype=dtype)
        assert got.cpu().equal(torch.from_numpy(y).to(dtype))


@pytest.mark.parametrize("m", [14, 40, 130])
def test_nan_and_zero_rows_stay_in_their_row(m):
    N, K = 96, 512
    a, w = _activations(m, K, 3), _weights(N, K, 4)
    a[0][5, 100] = 0x7F
    a[1][9, 3] = 0xFF
    a[0][11] = 0
    W = _upload(*w, N, K)
    A = _mx8(*a, K)
    rest = [i for i in range(m) if i not in (5, 9)]
    clean = (np.where((a[0] & 127) == 127, 0, a[0]).astype(np.uint8), np.where(a[1] == 255, 127, a[1]).astype(np.uint8))
    for gate in (None, "silu"):
        got = F.gemm_mx8(A, *W, N, gate=gate)
        assert got[[5, 9]].isnan().all() and got[11].eq(0).all()
        want, err = _expected(clean, w, K, gate)
        _check16(got[rest], want[rest], err[rest])
        eight = F.gemm_mx8(A, *W, N, gate=gate, mx8=True) if not gate else None
        if eight is not None:
            v = eight.codes[:, :N].float()
            assert v[[5, 9]].isnan().all() and not v[rest].isnan().any() and v[11].eq(0).all()


def test_gate_far_out():
    """Gates far from zero, both ways: the function keeps its limits."""
    m, N, K = 4, 64, 128
    ac, a_s = np.zeros((m, K), np.uint8), np.full((m, K // 32), 127, np.uint8)
    ac[:, 0] = 0x38                                                        # 1 at k = 0
    wc = np.zeros((N, K // 2), np.uint8)
    wc[:32, 0] = np.where(np.arange(32) % 2, 0x0F, 0x07)                   # gates -6, 6
    wc[32:, 0] = 0x02                                                      # up 1
    w_s = np.full((N, K // 32), 127, np.uint8)
    a_s[:, 0] = [127, 131, 140, 180]
    want, _ = oracle.gemm_mx8_reference(ac, a_s, wc, w_s, K)
    for gate in ("silu", "gelu"):
        v = oracle.gate_reference(want[:, :32], want[:, 32:], gate)
        got = F.gemm_mx8(_mx8(ac, a_s, K), *_upload(wc, w_s, N, K), N, gate=gate).double().cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - v) <= np.abs(v) * (2.0 ** -8 + 2.0 ** -16) + 2.0 ** -126).all()


def _columns(wq, sq, N, K, tiles):
    """Canonical codes and scales of the given weight tiles, taken from the packed bytes on the device."""
    KB = -(-K // 512) * 4
    cs, ss = [], []
    for t in tiles:
        one = F.native_unpack(wq[t * KB * 1024:(t + 1) * KB * 1024].cpu(), sq[t * KB * 64:(t + 1) * KB * 64].cpu(), 16, K)
        cs.append(one[0])
        ss.append(one[1])
    return np.concatenate(cs), np.concatenate(ss)


def _random_packed(N, K, seed):
    """Random weights in the packed layout, made on the device, zero behind K."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nw, ns = F.native_repack_size(N, K)
    Np, Kp = -(-N // 16) * 16, -(-K // 512) * 512
    wq = torch.randint(0, 256, (nw,), dtype=torch.uint8, device="cuda", generator=gen)
    sq = torch.randint(120, 130, (ns,), dtype=torch.uint8, device="cuda", generator=gen)
    if Kp != K:
        block = torch.arange(K // 128, Kp // 128, device="cuda")[:, None] * 4 + torch.arange(4, device="cuda")
        wq.view(Np // 16, Kp // 128, 4, 256)[:, K // 128:, :, :] *= (block * 32 < K)[None, :, :, None].to(torch.uint8)
    return wq, sq


def _check_sampled(m, N, K, gate, tiles):
    """16-bit and (where the columns allow) 8-bit results on the columns of the given output tiles."""
    wq, sq = _random_packed(N, K, m + N)
    a = _activations(m, K, 8)
    A = _mx8(*a, K)
    cols = N // 2 if gate else N
    tiles = sorted({min(max(t, 0), cols // 16 - 1) for t in tiles})
    got = F.gemm_mx8(A, wq, sq, N, gate=gate)
    pick = np.concatenate([np.arange(16 * t, 16 * t + 16) for t in tiles])
    w = _columns(wq, sq, N, K, tiles + ([t + cols // 16 for t in tiles] if gate else []))
    want, err = _expected(a, w, K, gate)
    _check16(got[:, torch.from_numpy(pick).cuda()], want, err)
    if cols % 32 == 0 and N < 1 << 20:
        eight = F.gemm_mx8(A, wq, sq, N, gate=gate, mx8=True)
        pair = sorted({t // 2 for t in tiles})
        p = np.concatenate([np.arange(32 * t, 32 * t + 32) for t in pair])
        two = [x for t in pair for x in (2 * t, 2 * t + 1)]
        w = _columns(wq, sq, N, K, two + ([t + cols // 16 for t in two] if gate else []))
        want, err = _expected(a, w, K, gate)
        codes = torch.zeros((m, F.mx8_padded(len(p))), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((m, F.mx8_padded(len(p)) // 32), dtype=torch.uint8, device="cuda")
        codes[:, :len(p)] = eight.codes.view(torch.uint8)[:, torch.from_numpy(p).cuda()]
        scales[:, :len(pair)] = eight.scales.view(torch.uint8)[:, pair]
        _check8(F.MX8(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), len(p)), want, err)
        assert not eight.codes.view(torch.uint8)[:, cols:].any() and not eight.scales.view(torch.uint8)[:, cols // 32:].any()


@pytest.mark.parametrize("m,N,K,gate", [(16, 57344, 8192, "silu"), (16, 10240, 8192, None), (256, 8192, 28672, None),
                                        (100, 28672, 4096, "gelu"), (700, 20480, 2880, None),
                                        (5, (1 << 20) + 16, 8192, None)])
def test_large_on_sampled_columns(m, N, K, gate):
    cols = N // 2 if gate else N
    _check_sampled(m, N, K, gate, [0, 1, cols // 48, cols // 16 - 1, cols // 32 + 1, min(cols // 16 - 1, 1 << 16)])


# one size for every kernel and split of K that the choice by the time model reaches besides
@pytest.mark.parametrize("m,N,K,gate", [
    (17, 11200, 32, None), (21, 17440, 32, "silu"), (25, 52928, 32, "silu"), (35, 39712, 32, None), (70, 5872, 4928, None),
    (1780, 160, 2784, "silu"), (17, 16, 14176, None), (65, 16064, 3840, "silu"), (125, 64, 1184, "silu"),
    (157, 64, 1600, "gelu"), (73, 39200, 32, "silu"), (132, 14080, 8192, "silu"), (67, 17632, 5952, None),
    (75, 8928, 11488, None), (2744, 64, 17888, "silu"), (320, 13152, 31648, "silu"), (1051, 3904, 12512, None),
    (261, 7920, 30752, None)])
def test_every_kernel_on_sampled_columns(m, N, K, gate):
    last = (N // 2 if gate else N) // 16 - 1
    _check_sampled(m, N, K, gate, [0, 1, last // 2, last - 1, last])


@pytest.mark.parametrize("m,N,K,gate", [(2754, 32, 2944, "silu"), (33, 10240, 8192, None), (64, 8192, 28672, None),
                                        (96, 10240, 8192, None), (64, 20480, 4096, "gelu")])
def test_narrow_tiles_on_sampled_columns(m, N, K, gate):
    last = (N // 2 if gate else N) // 16 - 1
    _check_sampled(m, N, K, gate, sorted({0, last // 2, max(last - 1, 0), last}))


@pytest.mark.parametrize("m", [3, 24, 70])
def test_longest_rows(m):
    _run_all(m, 32, 1 << 20, (None, "silu"), m)


def test_activations_near_the_size_limit():
    m, N, K = 130816, 32, 16384                                            # 2.14e9 bytes of codes
    few = _activations(64, K, 1)
    codes = torch.from_numpy(few[0]).cuda().repeat(m // 64, 1)
    scales = torch.from_numpy(few[1]).cuda().repeat(m // 64, 1)
    w = _weights(N, K, 2)
    got = F.gemm_mx8(F.MX8(codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), K), *_upload(*w, N, K), N)
    want, err = _expected(few, w, K)
    for at in (0, 64 * 777, m - 64):
        _check16(got[at:at + 64], want, err)
    assert got.reshape(m // 64, 64, N).eq(got[:64]).all()


def test_no_rows():
    W = _upload(*_weights(64, 128, 1), 64, 128)
    assert F.gemm_mx8(F.new_mx8(0, 128), *W, 64).shape == (0, 64)
    assert F.gemm_mx8(F.new_mx8(0, 128), *W, 64, gate="silu", mx8=True).codes.shape == (0, 128)

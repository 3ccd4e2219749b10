"""GPU parity of fp4_rms_norm and fp4_quantize_mx8 against the CPU oracle.

Bar: the same bits.  The definition rounds to FP32 at stated places and sums the
squares in FP64, so that 8-bit codes, scales, 16-bit results and the sum with the
residual are fixed (a NaN may have either sign)."""

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F

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


def _rows(rows, width, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, width), generator=g) * torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g).float())
    return (x * (1 + 20 * (torch.rand(width, generator=g) < 0.02))).to(dtype)


def _same(got, want, dtype):
    """16-bit results equal to the FP32 values `want` rounded once."""
    want = torch.from_numpy(np.asarray(want, dtype=np.float32)).to(dtype)
    got = got.cpu()
    assert got.shape == want.shape
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), (int((~same).sum()), got[~same][:4], want[~same][:4])


def _same_mx8(got, want, K):
    """8-bit rows equal to the quantized FP32 values `want`, padding included."""
    codes, scales = oracle.mx8_quantize_reference(want)
    gc = got.codes.view(torch.uint8).cpu().numpy()
    gs = got.scales.view(torch.uint8).cpu().numpy()
    assert gc.shape == codes.shape and gs.shape == scales.shape
    assert np.array_equal(gs, scales), np.argwhere(gs != scales)[:4]
    bad = (gc != codes) & ~(((gc & 127) == 127) & ((codes & 127) == 127))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], gc[bad][:4], codes[bad][:4])


SIZES = [(1, 32), (3, 64), (5, 96), (2, 512), (4, 544), (130, 128), (7, 2048), (33, 2080), (9, 2880), (3, 4096), (2, 8192),
         (2, 8224), (1, 16384), (3, 20000), (2, 32768), (2, 32800), (1, 65536)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,width", SIZES)
def test_norm_bits(rows, width, residual, dtype):
    x = _rows(rows, width, dtype, width + rows)
    r = _rows(rows, width, dtype, width + rows + 1) if residual else None
    w = _rows(1, width, dtype, 5)[0]
    y, h = oracle.rms_norm_reference(x.double().numpy(), w.double().numpy(), 1e-5,
                                     r.double().numpy() if residual else None)
    xc, wc, rc = x.cuda(), w.cuda(), r.cuda() if residual else None
    for mx8 in (False, True):
        got = F.rms_norm(xc, wc, 1e-5, residual=rc, mx8=mx8)
        torch.cuda.synchronize()
        if residual:
            got, total = got
            _same(total, h, dtype)
        if mx8:
            _same_mx8(got, y, width)
        else:
            _same(got, y, dtype)


@pytest.mark.parametrize("width", [8, 24, 40, 520, 1000, 8200])
def test_norm_of_any_vector_width_in_16_bits(width):
    x, w = _rows(6, width, BF16, width), _rows(1, width, BF16, 2)[0]
    y, _ = oracle.rms_norm_reference(x.double().numpy(), w.double().numpy(), 1e-6)
    _same(F.rms_norm(x.cuda(), w.cuda()), y, BF16)


def test_norm_without_weight_and_of_special_rows():
    x = _rows(8, 256, BF16, 3)
    x[0] = 0.0
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 3e38                                      # squares beyond FP32
    x[4] = 1e-40                                     # subnormal
    x[5, :] = 0.0
    x[5, 100] = -2.0
    y, _ = oracle.rms_norm_reference(x.double().numpy(), None, 1e-6)
    _same(F.rms_norm(x.cuda(), None, 1e-6), y, BF16)
    got = F.rms_norm(x.cuda(), None, 1e-6, mx8=True)
    _same_mx8(got, y, 256)


@pytest.mark.parametrize("width", [2880, 8192, 40960])
def test_norm_strides_and_places(width):
    """Strided rows; the sum in the residual's place, the result in x's; a residual
    of one row for all."""
    big = torch.zeros((5, width + 72), dtype=BF16)
    big[:, 8:8 + width] = _rows(5, width, BF16, 1)
    r = _rows(5, width, BF16, 2)
    w = _rows(1, width, BF16, 3)[0]
    y, h = oracle.rms_norm_reference(big[:, 8:8 + width].double().numpy(), w.double().numpy(), 1e-6, r.double().numpy())
    x, rc = big.cuda(), r.cuda()
    view = x[:, 8:8 + width]
    got, total = F.rms_norm(view, w.cuda(), residual=rc, sum_out=rc, out=view)
    assert total is rc and got is view
    _same(rc, h, BF16)
    _same(view, y, BF16)
    assert x[:, :8].eq(0).all() and x[:, 8 + width:].eq(0).all()
    x, rc = big.cuda(), r.cuda()
    view = x[:, 8:8 + width]
    got, total = F.rms_norm(view, w.cuda(), residual=rc, sum_out=view, mx8=True)     # the sum in x's place
    _same(view, h, BF16)
    _same_mx8(got, y, width)
    assert rc.cpu().equal(r)
    one = r[:1].expand(5, width)
    y, h = oracle.rms_norm_reference(big[:, 8:8 + width].double().numpy(), w.double().numpy(), 1e-6, one.double().numpy())
    got, total = F.rms_norm(big.cuda()[:, 8:8 + width], w.cuda(), residual=r[:1].cuda().expand(5, width))
    _same(total, h, BF16)
    _same(got, y, BF16)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantizer_on_every_value(dtype):
    """Every 16-bit value beside every kind of block maximum: the codes at each
    scale, the borders between codes, subnormals, NaN and infinities."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    tops = torch.tensor([0.0, 2.0 ** -9, 0.4375, 0.876, 1.0, 448.0, 449.0, 65504.0] +
                        ([1e-38, 3e38, 2.0 ** -130, 2.0 ** -118] if dtype == BF16 else [2.0 ** -24, 3e-5, 7e-4, 0.01]))
    for top in tops.tolist():
        x = torch.zeros((65536 // 31 + 1, 32), dtype=dtype)
        x[:, 0] = top
        flat = torch.zeros((len(x) * 31,), dtype=dtype)
        flat[:65536] = every
        x[:, 1:] = flat.reshape(-1, 31)
        _same_mx8(F.quantize_mx8(x.cuda()), x.double().numpy(), 32)
    # values alone in their block: every scale
    x = torch.zeros((65536, 32), dtype=dtype)
    x[:, 5] = every
    _same_mx8(F.quantize_mx8(x.cuda()), x.double().numpy(), 32)


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 160), (5, 2880), (2, 28672)])
def test_quantizer_rows(rows, K):
    x = torch.zeros((rows, K + 8), dtype=BF16)
    x[:, :K] = _rows(rows, K, BF16, K)
    got = F.quantize_mx8(x.cuda()[:, :K])
    _same_mx8(got, x[:, :K].double().numpy(), K)
    into = F.new_mx8(rows, K)
    into.codes.view(torch.uint8).fill_(255)
    into.scales.view(torch.uint8).fill_(255)
    assert F.quantize_mx8(x.cuda()[:, :K], out=into) is into
    _same_mx8(into, x[:, :K].double().numpy(), K)


def test_longest_rows():
    n = 1 << 20
    x, r = (torch.randn((2, n), generator=torch.Generator().manual_seed(i)).to(BF16) for i in (1, 2))
    y, h = oracle.rms_norm_reference(x.double().numpy(), None, 1e-6, r.double().numpy())
    got, total = F.rms_norm(x.cuda(), residual=r.cuda(), mx8=True)
    codes, scales = oracle.mx8_quantize_reference(y)
    assert np.array_equal(got.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(got.scales.view(torch.uint8).cpu().numpy(), scales)
    assert total.cpu().equal(torch.from_numpy(h.astype(np.float32)).to(BF16))
    codes, scales = oracle.mx8_quantize_reference(x.double().numpy())
    got = F.quantize_mx8(x.cuda())
    assert np.array_equal(got.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(got.scales.view(torch.uint8).cpu().numpy(), scales)


def test_many_rows():
    """More rows than one launch takes."""
    rows = (1 << 20) + 5
    x = torch.randn((997, 32), generator=torch.Generator().manual_seed(1)).to(BF16)
    big = x.cuda().repeat(-(-rows // 997), 1)[:rows].contiguous()
    y, _ = oracle.rms_norm_reference(x.double().numpy(), None, 1e-6)
    want = torch.from_numpy(y.astype(np.float32)).to(BF16).cuda()
    got = F.rms_norm(big)
    eight = F.rms_norm(big, mx8=True)
    ref = F.rms_norm(x.cuda(), mx8=True)
    for at in (0, (1 << 20) - 500, rows - 997):
        i = (torch.arange(at, min(at + 997, rows), device="cuda")) % 997
        assert got[at:at + 997].equal(want[i])
        assert eight.codes[at:at + 997].view(torch.uint8).equal(ref.codes.view(torch.uint8)[i])
        assert eight.scales[at:at + 997].view(torch.uint8).equal(ref.scales.view(torch.uint8)[i])


def test_no_rows():
    x = torch.empty((0, 64), dtype=BF16, device="cuda")
    assert F.rms_norm(x).shape == (0, 64)
    assert F.rms_norm(x, residual=x)[1].shape == (0, 64)
    assert F.quantize_mx8(x).codes.shape == (0, 128)

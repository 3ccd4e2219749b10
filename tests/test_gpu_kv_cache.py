"""GPU parity of fp4_kv_append and fp4_kv_read against the CPU oracle.

Bars: the cache's bytes equal to the oracle's, untouched ones included
(integer decisions taken in FP32 on both sides); rows read back equal to the
oracle's value rounded once where alpha is a power of two (then code x scale x
alpha is exact in FP32), else within half a step of the output type plus the
FP32 product's 2^-24."""

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


def _say(*a):
    print("[case]", *a, flush=True)


def _rows(n, H, D, dtype, seed, specials=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, H, D), generator=g) * torch.exp2(torch.randint(-6, 7, (n, H, 1), generator=g).float())
    if specials and n >= 4:
        x[0, 0, :32] = 0.0
        mids = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        x[1, 0, :8], x[1, 0, 8:16], x[1, 0, 16:32] = mids, -mids, 0.0
        x[2, -1, -32:] = -1e-6
        x[2, -1, -1] = 7.0
        x[3, 0, 3], x[3, 0, 4], x[3, 0, 40] = float("nan"), 2.0, float("nan")
        x[3, -1, -1], x[3, -1, -2] = float("inf"), float("-inf")
    return x.to(dtype)


def _slots(n, total, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    return torch.from_numpy(rng.permutation(total)[:n].astype(np.int64))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("fmt,D,H,page,n,ka,va", [
    (0, 64, 3, 32, 37, 1.0, 1.0), (0, 128, 8, 64, 64, 1.0, 0.5), (0, 256, 1, 96, 9, 0.02, 1.7),
    (1, 64, 1, 128, 1, 1.0, 1.0), (1, 128, 2, 32, 130, 2.0 ** -7, 0.3), (1, 256, 4, 64, 33, 3.0, 1.0)])
def test_append_bit_exact(dtype, fmt, D, H, page, n, ka, va):
    _say("append", dtype, fmt, D, H, page, n)
    pages = -(-n // page) + 2
    cache = F.new_kv_cache(pages, page, H, D, fmt, ka, va)
    start = torch.randint(0, 256, (cache.data.numel(),), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    cache.data.copy_(start)
    k, v = _rows(n, H, D, dtype, 10 * n + D), _rows(n, H, D, dtype, 10 * n + D + 1)
    slots = _slots(n, pages * page, n)
    if n > 8:
        slots[5], slots[7], slots[8] = -1, pages * page, 1 << 62
    F.kv_append(cache, k.cuda(), v.cuda(), slots.cuda())
    want = start.numpy().copy()
    oracle.kv_write_reference(want, slots.numpy(), k.float().numpy(), v.float().numpy(), page, fmt, ka, va)
    assert np.array_equal(cache.data.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", [0, 1])
def test_append_every_fp16_value(fmt):
    """Every FP16 bit pattern, in blocks with scales from small to large."""
    bits = np.arange(65536, dtype=np.uint16).astype(np.int16)
    x = torch.from_numpy(bits.copy()).view(FP16)
    rng = np.random.Generator(np.random.PCG64(3))
    x = torch.cat([x, x[torch.from_numpy(rng.permutation(65536))]]).reshape(-1, 1, 128)
    n = x.shape[0]
    cache = F.new_kv_cache(n // 64, 64, 1, 128, fmt)
    cache.data.zero_()
    F.kv_append(cache, x.cuda(), x.flip(0).contiguous().cuda(), torch.arange(n, device="cuda"))
    want = np.zeros(cache.data.numel(), np.uint8)
    f = x.float().numpy()
    oracle.kv_write_reference(want, np.arange(n), f, f[::-1].copy(), 64, fmt)
    assert np.array_equal(cache.data.cpu().numpy(), want)


def test_append_agrees_with_quantize():
    """The codes are fp4_quantize's: both are the same rule on the same rows."""
    x = _rows(64, 2, 128, BF16, 5).cuda()
    for fmt in (0, 1):
        cache = F.new_kv_cache(1, 64, 2, 128, fmt)
        F.kv_append(cache, x, x, torch.arange(64, device="cuda"))
        codes, scales = F.quantize(x.reshape(128, 128), fmt)
        kc, vc, ks, vs = oracle.kv_offsets(fmt, 128)
        data = cache.data.cpu().numpy().reshape(2, 2, -1)          # [head][tile]
        t = np.arange(64)
        for off, want in ((kc, codes), (vc, codes), (ks, scales), (vs, scales)):
            got = np.stack([np.stack([data[h, i // 32, off[i % 32]] for i in t]) for h in range(2)], 1)
            assert np.array_equal(got.reshape(128, -1), want.cpu().numpy())


@pytest.mark.parametrize("layout", ["packed", "heads_first", "broadcast"])
def test_append_strides(layout):
    n, H, D, page = 21, 4, 128, 32
    if layout == "packed":            # one projection's rows: q | k | v
        x = _rows(n, 3 * H, D, BF16, 7).cuda()
        k, v = x[:, H:2 * H], x[:, 2 * H:]
    elif layout == "heads_first":
        x = _rows(2 * H, n, D, BF16, 8).cuda()
        k, v = x[:H].transpose(0, 1), x[H:].transpose(0, 1)
    else:
        k = _rows(1, H, D, BF16, 9).cuda().expand(n, H, D)
        v = _rows(n, 1, D, BF16, 11).cuda().expand(n, H, D)
    cache = F.new_kv_cache(2, page, H, D, 0)
    cache.data.zero_()
    F.kv_append(cache, k, v, torch.arange(3, 3 + n, device="cuda"))
    want = np.zeros(cache.data.numel(), np.uint8)
    oracle.kv_write_reference(want, np.arange(3, 3 + n), k.float().cpu().numpy(), v.float().cpu().numpy(), page, 0)
    assert np.array_equal(cache.data.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("fmt,D,H,page,ka,va", [(0, 64, 2, 64, 1.0, 0.25), (0, 128, 8, 32, 1.0, 1.0),
                                                (0, 256, 3, 96, 0.37, 1.9), (1, 64, 5, 32, 1.0, 1.0),
                                                (1, 128, 1, 128, 0.011, 3.0), (1, 256, 2, 64, 1.0, 1.0)])
def test_read(dtype, fmt, D, H, page, ka, va):
    _say("read", dtype, fmt, D, H, page)
    pages = 3
    rng = np.random.Generator(np.random.PCG64(D + 7 * fmt))
    data = np.zeros(F.kv_cache_size(pages, page, H, D, fmt), np.uint8)
    total = pages * page
    x = rng.standard_normal((2, total, H, D)).astype(np.float32) * np.exp2(rng.integers(-5, 6, (2, total, H, 1)))
    oracle.kv_write_reference(data, np.arange(total), x[0], x[1], page, fmt)
    cache = F.KVCache(torch.from_numpy(data).cuda(), pages, page, H, D, fmt, ka, va)
    slots = _slots(total - 10, total, 4)
    slots[3], slots[-1] = -5, total
    k, v = F.kv_read(cache, slots.cuda(), dtype=dtype)
    inside = np.clip(slots.numpy(), 0, total - 1)
    want = oracle.kv_read_reference(data, inside, H, D, page, fmt, ka, va)
    for got, ref, alpha in ((k, want[0], ka), (v, want[1], va)):
        ref[[3, -1]] = 0.0
        got = got.double().cpu().numpy()
        if np.log2(alpha) == int(np.log2(alpha)):
            # exact in FP32: one rounding to the type (float64 -> float32 is exact here)
            assert np.array_equal(got, torch.from_numpy(ref.astype(np.float32)).to(dtype).double().numpy())
        else:
            half = torch.finfo(dtype).eps / 2
            tiny = 0.0 if dtype == BF16 else 2.0 ** -25   # half a step of FP16's subnormals
            assert np.all(np.abs(got - ref) <= np.abs(ref) * (half + 2.0 ** -23) + tiny)


def test_read_into_strided_outputs_and_one_of_them():
    n, H, D = 40, 2, 64
    cache = F.new_kv_cache(2, 32, H, D, 0)
    x = _rows(64, 2 * H, D, FP16, 2, specials=False).cuda()
    F.kv_append(cache, x[:, :H], x[:, H:], torch.arange(64, device="cuda"))
    slots = torch.arange(5, 5 + n, device="cuda")
    k, v = F.kv_read(cache, slots, dtype=FP16)
    both = torch.full((n, 2 * H + 1, D), 7.0, dtype=FP16, device="cuda")
    F.kv_read(cache, slots, k_out=both[:, :H], v_out=both[:, H:2 * H])
    assert torch.equal(both[:, :H], k) and torch.equal(both[:, H:2 * H], v) and torch.all(both[:, 2 * H] == 7.0)
    heads_first = torch.empty((H, n, D), dtype=FP16, device="cuda")
    F.kv_read(cache, slots, k_out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), k)
    only = torch.empty_like(v)
    st = F.lib().fp4_kv_read(cache._ref, slots.data_ptr(), n, None, only.data_ptr(), 0, 0, H * D, D, 1,
                             F._stream_handle(None))
    assert st == 0 and torch.equal(only, v)
    for bad in (lambda: F.kv_read(cache, slots, k_out=both[:, :H, ::2]), lambda: F.kv_read(cache, slots.int()),
                lambda: F.kv_read(cache, slots, k_out=both[:, 1:H + 1].flatten()),
                lambda: F.kv_read(cache, slots, dtype=torch.float32),
                lambda: F.kv_append(cache, x[:, :H], x[:, H:], slots),
                lambda: F.kv_append(cache, x[:n, :H], x[:n, H:].bfloat16(), slots),
                lambda: F.kv_append(cache, x[:n, :1], x[:n, H:], slots),
                lambda: F.kv_append(cache, x[:n, :H].cpu(), x[:n, H:], slots)):
        with pytest.raises(ValueError):
            bad()


def test_no_tokens_is_a_no_op():
    cache = F.new_kv_cache(1, 32, 1, 64, 0)
    cache.data.fill_(9)
    e = torch.empty((0, 1, 64), dtype=BF16, device="cuda")
    F.kv_append(cache, e, e, torch.empty(0, dtype=torch.int64, device="cuda"))
    k, v = F.kv_read(cache, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert torch.all(cache.data == 9) and k.shape == (0, 1, 64) == v.shape


def test_cache_past_4_gib():
    """Slots whose bytes lie past 2^32: first and last page, and a row before
    and after the 4 GiB border."""
    H, D, page = 8, 128, 64
    pages = (5 << 30) // (page * H * 144)
    cache = F.new_kv_cache(pages, page, H, D, 0)
    border = (1 << 32) // (H * 144)
    slots = torch.tensor([0, pages * page - 1, border - 1, border, border + page], device="cuda")
    x = _rows(5, 2 * H, D, BF16, 6, specials=False).cuda()
    F.kv_append(cache, x[:, :H], x[:, H:], slots)
    k, v = F.kv_read(cache, slots)
    small = F.new_kv_cache(1, page, H, D, 0)
    at = torch.arange(5, device="cuda")
    F.kv_append(small, x[:, :H], x[:, H:], at)
    ks, vs = F.kv_read(small, at)
    assert torch.equal(k, ks) and torch.equal(v, vs)


def test_more_tokens_than_one_launch_covers():
    n = (1 << 20) + 5
    cache = F.new_kv_cache(n // 32 + 1, 32, 1, 64, 1)
    x = torch.randn((n, 2, 64), dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    slots = torch.arange(n, device="cuda")
    F.kv_append(cache, x[:, :1], x[:, 1:], slots)
    k, v = F.kv_read(cache, slots)
    pick = torch.tensor([0, 1, n - 6, n - 5, n - 4, n - 1], device="cuda")
    small = F.new_kv_cache(1, 32, 1, 64, 1)
    F.kv_append(small, x[pick, :1], x[pick, 1:], torch.arange(6, device="cuda"))
    ks, vs = F.kv_read(small, torch.arange(6, device="cuda"))
    assert torch.equal(k[pick], ks) and torch.equal(v[pick], vs)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("ka,va", [(1.0, 0.37), (2.0 ** -20, 3000.0), (2.0 ** 60, 1e-30)])
def test_append_every_bf16_value(fmt, ka, va):
    """Every BF16 bit pattern, among its neighbours and mixed: all NaNs, the
    signalling ones too, become 0 and leave the rest of their block alone."""
    bits = np.arange(65536, dtype=np.uint16)
    mixed = np.random.Generator(np.random.PCG64(9)).permutation(bits)
    x = torch.from_numpy(np.concatenate([bits, mixed]).view(np.int16)).view(BF16).reshape(-1, 1, 128)
    n = x.shape[0]
    cache = F.new_kv_cache(n // 64, 64, 1, 128, fmt, ka, va)
    cache.data.zero_()
    F.kv_append(cache, x.cuda(), x.flip(0).contiguous().cuda(), torch.arange(n, device="cuda"))
    want = np.zeros(cache.data.numel(), np.uint8)
    f = x.float().numpy()
    with np.errstate(all="ignore"):
        oracle.kv_write_reference(want, np.arange(n), f, f[::-1].copy(), 64, fmt, ka, va)
    assert np.array_equal(cache.data.cpu().numpy(), want)

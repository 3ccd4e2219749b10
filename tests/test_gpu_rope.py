"""GPU parity of fp4_rope and fp4_kv_append_rope against the CPU oracle.

Bar: the same bits.  The definition rounds cosine and sine and every product and
sum to FP32; the float64 functions of two sides differ by an ulp of float64, which
moves an FP32 rounding once in 2^27 values.  The cache's bytes are those of the two
calls one after another."""

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


def _x(tokens, heads, D, dtype, seed):
    return torch.randn((tokens, heads, D), generator=torch.Generator().manual_seed(seed)).to(dtype)


def _positions(tokens, seed, far=200000):
    rng = np.random.Generator(np.random.PCG64(seed))
    p = rng.integers(0, far, tokens)
    p[: min(tokens, 3)] = [0, 1, far][: min(tokens, 3)]
    return torch.from_numpy(p.astype(np.int64))


def _want(x, pos, freq, inter, amp=1.0):
    y = oracle.rope_reference(x.double().numpy(), pos.numpy(), freq.cpu().numpy(), inter, amp)
    return torch.from_numpy(y.astype(np.float32)).to(x.dtype)


SHAPES = [(1, 1, 64, 64), (1, 72, 128, 128), (5, 9, 128, 64), (13, 3, 96, 24), (9, 4, 80, 20), (17, 2, 256, 192),
          (4, 5, 64, 62), (3, 2, 8, 2), (301, 7, 128, 96), (2100, 3, 64, 32), (2, 3, 1024, 1024), (6, 1, 128, 34)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,heads,D,R", SHAPES)
def test_rope_bits(tokens, heads, D, R, inter, dtype):
    x, pos = _x(tokens, heads, D, dtype, tokens + D), _positions(tokens, R)
    freq, _ = F.rope_frequencies(R, 500000.0)
    got = F.rope(x.cuda(), pos.cuda(), freq, interleaved=inter)
    want = _want(x, pos, freq, inter)
    assert got.cpu().equal(want)
    y = x.cuda()
    assert F.rope(y, pos.cuda(), freq, interleaved=inter, out=y) is y          # in place
    assert y.cpu().equal(want)


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 31 - 1, -5])
def test_far_positions(far):
    x = _x(4, 2, 64, BF16, 3)
    pos = torch.tensor([far, far - 1, far - 12345, far // 3], dtype=torch.int64)
    freq, _ = F.rope_frequencies(64)
    assert F.rope(x.cuda(), pos.cuda(), freq).cpu().equal(_want(x, pos, freq, False))


def test_special_values_amplitude_and_angles():
    x = _x(5, 2, 64, BF16, 9)
    x[0, 0, 3], x[1, 1, 40], x[2, 0, 0], x[3] = float("nan"), float("inf"), -0.0, 0.0
    pos = torch.tensor([0, 7, 0, 9, 100000], dtype=torch.int64)
    freq, amp = F.rope_frequencies(64, scaling="yarn", factor=16.0, original=4096)
    got, want = F.rope(x.cuda(), pos.cuda(), freq, amplitude=amp).cpu(), _want(x, pos, freq, False, amp)
    assert ((got == want) | (got.isnan() & want.isnan())).all()
    # multiples of pi / 4 and their FP32 neighbours as frequencies of position 1 and 3
    f = (torch.arange(1, 65, dtype=torch.float64) * np.pi / 4).float()
    f = torch.cat((f, torch.nextafter(f, torch.full_like(f, 1e9)), torch.nextafter(f, torch.zeros_like(f))))
    x = _x(2, 1, 2 * len(f), FP16, 4)
    pos = torch.tensor([1, 3], dtype=torch.int64)
    assert F.rope(x.cuda(), pos.cuda(), f.cuda()).cpu().equal(_want(x, pos, f, False))


def test_strides():
    """Queries and keys of one projection, turned in place; head-major output."""
    qkv = _x(11, 12, 128, BF16, 5)
    pos = _positions(11, 1)
    freq, _ = F.rope_frequencies(128)
    y = qkv.cuda()
    F.rope(y[:, :10], pos.cuda(), freq, out=y[:, :10])
    assert y[:, :10].cpu().equal(_want(qkv[:, :10], pos, freq, False)) and y[:, 10:].cpu().equal(qkv[:, 10:])
    out = torch.zeros((12, 11, 128), dtype=BF16, device="cuda")
    F.rope(qkv.cuda(), pos.cuda(), freq, out=out.transpose(0, 1))
    assert out.transpose(0, 1).cpu().equal(_want(qkv, pos, freq, False))
    one = qkv[:1].cuda().expand(11, 12, 128)                                       # one row for all tokens
    assert F.rope(one, pos.cuda(), freq).cpu().equal(_want(qkv[:1].expand(11, 12, 128), pos, freq, False))


CACHES = [(0, 64, 3, 6, 32, 37, 64), (0, 128, 8, 64, 64, 1, 128), (0, 128, 2, 10, 64, 130, 64), (0, 256, 1, 3, 96, 9, 192),
          (1, 64, 1, 5, 128, 1, 32), (1, 128, 2, 16, 32, 131, 128), (1, 256, 4, 4, 64, 33, 250), (0, 128, 4, 8, 32, 2050, 128),
          (1, 128, 1, 1, 32, 66, 36), (0, 64, 2, 0, 32, 5, 48)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("fmt,D,H,QH,page,n,R", CACHES)
def test_append_rope_is_rope_then_append(fmt, D, H, QH, page, n, R, inter, dtype):
    pages = n // page + 2
    rng = np.random.Generator(np.random.PCG64(n + D))
    slots = torch.from_numpy(rng.permutation(pages * page)[:n].astype(np.int64))
    if n > 4:
        slots[1], slots[4] = -1, pages * page                                       # padding
    x = _x(n, QH + 2 * H, D, dtype, 7 * n + D)
    if n > 6:
        x[6, QH, 3] = float("nan")
        x[5, QH, :] = 0.0
    pos = _positions(n, 3)
    freq, _ = F.rope_frequencies(R, 10000.0)
    start = torch.from_numpy(rng.integers(0, 256, F.kv_cache_size(pages, page, H, D, fmt), dtype=np.uint8))
    alphas = (1.0, 0.5) if inter else (0.02, 1.7)
    cache = F.KVCache(start.cuda(), pages, page, H, D, fmt, *alphas)
    y = x.cuda()
    got = F.kv_append_rope(cache, y[:, :QH], y[:, QH:QH + H], y[:, QH + H:], slots.cuda(), pos.cuda(), freq,
                           interleaved=inter)
    assert y.cpu().view(torch.int16).equal(x.view(torch.int16))
    want = start.numpy().copy()
    k = _want(x[:, QH:QH + H], pos, freq, inter)
    oracle.kv_write_reference(want, slots.numpy(), k.float().numpy(), x[:, QH + H:].float().numpy(), page, fmt, *alphas)
    assert np.array_equal(cache.data.cpu().numpy(), want)
    assert got.cpu().equal(_want(x[:, :QH], pos, freq, inter))
    # queries in place
    cache2 = F.KVCache(start.cuda(), pages, page, H, D, fmt, *alphas)
    assert F.kv_append_rope(cache2, y[:, :QH], y[:, QH:QH + H], y[:, QH + H:], slots.cuda(), pos.cuda(), freq,
                            interleaved=inter, q_out=y[:, :QH]) is not None
    assert y[:, :QH].equal(got) and cache2.data.equal(cache.data)


def test_no_tokens():
    freq, _ = F.rope_frequencies(64)
    x = torch.empty((0, 3, 64), dtype=BF16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert F.rope(x, none, freq).shape == (0, 3, 64)
    cache = F.new_kv_cache(1, 32, 3, 64, 0)
    assert F.kv_append_rope(cache, x, x, x, none, none, freq).shape == (0, 3, 64)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("inter", [False, True])
def test_large_outputs_are_those_of_their_parts(inter, dtype):
    """Queries of more than 64 MiB (stored past the caches), alone and with the cache's write."""
    n, QH, H, D, page = 4101, 64, 2, 128, 64
    x = torch.randn((n, QH + 2 * H, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(dtype)
    pos, freq = _positions(n, 5).cuda(), F.rope_frequencies(D, 10000.0)[0]
    slots = torch.randperm(65 * page, generator=torch.Generator().manual_seed(1))[:n].cuda()
    whole, parts = F.new_kv_cache(65, page, H, D, 0), F.new_kv_cache(65, page, H, D, 0)
    whole.data.zero_(), parts.data.zero_()
    got = F.kv_append_rope(whole, x[:, :QH], x[:, QH:QH + H], x[:, QH + H:], slots, pos, freq, interleaved=inter)
    alone = F.rope(x[:, :QH], pos, freq, interleaved=inter)
    for a in range(0, n, 1000):
        y, at = x[a:a + 1000], slice(a, a + 1000)
        q = F.kv_append_rope(parts, y[:, :QH], y[:, QH:QH + H], y[:, QH + H:], slots[at], pos[at], freq, interleaved=inter)
        assert q.equal(got[at]) and q.equal(alone[at])
    assert whole.data.equal(parts.data)
    F.rope(x[:, :QH], pos, freq, interleaved=inter, out=x[:, :QH])                 # in place
    assert x[:, :QH].equal(got)


def test_more_tokens_than_a_launch_takes():
    n, D, page = (1 << 20) + 6, 64, 32
    x = torch.randn((n, 3, D), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(BF16)
    pos = torch.arange(n, device="cuda")
    freq, _ = F.rope_frequencies(D, 500000.0)
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[:20], slots[-20:] = torch.arange(20, device="cuda"), torch.arange(64, 84, device="cuda")
    cache, few = F.new_kv_cache(3, page, 1, D, 0), F.new_kv_cache(3, page, 1, D, 0)
    cache.data.zero_(), few.data.zero_()
    got = F.kv_append_rope(cache, x[:, :1], x[:, 1:2], x[:, 2:], slots, pos, freq)
    alone = F.rope(x[:, :1], pos, freq)
    for at in (slice(0, 20), slice(n - 20, n)):
        y = x[at]
        q = F.kv_append_rope(few, y[:, :1], y[:, 1:2], y[:, 2:], slots[at], pos[at], freq)
        assert q.equal(got[at]) and q.equal(alone[at])
        assert q.cpu().equal(_want(y[:, :1].cpu(), pos[at].cpu(), freq, False))
    assert cache.data.equal(few.data) and got.equal(alone)

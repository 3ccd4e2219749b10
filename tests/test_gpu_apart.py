"""Overlapping outputs, and outputs of the other kind, are refused before anything is written; views of one array side
by side give the bits of separate arrays."""

import pytest

from mixed_precision_bf16_amd import fp4gemm as F

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gfx950():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    name = torch.cuda.get_device_properties(0).gcnArchName
    if not name.startswith("gfx950"):
        pytest.skip(f"needs gfx950, found {name}")
    F.lib()
    yield


def _randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def _rejects(call, *unchanged):
    before = [t.clone() for t in unchanged]
    with pytest.raises(F.Fp4Error) as e:
        call()
    assert e.value.status == 2
    torch.cuda.synchronize()
    assert all(a.view(torch.uint8).equal(b.view(torch.uint8)) for a, b in zip(before, unchanged))


@pytest.mark.parametrize("width", [512, 40960])
def test_norm(width):
    rows = 9
    x, r, w = _randn(rows + 1, width), _randn(rows + 1, width, seed=1), _randn(width, seed=2)
    _rejects(lambda: F.rms_norm(x[1:], w, out=x[:-1]), x)
    _rejects(lambda: F.rms_norm(x[:-1], w, residual=r[:-1], sum_out=r[1:]), x, r)
    _rejects(lambda: F.rms_norm(x[:-1], x[3], out=x[:-1]), x)
    want, total = F.rms_norm(x[:-1], w, residual=r[:-1])
    side = torch.zeros((rows, 4 * width), dtype=BF16, device="cuda")        # x, residual, out and sum, column by column
    part = side.split(width, 1)
    part[0].copy_(x[:-1])
    part[1].copy_(r[:-1])
    F.rms_norm(part[0], w, residual=part[1], out=part[2], sum_out=part[3])
    assert part[2].equal(want) and part[3].equal(total) and part[0].equal(x[:-1]) and part[1].equal(r[:-1])
    _rejects(lambda: F.rms_norm(part[0], w, residual=part[1], out=side[:, 2 * width - 8:3 * width - 8]), side)
    eight = F.new_mx8(rows, width)
    _rejects(lambda: F.rms_norm(eight.codes.view(BF16).view(-1)[:width].view(1, width).expand(rows, width), mx8=True, out=eight),
             eight.codes)


def test_quantizer():
    x = _randn(6, 512)
    codes = x.view(torch.uint8).view(-1)[512:512 + 4 * 512].view(4, 512).view(torch.float8_e4m3fn)
    out = F.MX8(codes, torch.zeros((4, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu), 512)
    _rejects(lambda: F.quantize_mx8(x[:4], out=out), x)
    got, want = F.quantize_mx8(x[4:], out=F.MX8(codes[:2], out.scales[:2], 512)), F.quantize_mx8(x[4:].clone())
    assert got.codes.view(torch.uint8).equal(want.codes.view(torch.uint8))
    assert got.scales.view(torch.uint8).equal(want.scales.view(torch.uint8))


def test_rotation():
    n, heads, dim = 37, 5, 64
    both = _randn(n, 3 * heads, dim)
    pos, (freq, _) = torch.arange(n, device="cuda"), F.rope_frequencies(dim)
    x = both[:, :heads]
    want = F.rope(x.clone(), pos, freq)
    _rejects(lambda: F.rope(x, pos, freq, out=both[:, 1:heads + 1]), both)
    _rejects(lambda: F.rope(x[1:], pos[1:], freq, out=x[:-1]), both)
    _rejects(lambda: F.rope(both[:, heads - 1:2 * heads - 1], pos, freq, out=x), both)
    rest = both[:, 2 * heads:].clone()
    F.rope(x, pos, freq, out=both[:, heads:2 * heads])                      # beside it in the same array
    assert both[:, heads:2 * heads].equal(want) and both[:, 2 * heads:].equal(rest)
    F.rope(x, pos, freq, out=x)
    assert x.equal(want)


def test_rotation_with_the_cache():
    n, qh, h, dim, page = 37, 4, 2, 64, 32
    qkv = _randn(n + 1, qh + 2 * h, dim)
    pos, (freq, _) = torch.arange(n, device="cuda"), F.rope_frequencies(dim)
    slots = torch.randperm(5 * page, generator=torch.Generator().manual_seed(1))[:n].cuda()
    cache, other = F.new_kv_cache(5, page, h, dim, 0), F.new_kv_cache(5, page, h, dim, 0)
    cache.data.zero_(), other.data.zero_()
    q, k, v = qkv[:n].split([qh, h, h], 1)
    want = F.kv_append_rope(other, q.clone(), k.clone(), v.clone(), slots, pos, freq)
    for out in (qkv[:n, 1:qh + 1], qkv[:n, qh:], qkv[1:, :qh]):
        _rejects(lambda: F.kv_append_rope(cache, q, k, v, slots, pos, freq, q_out=out), qkv, cache.data)
    room = cache.data[:n * qh * dim * 2].view(BF16).view(n, qh, dim)
    _rejects(lambda: F.kv_append_rope(cache, q, k, v, slots, pos, freq, q_out=room), qkv, cache.data)
    _rejects(lambda: F.kv_append_rope(cache, room, k, v, slots, pos, freq), qkv, cache.data)
    F.kv_append_rope(cache, q, k, v, slots, pos, freq, q_out=q)
    assert q.equal(want) and cache.data.equal(other.data)


def test_8_bit_rows_as_16_bit_outputs():
    x = _randn(3, 64)
    a = F.quantize_mx8(x)
    W = [torch.zeros(k, dtype=torch.uint8, device="cuda") for k in F.native_repack_size(64, 64)]
    for call in (lambda: F.rms_norm(x, out=F.new_mx8(3, 64)), lambda: F.gemm_mx8(a, *W, 64, out=F.new_mx8(3, 64)),
                 lambda: F.gemm_mx8(a, *W, 64, dtype=BF16, out=F.new_mx8(3, 64))):
        with pytest.raises(ValueError, match="mx8"):
            call()

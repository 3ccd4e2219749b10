"""Outputs that lie on other arrays of a call are refused, to the byte; views of one
array side by side, and outputs in an input's place, are not.  Calls of the C entries
with addresses that nothing stands behind: run only where no GPU could take them."""

import ctypes

import pytest

from mixed_precision_bf16_amd import fp4gemm as F

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for machines without a GPU")


G = 1 << 30
SHAPE, DEVICE, HIP = 2, 6, 7


def _refused(status):
    assert status in (SHAPE, DEVICE, HIP), status
    return status == SHAPE


# ------------------------------------------------------------------------ norm
FAR = dict(x=1 * G, residual=2 * G, weight=3 * G, out=4 * G, out_scales=5 * G, sum=6 * G, rows=5, width=64, x_stride=64,
           residual_stride=64, out_stride=64, sum_stride=64, eps=1e-6, act_type=0, out_type=0)
ROW = 128                                                                  # bytes of a row


def _norm(**over):
    return _refused(F.lib().fp4_rms_norm(F._PACK_NORM.pack(*(FAR | over).values()), None))


def test_norm_outputs_on_other_arrays():
    assert not _norm()
    for out in ("out", "sum"):
        for other in ("x", "residual"):
            assert not _norm(**{out: FAR[other]})                           # in its place
            for by in (16, -16, ROW, -ROW, 4 * ROW, -4 * ROW, 4 * ROW + 112, -4 * ROW - 112):
                assert _norm(**{out: FAR[other] + by}), (out, other, by)
            for by in (5 * ROW, -5 * ROW):
                assert not _norm(**{out: FAR[other] + by}), (out, other, by)
        for by in (-4 * ROW - 112, -16, 0, 16, 112):
            assert _norm(**{out: FAR["weight"] + by}), (out, by)
        for by in (-5 * ROW, 128):
            assert not _norm(**{out: FAR["weight"] + by}), (out, by)
    for by in (0, 16, -4 * ROW, 4 * ROW):
        assert _norm(sum=FAR["out"] + by)
    assert not _norm(sum=FAR["out"] + 5 * ROW)


def test_norm_views_of_one_array():
    """x, residual, out and sum as columns of one array; the same columns shifted."""
    side = dict(x=G, residual=G + 128, out=G + 256, sum=G + 384, x_stride=256, residual_stride=256, out_stride=256,
                sum_stride=256)
    assert not _norm(**side)
    assert _norm(**(side | dict(out=G + 240))) and _norm(**(side | dict(sum=G + 400 - 32)))
    assert _norm(**(side | dict(out=G + 128 + 512)))                        # the residual's columns, a row further
    assert not _norm(**(side | dict(out=G + 256 + 512)))                    # its own columns, a row further
    # rows of another stride inside one another: even rows of the array and all rows of its other half
    assert not _norm(x=G, x_stride=256, out=G + 128, out_stride=128)
    assert _norm(x=G, x_stride=256, out=G + 128, out_stride=64)
    # a residual of one row for all, beside the output
    assert not _norm(residual=7 * G, residual_stride=0, out=7 * G + ROW)
    assert _norm(residual=7 * G + ROW, residual_stride=0, out=7 * G)
    # one row: its stride means nothing
    assert not _norm(rows=1, x=G, out=G, x_stride=72) and _norm(rows=1, x=G, out=G + 16)


def test_norm_8_bit_outputs_on_other_arrays():
    codes, scales = 5 * 128, 5 * 4                                          # bytes: rows of 64 are padded to 128
    eight = dict(out_type=1, width=64)
    assert not _norm(**eight)
    for name, size in (("x", 5 * ROW), ("residual", 5 * ROW), ("sum", 5 * ROW), ("weight", ROW)):
        for by in (-codes + 16, 0, 16, size - 16):
            assert _norm(**eight, out=FAR[name] + by), (name, by)
        for by in (-scales + 4, 0, 4, size - 4):
            assert _norm(**eight, out_scales=FAR[name] + by), (name, by)
        assert not _norm(**eight, out=FAR[name] - codes) and not _norm(**eight, out=FAR[name] + size)
        assert not _norm(**eight, out_scales=FAR[name] - scales) and not _norm(**eight, out_scales=FAR[name] + size)
    for by in (-scales + 4, 0, codes - 4):
        assert _norm(**eight, out_scales=FAR["out"] + by)
    assert not _norm(**eight, out_scales=FAR["out"] + codes)
    # codes between the rows of a strided x
    assert not _norm(**eight, rows=1, x_stride=1024, out=G + ROW) and not _norm(**eight, x_stride=1024, out=G + ROW)


def test_norm_of_the_most_rows_is_checked_at_once():
    """Strides and counts at their limits, unlike strides inside one another."""
    most = dict(rows=1 << 24, width=1 << 20, x_stride=(1 << 40) - 8, out_stride=(1 << 40) - 16, residual=0, sum=0)
    _norm(**most)
    _norm(**(most | dict(x_stride=1 << 21, out_stride=(1 << 21) + 8, out=G + (1 << 21))))
    assert _norm(**(most | dict(x_stride=1 << 20, out_stride=1 << 20, out=G + 16)))


# ------------------------------------------------------------------- quantizer
def _quantize(x=G, rows=5, K=64, stride=64, codes=2 * G, scales=3 * G):
    return _refused(F.lib().fp4_quantize_mx8(x, rows, K, stride, 0, codes, scales, None))


def test_quantizer_outputs_on_other_arrays():
    n_codes, n_scales = 5 * 128, 5 * 4                                      # bytes: rows of 64 are padded to 128
    assert not _quantize()
    for by in (-n_codes + 16, 0, 16, 5 * ROW - 16):
        assert _quantize(codes=G + by), by
    for by in (-n_scales + 4, 0, 4, 5 * ROW - 4):
        assert _quantize(scales=G + by), by
    for by in (-n_scales + 4, 0, n_codes - 4):
        assert _quantize(scales=2 * G + by), by
    for by in (-n_codes, 5 * ROW):
        assert not _quantize(codes=G + by), by
    assert not _quantize(scales=2 * G + n_codes) and not _quantize(scales=G - n_scales)
    # in the gaps between x's rows
    assert not _quantize(stride=1024, codes=G + ROW) and not _quantize(stride=1024, scales=G + 4 * 2048 - 32)
    assert _quantize(stride=320, codes=G + ROW) and _quantize(stride=1024, scales=G + 4 * 2048 - 16)


# -------------------------------------------------------------------- rotation
def _rope(x=G, out=2 * G, tokens=3, heads=4, dim=64, xt=256, xh=64, ot=256, oh=64, positions=3 * G, frequencies=4 * G):
    r = F._PACK_ROPE.pack(positions, frequencies, 64, 1.0, 0)
    return _refused(F.lib().fp4_rope(r, x, out, tokens, heads, dim, xt, xh, ot, oh, 0, None))


def test_rotated_rows_on_other_arrays():
    token = 512                                                             # bytes of four heads
    assert not _rope() and not _rope(out=G)
    for by in (16, -16, 128, -128, token, -token, 3 * token - 16, 16 - 3 * token):
        assert _rope(out=G + by), by
    for by in (3 * token, -3 * token):
        assert not _rope(out=G + by), by
    # x and out side by side in one array of 12 heads; shifted by a head they meet
    side = dict(xt=768, ot=768)
    assert not _rope(out=G + token, **side) and not _rope(out=G + 1024, **side)
    assert _rope(out=G + token - 128, **side) and _rope(out=G + 1536 - 128, **side) and _rope(out=G + 128, **side)
    # head-major output of a token-major x: apart, inside it, and on its last element
    assert not _rope(ot=64, oh=192) and _rope(out=G, ot=64, oh=192) and _rope(out=G + 3 * token - 16, ot=64, oh=192)
    # one head, one token: their strides mean nothing
    assert not _rope(out=G, heads=1, xh=64, oh=72) and not _rope(out=G, tokens=1, xt=256, ot=512)
    # one row for all: outside it and on it
    assert not _rope(x=G, xt=0, xh=0, out=G + 128) and _rope(x=G + 128, xt=0, xh=0, out=G)
    for by in (-3 * token + 16, -16, 0, 16):
        assert _rope(out=3 * G + by) and _rope(out=4 * G + by), by
    assert _rope(out=4 * G + 112) and not _rope(out=4 * G + 128) and not _rope(out=3 * G + 32)


def _append(data=G, **over):
    c = F._KVCacheDesc(data=data, pages=2, page_size=32, kv_heads=2, head_dim=64, format=0, k_alpha=1.0, v_alpha=1.0)
    f = dict(q=2 * G, q_out=3 * G, k=4 * G, v=5 * G, slots=6 * G, tokens=3, q_heads=4, qt=256, qh=64, ot=256, oh=64,
             kt=128, kh=64, vt=128, vh=64, act=0, positions=7 * G, frequencies=8 * G) | over
    r = F._PACK_ROPE.pack(f.pop("positions"), f.pop("frequencies"), 64, 1.0, 0)
    return _refused(F.lib().fp4_kv_append_rope(ctypes.byref(c), r, F._PACK_APPEND_ROPE.pack(*f.values()), None))


def test_rotated_queries_and_the_cache_on_other_arrays():
    n_q, n_k = 3 * 512, 3 * 256                                             # bytes of the queries, of the keys
    size = F.kv_cache_size(2, 32, 2, 64, 0)
    assert not _append() and not _append(q_out=2 * G) and not _append(q=0, q_out=0, q_heads=0)
    for by in (16, -16, 512, n_q - 16, 16 - n_q):
        assert _append(q_out=2 * G + by), by
    assert not _append(q_out=2 * G + n_q) and not _append(q_out=2 * G - n_q)
    for other, last in ((4 * G, n_k), (5 * G, n_k), (G, size), (6 * G, 16), (7 * G, 16), (8 * G, 128)):
        for by in (16 - n_q, 0, last - 16):
            assert _append(q_out=other + by), (other // G, by)
        assert not _append(q_out=other - n_q) and not _append(q_out=other + (last + 31) // 16 * 16)
    for other, last in ((2 * G, n_q), (4 * G, n_k), (5 * G, n_k), (6 * G, 16), (7 * G, 16), (8 * G, 112)):
        for by in (16 - size, 0, last - 16):
            assert _append(data=other + by), (other // G, by)
        assert not _append(data=other - size) and not _append(data=other + n_q)
    # queries, keys and values side by side in the rows of one projection; in place; shifted by a head
    rows = dict(q=2 * G, k=2 * G + 512, v=2 * G + 768, qt=512, kt=512, vt=512)
    assert not _append(**rows) and not _append(**rows, q_out=2 * G, ot=512)
    for by in (128, -128, 1024 + 128):
        assert _append(**rows, q_out=2 * G + by, ot=512), by
    assert not _append(**rows, q_out=2 * G + 3 * 1024)
    # head-major keys that begin behind the queries
    assert not _append(k=2 * G + n_q, kt=64, kh=192, q_out=2 * G) and _append(k=2 * G + n_q - 128, kt=64, kh=192, q_out=2 * G)

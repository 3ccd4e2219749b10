"""FP4 key/value cache and attention: the oracle's layout and attention pinned
on small cases, sizes, and the argument checks of the C entries and of the
binding, which all run before any HIP call."""

import ctypes
import itertools

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F

torch = pytest.importorskip("torch")

SHAPES = list(itertools.product((0, 1), (64, 128, 256)))


@pytest.mark.parametrize("fmt,D", SHAPES)
def test_layout_gives_every_byte_of_a_tile_to_one_token(fmt, D):
    parts = oracle.kv_offsets(fmt, D)
    owner = {}
    for part in parts:
        for t in range(32):
            for o in part[t]:
                assert owner.setdefault(int(o), t) == t
        assert part.size == len(np.unique(part))
    assert sorted(owner) == list(range(32 * D + 64 * D // (16 if fmt == 0 else 32)))


@pytest.mark.parametrize("fmt,D", SHAPES)
def test_layout_is_fragment_order(fmt, D):
    """A lane's 16 key bytes are consecutive elements of one token (D = 64: of
    two), its value bytes consecutive elements of tokens 4 j .. 4 j + 3."""
    kc, vc, _, _ = oracle.kv_offsets(fmt, D)
    run = 16 if D >= 128 else 8
    for t in (0, 5, 17, 31):
        assert np.array_equal(kc[t, :run], kc[t, 0] + np.arange(run)) and kc[t, 0] % run == 0
        piece = 4 if D >= 128 else 2
        assert np.array_equal(vc[t, :piece], vc[t, 0] + np.arange(piece))
    for t in (0, 4, 20, 28):
        assert [vc[t + i, 0] - vc[t, 0] for i in range(4)] == [(4 if D >= 128 else 2) * i for i in range(4)]


@pytest.mark.parametrize("fmt,D", SHAPES)
def test_oracle_write_read_roundtrip_and_untouched_bytes(fmt, D):
    rng = np.random.Generator(np.random.PCG64(D + fmt))
    H, page = 2, 64
    data = rng.integers(0, 256, F.kv_cache_size(3, page, H, D, fmt), dtype=np.uint8)
    before = data.copy()
    slots = np.array([0, 191, -1, 70, 192, 33])
    k = rng.standard_normal((6, H, D)).astype(np.float32)
    v = rng.standard_normal((6, H, D)).astype(np.float32)
    oracle.kv_write_reference(data, slots, k, v, page, fmt)
    held = 2 * H * (D // 2 + D // (16 if fmt == 0 else 32))
    assert np.count_nonzero(data != before) <= 4 * held
    got_k, got_v = oracle.kv_read_reference(data, slots[[0, 1, 3, 5]], H, D, page, fmt)
    G = 16 if fmt == 0 else 32
    for got, x in ((got_k, k), (got_v, v)):
        x = x[[0, 1, 3, 5]].reshape(4, H, D // G, G)
        amax = np.abs(x).max(-1, keepdims=True)
        # nearest of E2M1: steps of 2 below 6 after a scale within amax / 6 (1 +- 2^-4), MXFP4 up to amax / 4
        assert np.all(np.abs(got.reshape(x.shape) - x) <= amax * (1.07 / 6 if fmt == 0 else 1 / 4))


def test_oracle_attention_small_cases():
    k = np.zeros((64, 1, 64))
    v = np.zeros((64, 1, 64))
    k[0, 0, 0], k[1, 0, 0] = 1.0, 3.0
    v[0, 0, :], v[1, 0, :] = 5.0, 9.0
    q = np.zeros((2, 2, 64))
    q[:, :, 0] = np.log(2.0)
    out, lse, w = oracle.attention_reference(q, k, v, np.array([[0]]), [2], [0, 2], 64)
    assert np.allclose(out[0, 0], 5.0) and np.allclose(lse[0], np.log(2.0))   # sees only key 0
    assert np.allclose(out[1, 1], (2 * 5 + 8 * 9) / 10) and np.allclose(lse[1], np.log(10.0))
    assert np.allclose(w, out)
    out, lse, _ = oracle.attention_reference(q, k, v, np.array([[0]]), [2], [0, 2], 64, window=1,
                                             sinks=np.log(np.array([8.0, 24.0])))
    assert np.allclose(out[1, 0], 9 / 2) and np.allclose(out[1, 1], 9 * 8 / 32) and np.allclose(lse[1, 0], np.log(16.0))
    out, lse, _ = oracle.attention_reference(q, k, v, np.array([[-1]]), [2], [0, 2], 64)
    assert np.all(out == 0) and np.all(lse == -np.inf)                        # a page that is not there
    out, lse, _ = oracle.attention_reference(q, k, v, np.array([[0]]), [1], [0, 2], 64)
    assert np.all(out[0] == 0) and np.all(out[1] == 5)                        # the first query lies before key 0


@pytest.mark.parametrize("pages,page,H,D,fmt", [(1, 32, 1, 64, 0), (7, 96, 3, 128, 0), (5, 64, 8, 256, 1),
                                                (1 << 20, 64, 8, 128, 0)])
def test_cache_size(pages, page, H, D, fmt):
    G = 16 if fmt == 0 else 32
    assert F.kv_cache_size(pages, page, H, D, fmt) == pages * page * H * 2 * (D // 2 + D // G)


@pytest.mark.parametrize("pages,page,H,D,fmt,status", [
    (0, 64, 1, 64, 0, 2), (1 << 31, 64, 1, 64, 0, 2), (1, 16, 1, 64, 0, 2), (1, 48, 1, 64, 0, 2),
    (1, 8192, 1, 64, 0, 2), (1, 64, 0, 64, 0, 2), (1, 64, 257, 64, 0, 2), (1, 64, 1, 96, 0, 2),
    (1, 64, 1, 0, 0, 2), (1, 64, 1, 64, 2, 3), (-1, 64, 1, 64, 1, 2)])
def test_cache_shape_errors(pages, page, H, D, fmt, status):
    b = ctypes.c_size_t(7)
    assert F.lib().fp4_kv_cache_size(pages, page, H, D, fmt, ctypes.byref(b)) == status
    assert b.value == 7
    c = F._KVCacheDesc(16, pages, page, H, D, fmt, 1.0, 1.0)
    d = ctypes.c_void_p(16)
    assert F.lib().fp4_kv_append(ctypes.byref(c), d, d, d, 1, 64, 64, 64, 64, 0, None) == status
    assert F.lib().fp4_kv_read(ctypes.byref(c), d, 1, d, d, 64, 64, 64, 64, 0, None) == status
    assert F.lib().fp4_attention(ctypes.byref(c), ctypes.byref(F._AttentionArgs()), None) == status
    assert F.lib().fp4_attention_workspace_size(ctypes.byref(c), ctypes.byref(F._AttentionArgs()),
                                                ctypes.byref(b)) == status


def _cache(**over):
    f = dict(data=16, pages=4, page_size=64, kv_heads=2, head_dim=128, format=0, k_alpha=1.0, v_alpha=1.0)
    f.update(over)
    return F._KVCacheDesc(**f)


def test_append_and_read_argument_errors():
    lib = F.lib()

    def append(c=None, k=16, v=16, slots=16, n=3, kt=256, kh=128, vt=256, vh=128, act=0):
        c = _cache() if c is None else c
        return lib.fp4_kv_append(ctypes.byref(c), k, v, slots, n, kt, kh, vt, vh, act, None)

    def read(c=None, k=16, v=16, slots=16, n=3, kt=256, kh=128, vt=256, vh=128, act=0):
        c = _cache() if c is None else c
        return lib.fp4_kv_read(ctypes.byref(c), slots, n, k, v, kt, kh, vt, vh, act, None)

    assert lib.fp4_kv_append(None, 16, 16, 16, 1, 8, 8, 8, 8, 0, None) == 1
    for call in (append, read):
        assert call(c=_cache(data=0)) == 1 and call(c=_cache(data=8)) == 2
        for a in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 101):
            assert call(c=_cache(k_alpha=a)) == 4 and call(c=_cache(v_alpha=a)) == 4
        assert call(act=2) == 3 and call(n=-1) == 2 and call(n=(1 << 24) + 1) == 2
        assert call(n=0, k=None, v=None, slots=None) == 0
        assert call(slots=None) == 1 and call(slots=20) == 2
        assert call(k=24) == 2 and call(v=24) == 2
        for s in ("kt", "kh", "vt", "vh"):
            assert call(**{s: 132}) == 2 and call(**{s: -128}) == 2 and call(**{s: 1 << 40}) == 2
    assert append(k=None) == 1 and append(v=None) == 1
    assert read(k=None, v=None) == 1
    # output rows that share elements
    assert read(kt=128) == 2 and read(vh=64) == 2 and read(kt=0) == 2 and read(kt=128, kh=256) == 2


def _args(**over):
    f = dict(q=16, out=16, page_table=16, seq_lens=16, batch=2, q_rows=2, q_heads=4, max_q=1, page_columns=3,
             page_stride=3, q_token_stride=512, q_head_stride=128, out_token_stride=512, out_head_stride=128,
             causal=1, scale=0.1, workspace=16, workspace_bytes=1 << 40)
    f.update(over)
    return F._AttentionArgs(**f)


def test_attention_argument_errors():
    lib = F.lib()

    def call(c=None, **over):
        c = _cache() if c is None else c
        return lib.fp4_attention(ctypes.byref(c), ctypes.byref(_args(**over)), None)

    assert lib.fp4_attention(ctypes.byref(_cache()), None, None) == 1
    assert call(c=_cache(data=0)) == 1
    for name in ("q", "out", "page_table", "seq_lens"):
        assert call(**{name: None}) == 1, name
    for name, bad in (("q", 24), ("out", 24), ("page_table", 18), ("seq_lens", 18), ("q_offsets", 18), ("lse", 18),
                      ("sinks", 18), ("batch", -1), ("batch", (1 << 24) + 1), ("q_rows", -2), ("q_rows", 3),
                      ("q_rows", (1 << 24) + 2), ("q_heads", 1), ("q_heads", 5), ("q_heads", 2 * 1025),
                      ("max_q", -1), ("page_columns", 0), ("page_columns", 1 << 25), ("page_stride", 2),
                      ("q_token_stride", 516), ("q_head_stride", -8), ("out_token_stride", 256),
                      ("out_head_stride", 64), ("out_token_stride", 0)):
        assert call(**{name: bad}) == 2, (name, bad)
    assert call(act_type=2) == 3
    for name, bad in (("causal", 2), ("window", -1), ("scale", 0.0), ("scale", -1.0), ("scale", float("nan")),
                      ("scale", float("inf")), ("scale", 2.0 ** 13), ("scale", 2.0 ** -101)):
        assert call(**{name: bad}) == 4, (name, bad)
    assert call(causal=0, window=5) == 4
    assert call(c=_cache(k_alpha=2.0 ** 20)) == 4      # scale * k_alpha above 2^12
    need = ctypes.c_size_t()
    assert lib.fp4_attention_workspace_size(ctypes.byref(_cache()), ctypes.byref(_args()), ctypes.byref(need)) == 0
    assert need.value > 0
    assert call(workspace=None) == 5 and call(workspace_bytes=need.value - 1) == 5 and call(workspace=24) == 5
    assert call(batch=0, q_rows=0, q=None, out=None, workspace=None) == 0
    assert call(q_rows=0, q=None, workspace=None) == 0
    assert lib.fp4_attention_workspace_size(None, ctypes.byref(_args()), ctypes.byref(need)) == 1


def test_workspace_depends_on_shapes_only():
    lib = F.lib()

    def size(**over):
        need = ctypes.c_size_t()
        assert lib.fp4_attention_workspace_size(ctypes.byref(_cache()), ctypes.byref(_args(**over)),
                                                ctypes.byref(need)) == 0
        return need.value
    assert size() == size(q=None, out=None, page_table=None, seq_lens=None, workspace=None, workspace_bytes=0)
    assert size() == size(causal=0, window=0, act_type=1, scale=3.0)


def test_packed_arguments_are_the_structure():
    values = list(range(1, 8)) + list(range(11, 22)) + [1, 0, 0.5, 31, 32]
    raw = F._pack_attention(*values)
    assert len(raw) == ctypes.sizeof(F._AttentionArgs)
    a = F._AttentionArgs.from_buffer_copy(raw)
    assert [getattr(a, n) for n, _ in F._AttentionArgs._fields_] == values
    for at, bad in ((17, 1 << 63), (10, 2.5)):
        with pytest.raises(ValueError):
            F._pack_attention(*values[:at], bad, *values[at + 1:])


def test_binding_refuses_host_tensors():
    c = torch.zeros(F.kv_cache_size(1, 32, 1, 64, 0), dtype=torch.uint8)
    with pytest.raises(ValueError):
        F.KVCache(c, 1, 32, 1, 64, 0)
    with pytest.raises(F.Fp4Error):
        F.kv_cache_size(1, 31, 1, 64, 0)


class _DeviceTensor:
    """What KVCache asks of its tensor, without a GPU."""
    dtype, is_cuda = torch.uint8, True

    def __init__(self, n, address=4096):
        self.numel, self.data_ptr, self.is_contiguous = (lambda: n), (lambda: address), (lambda: True)


def test_cache_fields_are_fixed():
    """The descriptor that the calls take holds the data's address, the shape
    and the scales: none of them can be set past it."""
    data = _DeviceTensor(F.kv_cache_size(3, 32, 2, 64, 1))
    c = F.KVCache(data, 3, 32, 2, 64, 1, 0.5, 2.0)
    want = dict(data=data, pages=3, page_size=32, kv_heads=2, head_dim=64, fmt=1, k_alpha=0.5, v_alpha=2.0)
    assert {n: getattr(c, n) for n in want} == want
    for name in want:
        with pytest.raises(AttributeError):
            setattr(c, name, _DeviceTensor(data.numel(), 8192) if name == "data" else 64)
        with pytest.raises(AttributeError):
            delattr(c, name)
    assert {n: getattr(c, n) for n in want} == want
    d = c._desc
    assert (d.data, d.pages, d.page_size, d.kv_heads, d.head_dim, d.format, d.k_alpha, d.v_alpha) == \
        (4096, 3, 32, 2, 64, 1, 0.5, 2.0)


def test_a_page_table_row_for_all_sequences_passes_the_checks():
    # the workspace is checked after the strides, and before any HIP call
    call = lambda **over: F.lib().fp4_attention(ctypes.byref(_cache()), ctypes.byref(_args(workspace=None, **over)),  # noqa: E731
                                                None)
    assert call() == 5 and call(page_stride=0) == 5 and call(page_stride=7) == 5
    assert call(page_stride=-1) == 2 and call(page_stride=1) == 2

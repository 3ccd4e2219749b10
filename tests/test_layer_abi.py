"""Norm, rotary positions and products of 8-bit activations: the oracle pinned on
small cases and by other arithmetic, sizes, frequencies, and the argument checks
of the C entries and of the binding, which all run before any HIP call."""

import ctypes
import math
import struct
from fractions import Fraction

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ the oracle
def test_oracle_e4m3_codes_are_the_library_cast():
    """Every border between codes and its FP32 neighbours, and random values, at scale 1
    (a 448 in the block)."""
    edges = (oracle.layer_oracle.E4M3[1:] + oracle.layer_oracle.E4M3[:-1]) / 2
    v = np.concatenate([edges, np.nextafter(edges.astype(np.float32), np.float32(0)),
                        np.nextafter(edges.astype(np.float32), np.float32(1e9)), oracle.layer_oracle.E4M3,
                        np.random.default_rng(1).standard_normal(4000) * 30])
    v = v[np.abs(v) <= 448].astype(np.float32)
    v = np.concatenate([v, -v])
    v = np.concatenate([v, np.zeros(-len(v) % 31, np.float32)]).reshape(-1, 31)
    x = np.concatenate([np.full((len(v), 1), 448, np.float32), v], 1)
    codes, scales = oracle.mx8_quantize_reference(x)
    assert (scales[:, 0] == 127).all()
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes[:, :32], want)


def test_oracle_scale_is_the_least_power_of_two():
    rng = np.random.default_rng(2)
    top = np.concatenate([np.exp2(rng.uniform(-100, 100, 300)), 448 * np.exp2(np.arange(-60.0, 60)),
                          np.nextafter((448 * np.exp2(np.arange(-60.0, 60))).astype(np.float32), np.float32(np.inf))])
    x = np.zeros((len(top), 32), np.float32)
    x[:, 7] = top.astype(np.float32)
    codes, scales = oracle.mx8_quantize_reference(x)
    for t, s in zip(x[:, 7], scales[:, 0]):
        e = int(s) - 127
        assert Fraction(float(t)) <= 448 * Fraction(2) ** e and Fraction(float(t)) > 448 * Fraction(2) ** (e - 1)
    back = oracle.mx8_value(codes, scales, 32)
    assert (np.abs(back - x) <= np.abs(x) * 2.0 ** -4).all()
    # all zero; NaN and infinities leave the scale to the others; padding zero
    x = np.zeros((3, 160), np.float32)
    x[1, :3] = [np.nan, 448, -np.inf]
    x[2, 159] = 1e-40
    codes, scales = oracle.mx8_quantize_reference(x)
    assert codes.shape == (3, 256) and scales.shape == (3, 8)
    assert not codes[0].any() and not scales[0].any() and not codes[:, 160:].any() and not scales[:, 5:].any()
    assert codes[1, 0] & 127 == 127 and codes[1, 1] == 0x7E and codes[1, 2] & 127 == 127 and scales[1, 0] == 127
    assert scales[2, 4] == 0


def test_oracle_norm_small_cases():
    x = np.array([[3.0, 4.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]])
    y, h = oracle.rms_norm_reference(x, np.full(8, 2.0), 1e-12)
    assert np.allclose(y[0, :2], np.array([6, 8]) / math.sqrt(25 / 8)) and np.array_equal(h, x)
    y, h = oracle.rms_norm_reference(x, None, 1e-12, residual=-x)
    assert not y.any() and not h.any()
    rng = np.random.default_rng(0)
    x, r, w = (rng.standard_normal((3, 64)).astype(np.float32) for _ in range(3))
    y, h = oracle.rms_norm_reference(x, w[0], 1e-5, r)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x + r).double(), (64,), torch.from_numpy(w[0]).double(), 1e-5)
    assert np.allclose(y, t.numpy(), rtol=1e-6, atol=1e-6)


def test_oracle_rope_is_a_turn():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 2, 12)).astype(np.float32)
    pos, freq = np.array([0, 1, 5, 40000]), np.array([1.0, 0.1, 0.003], np.float32)
    half = oracle.rope_reference(x, pos, freq, False)
    pairs = oracle.rope_reference(x, pos, freq, True)
    z = (x[..., :3] + 1j * x[..., 3:6]) * np.exp(1j * pos[:, None] * freq.astype(np.float64))[:, None]
    assert np.allclose(half[..., :3], z.real, atol=1e-6) and np.allclose(half[..., 3:6], z.imag, atol=1e-6)
    z = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) * np.exp(1j * pos[:, None] * freq.astype(np.float64))[:, None]
    assert np.allclose(pairs[..., 0:6:2], z.real, atol=1e-6) and np.allclose(pairs[..., 1:6:2], z.imag, atol=1e-6)
    assert np.array_equal(half[..., 6:], x[..., 6:]) and np.array_equal(half[0], x[0])
    assert np.allclose(oracle.rope_reference(x, pos, freq, False, 2.0)[..., :6], 2 * half[..., :6], rtol=1e-6)


def test_oracle_product_and_gates():
    codes = np.array([[0x38, 0xB8] + [0] * 126], np.uint8)                 # 1, -1
    scales = np.array([[128, 127, 127, 127]], np.uint8)                    # twice
    w = np.zeros((2, 16), np.uint8)
    w[0, 0], w[1, 0] = 0x42, 0x17                                          # (1, 2), (6, 0.5)
    ws = np.array([[127], [126]], np.uint8)
    y, total = oracle.gemm_mx8_reference(codes, scales, w, ws, 32, alpha=0.5)
    assert np.array_equal(y, [[-1.0, 2.75]]) and np.array_equal(total, [[3.0, 3.25]])
    g = torch.linspace(-9, 9, 201, dtype=torch.float64)
    u = torch.full_like(g, 1.5)
    assert np.allclose(oracle.gate_reference(g.numpy(), u.numpy(), "silu"), (torch.nn.functional.silu(g) * u).numpy())
    assert np.allclose(oracle.gate_reference(g.numpy(), u.numpy(), "gelu"),
                       (torch.nn.functional.gelu(g, approximate="tanh") * u).numpy())


# ----------------------------------------------------------------- frequencies
def test_frequencies():
    f, amp = F.rope_frequencies(128, 500000.0, device="cpu")
    i = np.arange(64)
    assert amp == 1.0 and f.dtype == torch.float32 and np.array_equal(f, (500000.0 ** (-i / 64)).astype(np.float32))
    lin, _ = F.rope_frequencies(128, 500000.0, "linear", 8.0, device="cpu")
    assert torch.equal(lin, f / 8)
    ntk, _ = F.rope_frequencies(128, 500000.0, "ntk", 8.0, device="cpu")
    assert ntk[0] == 1 and np.isclose(float(ntk[-1]), float(f[-1]) / 8, rtol=1e-6)
    bands, amp = F.rope_frequencies(128, 500000.0, "bands", 8.0, original=8192, device="cpu")
    turns = 8192 * f.double() / (2 * math.pi)
    assert amp == 1.0
    assert torch.equal(bands[turns > 4], f[turns > 4]) and torch.equal(bands[turns < 1], (f / 8)[turns < 1])
    mid = (turns >= 1) & (turns <= 4)
    assert mid.any() and (bands[mid] <= f[mid]).all() and (bands[mid] >= f[mid] / 8).all()
    yarn, amp = F.rope_frequencies(64, 10000.0, "yarn", 16.0, original=4096, device="cpu")
    f, _ = F.rope_frequencies(64, device="cpu")
    assert amp == 1 + 0.1 * math.log(16) and yarn[0] == f[0] and np.isclose(float(yarn[-1]), float(f[-1]) / 16, rtol=1e-6)
    assert (yarn <= f * 1.0000001).all() and (yarn >= f / 16 * 0.9999999).all()
    same, amp = F.rope_frequencies(64, scaling="yarn", device="cpu")
    assert amp == 1.0 and torch.allclose(same, f)
    for bad in (dict(rotary=0), dict(rotary=7), dict(rotary=8, scaling="other"), dict(rotary=8, factor=0.5),
                dict(rotary=8, base=1.0), dict(rotary=8, base=math.inf), dict(rotary=8, factor=math.inf),
                dict(rotary=8, scaling="bands", low=4.0), dict(rotary=8, scaling="yarn", slow=0.0),
                dict(rotary=8, scaling="yarn", original=0)):
        with pytest.raises(ValueError):
            F.rope_frequencies(device="cpu", **bad)


# ---------------------------------------------------------------- C argument checks
def _norm(**over):
    f = dict(x=16, residual=0, weight=16, out=16, out_scales=16, sum=0, rows=3, width=64, x_stride=64,
             residual_stride=64, out_stride=64, sum_stride=64, eps=1e-6, act_type=0, out_type=0)
    f.update(over)
    return F.lib().fp4_rms_norm(F._PACK_NORM.pack(*f.values()), None)


def test_norm_argument_errors():
    assert F.lib().fp4_rms_norm(None, None) == 1
    for name in ("x", "out"):
        assert _norm(**{name: 0}) == 1
    assert _norm(out_type=1, out_scales=0) == 1
    assert _norm(act_type=2) == 3 and _norm(out_type=2) == 3 and _norm(out_type=-1) == 3
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0):
        assert _norm(eps=bad) == 4
    for over in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(width=0), dict(width=4), dict(width=68),
                 dict(width=(1 << 20) + 8), dict(width=40, out_type=1), dict(x=24), dict(weight=24), dict(out=24),
                 dict(residual=24), dict(sum=24, residual=16), dict(x_stride=-64), dict(x_stride=68),
                 dict(x_stride=1 << 40), dict(residual=16, residual_stride=60), dict(out_stride=56), dict(out_stride=0),
                 dict(sum=32, sum_stride=56), dict(out_type=1, out=24), dict(out_type=1, out_scales=18)):
        assert _norm(**over) == 2, over
    assert _norm(rows=0, x=0, out=0) == 0


def test_quantizer_argument_errors_and_sizes():
    def call(x=16, rows=3, K=64, xs=64, act=0, codes=16, scales=16):
        return F.lib().fp4_quantize_mx8(x, rows, K, xs, act, codes, scales, None)
    assert call(x=None) == 1 and call(codes=None) == 1 and call(scales=None) == 1
    assert call(act=2) == 3
    for over in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(K=0), dict(K=16), dict(K=48), dict(K=(1 << 20) + 32),
                 dict(x=24), dict(xs=60), dict(xs=-8), dict(codes=24), dict(scales=18)):
        assert call(**over) == 2, over
    assert call(rows=0, x=None, codes=None, scales=None) == 0
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    for rows, K in ((0, 32), (1, 32), (5, 128), (7, 2880), (1 << 24, 1 << 20)):
        assert F.lib().fp4_mx8_size(rows, K, ctypes.byref(a), ctypes.byref(b)) == 0
        assert a.value == rows * oracle.mx8_padded(K) and b.value * 32 == a.value
        assert F.mx8_padded(K) == oracle.mx8_padded(K)
    assert F.lib().fp4_mx8_size(1, 32, None, None) == 0
    for rows, K in ((-1, 32), (1, 0), (1, 33), ((1 << 24) + 1, 32), (1, 1 << 21)):
        assert F.lib().fp4_mx8_size(rows, K, ctypes.byref(a), ctypes.byref(b)) == 2


def _product(**over):
    f = dict(codes=16, scales=16, wq=16, sq=16, out=16, out_scales=16, workspace=256, workspace_bytes=1 << 40, m=5, N=64,
             K=128, out_type=0, gate=0, alpha=1.0)
    f.update(over)
    return F.lib().fp4_gemm_mx8(F._PACK_MX8.pack(*f.values()), None)


def test_product_argument_errors():
    assert F.lib().fp4_gemm_mx8(None, None) == 1
    for name in ("codes", "scales", "wq", "sq", "out"):
        assert _product(**{name: 0}) == 1, name
    assert _product(out_type=2, out_scales=0) == 1
    for over in (dict(out_type=3), dict(out_type=-1), dict(gate=3), dict(gate=-1)):
        assert _product(**over) == 3, over
    for bad in (0.0, float("nan"), float("inf"), 2.0 ** 101, 2.0 ** -101):
        assert _product(alpha=bad) == 4, bad
    for over in (dict(m=-1), dict(m=(1 << 20) + 1), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=48),
                 dict(K=1 << 21), dict(N=48, gate=1), dict(N=33, gate=2), dict(N=48, out_type=2),
                 dict(N=96, gate=1, out_type=2), dict(m=1 << 20, K=2048), dict(m=1 << 20, N=1024), dict(codes=24),
                 dict(scales=18), dict(wq=24), dict(sq=24), dict(out=24), dict(out_type=2, out_scales=18)):
        assert _product(**over) == 2, over
    assert _product(m=0, codes=0, scales=0, wq=0, sq=0, out=0) == 0
    size = ctypes.c_size_t()

    def need(m=5, N=64, K=128, out_type=0, gate=0, at=ctypes.byref(size)):
        return F.lib().fp4_gemm_mx8_workspace_size(m, N, K, out_type, gate, at)
    assert need() == 0 and need(at=None) == 1 and need(N=0) == 2 and need(K=40) == 2 and need(gate=7) == 3
    assert need(m=0) == 0 and size.value == 0


def test_products_with_a_workspace_check_it():
    size = ctypes.c_size_t()
    for m, N, K in ((256, 8192, 28672), (256, 1024, 8192), (128, 2048, 16384)):
        assert F.lib().fp4_gemm_mx8_workspace_size(m, N, K, 0, 0, ctypes.byref(size)) == 0
        if size.value:
            assert _product(m=m, N=N, K=K, workspace=0) == 5 and _product(m=m, N=N, K=K, workspace=128) == 5
            assert _product(m=m, N=N, K=K, workspace_bytes=size.value - 1) == 5


def _rope(positions=16, frequencies=16, rotary=64, amplitude=1.0, interleaved=0):
    return F._PACK_ROPE.pack(positions, frequencies, rotary, amplitude, interleaved)


def test_rope_argument_errors():
    def call(r=None, x=16, out=16, tokens=3, heads=4, dim=64, xt=256, xh=64, ot=256, oh=64, act=0):
        return F.lib().fp4_rope(_rope() if r is None else r, x, out, tokens, heads, dim, xt, xh, ot, oh, act, None)
    assert F.lib().fp4_rope(None, 16, 16, 1, 1, 64, 64, 64, 64, 64, 0, None) == 1
    assert call(x=None) == 1 and call(out=None) == 1
    assert call(_rope(positions=0)) == 1 and call(_rope(frequencies=0)) == 1
    assert call(act=2) == 3
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 21, 2.0 ** -21):
        assert call(_rope(amplitude=bad)) == 4
    for r in (_rope(rotary=0), _rope(rotary=3), _rope(rotary=66), _rope(rotary=-2), _rope(positions=20),
              _rope(frequencies=18)):
        assert call(r) == 2
    for over in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(heads=-1), dict(heads=65537), dict(dim=60),
                 dict(dim=1032), dict(x=24), dict(out=24), dict(xt=252), dict(xh=-64), dict(ot=192), dict(oh=56),
                 dict(ot=0), dict(oh=0)):
        assert call(**over) == 2, over
    assert call(tokens=0, x=None, out=None) == 0 and call(heads=0, x=None, out=None) == 0


def test_append_rope_argument_errors():
    def cache(**over):
        f = dict(data=16, pages=4, page_size=64, kv_heads=2, head_dim=128, format=0, k_alpha=1.0, v_alpha=1.0)
        f.update(over)
        return F._KVCacheDesc(**f)

    def call(c=None, r=None, **over):
        f = dict(q=16, q_out=16, k=16, v=16, slots=16, tokens=3, q_heads=4, qt=512, qh=128, ot=512, oh=128, kt=256,
                 kh=128, vt=256, vh=128, act=0)
        f.update(over)
        return F.lib().fp4_kv_append_rope(ctypes.byref(cache() if c is None else c), _rope() if r is None else r,
                                          F._PACK_APPEND_ROPE.pack(*f.values()), None)
    c = cache()
    assert F.lib().fp4_kv_append_rope(None, _rope(), b"\0" * 128, None) == 1
    assert F.lib().fp4_kv_append_rope(ctypes.byref(c), None, b"\0" * 128, None) == 1
    assert F.lib().fp4_kv_append_rope(ctypes.byref(c), _rope(), None, None) == 1
    assert call(cache(data=0)) == 1 and call(cache(data=8)) == 2 and call(cache(head_dim=96)) == 2
    assert call(cache(k_alpha=0.0)) == 4 and call(cache(format=2)) == 3
    for name in ("q", "q_out", "k", "v", "slots"):
        assert call(**{name: 0}) == 1, name
    assert call(r=_rope(positions=0)) == 1 and call(r=_rope(rotary=130)) == 2 and call(r=_rope(amplitude=0.0)) == 4
    assert call(act=2) == 3
    for over in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(q_heads=-1), dict(q_heads=65537), dict(q=24),
                 dict(q_out=24), dict(k=24), dict(v=24), dict(slots=20), dict(qt=516), dict(ot=384), dict(oh=64),
                 dict(kt=-8), dict(vh=4), dict(vt=1 << 40)):
        assert call(**over) == 2, over
    assert call(tokens=0, q=0, q_out=0, k=0, v=0, slots=0) == 0


def test_outputs_on_other_arrays_are_refused():
    """Calls right but for an output that lies on another array of theirs."""
    far = dict(x=1 << 30, residual=2 << 30, weight=3 << 30, out=4 << 30, out_scales=5 << 30, sum=6 << 30)
    for over in (dict(out=1 << 30, x_stride=72), dict(out=2 << 30, residual_stride=72), dict(sum=1 << 30, sum_stride=72),
                 dict(sum=2 << 30, sum_stride=72), dict(sum=4 << 30), dict(out_type=1, out=1 << 30),
                 dict(out_type=1, out=2 << 30), dict(out_type=1, sum=4 << 30)):
        assert _norm(**(far | over)) == 2, over
    assert F.lib().fp4_quantize_mx8(1 << 30, 3, 64, 64, 0, 1 << 30, 2 << 30, None) == 2
    far = dict(codes=1 << 40, scales=2 << 40, wq=3 << 40, sq=4 << 40, out=5 << 40, out_scales=6 << 40, workspace=7 << 40)
    m, N, K = 256, 8192, 28672
    for name, last in (("codes", m * K), ("scales", m * K // 32), ("wq", N * K // 2), ("sq", N * K // 32)):
        for by in (0, last - 256, 256 - m * N * 2):
            assert _product(**(far | dict(out=far[name] + by)), m=m, N=N, K=K) == 2, (name, by)
        assert _product(**(far | dict(workspace=far[name])), m=m, N=N, K=K) == 2
        assert _product(**(far | dict(out_type=2, out_scales=far[name] + last - 4)), m=m, N=N, K=K) == 2
    assert _product(**(far | dict(workspace=5 << 40)), m=m, N=N, K=K) == 2
    assert _product(**(far | dict(out_type=2, out_scales=5 << 40)), m=m, N=N, K=K) == 2

    def turn(out=1 << 30, xt=256, xh=64, ot=256, oh=64):
        return F.lib().fp4_rope(_rope(), 1 << 30, out, 3, 4, 64, xt, xh, ot, oh, 0, None)
    assert turn(xt=512) == 2 and turn(xh=128, xt=512, ot=512) == 2
    c = F._KVCacheDesc(data=16, pages=4, page_size=64, kv_heads=2, head_dim=128, format=0, k_alpha=1.0, v_alpha=1.0)
    for over in (dict(q_out=2 << 30), dict(q_out=3 << 30), dict(q_out=1 << 30, qt=1024), dict(q_out=1 << 30, qt=1024, ot=1024, qh=256)):
        f = dict(q=1 << 30, q_out=5 << 30, k=2 << 30, v=3 << 30, slots=4 << 30, tokens=3, q_heads=4, qt=512, qh=128,
                 ot=512, oh=128, kt=256, kh=128, vt=256, vh=128, act=0) | over
        assert F.lib().fp4_kv_append_rope(ctypes.byref(c), _rope(), F._PACK_APPEND_ROPE.pack(*f.values()), None) == 2, over


def test_packed_arguments_have_the_structures_sizes():
    """Pointers and int64 first, the 4-byte fields at the end: no holes but the last."""
    for packer, eights, fours in ((F._PACK_NORM, 12, 3), (F._PACK_MX8, 11, 3), (F._PACK_ROPE, 4, 1),
                                  (F._PACK_APPEND_ROPE, 15, 1)):
        assert packer.size == (8 * eights + 4 * fours + 7) // 8 * 8
    with pytest.raises(ValueError):
        F._pack(struct.Struct("@Q"), "x", -1)


# ------------------------------------------------------------------- the binding
def test_binding_refuses():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    n = torch.zeros(4, dtype=torch.int64)
    f = torch.ones(32)
    for call in (lambda: F.rms_norm(x), lambda: F.quantize_mx8(x), lambda: F.rms_norm(x.float()),
                 lambda: F.rope(x.reshape(4, 1, 64), n, f), lambda: F.rope(x, n, f),
                 lambda: F.MX8(x, x, 64), lambda: F.MX8(x.to(torch.float8_e4m3fn), x, 64),
                 lambda: F.MX8(torch.zeros((4, 128), dtype=torch.float8_e4m3fn), x, 33)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(F.Fp4Error):
        F.gemm_mx8_workspace_size(1, 0, 32)
    for a, gate in ((x, None), (None, "silu")):
        with pytest.raises(ValueError):
            F.gemm_mx8(a, x, x, 32, gate=gate)
    with pytest.raises(ValueError):
        F.new_mx8(1, 48, "cpu")


def test_8_bit_rows_are_fixed():
    a = F.new_mx8(3, 160, "cpu")
    assert a.codes.shape == (3, 256) and a.scales.shape == (3, 8) and a.K == 160
    for name in ("codes", "scales", "K"):
        with pytest.raises(AttributeError):
            setattr(a, name, getattr(a, name))
        with pytest.raises(AttributeError):
            delattr(a, name)

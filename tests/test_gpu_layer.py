"""Norm, rotary positions, products of 8-bit activations and attention as a
decoder layer runs them: stage by stage against the oracle on the stage's own
inputs, eager against captured, on other streams and threads.

Bars per stage: the norm, the rotation and the cache's bytes bit for bit; products
as in tests/test_gpu_gemm_mx8.py; attention (tested on its own) by the roundings of
its kernel: half a step of BF16 on the result and on each probability, and the
scores' FP32 sums, e_s = (D + 4) 2^-24 scale max_j sum_d |q_d k_jd| + 2^-20, in
numerator and denominator (the scores of these rows reach thousands: e_s is no small
part)."""

import threading

import numpy as np
import pytest

import oracle
from mixed_precision_bf16_amd import fp4gemm as F
from mixed_precision_bf16_amd import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16 = torch.bfloat16
D, QH, H, HD, INNER, PAGE = 512, 8, 2, 64, 1408, 32
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def gfx950():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    name = torch.cuda.get_device_properties(0).gcnArchName
    if not name.startswith("gfx950"):
        pytest.skip(f"needs gfx950, found {name}")
    F.lib()
    yield


class Layer:
    def __init__(self, seed=0):
        self.canon, self.packed = {}, {}
        for i, (name, N, K) in enumerate((("qkv", (QH + 2 * H) * HD, D), ("o", D, QH * HD), ("up", 2 * INNER, D),
                                          ("down", D, INNER))):
            p = synth.make_random(1, N, K, 1, seed=100 * seed + i)
            scales = (p.scales.astype(np.int64) - 4).astype(np.uint8)          # results of about the size of their rows
            self.canon[name] = (p.codes, scales, N, K)
            self.packed[name] = tuple(t.cuda() for t in F.native_repack(p.codes, scales, N, K))
        g = torch.Generator().manual_seed(seed)
        self.norms = [(1 + 0.2 * torch.randn(D, generator=g)).to(BF16).cuda() for _ in range(2)]
        self.freq, self.amp = F.rope_frequencies(HD, 500000.0, "bands", 8.0, original=512)

    def product(self, name, a, **kw):
        return F.gemm_mx8(a, *self.packed[name], self.canon[name][2], **kw)

    def run(self, x, residual, cache, slots, positions, table, lens, offsets=None, max_q=None, stream=None, seen=None):
        kw = dict(stream=stream)
        n = x.shape[0]
        a, h = F.rms_norm(x, self.norms[0], EPS, residual=residual, mx8=True, **kw)
        qkv = self.product("qkv", a, **kw).view(n, QH + 2 * H, HD)
        q = F.kv_append_rope(cache, qkv[:, :QH], qkv[:, QH:QH + H], qkv[:, QH + H:], slots, positions, self.freq,
                             amplitude=self.amp, **kw)
        o = F.attention(q, cache, table, lens, q_offsets=offsets, max_q=max_q, **kw)
        a2 = F.quantize_mx8(o.view(n, QH * HD), **kw)
        y = self.product("o", a2, **kw)
        a3, h2 = F.rms_norm(y, self.norms[1], EPS, residual=h, mx8=True, **kw)
        f = self.product("up", a3, gate="silu", mx8=True, **kw)
        out = self.product("down", f, **kw)
        if seen is not None:
            seen.update(x=x, residual=residual, a=a, h=h, qkv=qkv, q=q, o=o, a2=a2, y=y, a3=a3, h2=h2, f=f, out=out)
        return out, h2

    # ------------------------------------------------------------- the oracle
    def check(self, s):
        def np64(t):
            return t.double().cpu().numpy()

        def codes(m):
            return m.codes.view(torch.uint8).cpu().numpy(), m.scales.view(torch.uint8).cpu().numpy()

        def same_mx8(m, want):
            for got, ref in zip(codes(m), oracle.mx8_quantize_reference(want)):
                assert np.array_equal(got, ref)

        def same(got, want):
            assert got.cpu().equal(torch.from_numpy(np.asarray(want, np.float32)).to(BF16))

        def product(name, a, got=None, gate=None):
            c, sc, N, K = self.canon[name]
            y, total = oracle.gemm_mx8_reference(*codes(a), c, sc, K)
            err = total * (2.0 ** -9 + K * 2.0 ** -24)
            if gate:
                half = N // 2
                u, g = np.abs(y[:, half:]), y[:, :half]
                v = oracle.gate_reference(g, y[:, half:], gate)
                act = np.abs(oracle.gate_reference(g, np.ones_like(g), gate))
                err = 1.13 * u * err[:, :half] + act * err[:, half:] + 1.13 * err[:, :half] * err[:, half:] + np.abs(v) * 2.0 ** -16
                y = v
            return y, err

        for first, x, r, w in (("a", "x", "residual", 0), ("a3", "y", "h", 1)):
            y, h = oracle.rms_norm_reference(np64(s[x]), np64(self.norms[w]), EPS, np64(s[r]))
            same_mx8(s[first], y)
            same(s["h" if w == 0 else "h2"], h)
        for name, a, got in (("qkv", "a", s["qkv"].reshape(len(s["x"]), -1)), ("o", "a2", s["y"]), ("down", "f", s["out"])):
            y, err = product(name, s[a])
            assert (np.abs(np64(got) - y) <= err + 2.0 ** -8 * (np.abs(y) + err)).all(), name
        same_mx8(s["a2"], np64(s["o"]).reshape(len(s["x"]), -1))
        y, err = product("up", s["a3"], gate="silu")
        c, sc = codes(s["f"])
        step = np.repeat(np.exp2(sc[:, :INNER // 32].astype(np.float64) - 127), 32, axis=1)
        far = np.abs(oracle.mx8_value(c, sc, INNER) - y)
        assert (far <= err + 2.0 ** -4 * (np.abs(y) + err) + 2.0 ** -10 * step).all()


class Sequences:
    """Two sequences in one cache, pages in turn."""

    def __init__(self, fmt=0, pages=16):
        self.fmt = fmt
        self.cache = F.new_kv_cache(pages, PAGE, H, HD, fmt)
        self.cache.data.fill_(0xFF)
        self.table = torch.arange(pages, dtype=torch.int32).view(-1, 2).T.contiguous()
        self.lens = [0, 0]

    def add(self, news):
        """(slots, positions, lens, offsets) of the next `news` tokens of each."""
        pos = [torch.arange(a, a + n) for a, n in zip(self.lens, news)]
        slots = torch.cat([self.table[b, p // PAGE].long() * PAGE + p % PAGE for b, p in enumerate(pos)])
        self.lens = [a + n for a, n in zip(self.lens, news)]
        off = torch.tensor([0, news[0], sum(news)], dtype=torch.int32)
        return (slots.cuda(), torch.cat(pos).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), off.cuda())

    def held(self):
        n = [torch.arange(x) for x in self.lens]
        return torch.cat([self.table[b, p // PAGE].long() * PAGE + p % PAGE for b, p in enumerate(n)])


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, D), generator=g)).to(BF16).cuda(), (torch.randn((n, D), generator=g) * 2).to(BF16).cuda()


@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_and_tokens_stage_by_stage(fmt):
    layer, seqs = Layer(), Sequences(fmt)
    keys, values = [], []
    want = np.full(seqs.cache.data.numel(), 0xFF, np.uint8)
    for step, news in enumerate(([41, 29], [1, 1], [1, 1])):
        n = sum(news)
        x, r = _rows(n, step)
        slots, pos, lens, off = seqs.add(news)
        seen = {}
        layer.run(x, r, seqs.cache, slots, pos, seqs.table.cuda(), lens, off, max(news), seen=seen)
        layer.check(seen)
        qkv = seen["qkv"].double().cpu().numpy()
        turn = lambda t: oracle.rope_reference(t, pos.cpu().numpy(), layer.freq.cpu().numpy(), False, layer.amp)  # noqa: E731
        bf = lambda t: torch.from_numpy(t.astype(np.float32)).to(BF16)  # noqa: E731
        assert seen["q"].cpu().equal(bf(turn(qkv[:, :QH])))
        k = bf(turn(qkv[:, QH:QH + H])).float().numpy()
        oracle.kv_write_reference(want, slots.cpu().numpy(), k, qkv[:, QH + H:].astype(np.float32), PAGE, fmt)
        assert np.array_equal(seqs.cache.data.cpu().numpy(), want)
        K, V = np.zeros((16 * PAGE, H, HD)), np.zeros((16 * PAGE, H, HD))
        at = seqs.held().numpy()
        K[at], V[at] = oracle.kv_read_reference(want, at, H, HD, PAGE, fmt)
        o, _, weight = oracle.attention_reference(seen["q"].double().cpu().numpy(), K, V, seqs.table.numpy(), seqs.lens,
                                                  off.cpu().numpy(), PAGE, scale=HD ** -0.5)
        q = np.abs(seen["q"].double().cpu().numpy()).reshape(n, H, QH // H, HD)
        mag = np.einsum("nhgd,khd->nhgk", q, np.abs(K[at])).max(-1).reshape(n, QH, 1)
        e_s = (HD + 4) * 2.0 ** -24 * HD ** -0.5 * mag + 2.0 ** -20 + sum(seqs.lens) * 2.0 ** -24
        # probabilities below 2^-14 are FP16 subnormals on the matrix core: half a step 2^-25 on each
        tiny = 2.0 ** -25 * np.repeat(np.abs(V[at]).sum(0), QH // H, axis=0)
        far = np.abs(seen["o"].double().cpu().numpy() - o) - ((2.0 ** -8 + 2 * e_s) * weight + 2.0 ** -8 * np.abs(o) + tiny)
        assert far.max() <= 0, (far.max(), np.argwhere(far > 0)[:4])


def test_captured_steps_follow_their_inputs():
    """A decode step in a graph: replayed with new rows, slots, positions and lengths,
    the program's own work between, and a second graph of the same step with other
    tensors; every replay equal to the eager call."""
    layer = Layer(1)

    class Step:
        def __init__(self):
            self.seqs = Sequences()
            self.x, self.r = _rows(2, 0)
            self.slots, self.pos, self.lens, _ = Sequences().add([1, 1])
            self.table = self.seqs.table.cuda()

        def call(self):
            return layer.run(self.x, self.r, self.seqs.cache, self.slots, self.pos, self.table, self.lens)

    steps = [Step(), Step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in steps:
            s.call()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.call())
        graphs.append(g)
    eager = [Sequences(), Sequences()]
    for e, s in zip(eager, steps):
        e.cache.data.copy_(s.seqs.cache.data)
    for turn in range(4):
        for i in (0, 1, 0)[turn % 2:]:
            x, r = _rows(2, 10 * turn + i)
            slots, pos, lens, _ = eager[i].add([1, 1])
            s = steps[i]
            for to, new in ((s.x, x), (s.r, r), (s.slots, slots), (s.pos, pos), (s.lens, lens)):
                to.copy_(new)
            graphs[i].replay()
            want = layer.run(x, r, eager[i].cache, slots, pos, s.table, lens)
            torch.cuda.synchronize()
            assert outs[i][0].equal(want[0]) and outs[i][1].equal(want[1])
            assert s.seqs.cache.data.equal(eager[i].cache.data)


def test_captured_products_with_a_split_of_k():
    """Two graphs, each with its own workspace, in turn and with eager calls between."""
    m, N, K = 96, 1024, 8192
    assert F.gemm_mx8_workspace_size(m, N, K) > 0
    p = synth.make_random(1, N, K, 1, seed=5)
    W = tuple(t.cuda() for t in F.native_repack(p.codes, p.scales, N, K))
    def rows(seed):
        return F.quantize_mx8(torch.randn((m, K), generator=torch.Generator().manual_seed(seed)).to(BF16).cuda())
    mine = [rows(0), rows(1)]
    ws = [torch.empty(F.gemm_mx8_workspace_size(m, N, K), dtype=torch.uint8, device="cuda").random_(0, 256) for _ in mine]
    F.gemm_mx8(mine[0], *W, N, workspace=ws[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a, w in zip(mine, ws):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(F.gemm_mx8(a, *W, N, workspace=w))
        graphs.append(g)
    for turn in range(4):
        for i in (0, 1):
            new = rows(10 * turn + i)
            mine[i].codes.copy_(new.codes)
            mine[i].scales.view(torch.uint8).copy_(new.scales.view(torch.uint8))
            want = F.gemm_mx8(new, *W, N)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert outs[i].equal(want)


def test_another_stream_and_dropped_inputs():
    """Calls on a busy stream: inputs that the caller drops keep their memory until it
    has read them."""
    layer, seqs = Layer(2), Sequences()
    x, r = _rows(70, 3)
    slots, pos, lens, off = seqs.add([41, 29])
    table = seqs.table.cuda()
    want = layer.run(x, r, seqs.cache, slots, pos, table, lens, off, 41)
    bytes_want = seqs.cache.data.clone()
    side = torch.cuda.Stream()
    for _ in range(3):
        inputs = [t.clone() for t in (x, r, slots, pos, lens, off)]
        other = Sequences()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = layer.run(inputs[0], inputs[1], other.cache, inputs[2], inputs[3], table, inputs[4], inputs[5], 41, stream=side)
        turned = F.rope(inputs[0].view(70, 8, 64), inputs[3], layer.freq, stream=side)
        held, sizes = [t.data_ptr() for t in inputs], [(t.shape, t.dtype) for t in inputs]
        del inputs
        reused = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
        assert not set(held) & {t.data_ptr() for t in reused}
        torch.cuda.current_stream().wait_stream(side)
        assert got[0].equal(want[0]) and got[1].equal(want[1]) and other.cache.data.equal(bytes_want)
        assert turned.equal(F.rope(x.view(70, 8, 64), pos, layer.freq))


def test_two_threads_at_once():
    layers = [Layer(3), Layer(4)]
    jobs = []
    for i, layer in enumerate(layers):
        seqs = Sequences(i)
        x, r = _rows(70, 20 + i)
        slots, pos, lens, off = seqs.add([41, 29])
        args = (x, r, seqs.cache, slots, pos, seqs.table.cuda(), lens, off, 41)
        jobs.append((layer, args, layer.run(*args)))
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                got[i].append(jobs[i][0].run(*jobs[i][1], stream=s))
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        assert len(got[i]) == 10
        for o in got[i]:
            assert o[0].equal(jobs[i][2][0]) and o[1].equal(jobs[i][2][1])


def test_tensors_off_the_device_are_refused():
    x = torch.zeros((4, 64), dtype=BF16, device="cuda")
    host = torch.zeros((4, 64), dtype=BF16)
    n, f = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(32, device="cuda")
    a = F.quantize_mx8(x)
    w = [torch.zeros(k, dtype=torch.uint8) for k in F.native_repack_size(32, 64)]
    W = [t.cuda() for t in w]
    cache = F.new_kv_cache(1, 32, 1, 64, 0)
    rows = x.view(4, 1, 64)
    for call in (lambda: F.rms_norm(x, residual=host), lambda: F.rms_norm(x, host[0]), lambda: F.rms_norm(x, out=host),
                 lambda: F.rms_norm(x, residual=x, sum_out=host), lambda: F.rms_norm(x, sum_out=x),
                 lambda: F.rms_norm(x, x[0].float()), lambda: F.rms_norm(x[:, 1:57]), lambda: F.rms_norm(x, mx8=True, out=x),
                 lambda: F.rms_norm(x[:, :40], mx8=True), lambda: F.rms_norm(x, mx8=True, out=F.new_mx8(4, 96)),
                 lambda: F.quantize_mx8(x, out=F.new_mx8(3, 64)), lambda: F.quantize_mx8(x[:, :40]),
                 lambda: F.gemm_mx8(a, *w, 32), lambda: F.gemm_mx8(a, W[0][:-1], W[1], 32),
                 lambda: F.gemm_mx8(a, *W, 32, gate="relu"), lambda: F.gemm_mx8(a, *W, 32, mx8=True, dtype=BF16),
                 lambda: F.gemm_mx8(a, *W, 32, dtype=torch.float32), lambda: F.gemm_mx8(a, *W, 32, out=x),
                 lambda: F.gemm_mx8(a, *W, 32, mx8=True, out=F.new_mx8(4, 64)),
                 lambda: F.gemm_mx8(a, *W, 32, workspace=torch.zeros(4)),
                 lambda: F.rope(rows, n.cpu(), f), lambda: F.rope(rows, n.int(), f), lambda: F.rope(rows, n[:3], f),
                 lambda: F.rope(rows, n, f.double()), lambda: F.rope(rows, n, torch.ones(33, device="cuda")),
                 lambda: F.rope(rows, n, f, out=host.view(4, 1, 64)), lambda: F.rope(rows, n, f, out=rows.half()),
                 lambda: F.kv_append_rope(cache, rows, rows, host.view(4, 1, 64), n, n, f),
                 lambda: F.kv_append_rope(cache, rows.half(), rows, rows, n, n, f),
                 lambda: F.kv_append_rope(cache, rows, rows, rows, n, n.cpu(), f),
                 lambda: F.kv_append_rope(cache, rows, rows, rows, n, n, f, q_out=host.view(4, 1, 64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: F.rms_norm(x, eps=0.0), lambda: F.rms_norm(x, eps=float("nan")),
                 lambda: F.gemm_mx8(a, *W, 32, alpha=0.0), lambda: F.rope(rows, n, f, amplitude=float("inf")),
                 lambda: F.rope(rows, n, f, out=rows[:1].expand(4, 1, 64))):
        with pytest.raises(F.Fp4Error):
            call()
    torch.cuda.synchronize()

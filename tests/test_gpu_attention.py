"""GPU parity of fp4_attention against the float64 oracle.

Inputs are written into the cache by the oracle, so the reference knows the
rows exactly.  Tolerance of one output, from the roundings of the kernel: half
a step u_o of the output type on the result, and on every probability half a
step u_p of the matrix-core type (BF16 for MXFP4 caches with BF16 activations,
else FP16) plus the error e_s of its score in FP32:

    |out - ref| <= u_o |ref| + (u_p + 2 e_s) sum_j p_j |v_j| / l + tiny

with e_s = (D + 4) 2^-24 scale max_j sum_d |q_d k_jd| + 2^-20 (the FP32 sums of
the products, and the exponential) plus (keys) 2^-24 for the FP32 sum over
the keys; tiny covers FP16 subnormals of the output (2^-25).  The numerator and
the denominator both carry e_s, hence the 2.  lse: e_s + 2^-22 |lse| +
(keys) 2^-24."""

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


class Problem:
    """Sequences of `lens` keys with `news` query tokens each, pages in random
    order, everything that no token was written to filled with 0xFF (NaN
    scales)."""

    def __init__(self, lens, news, fmt=0, dtype=BF16, D=128, H=2, group=4, page=64, seed=0, strength=1.5, ka=1.0,
                 va=1.0, extra_columns=0):
        rng = np.random.Generator(np.random.PCG64(seed))
        self.lens, self.fmt, self.dtype, self.D, self.H, self.page = list(lens), fmt, dtype, D, H, page
        self.ka, self.va, self.heads = ka, va, H * group
        per = [-(-x // page) for x in lens]
        self.pages = sum(per) + 2
        order = rng.permutation(self.pages)
        cols = max(per + [1]) + extra_columns
        self.table = np.full((len(lens), cols), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.data = np.full(F.kv_cache_size(self.pages, page, H, D, fmt), 0xFF, np.uint8)
        slots = np.concatenate([self.slots(b, np.arange(x)) for b, x in enumerate(lens)]).astype(np.int64)
        x = rng.standard_normal((2, len(slots), H, D)).astype(np.float32)
        x[0, :, :, :3] *= 4.0
        x[0] *= ka
        x[1] *= va
        oracle.kv_write_reference(self.data, slots, x[0], x[1], page, fmt, ka, va)
        self.k = np.zeros((self.pages * page, H, D))
        self.v = np.zeros_like(self.k)
        if len(slots):
            self.k[slots], self.v[slots] = oracle.kv_read_reference(self.data, slots, H, D, page, fmt, ka, va)
        self.offsets = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        q = rng.standard_normal((int(self.offsets[-1]), self.heads, D)) * strength / ka
        self.q = torch.from_numpy(q).to(dtype)
        self.uniform = len(set(news)) == 1
        self.scale = D ** -0.5

    def slots(self, b, pos):
        return self.table[b, pos // self.page].astype(np.int64) * self.page + pos % self.page

    def cache(self):
        return F.KVCache(torch.from_numpy(self.data).cuda(), self.pages, self.page, self.H, self.D, self.fmt, self.ka,
                         self.va)

    def run(self, q=None, **kw):
        off = kw.pop("offsets", None)
        if off is None and not self.uniform:
            off = torch.from_numpy(self.offsets).cuda()
        kw.setdefault("scale", self.scale)
        return F.attention(self.q.cuda() if q is None else q, self.cache(), torch.from_numpy(self.table).cuda(),
                           torch.tensor(self.lens, dtype=torch.int32, device="cuda"), q_offsets=off, return_lse=True,
                           **kw)

    def check(self, got, causal=True, window=0, sinks=None, scale=None):
        scale = float(np.float32(self.scale if scale is None else scale))
        q = self.q.double().numpy()
        ref, lse, weight = oracle.attention_reference(q, self.k, self.v, self.table, self.lens, self.offsets, self.page,
                                                      causal, window, scale, sinks)
        out = got[0].double().cpu().numpy()
        got_lse = got[1].double().cpu().numpy()
        group = self.heads // self.H
        u_o = torch.finfo(self.dtype).eps / 2
        u_p = 2.0 ** -8 if self.fmt == 1 and self.dtype == BF16 else 2.0 ** -11
        e_s = np.zeros(lse.shape)
        for b, n in enumerate(np.diff(self.offsets)):
            s = self.slots(b, np.arange(self.lens[b])) if self.lens[b] else np.zeros(0, np.int64)
            s = s[(s >= 0) & (s < len(self.k))]
            for h in range(self.heads):
                qa = np.abs(q[self.offsets[b]:self.offsets[b] + n, h])
                mag = (qa @ np.abs(self.k[s, h // group]).T).max(-1, initial=0.0) if n else 0.0
                e_s[self.offsets[b]:self.offsets[b] + n, h] = (self.D + 4) * 2.0 ** -24 * scale * mag + 2.0 ** -20
        keys = max(self.lens + [1]) * 2.0 ** -24
        bound = u_o * np.abs(ref) + (u_p + 2 * e_s[..., None] + keys) * weight + 2.0 ** -25
        assert np.all(np.isfinite(out))
        off = np.abs(out - ref)
        assert np.all(off <= bound), (float((off / bound).max()), np.argwhere(off > bound)[:4])
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        d = np.abs(got_lse[~empty] - lse[~empty])
        assert np.all(d <= (e_s + keys)[~empty] + 2.0 ** -22 * np.abs(lse[~empty])), float(d.max(initial=0))


def _go(p, **kw):
    sinks = kw.get("sinks")
    dev = dict(kw)
    if sinks is not None:
        dev["sinks"] = torch.from_numpy(sinks).cuda()
    got = p.run(**dev)
    torch.cuda.synchronize()
    kw.pop("max_q", None)
    p.check(got, **kw)
    return got


def _sinks(heads, seed):
    s = np.random.Generator(np.random.PCG64(seed)).standard_normal(heads).astype(np.float32)
    s[0] = -np.inf
    return s


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D,H,group,page", [(64, 1, 1, 32), (64, 8, 8, 64), (128, 2, 4, 96), (128, 8, 8, 64),
                                            (128, 1, 16, 128), (256, 2, 5, 32), (256, 1, 1, 256)])
def test_decode(D, H, group, page, fmt, dtype):
    """One query token a sequence, lengths from one key on."""
    print("[case] decode", D, H, group, page, fmt, dtype, flush=True)
    p = Problem([1, 31, 32, 33, 127, 129, 300, 64], [1] * 8, fmt, dtype, D, H, group, page, seed=D + group)
    _go(p)


@pytest.mark.parametrize("fmt,dtype,ka,va", [(0, BF16, 0.02, 0.7), (0, FP16, 1.3, 0.01), (1, BF16, 0.3, 1.9),
                                             (1, FP16, 2.0, 0.5)])
def test_alphas(fmt, dtype, ka, va):
    _go(Problem([70, 200], [1, 1], fmt, dtype, ka=ka, va=va, seed=3))


@pytest.mark.parametrize("fmt,dtype", [(0, BF16), (1, BF16), (1, FP16)])
@pytest.mark.parametrize("news,lens,D,group", [
    ([4, 4, 4], [4, 100, 257], 128, 8), ([2, 2], [2, 65], 64, 20), ([1, 5, 3, 0, 2], [9, 200, 3, 50, 64], 128, 4),
    ([17, 1, 40], [17, 500, 130], 128, 5), ([33, 70], [33, 200], 256, 3), ([7, 130], [64, 130], 64, 8)])
def test_several_query_tokens(news, lens, D, group, fmt, dtype):
    """Drafted tokens, ragged chunks and prompts; a sequence without queries."""
    print("[case] several", news, lens, D, group, fmt, dtype, flush=True)
    p = Problem(lens, news, fmt, dtype, D, 2, group, seed=len(lens) + D)
    _go(p)
    _go(p, max_q=max(news))


@pytest.mark.parametrize("max_q", [1, None])
@pytest.mark.parametrize("window", [1, 31, 33, 128, 5000])
@pytest.mark.parametrize("sinks", [False, True])
def test_window_and_sinks(window, sinks, max_q):
    p = Problem([1, 40, 333, 700], [1, 3, 2, 40], 1, BF16, 64, 2, 8, 32, seed=window)
    _go(p, window=window, sinks=_sinks(16, 5) if sinks else None, max_q=max_q)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 20, 1]])
def test_all_keys_without_causal_order(news):
    _go(Problem([5, 90, 260], news, 0, FP16, seed=8), causal=False)


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("max_q", [1, 40])
def test_rows_that_see_nothing(sinks, max_q):
    """Empty sequences, and query tokens that lie before the first key."""
    p = Problem([0, 2, 0, 70, 10], [1, 5, 3, 2, 33], 0, BF16, seed=9)
    got = _go(p, sinks=_sinks(8, 6) if sinks else None, max_q=max_q)
    assert torch.all(got[0][0] == 0) and torch.all(got[0][1:4] == 0)


@pytest.mark.parametrize("max_q", [2, 60])
def test_pages_that_are_not_there(max_q):
    """Entries outside [0, pages) hold no keys, wherever they are."""
    p = Problem([200, 300, 64], [2, 60, 1], 0, BF16, page=32, seed=10)
    p.table[0, 2], p.table[1, 0], p.table[1, 9], p.table[2, :] = -1, p.pages, np.iinfo(np.int32).min, -7
    _go(p, max_q=max_q)


def test_infinite_keys_stay_with_the_queries_that_see_them():
    """A token written with infinities does not reach earlier queries (NVFP4
    saturates them, an MXFP4 scale saturates in the value product)."""
    for fmt, dtype in ((0, BF16), (1, BF16), (1, FP16)):
        p = Problem([40], [3], fmt, dtype, 128, 1, 4, 64, seed=11)
        clean = p.run()
        bad = np.full((1, 1, 128), np.inf, np.float32)
        oracle.kv_write_reference(p.data, p.slots(0, np.array([39])), bad, bad, 64, fmt)
        got = p.run()
        assert torch.equal(got[0][:2], clean[0][:2]) and torch.equal(got[1][:2], clean[1][:2])


@pytest.mark.parametrize("fmt,dtype,strength", [(0, BF16, 200.0), (0, BF16, 1e-20), (1, BF16, 200.0), (0, FP16, 100.0),
                                                (1, FP16, 1e-3)])
def test_strong_and_weak_queries(fmt, dtype, strength):
    """Peaked and flat softmax; BF16 queries far from FP16's range."""
    _go(Problem([130, 513], [1, 4], fmt, dtype, strength=strength, seed=12))


def test_growing_scores_rescale():
    """Scores that grow along the sequence: the running maximum moves in every
    tile, and early keys vanish."""
    p = Problem([600], [1], 0, BF16, 128, 1, 4, 64, seed=13)
    slots = p.slots(0, np.arange(600))
    k = np.random.Generator(np.random.PCG64(1)).standard_normal((600, 1, 128)).astype(np.float32) * 0.05
    k[:, 0, 0] = np.arange(600) * 0.2
    v = np.random.Generator(np.random.PCG64(2)).standard_normal((600, 1, 128)).astype(np.float32)
    oracle.kv_write_reference(p.data, slots, k, v, 64, 0)
    p.k[slots], p.v[slots] = oracle.kv_read_reference(p.data, slots, 1, 128, 64, 0)
    p.q[..., 0] = 6.0
    _go(p)
    p.q[..., 0] = -6.0
    _go(p)


@pytest.mark.parametrize("lens,H", [([9000], 1), ([4000, 1, 70, 2500], 2), ([700] * 40, 4)])
def test_items_split_over_workgroups(lens, H):
    """Long sequences are joined from partial sums; repeated calls with a used
    workspace give the same bits."""
    p = Problem(lens, [1] * len(lens), 0, BF16, 128, H, 8, 64, seed=H)
    size = F.attention_workspace_size(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
                                      torch.tensor(p.lens, dtype=torch.int32, device="cuda"))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    first = _go(p)
    for _ in range(3):
        again = p.run(workspace=ws)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("B", [300, 1000])
def test_large_batches(B):
    """More sequences than one pass of the work scan covers, most of them short."""
    rng = np.random.Generator(np.random.PCG64(B))
    lens = [int(x) for x in rng.integers(0, 40, B)]
    lens[B // 2] = 2000
    _go(Problem(lens, [1] * B, 1, BF16, 64, 1, 2, 32, seed=B))


def test_strides_rows_of_no_sequence_and_longer_tables():
    p = Problem([100, 80], [2, 3], 0, BF16, 128, 2, 4, 64, seed=14, extra_columns=3)
    want = p.run()
    q = torch.randn((8, 3 * 8, 128), device="cuda").to(BF16)
    q[1:6, 8:16] = p.q.cuda()
    out = torch.full((8, 8 * 2, 128), 5.0, dtype=BF16, device="cuda")
    lse = torch.full((8, 8), 5.0, device="cuda")
    wide = torch.full((2, 2 * p.table.shape[1]), 1 << 20, dtype=torch.int32, device="cuda")
    wide[:, :p.table.shape[1]] = torch.from_numpy(p.table).cuda()
    off = torch.tensor([1, 3, 6], dtype=torch.int32, device="cuda")
    F.attention(q[:, 8:16], p.cache(), wide[:, :p.table.shape[1]],
                torch.tensor(p.lens, dtype=torch.int32, device="cuda"), q_offsets=off, out=out[:, ::2], lse=lse,
                scale=p.scale)
    assert torch.equal(out[1:6, ::2], want[0]) and torch.equal(lse[1:6], want[1])
    assert torch.all(out[:, 1::2] == 5) and torch.all(out[[0, 6, 7]] == 5) and torch.all(lse[[0, 6, 7]] == 5)


def test_lengths_past_the_table_are_clamped():
    p = Problem([64, 128], [1, 1], 0, BF16, page=64, seed=15)
    p.table = np.where(p.table < 0, -1, p.table)
    got = F.attention(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
                      torch.tensor([64, 1 << 30], dtype=torch.int32, device="cuda"), return_lse=True)
    p.check(got)
    got = F.attention(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
                      torch.tensor([-5, 128], dtype=torch.int32, device="cuda"), return_lse=True)
    assert torch.all(got[0][0] == 0) and torch.all(torch.isneginf(got[1][0]))


def test_offsets_out_of_range_are_clamped():
    p = Problem([50, 60], [1, 2], 0, BF16, seed=16)
    off = torch.tensor([-4, 1, 1 << 30], dtype=torch.int32, device="cuda")
    p.check(p.run(offsets=off))


@pytest.mark.parametrize("rows,max_q,off", [(6, 1, [0, 6, 2, 6]), (1400, 1400, [0, 1400, 700, 1400])])
def test_offsets_that_decrease_write_nothing(rows, max_q, off):
    p = Problem([50, 60, 70], [2, 2, 2], 0, BF16, seed=22)
    q = torch.zeros((rows, 8, 128), dtype=BF16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((rows, 8), 7.0, device="cuda")
    args = (q, p.cache(), torch.from_numpy(p.table).cuda(), torch.tensor(p.lens, dtype=torch.int32, device="cuda"))
    F.attention(*args, q_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), max_q=max_q, out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(out == 7) and torch.all(lse == 7)


def test_a_query_of_nan_stays_alone():
    for news, max_q in (([3, 1], 3), ([70, 64], None)):
        p = Problem([200, 300], news, 0, BF16, seed=23)
        want = p.run(max_q=max_q)
        p.q[1, 2, 5] = float("nan")
        p.q[2, 3, :] = float("inf")
        got = p.run(max_q=max_q)
        keep = torch.ones(got[1].shape, dtype=torch.bool, device="cuda")
        keep[1, 2] = keep[2, 3] = False
        assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
        assert torch.all(torch.isnan(got[0][1, 2])) and torch.all(torch.isnan(got[0][2, 3]))


@pytest.mark.parametrize("B", [70, 600])
def test_prompts_of_many_sequences(B):
    """More sequences than a wave's lanes: blocks in the order of the sequences."""
    rng = np.random.Generator(np.random.PCG64(B))
    news = [int(x) for x in rng.integers(0, 40, B)]
    lens = [n + int(x) for n, x in zip(news, rng.integers(0, 60, B))]
    p = Problem(lens, news, 1, BF16, 64, 4, 4, 32, seed=B)
    got = p.run(max_q=64)
    few = sorted({0, 1, B // 2, 63, 64, 65, B - 2, B - 1})
    one = Problem.__new__(Problem)
    for b in few:
        one.__dict__.update(p.__dict__)
        lo, hi = int(p.offsets[b]), int(p.offsets[b + 1])
        if lo == hi:
            continue
        one.lens, one.table, one.q = [p.lens[b]], p.table[b:b + 1], p.q[lo:hi]
        one.offsets = np.array([0, hi - lo], np.int32)
        one.check((got[0][lo:hi], got[1][lo:hi]))


def test_graph_replay_follows_the_data():
    """A captured step (append, attention) replayed with other lengths, tokens
    and queries, the program's own work between the replays; a second graph
    shares the workspace."""
    H, D, group, page, B = 2, 128, 4, 64, 3
    cache = F.new_kv_cache(40, page, H, D, 0)
    gen = torch.Generator("cuda").manual_seed(3)
    fill = torch.randn((40 * page, 2 * H, D), device="cuda", generator=gen).to(BF16)
    F.kv_append(cache, fill[:, :H], fill[:, H:], torch.arange(40 * page, device="cuda"))
    table = torch.randperm(36, device="cuda", generator=gen).to(torch.int32).reshape(3, 12)
    q = torch.empty((B, H * group, D), dtype=BF16, device="cuda")
    kv = torch.empty((B, 2 * H, D), dtype=BF16, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int64, device="cuda")
    ws = torch.empty(F.attention_workspace_size(q, cache, table, lens), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(q), torch.empty((B, H * group), device="cuda")) for _ in range(2)]

    def step(i):
        F.kv_append(cache, kv[:, :H], kv[:, H:], slots)
        F.attention(q, cache, table, lens, out=outs[i][0], lse=outs[i][1], workspace=ws)

    def load(seed):
        g = torch.Generator("cuda").manual_seed(seed)
        q.copy_(torch.randn(q.shape, device="cuda", generator=g))
        kv.copy_(torch.randn(kv.shape, device="cuda", generator=g))
        n = torch.randint(1, 12 * page, (B,), device="cuda", generator=g)
        lens.copy_(n)
        slots.copy_(table.gather(1, ((n - 1) // page)[:, None])[:, 0].long() * page + (n - 1) % page)

    load(0)
    step(0)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(i)
        graphs.append(g)
    for seed in range(1, 7):
        load(seed)
        want = F.attention(q, _appended(cache, kv, H, slots), table, lens, return_lse=True)
        torch.cuda.synchronize()
        i = seed % 2
        outs[i][0].fill_(9.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])


def test_graph_replay_of_a_split_chunk():
    """The tiled kernel with shares of the keys, captured once, replayed over
    other lengths (also ones too short to share)."""
    p = Problem([3000, 2000], [70, 70], 1, FP16, 128, 1, 8, 64, seed=24)
    q, cache, table = p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(F.attention_workspace_size(q, cache, table, lens), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    out, lse = torch.empty_like(q), torch.empty((140, 8), device="cuda")
    F.attention(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        F.attention(q, cache, table, lens, out=out, lse=lse, workspace=ws)
    for a, b in ((3000, 2000), (70, 1999), (513, 69), (0, 2000), (2999, 128)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        want = F.attention(q, cache, table, lens, return_lse=True)
        torch.cuda.synchronize()
        out.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, interleaved."""
    ps = [Problem([4000, 50], [1, 1], 0, BF16, seed=25), Problem([2500], [70], 0, BF16, 128, 1, 8, seed=26)]
    want = [p.run() for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    args = [(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
             torch.tensor(p.lens, dtype=torch.int32, device="cuda")) for p in ps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(F.attention(*args[i], scale=ps[i].scale, stream=s, return_lse=True))
    torch.cuda.synchronize()
    for i in range(2):
        for o in got[i]:
            assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])


def _appended(cache, kv, H, slots):
    c = F.KVCache(cache.data.clone(), cache.pages, cache.page_size, cache.kv_heads, cache.head_dim, cache.fmt)
    F.kv_append(c, kv[:, :H], kv[:, H:], slots)
    return c


def test_another_stream():
    p = Problem([500, 3000], [1, 1], 0, BF16, seed=17)
    want = p.run()
    q, cache, table = p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [F.attention(q, cache, table, lens, scale=p.scale, stream=side, return_lse=True) for _ in range(4)]
    k, v = F.kv_read(cache, torch.from_numpy(p.slots(1, np.arange(100))).cuda(), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    assert np.array_equal(k.double().cpu().numpy(), p.k[p.slots(1, np.arange(100))])


def test_no_queries_is_a_no_op():
    p = Problem([5], [1], seed=18)
    e = torch.empty((0, 8, 128), dtype=BF16, device="cuda")
    out = F.attention(e, p.cache(), torch.from_numpy(p.table).cuda(),
                      torch.tensor([5], dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 8, 128)


def test_binding_refusals():
    p = Problem([50, 60], [1, 1], seed=19)
    q, c, t = p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda()
    n = torch.tensor([50, 60], dtype=torch.int32, device="cuda")
    for bad in (lambda: F.attention(q.float(), c, t, n), lambda: F.attention(q[:, :, :64], c, t, n),
                lambda: F.attention(q, c, t.long(), n), lambda: F.attention(q, c, t, n.long()),
                lambda: F.attention(q, c, t, n[:1]), lambda: F.attention(q, c, t.cpu(), n),
                lambda: F.attention(q.cpu(), c, t, n), lambda: F.attention(q[0], c, t, n),
                lambda: F.attention(q[:1], c, t, n), lambda: F.attention(q, c, t, n, q_offsets=n),
                lambda: F.attention(q, c, t, n, sinks=torch.zeros(7, device="cuda")),
                lambda: F.attention(q, c, t, n, out=torch.empty_like(q, dtype=FP16)),
                lambda: F.attention(q, c, t, n, lse=torch.empty((2, 7), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(window=3, causal=False), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(F.Fp4Error):
            F.attention(q, c, t, n, **bad)
    with pytest.raises(F.Fp4Error):
        F.attention(torch.cat([q, q], 1)[:, :9], c, t, n)


@pytest.mark.parametrize("fmt,dtype", [(0, BF16), (1, FP16)])
def test_projection_cache_attention_projection(fmt, dtype):
    """The operators as a decode step uses them: an FP4 projection makes q, k
    and v, the new tokens go into the cache, attention reads it, and an FP4
    projection follows; each stage against its oracle on the stage's inputs."""
    B, H, group, D, page, width = 3, 2, 4, 64, 32, 256
    heads = H * group
    rng = np.random.Generator(np.random.PCG64(21))
    p = Problem([33, 70, 5], [1, 1, 1], fmt, dtype, D, H, group, page, seed=20)

    def weight(N, K):
        w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32) * K ** -0.5).to(BF16)
        codes, scales = oracle.quantize_reference(w.view(torch.int16).numpy().view(np.uint16), fmt)
        return codes, scales, F.upload(*F.repack(codes, scales, N, K, fmt))

    c1, s1, (w1, z1) = weight((heads + 2 * H) * D, width)
    c2, s2, (w2, z2) = weight(width, heads * D)
    x = torch.from_numpy(rng.standard_normal((B, width)).astype(np.float32)).to(dtype).cuda()
    qkv = F.gemm(x, w1, z1, (heads + 2 * H) * D, width, fmt).reshape(B, heads + 2 * H, D)
    cache = p.cache()
    table = torch.from_numpy(p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    at = np.array([p.slots(b, np.array([n - 1]))[0] for b, n in enumerate(p.lens)])
    F.kv_append(cache, qkv[:, heads:heads + H], qkv[:, heads + H:], torch.from_numpy(at).cuda())
    out, lse = F.attention(qkv[:, :heads], cache, table, lens, scale=p.scale, return_lse=True)
    y = F.gemm(out.reshape(B, heads * D), w2, z2, width, heads * D, fmt)
    torch.cuda.synchronize()

    new = qkv[:, heads:].float().cpu().numpy()
    oracle.kv_write_reference(p.data, at, new[:, :H], new[:, H:], page, fmt)
    assert np.array_equal(cache.data.cpu().numpy(), p.data)
    p.k[at], p.v[at] = oracle.kv_read_reference(p.data, at, H, D, page, fmt)
    p.q = qkv[:, :heads].cpu()
    p.check((out, lse))
    bits = lambda t: t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    act = "bf16" if dtype == BF16 else "f16"
    for a, c, s, K, got in ((x, c1, s1, width, qkv.reshape(B, -1)), (out.reshape(B, -1), c2, s2, heads * D, y)):
        ref = oracle.act_bits_to_f64(bits(a), act) @ oracle.dequant_weights(c, s, K, fmt).T
        mag = np.abs(oracle.act_bits_to_f64(bits(a), act)) @ np.abs(oracle.dequant_weights(c, s, K, fmt)).T
        assert np.all(np.abs(got.double().cpu().numpy() - ref) <= 8e-3 * np.abs(ref) + 2e-3 * mag)


@pytest.mark.parametrize("fmt,dtype", [(0, BF16), (1, BF16), (0, FP16), (1, FP16)])
@pytest.mark.parametrize("D,H,group,lens,news", [
    (128, 1, 8, [3000, 100], [70, 64]), (64, 2, 8, [2500], [65]), (256, 1, 8, [1900], [100]),
    (128, 2, 2, [200] * 64, [64] * 64), (128, 8, 8, [300, 700], [300, 260]), (64, 16, 4, [1, 513, 130, 200], [1, 513, 77, 130]),
    (256, 4, 4, [900, 64, 33], [900, 64, 20]), (128, 8, 5, [640, 40], [600, 40]), (128, 32, 1, [1100], [1050])])
def test_prompts(D, H, group, lens, news, fmt, dtype):
    """Query rows enough for the tiled kernel, with and without shares of the keys; sampled rows against the oracle."""
    print("[case] prompts", D, H, group, lens, news, fmt, dtype, flush=True)
    p = Problem(lens, news, fmt, dtype, D, H, group, 32 if D == 64 else 96, seed=D + H)
    got = p.run()
    torch.cuda.synchronize()
    _check_sampled(p, got)
    again = p.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def _check_sampled(p, got, **kw):
    """p.check on a few query tokens and heads (the oracle is slow)."""
    rows = int(p.offsets[-1])
    rng = np.random.Generator(np.random.PCG64(rows))
    heads = sorted({0, p.heads - 1, int(rng.integers(p.heads))})
    group = p.heads // p.H
    for b, n in enumerate(np.diff(p.offsets)):
        for i in sorted({0, 1, int(n) - 1, int(n) // 2, *(int(x) for x in rng.integers(0, max(n, 1), 6))} & set(range(n))):
            for h in heads:
                one = Problem.__new__(Problem)
                one.__dict__.update(p.__dict__)
                row = int(p.offsets[b]) + i
                one.lens, one.table = [max(0, p.lens[b] - int(n) + i + 1)], p.table[b:b + 1]
                one.offsets = np.array([0, 1], np.int32)
                one.q = p.q[row:row + 1, h:h + 1]
                one.H, one.heads = 1, 1
                one.k, one.v = p.k[:, h // group:h // group + 1], p.v[:, h // group:h // group + 1]
                one.check((got[0][row:row + 1, h:h + 1], got[1][row:row + 1, h:h + 1]),
                          **({**kw, "sinks": kw["sinks"][h:h + 1]} if kw.get("sinks") is not None else kw))


@pytest.mark.parametrize("window,sinks", [(0, True), (1, False), (70, True), (300, False)])
def test_prompts_with_window_and_sinks(window, sinks):
    p = Problem([700, 90], [650, 90], 1, BF16, 64, 16, 4, 32, seed=window + 2)
    s = _sinks(64, 4) if sinks else None
    got = p.run(window=window, sinks=None if s is None else torch.from_numpy(s).cuda())
    _check_sampled(p, got, window=window, sinks=s)


def test_prompts_with_empty_rows_missing_pages_and_strides():
    """Queries before the first key, pages that are not there and rows of no
    sequence, in the tiled kernel."""
    p = Problem([600, 100, 0], [600, 180, 9], 0, BF16, 128, 8, 8, 32, seed=33)
    p.table[0, 3], p.table[0, 10], p.table[1, 0] = -1, p.pages + 4, -2
    q = torch.full((800, 2 * 64, 128), float("nan"), dtype=BF16, device="cuda")
    q[4:793, :64] = p.q.cuda()
    out = torch.full((800, 64, 256), 5.0, dtype=BF16, device="cuda")[:, :, :128]
    lse = torch.full((800, 64), 5.0, device="cuda")
    F.attention(q[:, :64], p.cache(), torch.from_numpy(p.table).cuda(),
                torch.tensor(p.lens, dtype=torch.int32, device="cuda"),
                q_offsets=torch.from_numpy(p.offsets + 4).cuda(), out=out, lse=lse, scale=p.scale)
    assert torch.all(out[:4] == 5) and torch.all(out[793:] == 5) and torch.all(lse[:4] == 5) and torch.all(lse[793:] == 5)
    _check_sampled(p, (out[4:793], lse[4:793]))
    assert torch.all(out[604:684] == 0) and torch.all(torch.isneginf(lse[604:684]))
    assert torch.all(out[784:793] == 0) and torch.all(torch.isneginf(lse[784:793]))


def test_prompts_without_causal_order():
    p = Problem([520], [513], 1, FP16, 128, 8, 8, 64, seed=34)
    got = p.run(causal=False)
    q = p.q[:3].double().numpy()
    ref, lse, w = oracle.attention_reference(q, p.k, p.v, p.table, p.lens, [0, 3], 64, False, 0,
                                             float(np.float32(p.scale)))
    off = np.abs(got[0][:3].double().cpu().numpy() - ref)
    assert np.all(off <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -10 * w + 2.0 ** -25)


def test_kernels_agree():
    """max_q only chooses the kernel: both give the same rows up to rounding."""
    p = Problem([900, 333], [700, 333], 0, FP16, 128, 8, 8, 64, seed=35)
    a, b = p.run(max_q=1), p.run()
    assert torch.all((a[0].float() - b[0].float()).abs() <= 2.0 ** -9 * b[0].float().abs() + 2.0 ** -10)
    assert torch.all((a[1] - b[1]).abs() <= 2.0 ** -18 * (1 + b[1].abs()))


PAIRS = [(0, BF16), (0, FP16), (1, BF16), (1, FP16)]


def _rows_of_all_sizes(fmt, dtype, D, alpha, seed):
    """One key a sequence, 2 heads, the size of its rows 2^-13 .. 2^14: (cache, table, slots)."""
    B, H = 28, 2
    gen = torch.Generator("cuda").manual_seed(seed)
    kv = torch.rand((2, B, H, D), device="cuda", generator=gen) * 2 - 1
    kv *= 2.0 ** torch.arange(-13, 15, device="cuda")[:, None, None]
    cache = F.new_kv_cache(B, 32, H, D, fmt, alpha, alpha)
    cache.data.fill_(0xFF)
    slots = torch.randperm(B, device="cuda", generator=gen) * 32
    F.kv_append(cache, kv[0].to(dtype), kv[1].to(dtype), slots)
    return cache, (slots // 32).to(torch.int32)[:, None].contiguous(), slots


ALPHAS = [1.0, 0.37, 1e-3, 2.0 ** -20, 3000.0, 4096.0]


@pytest.mark.parametrize("alpha", ALPHAS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,dtype", PAIRS)
@pytest.mark.parametrize("n", [1, 96])
def test_values_come_out_as_they_are_read_back(fmt, dtype, D, alpha, n):
    """One key and queries of zero: its weight is exactly 1, and the output is
    its value row, the same bits as the read-back gives, whatever alpha and the
    rows' size are (both scale the exact code x scale by alpha in FP32, once)."""
    cache, table, slots = _rows_of_all_sizes(fmt, dtype, D, alpha, D)
    v = F.kv_read(cache, slots, dtype=dtype)[1]
    B = len(slots)
    q = torch.zeros((B * n, 2 * 8, D), dtype=dtype, device="cuda")
    out = F.attention(q, cache, table, torch.ones(B, dtype=torch.int32, device="cuda"), causal=False)
    want = v.repeat_interleave(8, 1).repeat_interleave(n, 0)
    assert torch.equal(out, want)


@pytest.mark.parametrize("alpha", ALPHAS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt,dtype", PAIRS)
@pytest.mark.parametrize("n", [1, 96])
def test_keys_weigh_as_they_are_read_back(fmt, dtype, D, alpha, n):
    """One key and queries with a single 1: the log-sum-exp is scale times one
    element x of the key row, exact but for these FP32 roundings (half a step,
    2^-24 relative, each): scale alpha, log2 e itself, times it, the score, 8 - m
    (its share of m), m plus the logarithm, ln 2 itself, times it, 8 in all; and
    next to 0 those that stay, in units of 2^-24: 8 - m in [8, 16) 8 ln 2, the
    exponential 2, the logarithm of a sum next to 1 2, at most 12."""
    cache, table, slots = _rows_of_all_sizes(fmt, dtype, D, alpha, D + 1)
    B = len(slots)
    q = torch.zeros((B, n, 2 * 8, D), dtype=dtype, device="cuda")
    at = torch.arange(16, device="cuda") * 37 % D
    q[:, :, torch.arange(16, device="cuda"), at] = 1.0
    _, lse = F.attention(q.reshape(B * n, 16, D), cache, table, torch.ones(B, dtype=torch.int32, device="cuda"),
                         causal=False, return_lse=True)
    k = oracle.kv_read_reference(cache.data.cpu().numpy(), slots.cpu().numpy(), 2, D, 32, fmt, alpha, alpha)[0]
    k = k.repeat(8, 1)[:, np.arange(16), at.cpu().numpy()]
    want = np.repeat(k * float(np.float32(D ** -0.5)), n, 0)
    off = np.abs(lse.double().cpu().numpy() - want)
    assert np.all(off <= 8 * 2.0 ** -24 * np.abs(want) + 12 * 2.0 ** -24)


def _of_size(lens, news, k_size, v_size, ka, va, fmt, dtype, D=128, H=2, group=4, seed=0):
    """A Problem whose rows have the given sizes, whatever the alphas are."""
    p = Problem(lens, news, fmt, dtype, D, H, group, 64, seed, strength=1.5 / k_size)
    p.ka, p.va = ka, va
    slots = np.concatenate([p.slots(b, np.arange(x)) for b, x in enumerate(lens)])
    x = np.random.Generator(np.random.PCG64(seed + 1)).standard_normal((2, len(slots), H, D)).astype(np.float32)
    x[0] *= k_size
    x[1] *= v_size
    p.data[:] = 0xFF
    oracle.kv_write_reference(p.data, slots, x[0], x[1], 64, fmt, ka, va)
    p.k[slots], p.v[slots] = oracle.kv_read_reference(p.data, slots, H, D, 64, fmt, ka, va)
    return p


@pytest.mark.parametrize("ka,va,k_size,v_size", [(1e-3, 1e-3, 100.0, 100.0), (1024.0, 1024.0, 0.01, 1e-4),
                                                 (4096.0, 2.0 ** 20, 1.0, 0.03), (2.0 ** -20, 2.0 ** -30, 1.0, 50.0)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("news,lens,group", [([1, 1], [70, 100], 4), ([70, 64], [100, 70], 8)])
def test_alphas_far_from_the_rows_size(ka, va, k_size, v_size, dtype, news, lens, group):
    p = _of_size(lens, news, k_size, v_size, ka, va, 1, dtype, group=group, seed=41)
    got = p.run()
    torch.cuda.synchronize()
    _check_sampled(p, got)


@pytest.mark.parametrize("fmt,dtype,ka,va", [(0, BF16, 0.02, 0.7), (0, FP16, 1.3, 0.01), (1, BF16, 0.3, 1.9),
                                             (1, FP16, 2.0, 0.5), (1, FP16, 0.003, 700.0)])
def test_alphas_of_prompts(fmt, dtype, ka, va):
    p = Problem([90, 120], [80, 64], fmt, dtype, 128, 2, 8, ka=ka, va=va, seed=42)
    got = p.run()
    torch.cuda.synchronize()
    _check_sampled(p, got)


@pytest.mark.parametrize("at", [66, 650])
def test_offsets_that_decrease_late_write_nothing(at):
    """The same in the tiled kernel where the decrease lies past the sequences
    that its search for a block looks at in one go."""
    B = 700
    p = Problem([40] * B, [1] * B, 0, BF16, 64, 1, 8, 64, seed=45)
    off = p.offsets.copy()
    off[at] = 10
    q = p.q.cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((B, 8), 7.0, device="cuda")
    F.attention(q, p.cache(), torch.from_numpy(p.table).cuda(), torch.tensor(p.lens, dtype=torch.int32, device="cuda"),
                q_offsets=torch.from_numpy(off).cuda(), max_q=64, out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.all(out == 7) and torch.all(lse == 7)


def test_prompts_of_many_sequences_in_shares():
    """More sequences than a wave's lanes, and few enough blocks that their
    keys are cut into shares."""
    news = [1] * 66
    news[5], news[65], news[40] = 64, 60, 0
    lens = [70] * 66
    lens[5], lens[65], lens[0] = 2000, 1300, 900
    p = Problem(lens, news, 0, BF16, 128, 1, 8, 64, seed=48)
    got = p.run(max_q=64)
    torch.cuda.synchronize()
    _check_sampled(p, got)
    size = F.attention_workspace_size(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
                                      torch.tensor(p.lens, dtype=torch.int32, device="cuda"),
                                      q_offsets=torch.from_numpy(p.offsets).cuda(), max_q=64)
    assert size > 0                                                  # partial sums: shares are used
    again = p.run(max_q=64, workspace=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("size", [-1e35, 1e35, -3e30, 1e12, -1e9, 1e8])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [1, 64])
def test_scores_far_from_zero(fmt, n, size):
    """Scores of any size, of BF16 queries: of keys whose scores are further
    apart than 2^20 the highest takes all, rounding included (v's own in the
    output: half a step), and the log-sum-exp is its score (eight roundings in FP32)."""
    p = Problem([40, 3], [n, n], fmt, BF16, 128, 1, 8, 64, seed=43)
    q = torch.zeros((2 * n, 8, 128), dtype=BF16)
    q[:, :, 5] = size
    for b in range(2):
        at = p.slots(b, np.arange(p.lens[b]))
        k = np.ones((p.lens[b], 1, 128), np.float32)
        k[:, :, 5] = 2.0 if size < 0 else 1.0
        k[1, :, 5] = 1.0 if size < 0 else 2.0
        oracle.kv_write_reference(p.data, at, k, p.v[at].astype(np.float32), 64, fmt)
        p.k[at], p.v[at] = oracle.kv_read_reference(p.data, at, 1, 128, 64, fmt)
    p.q = q
    out, lse = p.run(causal=False)
    for b in range(2):
        at = p.slots(b, np.array([1]))
        v = torch.from_numpy(p.v[at, 0]).cuda().double()[None]
        s = float(p.k[at, 0, 5][0]) * float(q[0, 0, 5].double()) * float(np.float32(p.scale))
        assert torch.all((out[b * n:b * n + n].double() - v).abs() <= 2.0 ** -8 * v.abs())
        assert torch.all((lse[b * n:b * n + n].double() - s).abs() <= 2.0 ** -21 * abs(s))


@pytest.mark.parametrize("max_q", [1, 64])
def test_sinks_of_the_lowest_values(max_q):
    """Sinks far below every score add nothing; where no key is seen the
    log-sum-exp is the sink itself, also at the type's lowest value."""
    p = Problem([0, 2, 50], [1, 4, 2], 0, BF16, 128, 1, 4, 64, seed=44)
    low = torch.finfo(torch.float32).min
    sinks = torch.tensor([low, -2e38, -1e31, -np.inf], device="cuda")
    plain = p.run(max_q=max_q)
    out, lse = p.run(max_q=max_q, sinks=sinks)
    empty = torch.isneginf(plain[1])
    assert torch.equal(out, plain[0]) and torch.equal(lse[~empty], plain[1][~empty])
    want = sinks.expand(lse.shape)[empty].double()
    got = lse[empty].double()
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    near = ~torch.isinf(want)
    assert torch.all((got[near] - want[near]).abs() <= 2.0 ** -22 * want[near].abs())


def test_a_page_table_that_sequences_share():
    p = Problem([100], [1], 0, BF16, seed=46)
    q = torch.cat([p.q] * 3).cuda()
    table = torch.from_numpy(p.table).cuda()
    n = torch.tensor([100, 64, 7], dtype=torch.int32, device="cuda")
    want = F.attention(q, p.cache(), table.repeat(3, 1), n, return_lse=True)
    got = F.attention(q, p.cache(), table.expand(3, -1), n, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("group", [100, 1024])
@pytest.mark.parametrize("news,lens", [([1, 1], [40, 300]), ([3, 1], [3, 150])])
def test_many_query_heads_a_kv_head(group, news, lens):
    """More query heads of a KV head than a row block holds."""
    p = Problem(lens, news, 0, FP16, 64, 1, group, seed=group)
    got = p.run()
    torch.cuda.synchronize()
    _check_sampled(p, got)


@pytest.mark.parametrize("fmt,dtype", PAIRS)
@pytest.mark.parametrize("D,group", [(64, 8), (128, 8), (256, 16)])
@pytest.mark.parametrize("news,lens", [([1, 2], [90, 700]), ([70, 50], [90, 600])])
def test_windows_and_sinks_of_every_kind(news, lens, D, group, fmt, dtype):
    """Window and sinks for each pair of types and head size, in both kernels."""
    p = Problem(lens, news, fmt, dtype, D, 2, group, 32, seed=D + group)
    s = _sinks(2 * group, 7)
    got = p.run(window=45, sinks=torch.from_numpy(s).cuda())
    torch.cuda.synchronize()
    _check_sampled(p, got, window=45, sinks=s)


@pytest.mark.parametrize("fmt,news", [(0, [1, 1]), (1, [70, 70])])
def test_pages_past_4_gib(fmt, news):
    """The same pages at the start of a small cache and at the end of a large
    one, and in the order reversed: the same bits."""
    H, D, page = 8, 256, 256
    p = Problem([600, 513], news, fmt, BF16, D, H, 2, page, seed=49)
    want = p.run()
    size = F.kv_cache_size(1, page, H, D, fmt)
    pages = (5 << 30) // size
    assert (pages - p.pages) * size > 1 << 32
    big = F.new_kv_cache(pages, page, H, D, fmt)
    last = pages - 1 - np.arange(p.pages)
    small = torch.from_numpy(p.data).cuda().reshape(p.pages, size)
    big.data.reshape(pages, size)[torch.from_numpy(last).cuda()] = small
    table = np.where(p.table >= 0, last[np.clip(p.table, 0, p.pages - 1)], -1).astype(np.int32)
    got = F.attention(p.q.cuda(), big, torch.from_numpy(table).cuda(),
                      torch.tensor(p.lens, dtype=torch.int32, device="cuda"), scale=p.scale, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_threads_at_once():
    """Calls from two host threads, each on a stream of its own."""
    import threading
    ps = [Problem([4000, 50], [1, 1], 0, BF16, seed=50), Problem([900, 700], [1, 1], 1, FP16, seed=51)]
    want = [p.run() for p in ps]
    args = [(p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda(),
             torch.tensor(p.lens, dtype=torch.int32, device="cuda")) for p in ps]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[i].append(F.attention(*args[i], scale=ps[i].scale, stream=s, return_lse=True))
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
        assert len(got[i]) == 20
        for o in got[i]:
            assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])


@pytest.mark.parametrize("news,lens", [([1, 1], [4000, 70]), ([70, 64], [1500, 300])])
def test_out_in_place_of_q(news, lens):
    """Every workgroup has read its query rows before any of them is written."""
    p = Problem(lens, news, 0, BF16, 128, 1, 8, seed=52)
    want = p.run()
    q = p.q.cuda()
    got = p.run(q=q, out=q)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(got[1], want[1])


def test_temporaries_of_calls_on_another_stream():
    """Inputs that the caller drops right after a call on a busy stream keep
    their memory until that stream has read them, and so do outputs dropped
    while the caller's stream still reads them."""
    p = Problem([300, 200], [1, 1], 0, BF16, seed=53)
    want = p.run()
    q, table = p.q.cuda(), torch.from_numpy(p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    slots = torch.from_numpy(p.slots(0, np.arange(300))).cuda()
    cache = p.cache()
    rows = F.kv_read(cache, slots)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        inputs = [q.clone(), table.clone(), lens.clone(), slots.clone()]
        sizes = [(t.shape, t.dtype) for t in inputs]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = F.attention(inputs[0], cache, inputs[1], inputs[2], scale=p.scale, stream=side, return_lse=True)
        back = F.kv_read(cache, inputs[3], stream=side)
        held = [t.data_ptr() for t in inputs]
        del inputs
        reused = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
        assert not set(held) & {t.data_ptr() for t in reused}
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*got, *back), (*want, *rows)):
            assert torch.equal(a, b)
        # the other way round: the caller's stream is late
        torch.cuda._sleep(20_000_000)
        copies = [t.clone() for t in got]
        held = [t.data_ptr() for t in got]
        shapes = [(t.shape, t.dtype) for t in got]
        del got, a, b
        with torch.cuda.stream(side):
            reused = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in shapes]
        assert not set(held) & {t.data_ptr() for t in reused}
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
        del copies, reused, back, a, b


def test_capture_that_forks_to_another_stream():
    """A captured step whose attention runs on a second stream, with
    temporaries of both; replayed over other queries, eager work in between."""
    p = Problem([2000, 300], [1, 1], 0, BF16, seed=54)
    q, cache, table = p.q.cuda(), p.cache(), torch.from_numpy(p.table).cuda()
    lens = torch.tensor(p.lens, dtype=torch.int32, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    F.attention(q, cache, table, lens, return_lse=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        got = F.attention(q * 1.0, cache, table + 0, lens, stream=side, return_lse=True)
        main.wait_stream(side)
        got = [t.clone() for t in got]
    for seed in range(4):
        q.copy_(torch.randn(q.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        want = F.attention(q, cache, table, lens, return_lse=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

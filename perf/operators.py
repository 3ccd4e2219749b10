"""Cases of the FP4 key/value-cache operators: writing the cache, reading it
back, and attention over it.

``run`` computes each case in elementary torch operations (FP32), or, where
``own`` is true, through ``mixed_precision_bf16_amd.fp4gemm``.  The cache bytes
that ``prepare`` makes are in the library's documented layout, so both take the
same inputs.  ``exact`` evaluates the definitions in float64.
"""

import math

import torch

own = False

_DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}
_GROUP = {"nvfp4": 16, "mxfp4": 32}
_FORMAT = {"nvfp4": 0, "mxfp4": 1}
_TILE = 32  # tokens of a layout tile


def _case(name, kind, **over):
    c = {"name": name, "kind": kind, "fmt": "nvfp4", "dtype": "bfloat16", "head_dim": 128, "q_heads": 64, "kv_heads": 8,
         "page": 64, "batch": 1, "shortest": 1, "longest": 1, "new_min": 1, "new": 1, "window": 0, "sinks": False,
         "k_alpha": 1.0, "v_alpha": 1.0}
    c.update(over)
    return c


def listed():
    return [
        # the keys and values of one sequence's next token (single-stream decode); a two-level NVFP4 scale
        _case("write_1_token", "write", longest=1, k_alpha=0.02, v_alpha=0.01),
        # a prompt chunk of odd length written into a cache with small heads
        _case("write_4095_mx_d64", "write", longest=4095, fmt="mxfp4", dtype="float16", head_dim=64),
        # a long prompt chunk of a 64/8-head layer of width 8192
        _case("write_8192", "write", longest=8192),
        # a short prefix read back (moving one sequence, checking a cache)
        _case("read_777_mx_d64", "read", longest=777, fmt="mxfp4", dtype="float16", head_dim=64),
        # a long context read back to BF16
        _case("read_65536", "read", longest=65536),
        # single-stream decode over a short context: latency
        _case("decode_b1_1000", "attend", shortest=1000, longest=1000),
        # a serving batch's decode step: append the new token of each sequence, then attend
        _case("step_b64_8192", "step", batch=64, shortest=16, longest=8192),
        # single-stream decode over a long context
        _case("decode_b1_131071_mx", "attend", shortest=131071, longest=131071, fmt="mxfp4"),
        # sliding-window layer with attention sinks, small heads
        _case("window128_b128_mx_d64", "attend", batch=128, shortest=100, longest=4000, window=128, sinks=True,
              fmt="mxfp4", head_dim=64, page=32),
        # four tokens a sequence (drafted tokens being checked)
        _case("draft4_b16", "attend", batch=16, shortest=1000, longest=5000, new_min=4, new=4, dtype="float16", page=32),
        # a prompt chunk over an earlier context
        _case("chunk2048_of_8192", "attend", shortest=8192, longest=8192, new_min=2048, new=2048),
        # several whole prompts of odd lengths, wide heads
        _case("prompts6_mx_d256", "attend", batch=6, shortest=0, longest=0, new_min=101, new=1999, fmt="mxfp4",
              head_dim=256, q_heads=16, kv_heads=4, page=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["write", "read", "attend", "attend", "attend", "step"])
    d = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    c = _case("", kind, fmt=rng.choice(["nvfp4", "mxfp4"]), dtype=rng.choice(["bfloat16", "float16"]), head_dim=d,
              kv_heads=kv, q_heads=kv * group, page=rng.choice([32, 64, 96, 128, 256]))
    del c["name"]
    if rng.random() < 0.3:
        c["k_alpha"], c["v_alpha"] = rng.choice([(0.02, 0.01), (0.5, 0.25), (1.7, 0.3)])
    if kind in ("write", "read"):
        c["longest"] = _log(rng, 1, 8192 * 1024 // (kv * d) if kind == "write" else 32768 * 1024 // (kv * d))
        c["longest"] = min(c["longest"], 60000)
        return c
    c["sinks"] = rng.random() < 0.25
    if kind == "attend" and rng.random() < 0.45:  # prompts and chunks
        c["batch"] = _log(rng, 1, 8)
        most = min(2048, int(math.sqrt(2.0 ** 38 / (c["batch"] * kv * group * d * 4))))
        c["new"] = _log(rng, 17, most)
        c["new_min"] = rng.randint(1, c["new"])
        extra = rng.choice([0, 0, _log(rng, 1, 4 * most)])
        c["shortest"], c["longest"] = (extra // 2, extra)  # at least the new tokens: see _lengths
    else:
        c["batch"] = _log(rng, 1, 96)
        c["longest"] = _log(rng, 2, max(2, min(100000, 2 ** 28 // (c["batch"] * kv * d))))
        c["shortest"] = rng.randint(1, c["longest"])
        if kind == "attend":
            c["new"] = c["new_min"] = rng.choice([1, 1, 2, 3, 8])
    if rng.random() < 0.25:
        c["window"] = _log(rng, 1, 4096)
    return c


def _spread(lo, hi, n, salt):
    """n sizes in [lo, hi], the last one hi: the same for every seed."""
    v = [lo + (i * 2654435761 + salt * 40503 + 12345) % (1 << 20) * (hi - lo + 1) // (1 << 20) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(c):
    """(new tokens, whole length) of each sequence."""
    news = _spread(c["new_min"], c["new"], c["batch"], 1)
    lens = _spread(min(c["shortest"], c["longest"]), c["longest"], c["batch"], 2)
    return news, [max(n, x) for n, x in zip(news, lens)]


def _cache_bytes(c):
    """Bytes of one token of one head, keys and values."""
    return 2 * (c["head_dim"] // 2 + c["head_dim"] // _GROUP[c["fmt"]])


def _visible(c):
    """(keys read, query-key pairs) over all sequences."""
    keys = pairs = 0
    for n, x in zip(*_lengths(c)):
        w = c["window"]
        keys += x if not w else min(x, w + n - 1)
        if not w:
            pairs += n * x - n * (n - 1) // 2
        else:
            pairs += sum(min(x - n + i + 1, w) for i in range(n))
    return keys, pairs


def work(c):
    row = c["kv_heads"] * c["head_dim"] * 2 * 2
    held = c["kv_heads"] * _cache_bytes(c)
    if c["kind"] == "write":
        return {"bytes": c["longest"] * (2 * row + 2 * held + 16), "flops": 0}
    if c["kind"] == "read":
        return {"bytes": c["longest"] * (row + held + 8), "flops": 0}
    keys, pairs = _visible(c)
    rows = sum(_lengths(c)[0])
    total = keys * held + rows * c["q_heads"] * (c["head_dim"] * 4 + 4) + c["batch"] * 8 + keys // c["page"] * 4
    if c["kind"] == "step":
        total += c["batch"] * (row + held + 8)
    return {"bytes": total, "flops": 4 * c["head_dim"] * c["q_heads"] * pairs}


# ------------------------------------------------------------------ the layout
def _places(c, slots):
    """Byte indices into the cache of the rows at `slots`: codes of K and V
    [n][heads][D/2], scales of K and V [n][heads][D/G]."""
    D, H, G = c["head_dim"], c["kv_heads"], _GROUP[c["fmt"]]
    dev = slots.device
    tile_bytes = 32 * D + 64 * D // G
    tok = slots % c["page"]
    page = slots // c["page"]
    h = torch.arange(H, device=dev)
    base = ((page[:, None] * H + h) * (c["page"] // _TILE) + (tok // _TILE)[:, None]) * tile_bytes
    t = (tok % _TILE)[:, None]
    u, r, j, i = t // 16, t % 16, t % 16 // 4, t % 4
    d = torch.arange(0, D, 2, device=dev)[None, :]
    g = torch.arange(D // G, device=dev)[None, :]
    if D == 64:
        kc = (d // 16 * 16 + r) * 16 + u * 8 + d % 16 // 2
        vc = (16 * j + d // 4) * 16 + u * 8 + i * 2 + d % 4 // 2
        ks = (g * 16 + r) * 2 + u
    else:
        C = D // 128
        kc = (d // 128 * 2 + u) * 1024 + (d % 128 // 32 * 16 + r) * 16 + d % 32 // 2
        vc = (d // 128 * 2 + u) * 1024 + (16 * j + d % 128 // 8) * 16 + i * 4 + d % 8 // 2
        per = 32 // G  # scales of a lane's 32 elements
        ks = (g % (4 * per) // per * 16 + r) * (2 * C * per) + g // (4 * per) * 2 * per + u * per + g % per
    vs = (g * 4 + j) * 8 + u * 4 + i
    at = [kc, 16 * D + vc, 32 * D + ks, 32 * D + 32 * D // G + vs]
    return [base[:, :, None] + x[:, None, :] for x in at]


def _quantize(x, fmt, alpha):
    """x [n][heads][D] FP32 -> (bytes of two codes [n][heads][D/2], scale bytes [n][heads][D/G])."""
    G = _GROUP[fmt]
    b = x.reshape(*x.shape[:-1], -1, G)
    alpha = torch.full((1,), alpha, dtype=torch.float32, device=x.device)
    amax = b.abs().amax(-1)
    if fmt == "nvfp4":
        t = amax / torch.full_like(alpha, 6.0) / alpha
        s = t.clamp(max=448.0).to(torch.float8_e4m3fn).view(torch.uint8).clamp(min=1)
        value = s.view(torch.float8_e4m3fn).float()
    else:
        field = ((amax / alpha).view(torch.int32) >> 23) & 255
        s = torch.where(field == 255, 254, (field - 2).clamp(min=0))
        value = torch.where(s == 0, 0x00400000, s << 23).to(torch.int32).view(torch.float32)
        s = s.to(torch.uint8)
    q = b.abs() / (alpha * value)[..., None]
    code = (q > 0.25).to(torch.uint8)
    for edge, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (q >= edge) if closed else (q > edge)
    code = (code | ((b < 0) & (code > 0)).to(torch.uint8) << 3).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _write(c, data, slots, k, v):
    kc, vc, ks, vs = _places(c, slots)
    for x, alpha, codes, scales in ((k, c["k_alpha"], kc, ks), (v, c["v_alpha"], vc, vs)):
        cb, sb = _quantize(x.float(), c["fmt"], alpha)
        data[codes] = cb
        data[scales] = sb


def _values(c, data, slots):
    """The FP32 values alpha * code * scale of the rows at `slots`: K and V [n][heads][D]."""
    D, G = c["head_dim"], _GROUP[c["fmt"]]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    kc, vc, ks, vs = _places(c, slots)
    out = []
    for codes, scales, alpha in ((kc, ks, c["k_alpha"]), (vc, vs, c["v_alpha"])):
        b = data[codes]
        x = grid[torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], D).int()]
        s = data[scales]
        if c["fmt"] == "nvfp4":
            s = s.view(torch.float8_e4m3fn).float()
        else:
            s = s.to(torch.int32)
            s = torch.where(s == 0, 0x00400000, s << 23).to(torch.int32).view(torch.float32)
        a = torch.full((1,), alpha, dtype=torch.float32, device=data.device)
        out.append((x.reshape(*s.shape, G) * s[..., None] * a).reshape(x.shape))
    return out


# ---------------------------------------------------------------------- inputs
def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    D, H, page = c["head_dim"], c["kv_heads"], c["page"]
    dtype = _DTYPES[c["dtype"]]
    attend = c["kind"] in ("attend", "step")
    news, lens = _lengths(c) if attend else ([c["longest"]], [c["longest"]])
    per = [-(-x // page) for x in lens]
    pages = sum(per) + 1
    order = torch.randperm(pages, generator=gen, device="cuda")
    columns = max(per)
    table = torch.zeros((len(lens), columns), dtype=torch.int32)  # the pages of each sequence, anywhere in the cache
    at, rows = 0, order.to(torch.int32).cpu()
    for b, n in enumerate(per):
        table[b, :n] = rows[at:at + n]
        at += n
    s = {"case": c, "pages": pages, "page_table": table.cuda(),
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    # keys with a few strong channels, as projections give them; every slot has held a token before
    strength = 1.0 + 2.0 * (torch.rand((2, H, D), generator=gen, device="cuda") < 0.04)
    group = _GROUP[c["fmt"]]
    s["cache"] = torch.zeros(pages * page * H * _cache_bytes(c), dtype=torch.uint8, device="cuda")
    if c["kind"] != "write":
        step = max(1, (1 << 25) // (H * D))
        for first in range(0, pages * page, step):
            slots = torch.arange(first, min(first + step, pages * page), device="cuda")
            kv = torch.randn((2, len(slots), H, D), generator=gen, device="cuda") * strength[:, None]
            _write(c, s["cache"], slots, (kv[0] * c["k_alpha"]).to(dtype), (kv[1] * c["v_alpha"]).to(dtype))
    if c["kind"] != "attend":
        pos = torch.cat([torch.arange(c["longest"])] if not attend else [torch.tensor([x - 1]) for x in lens])
        seq = torch.zeros(len(pos), dtype=torch.int64) if not attend else torch.arange(len(lens))
        s["slots"] = (table[seq, pos // page].long() * page + pos % page).cuda()
    if c["kind"] in ("write", "step"):
        # rows in hand: one projection's output [tokens][K heads | V heads][D], cut into K and V
        kv = torch.randn((len(pos), 2 * H, D), generator=gen, device="cuda")
        kv = (kv * strength.reshape(1, 2 * H, D)).reshape(len(pos), 2, H, D)
        kv = kv * torch.tensor([c["k_alpha"], c["v_alpha"]], device="cuda")[None, :, None, None]
        kv = kv.reshape(len(pos), 2 * H, D).to(dtype)
        s["k"], s["v"] = kv[:, :H], kv[:, H:]
    if attend:
        rows = sum(news)
        q = torch.randn((rows, c["q_heads"], D), generator=gen, device="cuda") * (1.5 / c["k_alpha"])
        s["q"] = q.to(dtype)
        ends = [0]
        for n in news:
            ends.append(ends[-1] + n)
        s["q_offsets"] = None if min(news) == max(news) else torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["max_q"], s["max_len"] = max(news), max(lens)
        s["scale"] = 1.0 / math.sqrt(D)
        s["sinks"] = torch.randn(c["q_heads"], generator=gen, device="cuda") if c["sinks"] else None
    return s


# ------------------------------------------------------------------ one pass
def _attend(c, s):
    D, H, G = c["head_dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    B, M, X = c["batch"], s["max_q"], s["max_len"]
    dev = s["q"].device
    lens = s["seq_lens"].long()[:, None]
    starts = torch.arange(B + 1, device=dev) * M if s["q_offsets"] is None else s["q_offsets"].long()
    count = (starts[1:] - starts[:-1])[:, None]
    i = torch.arange(M, device=dev)
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [B][M]
    j = torch.arange(X, device=dev)
    slot = s["page_table"].long()[:, j // c["page"]] * c["page"] + j % c["page"]  # [B][X]
    k, v = _values(c, s["cache"], slot.reshape(-1))
    k = k.reshape(B, X, H, D).permute(0, 2, 3, 1).contiguous()
    v = v.reshape(B, X, H, D).permute(0, 2, 1, 3).contiguous()
    q = s["q"][row].float().reshape(B, M, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, M * G, D)
    pos = lens - count + i                                                   # [B][M]
    seen = (j <= pos[..., None]) & (j < lens[..., None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    score = torch.matmul(q, k).mul_(s["scale"]).reshape(B, H, M, G, X)
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1)
    if s["sinks"] is not None:
        sink = s["sinks"].reshape(1, H, 1, G)
        top = torch.maximum(top, sink)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top[..., None]).exp_()
    total = p.sum(-1)
    if s["sinks"] is not None:
        total = total + (sink - top).exp()
    out = torch.matmul(p.reshape(B, H, M * G, X), v).reshape(B, H, M, G, D)
    out = out / torch.where(total == 0, 1.0, total)[..., None]
    lse = top + total.log()
    where = (i < count).reshape(-1).nonzero()[:, 0] if s["q_offsets"] is not None else slice(None)
    out = out.permute(0, 2, 1, 3, 4).reshape(B * M, H * G, D)[where]
    lse = lse.permute(0, 2, 1, 3).reshape(B * M, H * G)[where]
    return out.to(s["q"].dtype), lse


def run(s):
    c = s["case"]
    if own:
        from mixed_precision_bf16_amd import fp4gemm as F
        cache = F.KVCache(s["cache"], s["pages"], c["page"], c["kv_heads"], c["head_dim"], _FORMAT[c["fmt"]],
                          c["k_alpha"], c["v_alpha"])
        if c["kind"] in ("write", "step"):
            F.kv_append(cache, s["k"], s["v"], s["slots"])
        if c["kind"] in ("write", "read"):
            return F.kv_read(cache, s["slots"], dtype=_DTYPES[c["dtype"]])
        return F.attention(s["q"], cache, s["page_table"], s["seq_lens"], q_offsets=s["q_offsets"], max_q=s["max_q"],
                           scale=s["scale"], window=c["window"], sinks=s["sinks"], return_lse=True)
    if c["kind"] in ("write", "step"):
        _write(c, s["cache"], s["slots"], s["k"], s["v"])
    if c["kind"] in ("write", "read"):
        k, v = _values(c, s["cache"], s["slots"])
        return k.to(_DTYPES[c["dtype"]]), v.to(_DTYPES[c["dtype"]])
    return _attend(c, s)


# --------------------------------------------------------------- the definition
def _opened(c, data):
    """The whole cache in float64, K and V [slots][heads][D], by taking the
    bytes apart as a nested array."""
    D, H, G = c["head_dim"], c["kv_heads"], _GROUP[c["fmt"]]
    tiles = c["page"] // _TILE
    x = data.reshape(-1, H, tiles, 32 * D + 64 * D // G)
    P = x.shape[0]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=data.device)
    grid = torch.cat((grid, -grid))
    if c["fmt"] == "nvfp4":
        byte = torch.arange(256, device=data.device)
        m, e = (byte & 7).double(), (byte >> 3) & 15
        level = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    else:
        level = torch.exp2(torch.arange(256, device=data.device).double() - 127)

    def nibbles(y):
        return grid[torch.stack((y & 15, y >> 4), -1).flatten(-2).int()]

    kc, vc, ks, vs = x.split([16 * D, 16 * D, 32 * D // G, 32 * D // G], -1)
    n = D // G
    if D == 64:
        k = nibbles(kc.reshape(P, H, tiles, 4, 16, 2, 8)).permute(0, 2, 5, 4, 1, 3, 6)      # j r u d -> u r | j d
        v = nibbles(vc.reshape(P, H, tiles, 4, 16, 2, 4, 2)).permute(0, 2, 5, 3, 6, 1, 4, 7)  # j rv u i d -> u j i | rv d
        ks = level[ks.reshape(P, H, tiles, n, 16, 2).int()].permute(0, 2, 5, 4, 1, 3)
    else:
        C, per = D // 128, 32 // G
        k = nibbles(kc.reshape(P, H, tiles, C, 2, 4, 16, 16)).permute(0, 2, 4, 6, 1, 3, 5, 7)
        v = nibbles(vc.reshape(P, H, tiles, C, 2, 4, 16, 4, 4)).permute(0, 2, 4, 5, 7, 1, 3, 6, 8)
        ks = level[ks.reshape(P, H, tiles, 4, 16, C, 2, per).int()].permute(0, 2, 6, 4, 1, 5, 3, 7)
    vs = level[vs.reshape(P, H, tiles, n, 4, 2, 4).int()].permute(0, 2, 5, 4, 6, 1, 3)
    S = P * c["page"]
    a, b = (float(torch.tensor(c[w], dtype=torch.float32)) for w in ("k_alpha", "v_alpha"))
    k = k.reshape(S, H, n, G) * ks.reshape(S, H, n, 1) * a
    v = v.reshape(S, H, n, G) * vs.reshape(S, H, n, 1) * b
    return k.reshape(S, H, D), v.reshape(S, H, D)


def _rounded(x, fmt, alpha):
    """x [..., D] -> the values alpha * code * scale that the cache then holds,
    float64.  The definition takes its decisions on FP32 quotients: a quotient
    of FP32 numbers formed in float64 and rounded to FP32 is the correctly
    rounded one."""
    f32 = lambda y: y.float().double()  # noqa: E731
    G = _GROUP[fmt]
    b = x.double().reshape(*x.shape[:-1], -1, G)
    a = float(torch.tensor(alpha, dtype=torch.float32))
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        byte = torch.arange(1, 127, device=x.device)
        m, e = (byte & 7).double(), byte >> 3
        levels = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
        t = f32(f32(top / 6) / a)
        mid = (levels[1:] + levels[:-1]) / 2  # midpoint above levels[i]; byte i + 1: a tie goes to the even byte
        low, high = torch.bucketize(t, mid), torch.bucketize(t, mid, right=True)
        at = torch.where(low == high, low, torch.where((low + 1) % 2 == 0, low, high))
        scale = levels[at]
    else:
        t = f32(top / a)
        scale = torch.exp2((torch.frexp(t)[1] - 1 - 2).clamp(min=-127).double())
        scale = torch.where(t == 0, 2.0 ** -127, scale)
    S = f32(a * scale)[..., None]
    q = f32(b.abs() / S)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.bucketize(q, mid), torch.bucketize(q, mid, right=True)
    at = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return (grid[at] * torch.sign(b) * scale[..., None] * a).reshape(x.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "write":
        return _rounded(s["k"], c["fmt"], c["k_alpha"]), _rounded(s["v"], c["fmt"], c["v_alpha"])
    k, v = _opened(c, s["cache"])
    if c["kind"] == "read":
        return k[s["slots"]], v[s["slots"]]
    if c["kind"] == "step":
        k[s["slots"]] = _rounded(s["k"], c["fmt"], c["k_alpha"])
        v[s["slots"]] = _rounded(s["v"], c["fmt"], c["v_alpha"])
    G = c["q_heads"] // c["kv_heads"]
    news, lens = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, x) in enumerate(zip(news, lens)):
        j = torch.arange(x, device="cuda")
        at = s["page_table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
        for h in range(c["kv_heads"]):
            kk, vv = k[at, h], v[at, h]
            for i in range(0, n, 256):
                m = min(256, n - i)
                q = s["q"][first + i:first + i + m, h * G:(h + 1) * G].double()
                z = (q.reshape(m * G, -1) @ kk.T).reshape(m, G, x) * s["scale"]
                pos = (x - n + i + torch.arange(m, device="cuda"))[:, None]
                hide = j > pos
                if c["window"]:
                    hide |= j <= pos - c["window"]
                z = z.masked_fill(hide[:, None], -math.inf)
                if s["sinks"] is not None:
                    more = s["sinks"][h * G:(h + 1) * G].double().reshape(1, G, 1).expand(m, G, 1)
                    z = torch.cat((z, more), -1)
                t = torch.logsumexp(z, -1)
                w = torch.exp(z - t[..., None])[..., :x]
                out[first + i:first + i + m, h * G:(h + 1) * G] = (w.reshape(m * G, x) @ vv).reshape(m, G, -1)
                lse[first + i:first + i + m, h * G:(h + 1) * G] = t
        first += n
    return out, lse

"""Cases of the operators around the FP4 products of a decoder layer: the
root-mean-square norm with the residual's addition and 8-bit output, rotary
positions (alone, and with the write into the FP4 key/value cache), and the
products of 8-bit activations with FP4 weights (plain, and gated).

``run`` computes each case in elementary torch operations (FP32; angles and sums
of squares in FP64), or, where ``own`` is true, through
``mixed_precision_bf16_amd.fp4gemm``.  Weights and caches that ``prepare`` makes
are in the library's documented layouts, so both take the same inputs.
``exact`` evaluates the definitions in float64.

8-bit activations (MX8): E4M3 codes [rows][Kp] and one E8M0 scale for each 32 of
them [rows][Kp / 32], Kp = K rounded up to 128, zeros behind K.
"""

import math

import torch

own = False

_DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}
_GROUP = {"nvfp4": 16, "mxfp4": 32}
_FORMAT = {"nvfp4": 0, "mxfp4": 1}
_EPS = 1e-5


def _norm(name, rows, width, **over):
    return {"name": name, "kind": "norm", "rows": rows, "width": width, "dtype": "bfloat16", "residual": True,
            "mx8": True, **over}


def _rope(name, tokens, **over):
    return {"name": name, "kind": "rope", "tokens": tokens, "first": 0, "cache": True, "fmt": "nvfp4",
            "dtype": "bfloat16", "head_dim": 128, "q_heads": 64, "kv_heads": 8, "rotary": 128, "interleaved": False,
            "stretch": 1.0, "page": 64, "k_alpha": 1.0, "v_alpha": 1.0, **over}


def _product(name, m, N, K, **over):
    return {"name": name, "kind": "product", "m": m, "N": N, "K": K, "gate": "", "out": "bfloat16", "alpha": 1.0,
            **over}


def listed():
    return [
        # the residual and norm before a product, single-stream decode: latency
        _norm("norm_1x8192_mx8", 1, 8192),
        # the same for a prompt chunk
        _norm("norm_4095x8192_mx8", 4095, 8192),
        # a narrow model's norm without a residual, kept in 16 bits
        _norm("norm_777x2880_f16", 777, 2880, dtype="float16", residual=False, mx8=False),
        # the next token of one sequence, far into its context: rotated, its key and value written
        _rope("rope_append_1_far", 1, first=131071, k_alpha=0.02, v_alpha=0.01),
        # a prompt chunk of a 64/8-head layer
        _rope("rope_append_8191", 8191, first=4096),
        # queries and keys alone: neighbouring pairs, half of the head, stretched for a long context
        _rope("rope_1001_pairs_part", 1001, cache=False, dtype="float16", q_heads=32, kv_heads=4, rotary=64,
              interleaved=True, stretch=4.0, first=20000),
        # one token, odd sizes
        _product("product_1x5000x2880_f16", 1, 5000, 2880, out="float16", alpha=0.02),
        # a decode batch's query/key/value projection
        _product("product_16x10240x8192", 16, 10240, 8192),
        # a decode batch's gated projection, its output in 8 bits for the next product
        _product("gated_16x57344x8192_mx8", 16, 57344, 8192, gate="silu", out="mx8"),
        # a short prompt's down projection
        _product("product_256x8192x28672", 256, 8192, 28672),
        # a prompt chunk's gated projection
        _product("gated_2048x57344x8192", 2048, 57344, 8192, gate="silu"),
        # norm, gated projection and down projection of a batch, as they follow each other
        {"name": "feed_forward_61x8192x28672", "kind": "feed_forward", "rows": 61, "width": 8192, "inner": 28672,
         "dtype": "bfloat16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "rope", "product", "product", "feed_forward"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if kind == "norm":
        mx8 = rng.random() < 0.6
        step = 32 if mx8 else 8
        width = step * _log(rng, 128 // step, 16384 // step)
        c = _norm("", _log(rng, 1, min(32768, 4095 * 8192 // width)), width, dtype=dtype, mx8=mx8,
                  residual=rng.random() < 0.6)
    elif kind == "rope":
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8])
        c = _rope("", 1, dtype=dtype, head_dim=dim, q_heads=heads, kv_heads=kv, fmt=rng.choice(["nvfp4", "mxfp4"]),
                  rotary=rng.choice([dim, dim, dim // 2, dim // 4, dim * 3 // 4]), interleaved=rng.random() < 0.4,
                  stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), page=rng.choice([32, 64, 96, 256]),
                  cache=rng.random() < 0.6, first=_log(rng, 1, 500000))
        c["tokens"] = _log(rng, 1, min(30000, 8191 * 80 * 128 // ((heads + 2 * kv) * dim)))
        if rng.random() < 0.3:
            c["k_alpha"], c["v_alpha"] = rng.choice([(0.02, 0.01), (0.5, 0.25), (1.7, 0.3)])
    elif kind == "product":
        gate = rng.choice(["", "", "silu", "gelu"])
        m = _log(rng, 1, 2048)
        K = 32 * _log(rng, 4, 896)
        most = min(57344, 2 ** 41 // (2 * m * K), 57344 * 8192 // K)
        N = _log(rng, 64, max(64, most))
        out = rng.choice(["bfloat16", "float16", "mx8"])
        if out == "mx8":
            N = (N + 31) // 32 * 32
        if gate:
            N = (N + 63) // 64 * 64
        c = _product("", m, N, K, gate=gate, out=out, alpha=rng.choice([1.0, 1.0, 0.02]))
    else:
        width = 32 * _log(rng, 16, 256)
        inner = 32 * _log(rng, 16, min(896, 28672 * 8192 // (32 * width)))
        c = {"kind": kind, "rows": _log(rng, 1, 512), "width": width, "inner": inner, "dtype": dtype}
    c.pop("name", None)
    return c


def _up(n, step):
    return (n + step - 1) // step * step


def _weight_bytes(N, K):
    return N * K // 2 + N * K // 32


def work(c):
    if c["kind"] == "norm":
        elem = c["rows"] * c["width"]
        out = elem + elem // 32 if c["mx8"] else 2 * elem
        return {"bytes": 2 * elem + c["width"] * 2 + (4 * elem if c["residual"] else 0) + out, "flops": 4 * elem}
    if c["kind"] == "rope":
        q, kv = c["q_heads"] * c["head_dim"], c["kv_heads"] * c["head_dim"]
        if not c["cache"]:
            return {"bytes": c["tokens"] * (4 * (q + kv) + 8), "flops": c["tokens"] * 3 * (q + kv)}
        held = 2 * c["kv_heads"] * (c["head_dim"] // 2 + c["head_dim"] // _GROUP[c["fmt"]])
        # rotated and written; then the keys and values held are read back
        return {"bytes": c["tokens"] * (4 * q + 4 * kv + held + 16 + held + 4 * kv),
                "flops": c["tokens"] * 3 * (q + kv)}
    if c["kind"] == "product":
        m, N, K = c["m"], c["N"], c["K"]
        cols = N // 2 if c["gate"] else N
        out = m * cols + m * cols // 32 if c["out"] == "mx8" else 2 * m * cols
        return {"bytes": _weight_bytes(N, K) + m * K + m * K // 32 + out, "flops": 2 * m * N * K}
    m, D, F = c["rows"], c["width"], c["inner"]
    return {"bytes": _weight_bytes(2 * F, D) + _weight_bytes(D, F) + 6 * m * D + 2 * D + 2 * m * D,
            "flops": 2 * m * 3 * F * D}


# ------------------------------------------------------- FP4 weights (native layout)
def _e2m1(q):
    """Codes of the nearest E2M1 values to q (FP32), ties to the even code."""
    a = q.abs()
    code = (a > 0.25).to(torch.uint8)
    for edge, closed in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if closed else (a > edge)
    return code | ((q < 0) & (code > 0)).to(torch.uint8) << 3


def _weights(N, K, gen):
    """Gaussian weights in MXFP4, laid out once as fp4_native_repack does: code
    block (tile t of 16 rows, chunk c of 128 k), 16-byte slot 16 j + r = bytes
    64 c + 16 j .. + 15 of row 16 t + r; scale block (t, 512 k), dword 16 j + r,
    byte s = scale of block 16 q + 4 s + j."""
    Np, Kp = _up(N, 16), _up(K, 512)
    codes = torch.zeros((Np, Kp // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((Np, Kp // 32), dtype=torch.uint8, device="cuda")
    step = max(16, (1 << 26) // K)
    for n in range(0, N, step):
        w = torch.randn((min(step, N - n), K // 32, 32), generator=gen, device="cuda") * (K ** -0.5)
        e = torch.frexp(w.abs().amax(-1))[1] - 1 - 2
        c = _e2m1(torch.ldexp(w, -e[..., None])).reshape(-1, K)
        codes[n:n + len(w), :K // 2] = c[:, 0::2] | c[:, 1::2] << 4
        scales[n:n + len(w), :K // 32] = (e + 127).to(torch.uint8)
    codes = codes.reshape(Np // 16, 16, Kp // 128, 4, 16).permute(0, 2, 3, 1, 4).contiguous()
    scales = scales.reshape(Np // 16, 16, Kp // 512, 4, 4).permute(0, 2, 4, 1, 3).contiguous()
    return codes.reshape(-1), scales.reshape(-1)


def _weight_values(wq, sq, N, K):
    """The FP32 weights [N][K]."""
    Np, Kp = _up(N, 16), _up(K, 512)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=wq.device)
    pairs = torch.stack((grid.repeat(16), grid.repeat_interleave(16)), -1)  # of each byte
    b = wq.reshape(Np // 16, Kp // 128, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(Np, Kp // 2)[:N, :K // 2]
    s = sq.reshape(Np // 16, Kp // 512, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(Np, Kp // 32)[:N, :K // 32]
    s = (s.int() << 23).view(torch.float32)
    return (pairs[b.int()].reshape(N, K // 32, 32) * s[..., None]).reshape(N, K)


# ------------------------------------------------------------ 8-bit activations
def _power(e):
    """2^e, e a tensor of integers in -127 .. 127, in FP32."""
    return torch.where(e > -127, (e + 127) << 23, 0x00400000).to(torch.int32).view(torch.float32)


def _mx8(x):
    """FP32 [m][K] -> E4M3 codes [m][Kp], E8M0 scales [m][Kp / 32]: the scale of 32
    elements is the least power of two that brings their maximum to 448 or below."""
    m, K = x.shape
    b = torch.zeros((m, _up(K, 128)), dtype=torch.float32, device=x.device)
    b[:, :K] = x
    b = b.reshape(m, -1, 32)
    part, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(part == 0, -127, (e - 9 + (part > 0.875).int()).clamp(-127, 127)).int()
    codes = (b * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(m, -1), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _mx8_values(codes, scales, K):
    s = _power(scales.view(torch.uint8).int() - 127)
    return (codes.float().reshape(len(codes), -1, 32) * s[..., None]).reshape(len(codes), -1)[:, :K]


# -------------------------------------------------------------- the cache's layout
def _places(c, slots):
    """Byte indices into the cache of the rows at `slots`: codes of K and V
    [n][heads][D/2], scales of K and V [n][heads][D/G]."""
    D, H, G = c["head_dim"], c["kv_heads"], _GROUP[c["fmt"]]
    dev = slots.device
    tile_bytes = 32 * D + 64 * D // G
    tok = slots % c["page"]
    h = torch.arange(H, device=dev)
    base = (((slots // c["page"])[:, None] * H + h) * (c["page"] // 32) + (tok // 32)[:, None]) * tile_bytes
    t = (tok % 32)[:, None]
    u, r, j, i = t // 16, t % 16, t % 16 // 4, t % 4
    d = torch.arange(0, D, 2, device=dev)[None, :]
    g = torch.arange(D // G, device=dev)[None, :]
    if D == 64:
        kc = (d // 16 * 16 + r) * 16 + u * 8 + d % 16 // 2
        vc = (16 * j + d // 4) * 16 + u * 8 + i * 2 + d % 4 // 2
        ks = (g * 16 + r) * 2 + u
    else:
        C, per = D // 128, 32 // G
        kc = (d // 128 * 2 + u) * 1024 + (d % 128 // 32 * 16 + r) * 16 + d % 32 // 2
        vc = (d // 128 * 2 + u) * 1024 + (16 * j + d % 128 // 8) * 16 + i * 4 + d % 8 // 2
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
        e = torch.where(field == 255, 254, (field - 2).clamp(min=0)) - 127
        value, s = _power(e), (e + 127).to(torch.uint8)
    code = _e2m1(b / (alpha * value)[..., None]).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _write(c, data, slots, k, v):
    kc, vc, ks, vs = _places(c, slots)
    for x, alpha, codes, scales in ((k, c["k_alpha"], kc, ks), (v, c["v_alpha"], vc, vs)):
        cb, sb = _quantize(x.float(), c["fmt"], alpha)
        data[codes] = cb
        data[scales] = sb


def _held(c, data, slots):
    """The values alpha * code * scale of the rows at `slots`: K and V [n][heads][D]."""
    D, G = c["head_dim"], _GROUP[c["fmt"]]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    kc, vc, ks, vs = _places(c, slots)
    out = []
    for codes, scales, alpha in ((kc, ks, c["k_alpha"]), (vc, vs, c["v_alpha"])):
        b = data[codes]
        x = grid[torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], D).int()]
        s = data[scales]
        s = s.view(torch.float8_e4m3fn).float() if c["fmt"] == "nvfp4" else _power(s.int() - 127)
        a = torch.full((1,), alpha, dtype=torch.float32, device=data.device)
        out.append((x.reshape(*s.shape, G) * s[..., None] * a).reshape(x.shape).to(_DTYPES[c["dtype"]]))
    return out


# ---------------------------------------------------------------------- inputs
def _activations(shape, gen, strong=0.01):
    """Rows with a few strong channels, as the layers of a model give them."""
    channel = 1.0 + 9.0 * (torch.rand(shape[-1:], generator=gen, device="cuda") < strong)
    return torch.randn(shape, generator=gen, device="cuda") * channel


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["kind"] in ("norm", "feed_forward"):
        dtype, shape = _DTYPES[c["dtype"]], (c["rows"], c["width"])
        s["x"] = (0.3 * _activations(shape, gen)).to(dtype)
        s["weight"] = (1.0 + 0.2 * torch.randn(c["width"], generator=gen, device="cuda")).to(dtype)
        s["residual"] = _activations(shape, gen).to(dtype) if c.get("residual", True) else None
        if c["kind"] == "feed_forward":
            s["up"] = _weights(2 * c["inner"], c["width"], gen)
            s["down"] = _weights(c["width"], c["inner"], gen)
    elif c["kind"] == "product":
        s["codes"], s["scales"] = _mx8(_activations((c["m"], c["K"]), gen))
        s["weights"] = _weights(c["N"], c["K"], gen)
    else:
        T, D, H, dtype = c["tokens"], c["head_dim"], c["kv_heads"], _DTYPES[c["dtype"]]
        # rows in hand: one projection's output [tokens][Q heads | K heads | V heads][D]
        x = _activations((T, c["q_heads"] + 2 * H, D), gen, 0.04)
        x[:, -2 * H:-H] *= c["k_alpha"]
        x[:, -H:] *= c["v_alpha"]
        x = x.to(dtype)
        s["q"], s["k"], s["v"] = x.split([c["q_heads"], H, H], 1)
        s["qk"] = x[:, :c["q_heads"] + H]
        s["positions"] = c["first"] + torch.arange(T, device="cuda")
        pair = torch.arange(c["rotary"] // 2, device="cuda").double() * 2 / c["rotary"]
        s["frequencies"] = (500000.0 ** -pair / c["stretch"]).float()
        s["amplitude"] = 1.0 + 0.1 * math.log(c["stretch"])
        pages = -(-T // c["page"]) + 1
        table = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(T, device="cuda")
        s["slots"] = table[at // c["page"]] * c["page"] + at % c["page"]
        s["pages"] = pages
        held = 2 * (D // 2 + D // _GROUP[c["fmt"]])
        s["cache"] = torch.zeros(pages * c["page"] * H * held if c["cache"] else 0, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def _normed(s):
    """(the norm's FP32 output, the sum with the residual in FP32)."""
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    root = (1.0 / (h.double().square().mean(-1, keepdim=True) + _EPS).sqrt()).float()
    return h * root * s["weight"].float(), h


def _gated(y, kind):
    g, u = y.chunk(2, -1)
    if kind == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u


def _rotated(x, c, s):
    angle = s["positions"].double()[:, None] * s["frequencies"].double()
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    y, R = x.float().clone(), c["rotary"]
    at = (slice(0, R, 2), slice(1, R, 2)) if c["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    a, b = (x[..., i].float() for i in at)
    y[..., at[0]] = a * cos - b * sin
    y[..., at[1]] = b * cos + a * sin
    return y.to(x.dtype)


def run(s):
    c = s["case"]
    if own:
        from mixed_precision_bf16_amd import fp4gemm as F
        if c["kind"] == "norm":
            got = F.rms_norm(s["x"], s["weight"], _EPS, residual=s["residual"], mx8=c["mx8"])
            y, h = got if c["residual"] else (got, None)
            if not c["mx8"]:
                return y, h
            return y.codes[:, :c["width"]], y.scales[:, :c["width"] // 32], h
        if c["kind"] == "rope" and not c["cache"]:
            return F.rope(s["qk"], s["positions"], s["frequencies"], interleaved=c["interleaved"],
                          amplitude=s["amplitude"])
        if c["kind"] == "rope":
            cache = F.KVCache(s["cache"], s["pages"], c["page"], c["kv_heads"], c["head_dim"], _FORMAT[c["fmt"]],
                              c["k_alpha"], c["v_alpha"])
            q = F.kv_append_rope(cache, s["q"], s["k"], s["v"], s["slots"], s["positions"], s["frequencies"],
                                 interleaved=c["interleaved"], amplitude=s["amplitude"])
            return (q, *F.kv_read(cache, s["slots"], dtype=_DTYPES[c["dtype"]]))
        if c["kind"] == "product":
            mx8 = c["out"] == "mx8"
            y = F.gemm_mx8(F.MX8(s["codes"], s["scales"], c["K"]), *s["weights"], c["N"], gate=c["gate"] or None,
                           alpha=c["alpha"], mx8=mx8, dtype=None if mx8 else _DTYPES[c["out"]])
            cols = c["N"] // 2 if c["gate"] else c["N"]
            return (y.codes[:, :cols], y.scales[:, :cols // 32]) if mx8 else y
        a, h = F.rms_norm(s["x"], s["weight"], _EPS, residual=s["residual"], mx8=True)
        a = F.gemm_mx8(a, *s["up"], 2 * c["inner"], gate="silu", mx8=True)
        return F.gemm_mx8(a, *s["down"], c["width"], dtype=_DTYPES[c["dtype"]]), h
    if c["kind"] == "norm":
        y, h = _normed(s)
        h = h.to(s["x"].dtype) if c["residual"] else None
        if not c["mx8"]:
            return y.to(s["x"].dtype), h
        codes, scales = _mx8(y)
        return codes[:, :c["width"]], scales[:, :c["width"] // 32], h
    if c["kind"] == "rope" and not c["cache"]:
        return _rotated(s["qk"], c, s)
    if c["kind"] == "rope":
        _write(c, s["cache"], s["slots"], _rotated(s["k"], c, s), s["v"])
        return (_rotated(s["q"], c, s), *_held(c, s["cache"], s["slots"]))
    if c["kind"] == "product":
        y = _mx8_values(s["codes"], s["scales"], c["K"]) @ _weight_values(*s["weights"], c["N"], c["K"]).T
        y = y * c["alpha"]
        if c["gate"]:
            y = _gated(y, c["gate"])
        if c["out"] != "mx8":
            return y.to(_DTYPES[c["out"]])
        codes, scales = _mx8(y)
        return codes[:, :y.shape[1]], scales[:, :y.shape[1] // 32]
    y, h = _normed(s)
    D, inner = c["width"], c["inner"]
    y = _gated(_mx8_values(*_mx8(y), D) @ _weight_values(*s["up"], 2 * inner, D).T, "silu")
    y = _mx8_values(*_mx8(y), inner) @ _weight_values(*s["down"], D, inner).T
    return y.to(s["x"].dtype), h.to(s["x"].dtype)


# --------------------------------------------------------------- the definition
def _exact_weights(wq, sq, N, K):
    """The weights [N][K] in float64: each taken from its byte's address."""
    KB = _up(K, 512) // 128
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=wq.device)
    level = torch.cat((level, -level))
    k = torch.arange(K, device=wq.device)
    w = torch.empty((N, K), dtype=torch.float64, device=wq.device)
    step = max(1, (1 << 26) // K)
    for first in range(0, N, step):
        n = torch.arange(first, min(first + step, N), device=wq.device)[:, None]
        lane = 16 * (k % 128 // 32) + n % 16
        byte = wq[((n // 16 * KB + k // 128) * 64 + lane) * 16 + k % 32 // 2].int()
        code = torch.where(k % 2 == 0, byte & 15, byte >> 4)
        power = sq[((n // 16 * (KB // 4) + k // 512) * 64 + lane) * 4 + k % 512 // 128].double() - 127
        w[first:first + step] = level[code] * torch.exp2(power)
    return w


def _block_scale(y):
    """The powers of two of a row's blocks of 32, float64 [m][K / 32]."""
    top = y.abs().reshape(len(y), -1, 32).amax(-1)
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)  # log2 next to a power of two
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(-127, 127))


def _exact_mx8(y):
    """What the 8 bits stand for before their rounding: (codes, scales)."""
    s = _block_scale(y)
    return y / s.repeat_interleave(32, -1), s


def _exact_held(y):
    """The values that 8 bits then hold: E4M3 is 2^e / 8 apart in [2^e, 2^(e + 1)), 2^-9 below 2^-6."""
    z, s = _exact_mx8(y)
    step = torch.exp2((torch.frexp(z)[1] - 1).clamp(min=-6).double() - 3)
    return torch.round(z / step) * step * s.repeat_interleave(32, -1)


def _exact_gate(y, kind):
    F = y.shape[1] // 2
    g, u = y[:, :F], y[:, F:]
    if kind == "silu":
        return g * torch.sigmoid(g) * u
    return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)) * u


def _exact_norm(s):
    h = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0.0)
    return h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[1] + _EPS) * s["weight"].double(), h


def _exact_rope(x, c, s, held=False):
    """The rotation as a product of complex numbers; `held`: as the row that the
    cache's rule takes, every product and sum rounded to FP32, then to the type."""
    R = c["rotary"]
    angle = s["positions"].double()[:, None, None] * s["frequencies"].double()
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)
    y = x[..., :R].double()
    y = y.unflatten(-1, (R // 2, 2)) if c["interleaved"] else y.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    if held:
        f32 = lambda z: z.float().double()  # noqa: E731
        re, im = f32(turn.real), f32(turn.imag)
        a, b = y[..., 0], y[..., 1]
        y = torch.stack((f32(f32(a * re) - f32(b * im)), f32(f32(b * re) + f32(a * im))), -1)
    else:
        y = torch.view_as_real(torch.view_as_complex(y.contiguous()) * turn)
    y = y.flatten(-2) if c["interleaved"] else y.transpose(-1, -2).flatten(-2)
    y = torch.cat((y, x[..., R:].double()), -1)
    return y.float().to(x.dtype) if held else y


def _exact_cached(x, fmt, alpha):
    """x [..., D] -> the values alpha * code * scale that the cache then holds,
    float64.  The definition takes its decisions on FP32 quotients: a quotient
    of FP32 numbers formed in float64 and rounded to FP32 is the correctly
    rounded one."""
    f32 = lambda y: y.float().double()  # noqa: E731
    b = x.double().reshape(*x.shape[:-1], -1, _GROUP[fmt])
    a = float(torch.tensor(alpha, dtype=torch.float32))
    top = b.abs().amax(-1)

    def nearest(t, levels):  # ties to the even index
        mid = (levels[1:] + levels[:-1]) / 2
        low, high = torch.bucketize(t, mid), torch.bucketize(t, mid, right=True)
        return levels[torch.where(low == high, low, torch.where(low % 2 == 0, low, high))]

    if fmt == "nvfp4":
        byte = torch.arange(0, 127, device=x.device)
        m, e = (byte & 7).double(), byte >> 3
        levels = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
        scale = nearest(f32(f32(top / 6) / a), levels).clamp(min=2.0 ** -9)
    else:
        t = f32(top / a)
        scale = torch.exp2((torch.frexp(t)[1] - 1 - 2).clamp(min=-127).double())
        scale = torch.where(t == 0, 2.0 ** -127, scale)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    q = nearest(f32(b.abs() / f32(a * scale)[..., None]), grid)
    return (q * torch.sign(b) * scale[..., None] * a).reshape(x.shape)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "norm":
        y, h = _exact_norm(s)
        h = h if c["residual"] else None
        return (*_exact_mx8(y), h) if c["mx8"] else (y, h)
    if c["kind"] == "rope":
        if not c["cache"]:
            return _exact_rope(s["qk"], c, s)
        return (_exact_rope(s["q"], c, s), _exact_cached(_exact_rope(s["k"], c, s, True), c["fmt"], c["k_alpha"]),
                _exact_cached(s["v"], c["fmt"], c["v_alpha"]))
    if c["kind"] == "product":
        K = c["K"]
        power = s["scales"].view(torch.uint8).double() - 127
        a = s["codes"].double() * torch.exp2(power).repeat_interleave(32, -1)
        y = a[:, :K] @ _exact_weights(*s["weights"], c["N"], K).T * c["alpha"]
        y = _exact_gate(y, c["gate"]) if c["gate"] else y
        return _exact_mx8(y) if c["out"] == "mx8" else y
    y, h = _exact_norm(s)
    y = _exact_held(y) @ _exact_weights(*s["up"], 2 * c["inner"], c["width"]).T
    return _exact_held(_exact_gate(y, "silu")) @ _exact_weights(*s["down"], c["width"], c["inner"]).T, h

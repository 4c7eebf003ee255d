"""Cases of the operators around the Gated DeltaNet core: the block norm
(residual add and norm in front of a block), the gated head norm behind the
core, the 4-bit weight format (quantising and reading back) and the
projections with 4-bit weights.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU,
`run()` one pass, in plain torch operations or, with `own` true, through the
framework's calls.  `exact()` is the same result in float64 and `work()` the
bytes and operations a pass cannot do without.

The 4-bit format: groups of 32 weights along the input axis share one scale
byte s, worth 2**(s - 127) (255 marks a group that held an infinity or NaN);
a weight is one 4-bit code, sign bit and magnitude index into 0, 0.5, 1, 1.5,
2, 3, 4, 6.  Codes are stored two to a byte, the even weight in the low half.
"""
import math

import torch

own = False

GROUP = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MAX_FLOPS = 2 * 8192 * 12352 * 2048
MAX_BYTES = 1 << 29


# ---------------------------------------------------------------- the cases

def _norm(name, tokens, hidden, io, res, add=True, post=False):
    return {"name": name, "op": "block_norm", "tokens": tokens, "hidden": hidden, "io": io,
            "res": res, "add": add, "post": post}


def _gated(name, tokens, h_v, d, io, out):
    return {"name": name, "op": "gated_norm", "tokens": tokens, "h_v": h_v, "d": d, "io": io,
            "out": out}


def _format(name, rows, cols, src):
    return {"name": name, "op": "mx_format", "rows": rows, "cols": cols, "src": src}


def _proj(name, tokens, n_in, n_out, out):
    return {"name": name, "op": "mx_proj", "tokens": tokens, "in": n_in, "n_out": n_out, "out": out}


def _in_proj(name, tokens, hidden, h_k, h_v, d, out):
    return {"name": name, "op": "mx_in_proj", "tokens": tokens, "in": hidden, "h_k": h_k,
            "h_v": h_v, "d": d, "out": out}


def listed():
    return [
        # one decoded token of one request: latency
        _norm("norm_1x2048", 1, 2048, "bf16", "bf16"),
        # a prompt of 8192 tokens, the residual stream kept in fp32
        _norm("norm_8192x2048", 8192, 2048, "bf16", "f32"),
        # an odd width with a norm on both sides of the block, a packed batch of prompts
        _norm("norm_1237x1999_post", 1237, 1999, "f32", "f32", post=True),
        # one decode step of 64 requests
        _gated("gate_64x32x128", 64, 32, 128, "bf16", "bf16"),
        # a prompt of 8192 tokens
        _gated("gate_8192x32x128", 8192, 32, 128, "bf16", "bf16"),
        # the out-projection's weights, converted when a checkpoint is loaded
        _format("format_2048x4096", 2048, 4096, "bf16"),
        # the in-projection's weights (q, k, v, z and the gates), from an fp32 checkpoint
        _format("format_12352x2048", 12352, 2048, "f32"),
        # in-projection of one decoded token of one request
        _in_proj("in_proj_1", 1, 2048, 16, 32, 128, "bf16"),
        # out-projection of one decode step of 64 requests
        _proj("proj_64x4096x2048", 64, 4096, 2048, "bf16"),
        # an odd number of tokens and channels: a small verify step, fp32 results
        _proj("proj_37x1056x1001", 37, 1056, 1001, "f32"),
        # in-projection of a scheduler's chunk of a prompt
        _in_proj("in_proj_500", 500, 2048, 16, 32, 128, "bf16"),
        # in-projection of a prompt of 8192 tokens
        _in_proj("in_proj_8192", 8192, 2048, 16, 32, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("block_norm", "gated_norm", "mx_format", "mx_proj", "mx_in_proj"))
        tokens = _log_int(rng, 1, 8192)
        out = rng.choice(("bf16", "bf16", "f32"))
        if op == "block_norm":
            hidden = _log_int(rng, 32, 8192)
            if rng.random() < 0.6:
                hidden = max(32, hidden // 32 * 32)
            case = _norm("", tokens, hidden, out, rng.choice(("bf16", "f32")),
                         rng.random() < 0.8, rng.random() < 0.4)
            case["post"] = case["post"] and case["add"]
        elif op == "gated_norm":
            case = _gated("", tokens, rng.randint(1, 48), rng.choice((32, 64, 128)),
                          rng.choice(("bf16", "f32")), out)
        elif op == "mx_format":
            case = _format("", _log_int(rng, 16, 16384), 32 * _log_int(rng, 2, 256),
                           rng.choice(("bf16", "f32")))
        elif op == "mx_proj":
            case = _proj("", tokens, 32 * _log_int(rng, 2, 256), _log_int(rng, 16, 16384), out)
        else:
            h_k = rng.choice((1, 2, 4, 8, 16))
            case = _in_proj("", tokens, 32 * _log_int(rng, 2, 128), h_k, h_k * rng.randint(1, 4),
                            rng.choice((32, 64, 128)), out)
        del case["name"]
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES:
            return case


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _channels(case):
    """Output channels of a projection."""
    if case["op"] == "mx_proj":
        return case["n_out"]
    return 2 * case["h_k"] * case["d"] + 2 * case["h_v"] * case["d"] + 2 * case["h_v"]


def work(case):
    op = case["op"]
    if op == "block_norm":
        n = case["tokens"] * case["hidden"]
        per = _size(case["res"]) + _size(case["io"])                  # r in, x out
        if case["add"]:
            per += _size(case["io"]) + _size(case["res"])             # y in, r' out
        vectors = 1 + (1 if case["post"] else 0)
        return {"bytes": n * per + 4 * case["hidden"] * vectors,
                "flops": n * (4 + (2 if case["add"] else 0) + (4 if case["post"] else 0))}
    if op == "gated_norm":
        n = case["tokens"] * case["h_v"] * case["d"]
        return {"bytes": n * (2 * _size(case["io"]) + _size(case["out"])) + 4 * case["d"],
                "flops": 9 * n}
    if op == "mx_format":
        n = case["rows"] * case["cols"]
        packed = n // 2 + n // GROUP
        return {"bytes": n * 2 * _size(case["src"]) + 2 * packed, "flops": 6 * n}
    n_out, n_in, t = _channels(case), case["in"], case["tokens"]
    y = t * n_out * _size(case["out"])
    if op == "mx_in_proj":
        y += 2 * t * case["h_v"] * (4 - _size(case["out"]))           # the gates are fp32
    return {"bytes": n_out * (n_in // 2 + n_in // GROUP) + 2 * t * n_in + y,
            "flops": 2 * t * n_in * n_out}


# --------------------------------------------------------------- the inputs

def _encode(w):
    """Codes [rows, cols] (one to a byte) and scale bytes [rows, cols / 32] of
    the finite fp32 matrix w: the shared exponent is the largest magnitude's
    less 2, and codes round to nearest, ties to the even code, saturating."""
    groups = w.reshape(w.shape[0], -1, GROUP)
    amax = groups.abs().amax(-1)
    exponent = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    exponent = torch.where(amax > 0, exponent, torch.zeros_like(exponent))
    # exact: a power of two apart
    v = torch.ldexp(groups.double(), -exponent.unsqueeze(-1)).abs()
    index = torch.zeros(groups.shape, dtype=torch.uint8, device=w.device)
    for i in range(7):
        mid = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        index += ((v > mid) if i % 2 == 0 else (v >= mid)).to(torch.uint8)
    sign = (torch.signbit(groups)).to(torch.uint8) * 8
    return (index + sign).reshape(w.shape), (exponent + 127).to(torch.uint8)


def _pack(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def _decode(packed, scales):
    """The fp32 weights that packed codes and scale bytes stand for."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1, GROUP)
    scale = torch.ldexp(torch.ones((), device=packed.device), scales.int() - 127)
    return (table[codes.int()] * scale.unsqueeze(-1)).reshape(packed.shape[0], -1)


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    op = case["op"]
    t = case.get("tokens")
    if op == "block_norm":
        h = case["hidden"]
        # a residual stream has a few channels much larger than the others
        r = normal(t, h)
        r[:, :: max(1, h // 8)] *= 20.0
        d = {"r": r.to(_type(case["res"])), "w_pre": normal(h, scale=0.1)}
        if case["add"]:
            d["y"] = normal(t, h, scale=0.5).to(_type(case["io"]))
        if case["post"]:
            d["w_post"] = 1.0 + normal(h, scale=0.1)
        return d
    if op == "gated_norm":
        io = _type(case["io"])
        # outputs of the core differ in size from token to token and head to head
        o = normal(t, case["h_v"], case["d"]) * torch.exp(normal(t, case["h_v"], 1))
        return {"o": o.to(io), "z": normal(t, case["h_v"], case["d"], scale=1.5).to(io),
                "w": 1.0 + normal(case["d"], scale=0.1)}
    if op == "mx_format":
        w = normal(case["rows"], case["cols"], scale=case["cols"] ** -0.5)
        return {"w": w.to(_type(case["src"]))}
    w = normal(_channels(case), case["in"], scale=case["in"] ** -0.5)
    codes, scales = _encode(w)
    return {"x": normal(t, case["in"]).bfloat16(), "codes": _pack(codes), "scales": scales}


RES_SCALE = 0.75      # of a block's output as it joins the residual
EPS = 1e-6


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=dict(case))
    if not own:
        return s
    import gated_deltanet_state_layer_amd as G
    s["G"] = G
    op, t = case["op"], case.get("tokens")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "block_norm":
        s["x"] = empty(t, case["hidden"], dtype=_type(case["io"]))
        s["r_out"] = torch.empty_like(s["r"]) if case["add"] else None
    elif op == "gated_norm":
        io = G.GDN_BF16 if case["io"] == "bf16" else G.GDN_F32
        s["pool"] = G.Pool(G.make_desc(1, 1, 1, case["h_v"], case["d"], case["d"], 4, io))
        s["out"] = empty(t, case["h_v"], case["d"], dtype=_type(case["out"]))
    elif op == "mx_format":
        rows, cols = case["rows"], case["cols"]
        s["codes"] = empty(rows, cols // 2, dtype=torch.uint8)
        s["scales"] = empty(rows, cols // GROUP, dtype=torch.uint8)
        s["back"] = empty(rows, cols, dtype=_type(case["src"]))
    elif op == "mx_proj":
        s["y"] = empty(t, case["n_out"], dtype=_type(case["out"]))
        n = G.mx_proj_workspace_bytes(t, case["in"], case["n_out"])
        s["ws"] = empty(n, dtype=torch.uint8) if n else None
    else:
        io, ot = (G.GDN_BF16 if case["out"] == "bf16" else G.GDN_F32), _type(case["out"])
        h_k, h_v, d = case["h_k"], case["h_v"], case["d"]
        pool = s["pool"] = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, io))
        s["outs"] = {"q": empty(t, h_k, d, dtype=ot), "k": empty(t, h_k, d, dtype=ot),
                     "v": empty(t, h_v, d, dtype=ot), "z": empty(t, h_v, d, dtype=ot),
                     "a": empty(t, h_v), "b": empty(t, h_v)}
        n = pool.mx_in_proj_workspace_bytes(t, case["in"])
        s["ws"] = empty(n, dtype=torch.uint8) if n else None
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    case, G = s["case"], s["G"]
    op = case["op"]
    if op == "block_norm":
        G.block_norm(s["r"], s["w_pre"], s["x"], y=s.get("y"), w_post=s.get("w_post"),
                     residual_out=s["r_out"], res_scale=RES_SCALE, w_offset=1.0, eps=EPS)
        return (s["x"], s["r_out"]) if case["add"] else (s["x"],)
    if op == "gated_norm":
        return s["pool"].gated_norm(s["o"], s["z"], s["w"], s["out"], eps=EPS)
    if op == "mx_format":
        G.mx_quantize(s["w"], s["codes"], s["scales"])
        G.mx_dequantize(s["codes"], s["scales"], s["back"])
        return s["back"]
    if op == "mx_proj":
        return G.mx_proj(s["x"], s["codes"], s["scales"], s["y"], workspace=s["ws"])
    o = s["outs"]
    s["pool"].mx_in_proj(s["x"], s["codes"], s["scales"], o["q"], o["k"], o["v"], o["a"], o["b"],
                         z=o["z"], workspace=s["ws"])
    return dict(o)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "block_norm":
        r = s["r"].float()
        if case["add"]:
            u = s["y"].float()
            if case["post"]:
                u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * s["w_post"]
            r = r + RES_SCALE * u
        x = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * (1.0 + s["w_pre"])
        x = x.to(_type(case["io"]))
        return (x, r.to(_type(case["res"]))) if case["add"] else (x,)
    if op == "gated_norm":
        o, z = s["o"].float(), s["z"].float()
        n = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["w"]
        return (n * (z / (1.0 + torch.exp(-z)))).to(_type(case["out"]))
    if op == "mx_format":
        codes, scales = _encode(s["w"].float())
        return _decode(_pack(codes), scales).to(_type(case["src"]))
    y = s["x"].float() @ _decode(s["codes"], s["scales"]).T
    if op == "mx_proj":
        return y.to(_type(case["out"]))
    ot = _type(case["out"])
    t, h_k, h_v, d = case["tokens"], case["h_k"], case["h_v"], case["d"]
    q, k, v, z, a, b = torch.split(y, [h_k * d, h_k * d, h_v * d, h_v * d, h_v, h_v], -1)
    return {"q": q.reshape(t, h_k, d).to(ot), "k": k.reshape(t, h_k, d).to(ot),
            "v": v.reshape(t, h_v, d).to(ot), "z": z.reshape(t, h_v, d).to(ot),
            "a": 1.0 / (1.0 + torch.exp(a)), "b": 1.0 / (1.0 + torch.exp(-b))}


# ------------------------------------------------------- the result in 64 bits

def _exact_weights(packed, scales):
    """Weights by the format's bits: sign, two exponent bits, one fraction bit."""
    n, half = packed.shape
    codes = torch.empty((n, 2 * half), dtype=torch.int64, device=packed.device)
    codes[:, 0::2] = packed.long() % 16
    codes[:, 1::2] = packed.long() // 16
    sign = 1.0 - 2.0 * (codes // 8).double()
    e, f = (codes % 8) // 2, (codes % 2).double()
    mag = torch.where(e == 0, 0.5 * f, (1.0 + 0.5 * f) * torch.pow(2.0, (e - 1).double()))
    scale = torch.pow(torch.full((), 2.0, dtype=torch.float64, device=packed.device),
                      scales.double() - 127.0)
    return sign * mag * scale.repeat_interleave(GROUP, 1)


def exact(case, seed):
    i = _inputs(case, seed)
    op = case["op"]
    if op == "block_norm":
        h = case["hidden"]
        r = i["r"].double()
        if case["add"]:
            y = i["y"].double()
            if case["post"]:
                y = i["w_post"].double() * y / (y.square().sum(1, keepdim=True) / h + EPS).sqrt()
            r = r + RES_SCALE * y
        x = r / (r.square().sum(1, keepdim=True) / h + EPS).sqrt() * (i["w_pre"].double() + 1.0)
        return (x, r) if case["add"] else (x,)
    if op == "gated_norm":
        o, z = i["o"].double(), i["z"].double()
        rms = (o.square().sum(2, keepdim=True) / case["d"] + EPS).sqrt()
        return o / rms * i["w"].double() * z * torch.sigmoid(z)
    if op == "mx_format":
        w = i["w"].double().reshape(case["rows"], -1, GROUP)
        top = w.abs().max(2, keepdim=True).values
        # 2**e is the largest power of two not above the largest magnitude, over 4
        e = torch.where(top > 0, torch.floor(torch.log2(top)) - 2.0, torch.zeros_like(top))
        unit = torch.pow(2.0, e.clamp(-127, 127))
        v = (w / unit).abs().clamp(max=6.0)
        # steps of 0.5 below 2, 1 below 4, 2 above; round() ties to the even step
        step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
        return (torch.sign(w) * torch.round(v / step) * step * unit).reshape(case["rows"], -1)
    y = torch.matmul(i["x"].double(), _exact_weights(i["codes"], i["scales"]).t())
    if op == "mx_proj":
        return y
    t, h_k, h_v, d = case["tokens"], case["h_k"], case["h_v"], case["d"]
    c, v0 = h_k * d, h_v * d
    y_a, y_b = y[:, 2 * c + 2 * v0:][:, :h_v], y[:, 2 * c + 2 * v0 + h_v:]
    return {"q": y[:, :c].reshape(t, h_k, d), "k": y[:, c:2 * c].reshape(t, h_k, d),
            "v": y[:, 2 * c:2 * c + v0].reshape(t, h_v, d),
            "z": y[:, 2 * c + v0:2 * c + 2 * v0].reshape(t, h_v, d),
            "a": torch.sigmoid(-y_a), "b": torch.sigmoid(y_b)}

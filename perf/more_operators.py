"""Cases of the operators for batches of many requests: the maps of a batch
built from the requests' lengths, projections with 4-bit weights and a low-rank
adapter per request, beam selection over beams and vocabulary, and the
reordering of beams' states in the slot pool.

`listed()` and `draw()` give cases, `prepare()` a case's inputs on the GPU,
`run()` one pass, in plain torch operations or, with `own` true, through the
framework's calls.  `exact()` is the same result in float64 and `work()` the
bytes and operations a pass cannot do without.

The 4-bit format is that of gdn_mx_quantize: groups of 32 weights along the
input axis share one scale byte s, worth 2**(s - 127); a weight is a sign bit
and a magnitude index into 0, 0.5, 1, 1.5, 2, 3, 4, 6, two codes to a byte, the
even weight in the low half.
"""
import math

import torch

own = False

GROUP = 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CONV_K = 4
MAX_FLOPS = 2 * 8192 * 12352 * 2048
MAX_BYTES = 1 << 30


# ---------------------------------------------------------------- the cases

def _maps(name, seqs, tokens, cap, every, adapters):
    """`seqs` requests of `tokens` tokens in all, in arrays of `cap` rows;
    checkpoints every `every` tokens (0: none); `adapters` adapters."""
    return {"name": name, "op": "maps", "seqs": seqs, "tokens": tokens, "cap": cap, "every": every,
            "adapters": adapters}


def _proj(name, tokens, seqs, adapters, rank, n_in, n_out, out):
    return {"name": name, "op": "lora_proj", "tokens": tokens, "seqs": seqs, "adapters": adapters,
            "rank": rank, "in": n_in, "n_out": n_out, "out": out}


def _in_proj(name, tokens, seqs, adapters, rank, hidden, h_k, h_v, d, out):
    return {"name": name, "op": "lora_in_proj", "tokens": tokens, "seqs": seqs, "adapters": adapters,
            "rank": rank, "in": hidden, "h_k": h_k, "h_v": h_v, "d": d, "out": out}


def _beam(name, reqs, width, vocab, keep, io):
    return {"name": name, "op": "beam", "reqs": reqs, "width": width, "vocab": vocab, "keep": keep,
            "io": io}


def _reorder(name, reqs, width, live, layers, h_k, h_v, d, io):
    """`live` of the `width` beams of each request have children."""
    return {"name": name, "op": "reorder", "reqs": reqs, "width": width, "live": live,
            "layers": layers, "h_k": h_k, "h_v": h_v, "d": d, "io": io}


def listed():
    return [
        # one decode step of 64 requests with adapters: latency
        _maps("maps_64", 64, 64, 64, 0, 8),
        # the packed prompts of 16 requests, a state checkpoint every 512 tokens
        _maps("maps_16x36080", 16, 36080, 36864, 512, 8),
        # a long queue of prompts, an odd number of tokens, checkpoints every 64
        _maps("maps_2000x300001", 2000, 300001, 300001, 64, 100),
        # out-projection of one decoded token of one request
        _proj("lora_proj_1", 1, 1, 4, 16, 4096, 2048, "bf16"),
        # in-projection of one decode step of 64 requests with 40 adapters
        _in_proj("lora_in_proj_64", 64, 64, 40, 16, 2048, 16, 32, 128, "bf16"),
        # odd tokens and channels, seven requests of a scheduler's chunk, fp32 results
        _proj("lora_proj_500x1056x1001", 500, 7, 5, 24, 1056, 1001, "f32"),
        # in-projection of packed prompts of 8192 tokens, 16 requests with 8 adapters
        _in_proj("lora_in_proj_8192", 8192, 16, 8, 32, 2048, 16, 32, 128, "bf16"),
        # one request's beams: latency
        _beam("beam_1x4x32000", 1, 4, 32000, 4, "bf16"),
        # an odd vocabulary and fp32 logits, twice as many candidates kept as beams
        _beam("beam_3x5x50001", 3, 5, 50001, 10, "f32"),
        # a batch of 64 requests over a large vocabulary
        _beam("beam_64x8x131072", 64, 8, 131072, 16, "bf16"),
        # one request's four beams, one layer
        _reorder("reorder_1x4x1", 1, 4, 2, 1, 16, 32, 128, "bf16"),
        # 16 requests of eight beams, four layers
        _reorder("reorder_16x8x4", 16, 8, 5, 4, 16, 32, 128, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(("maps", "lora_proj", "lora_in_proj", "beam", "reorder"))
        if op == "maps":
            seqs = _log_int(rng, 1, 4096)
            tokens = seqs if rng.random() < 0.3 else _log_int(rng, seqs, 300000)
            cap = tokens if rng.random() < 0.5 else (tokens + 63) // 64 * 64
            case = _maps("", seqs, tokens, cap, rng.choice((0, 16, 64, 192, 512)),
                         rng.randint(0, 100))
        elif op in ("lora_proj", "lora_in_proj"):
            tokens = _log_int(rng, 1, 8192)
            # a decode step has one token a request, packed prompts few requests
            seqs = tokens if tokens <= 256 and rng.random() < 0.5 else rng.randint(1, min(tokens, 32))
            adapters, rank = _log_int(rng, 1, 64), rng.choice((8, 16, 16, 32, 40, 64))
            out = rng.choice(("bf16", "bf16", "f32"))
            if op == "lora_proj":
                case = _proj("", tokens, seqs, adapters, rank, 32 * _log_int(rng, 4, 128),
                             _log_int(rng, 16, 8192), out)
            else:
                h_k = rng.choice((1, 2, 4, 8, 16))
                case = _in_proj("", tokens, seqs, adapters, rank, 32 * _log_int(rng, 4, 128), h_k,
                                h_k * rng.randint(1, 4), rng.choice((32, 64, 128)), out)
        elif op == "beam":
            width = rng.randint(1, 16)
            case = _beam("", _log_int(rng, 1, 64), width, _log_int(rng, 1000, 160000),
                         width * rng.randint(1, 2), rng.choice(("bf16", "f32")))
        else:
            width = rng.randint(1, 16)
            h_k = rng.choice((1, 2, 4, 8, 16))
            case = _reorder("", _log_int(rng, 1, 32), width, rng.randint(1, width), rng.randint(1, 6),
                            h_k, h_k * rng.randint(1, 4), rng.choice((32, 64, 128)),
                            rng.choice(("bf16", "f32")))
        del case["name"]
        w = work(case)
        if w["flops"] <= MAX_FLOPS and w["bytes"] <= MAX_BYTES and _held(case) <= 2 * MAX_BYTES:
            return case


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


def _channels(case):
    """Output channels of a projection."""
    if case["op"] == "lora_proj":
        return case["n_out"]
    return 2 * case["h_k"] * case["d"] + 2 * case["h_v"] * case["d"] + 2 * case["h_v"]


def _slot_bytes(case):
    """State and conv window of all layers of one slot."""
    h_k, h_v, d = case["h_k"], case["h_v"], case["d"]
    return case["layers"] * (4 * h_v * d * d + (CONV_K - 1) * (2 * h_k + h_v) * d * _size(case["io"]))


def _held(case):
    """Bytes of the largest thing a case's inputs hold."""
    if case["op"] == "reorder":
        return case["reqs"] * case["width"] * _slot_bytes(case)
    return work(case)["bytes"]


def work(case):
    op = case["op"]
    if op == "maps":
        n, cap = case["seqs"], case["cap"]
        maps = 3 if case["adapters"] else 2
        ckpt = 0
        if case["every"]:
            rows = max(0, (case["tokens"] - n * (case["every"] - 1)) // case["every"])   # at least
            ckpt = 4 * (n + 1) + 8 * rows
        return {"bytes": 4 * (2 * n + (n if case["adapters"] else 0)) + 4 * (n + 1) + 4 * n +
                4 * maps * cap + ckpt, "flops": 2 * n + maps * cap}
    if op == "beam":
        rows = case["reqs"] * case["width"]
        n = rows * case["vocab"]
        # each logit: a difference, an exponential (counted as one), a sum, a comparison
        return {"bytes": n * _size(case["io"]) + 4 * rows + 12 * case["reqs"] * case["keep"],
                "flops": 4 * n}
    if op == "reorder":
        copies = case["reqs"] * (case["width"] - case["live"])
        return {"bytes": 2 * copies * _slot_bytes(case) + 12 * case["reqs"] * case["width"], "flops": 0}
    n_out, n_in, t, rank = _channels(case), case["in"], case["tokens"], case["rank"]
    y = t * n_out * _size(case["out"])
    if op == "lora_in_proj":
        y += 2 * t * case["h_v"] * (4 - _size(case["out"]))           # the gates are fp32
    used = min(case["seqs"], case["adapters"])
    return {"bytes": n_out * (n_in // 2 + n_in // GROUP) + 2 * t * n_in + y + 4 * t +
            used * 2 * rank * (n_in + n_out),
            "flops": 2 * t * n_in * n_out + 2 * t * rank * (n_in + n_out)}


# --------------------------------------------------------------- the inputs

def _encode(w):
    """Packed codes [rows, cols / 2] and scale bytes [rows, cols / 32] of the
    finite fp32 matrix w."""
    groups = w.reshape(w.shape[0], -1, GROUP)
    amax = groups.abs().amax(-1)
    exponent = torch.where(amax > 0, (torch.frexp(amax).exponent - 3).clamp(-127, 127), 0)
    v = torch.ldexp(groups, -exponent.unsqueeze(-1)).abs()
    index = torch.zeros(groups.shape, dtype=torch.uint8, device=w.device)
    for i in range(7):
        mid = (MAGNITUDES[i] + MAGNITUDES[i + 1]) / 2
        index += ((v > mid) if i % 2 == 0 else (v >= mid)).to(torch.uint8)
    codes = (index + torch.signbit(groups).to(torch.uint8) * 8).reshape(w.shape)
    return codes[:, 0::2] | codes[:, 1::2] << 4, (exponent + 127).to(torch.uint8)


def _decode(packed, scales):
    """The fp32 weights that packed codes and scale bytes stand for."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[0], -1, GROUP)
    scale = torch.ldexp(torch.ones((), device=packed.device), scales.int() - 127)
    return (table[codes.int()] * scale.unsqueeze(-1)).reshape(packed.shape[0], -1)


def _lengths(g, seqs, tokens):
    """Random lengths of `seqs` requests that sum to `tokens`; with as many
    tokens as requests one each, otherwise some may be empty."""
    if tokens == seqs:
        return torch.ones(seqs, dtype=torch.int32, device="cuda")
    cuts = torch.randint(0, tokens + 1, (seqs - 1,), generator=g, device="cuda").sort().values
    ends = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), cuts,
                      torch.full((1,), tokens, dtype=torch.int64, device="cuda")))
    return (ends[1:] - ends[:-1]).int()


def _adapter_ids(g, seqs, adapters):
    """Adapters 0, 1, .. and none (-1) in turn, in random order past the first."""
    ids = torch.arange(seqs, device="cuda") % (adapters + 1)
    ids = torch.where(ids == adapters, -1, ids)
    return ids[torch.randperm(seqs, generator=g, device="cuda")].int()


def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    def integers(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda").int()

    op = case["op"]
    if op == "maps":
        n = case["seqs"]
        d = {"lens": _lengths(g, n, case["tokens"]),
             "past": integers(0, 100, n) * max(case["every"], 1)}
        if case["adapters"]:
            d["adapter_ids"] = _adapter_ids(g, n, case["adapters"])
        if case["every"]:
            # a free list that runs out before the last checkpoint
            rows = case["tokens"] // case["every"]
            d["free"] = torch.randperm(max(1, rows - 3), generator=g, device="cuda").int()
        return d
    if op == "beam":
        r, w, v = case["reqs"], case["width"], case["vocab"]
        # a model's logits, some tokens ruled out by a grammar
        logits = normal(r, w, v, scale=2.5)
        logits[:, :, integers(0, v, v // 16).long()] = -math.inf
        finished = (torch.rand((r, w), generator=g, device="cuda") < 0.1).to(torch.uint8)
        return {"logits": logits.to(_type(case["io"])), "finished": finished,
                "scores": -normal(r, w, scale=4.0).abs().sort(-1).values}
    if op == "reorder":
        r, w, live, n = case["reqs"], case["width"], case["live"], case["reqs"] * case["width"]
        h_k, h_v, d = case["h_k"], case["h_v"], case["d"]
        window = normal(n, case["layers"], CONV_K - 1, (2 * h_k + h_v) * d).to(_type(case["io"]))
        # `live` beams of each request, every one of them a parent
        alive = torch.rand((r, w), generator=g, device="cuda").argsort(-1)[:, :live]
        pick = torch.cat((torch.arange(live, device="cuda").expand(r, live),
                          torch.randint(0, live, (r, w - live), generator=g, device="cuda")), 1)
        pick = pick.gather(1, torch.rand((r, w), generator=g, device="cuda").argsort(-1))
        return {"state": normal(n, case["layers"], h_v, d, d), "window": window,
                "slots": torch.randperm(n, generator=g, device="cuda").int().view(r, w),
                "parents": alive.gather(1, pick).int()}
    t, n_in, n_out, rank = case["tokens"], case["in"], _channels(case), case["rank"]
    codes, scales = _encode(normal(n_out, n_in, scale=n_in ** -0.5))
    ids = _adapter_ids(g, case["seqs"], case["adapters"])
    lens = _lengths(g, case["seqs"], t)
    ends = lens.long().cumsum(0)
    seq = (torch.arange(t, device="cuda").unsqueeze(1) >= ends).sum(1)
    return {"x": normal(t, n_in).bfloat16(), "codes": codes, "scales": scales,
            "a": normal(case["adapters"], rank, n_in, scale=n_in ** -0.5).bfloat16(),
            "b": normal(case["adapters"], n_out, rank, scale=0.5 * rank ** -0.5).bfloat16(),
            "s": 0.5 + torch.rand(case["adapters"], generator=g, device="cuda"), "ids": ids[seq]}


EOS = 2


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=dict(case))
    if not own:
        return s
    import gated_deltanet_state_layer_amd as G
    s["G"] = G
    op = case["op"]

    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "maps":
        n, cap, i32 = case["seqs"], case["cap"], torch.int32
        s["pool"] = G.Pool(G.make_desc(1, 1, 1, 1, 32, 32, CONV_K))
        s["out"] = {"cu_seqlens": empty(n + 1, dtype=i32), "last_rows": empty(n, dtype=i32),
                    "token_seq": empty(cap, dtype=i32), "token_pos": empty(cap, dtype=i32)}
        if case["adapters"]:
            s["out"]["token_adapter"] = empty(cap, dtype=i32)
        if case["every"]:
            s["out"]["ckpt_offsets"] = empty(n + 1, dtype=i32)
            s["out"]["ckpt_slots"] = empty(max(1, case["tokens"] // case["every"]), dtype=i32)
    elif op == "beam":
        r, w, k = case["reqs"], case["width"], case["keep"]
        s["out"] = (empty(r, k, dtype=torch.int32), empty(r, k, dtype=torch.int32), empty(r, k),
                    empty(r, k, dtype=torch.uint8))
        s["ws"] = empty(G.beam_select_workspace_bytes(r, w, case["vocab"], k), dtype=torch.uint8)
    elif op == "reorder":
        io = G.GDN_BF16 if case["io"] == "bf16" else G.GDN_F32
        n, d = case["reqs"] * case["width"], case["d"]
        pool = s["pool"] = G.Pool(G.make_desc(n, case["layers"], case["h_k"], case["h_v"], d, d, CONV_K, io))
        pool.state.copy_(s.pop("state"))
        pool.window.copy_(s.pop("window"))
        s["out"] = torch.empty_like(s["slots"])
    elif op == "lora_proj":
        s["y"] = empty(case["tokens"], case["n_out"], dtype=_type(case["out"]))
        s["ws"] = empty(G.mx_proj_lora_workspace_bytes(case["tokens"], case["in"], case["n_out"],
                                                       case["rank"]), dtype=torch.uint8)
    else:
        t, h_k, h_v, d = case["tokens"], case["h_k"], case["h_v"], case["d"]
        io, ot = (G.GDN_BF16 if case["out"] == "bf16" else G.GDN_F32), _type(case["out"])
        pool = s["pool"] = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, CONV_K, io))
        s["outs"] = {"q": empty(t, h_k, d, dtype=ot), "k": empty(t, h_k, d, dtype=ot),
                     "v": empty(t, h_v, d, dtype=ot), "z": empty(t, h_v, d, dtype=ot),
                     "a": empty(t, h_v), "b": empty(t, h_v)}
        s["ws"] = empty(pool.mx_in_proj_lora_workspace_bytes(t, case["in"], case["rank"]),
                        dtype=torch.uint8)
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    case, G = s["case"], s["G"]
    op = case["op"]
    if op == "maps":
        s["pool"].batch_maps(s["lens"], past=s["past"], adapter_ids=s.get("adapter_ids"),
                             n_adapters=case["adapters"], ckpt_every=case["every"],
                             free_slots=s.get("free"), **s["out"])
        return dict(s["out"])
    if op == "beam":
        parents, tokens, scores, finished = s["out"]
        G.beam_select(s["logits"], s["scores"], parents, tokens, scores, finished=s["finished"],
                      finished_out=finished, eos=EOS, workspace=s["ws"])
        return s["out"]
    if op == "reorder":
        s["pool"].reorder(s["slots"], s["parents"], s["out"])
        return s["pool"].state, s["pool"].window, s["out"]
    if op == "lora_proj":
        return G.mx_proj_lora(s["x"], s["codes"], s["scales"], s["a"], s["b"], s["s"], s["ids"], s["y"],
                              workspace=s["ws"])
    o = s["outs"]
    s["pool"].mx_in_proj_lora(s["x"], s["codes"], s["scales"], s["a"], s["b"], s["s"], s["ids"], o["q"],
                              o["k"], o["v"], o["a"], o["b"], z=o["z"], workspace=s["ws"])
    return dict(o)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "maps":
        return _plain_maps(case, s)
    if op == "beam":
        return _plain_beam(case, s)
    if op == "reorder":
        return _plain_reorder(s)
    x = s["x"].float()
    y = x @ _decode(s["codes"], s["scales"]).T
    for i in range(case["adapters"]):
        delta = (x @ s["a"][i].float().T) @ s["b"][i].float().T
        y = torch.where((s["ids"] == i).unsqueeze(1), y + s["s"][i] * delta, y)
    if op == "lora_proj":
        return y.to(_type(case["out"]))
    ot = _type(case["out"])
    t, h_k, h_v, d = case["tokens"], case["h_k"], case["h_v"], case["d"]
    q, k, v, z, a, b = torch.split(y, [h_k * d, h_k * d, h_v * d, h_v * d, h_v, h_v], -1)
    return {"q": q.reshape(t, h_k, d).to(ot), "k": k.reshape(t, h_k, d).to(ot),
            "v": v.reshape(t, h_v, d).to(ot), "z": z.reshape(t, h_v, d).to(ot),
            "a": 1.0 / (1.0 + torch.exp(a)), "b": 1.0 / (1.0 + torch.exp(-b))}


def _plain_maps(case, s):
    lens, cap = s["lens"].long(), case["cap"]
    zero = torch.zeros(1, dtype=torch.int64, device=lens.device)
    cu = torch.cat((zero, lens.cumsum(0)))
    row = torch.arange(cap, device=lens.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    inside, j = seq < case["seqs"], seq.clamp(max=case["seqs"] - 1)

    def per_token(v):
        return torch.where(inside, v, -1).int()

    out = {"cu_seqlens": cu.int(), "last_rows": torch.where(lens > 0, cu[1:] - 1, -1).int(),
           "token_seq": per_token(j), "token_pos": per_token(s["past"].long()[j] + row - cu[j])}
    if case["adapters"]:
        out["token_adapter"] = per_token(s["adapter_ids"].long()[j])
    if case["every"]:
        off = torch.cat((zero, (lens // case["every"]).cumsum(0)))
        rows, free = max(1, case["tokens"] // case["every"]), s["free"].long()
        i = torch.arange(rows, device=lens.device)
        slots = torch.where((i < off[-1]) & (i < free.numel()), free[i.clamp(max=free.numel() - 1)], -1)
        out["ckpt_offsets"], out["ckpt_slots"] = off.int(), slots.int()
    return out


def _plain_beam(case, s):
    # in 64 bits: scores of different beams may lie closer than 32 bits resolve
    v, k = case["vocab"], case["keep"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    score = s["scores"].double().unsqueeze(-1)
    c = score + (x - lse)
    done = s["finished"].bool().unsqueeze(-1)
    is_eos = torch.arange(v, device=x.device) == EOS
    c = torch.where(done, torch.where(is_eos, score, -math.inf), c).flatten(1)
    value, index = torch.sort(c, dim=-1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    some = value > -math.inf
    parent = torch.where(some, index // v, -1)
    token = torch.where(some, index % v, -1)
    ended = some & (s["finished"].gather(1, parent.clamp(min=0)).bool() | (token == EOS))
    return parent.int(), token.int(), value.float(), ended.to(torch.uint8)


def _plain_reorder(s):
    slots, parents = s["slots"].long(), s["parents"].long()
    w = parents.shape[1]
    same = parents.unsqueeze(2) == parents.unsqueeze(1)
    earlier = torch.ones(w, w, dtype=torch.bool, device=slots.device).tril(-1)
    first = ~(same & earlier).any(2)
    has_child = (parents.unsqueeze(2) == torch.arange(w, device=slots.device)).any(1)
    childless = torch.sort(has_child.int(), dim=1, stable=True).indices
    turn = ((~first).int().cumsum(1) - 1).clamp(min=0)
    source = slots.gather(1, parents)
    out = torch.where(first, source, slots.gather(1, childless.gather(1, turn)))
    s["state"][out.flatten()] = s["state"][source.flatten()]
    s["window"][out.flatten()] = s["window"][source.flatten()]
    return s["state"], s["window"], out.int()


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


def _exact_maps(case, i):
    lens = i["lens"].tolist()
    seq, pos, starts, off = [], [], [0], [0]
    for j, (n, p) in enumerate(zip(lens, i["past"].tolist())):
        seq += [j] * n
        pos += range(p, p + n)
        starts.append(starts[-1] + n)
        if case["every"]:
            off.append(off[-1] + n // case["every"])
    pad = [-1] * (case["cap"] - len(seq))
    out = {"cu_seqlens": starts, "last_rows": [e - 1 if n else -1 for n, e in zip(lens, starts[1:])],
           "token_seq": seq + pad, "token_pos": pos + pad}
    if case["adapters"]:
        ids = i["adapter_ids"].tolist()
        out["token_adapter"] = [ids[j] for j in seq] + pad
    if case["every"]:
        rows = max(1, case["tokens"] // case["every"])
        used = i["free"].tolist()[:off[-1]]
        out["ckpt_offsets"], out["ckpt_slots"] = off, (used + [-1] * rows)[:rows]
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in out.items()}


def _exact_beam(case, i):
    r, w, v, k = case["reqs"], case["width"], case["vocab"], case["keep"]
    logp = torch.log_softmax(i["logits"].double(), -1)
    outs = [], [], [], []
    for q in range(r):
        entries = []
        for b in range(w):
            base = float(i["scores"][q, b])
            if int(i["finished"][q, b]):
                entries.append((-base, b, EOS, True))
                continue
            row = logp[q, b] + base
            # the kept ones and every one as good as the last of them
            least = row.topk(min(k, v)).values[-1]
            at = torch.nonzero((row >= least) & (row > -math.inf)).flatten()
            entries += [(-c, b, t, t == EOS) for c, t in zip(row[at].tolist(), at.tolist())]
        entries = sorted(entries)[:k]
        entries += [(math.inf, -1, -1, False)] * (k - len(entries))
        for o, values in zip(outs, zip(*[(b, t, -c, int(e)) for c, b, t, e in entries])):
            o.append(values)
    kinds = torch.int32, torch.int32, torch.float64, torch.uint8
    return tuple(torch.tensor(o, dtype=kind, device="cuda") for o, kind in zip(outs, kinds))


def _exact_reorder(i):
    state, window, out = i["state"], i["window"], i["slots"].clone()
    for r, (slots, parents) in enumerate(zip(i["slots"].tolist(), i["parents"].tolist())):
        spare = [s for b, s in enumerate(slots) if b not in parents]
        taken = set()
        for j, p in enumerate(parents):
            dst = slots[p]
            if p in taken:
                dst = spare.pop(0)
                state[dst], window[dst] = state[slots[p]], window[slots[p]]
            taken.add(p)
            out[r, j] = dst
    return state, window, out


def exact(case, seed):
    i = _inputs(case, seed)
    op = case["op"]
    if op == "maps":
        return _exact_maps(case, i)
    if op == "beam":
        return _exact_beam(case, i)
    if op == "reorder":
        return _exact_reorder(i)
    x, ids = i["x"].double(), i["ids"].long()
    y = torch.matmul(x, _exact_weights(i["codes"], i["scales"]).t())
    for n in ids.unique().tolist():
        if n >= 0:
            rows = torch.nonzero(ids == n).flatten()
            inner = torch.matmul(x[rows], i["a"][n].double().t()) * i["s"][n].double()
            y[rows] += torch.matmul(inner, i["b"][n].double().t())
    if op == "lora_proj":
        return y
    t, h_k, h_v, d = case["tokens"], case["h_k"], case["h_v"], case["d"]
    c, v0 = h_k * d, h_v * d
    y_a, y_b = y[:, 2 * c + 2 * v0:][:, :h_v], y[:, 2 * c + 2 * v0 + h_v:]
    return {"q": y[:, :c].reshape(t, h_k, d), "k": y[:, c:2 * c].reshape(t, h_k, d),
            "v": y[:, 2 * c:2 * c + v0].reshape(t, h_v, d),
            "z": y[:, 2 * c + v0:2 * c + 2 * v0].reshape(t, h_v, d),
            "a": torch.sigmoid(-y_a), "b": torch.sigmoid(y_b)}

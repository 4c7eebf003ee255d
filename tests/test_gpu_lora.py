"""GPU: projections with 4-bit weights and a low-rank adapter per token, against
their definition in float64."""
import pytest

from mx_plan import TILE_CASES, paths, plan

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _unpack(codes, scales):
    c, s = codes.cpu().long(), scales.cpu().long()
    idx = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)
    v = torch.where(idx >= 8, -LEVELS[idx & 7], LEVELS[idx & 7])
    return (v * torch.ldexp(torch.ones((), dtype=torch.float64), (s - 127).double()).repeat_interleave(32, 1)).cuda()


def _weights(n_out, n_in, gen):
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 124, (n_out, n_in // 32), generator=gen, device="cuda").to(torch.uint8)
    return codes, scales


def _adapters(n, rank, n_in, n_out, gen):
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return ((rnd(n, rank, n_in) * n_in ** -0.5).to(BF), rnd(n, n_out, rank).to(BF),
            torch.rand(n, generator=gen, device="cuda") * 2 - 0.5)


def _reference(x, codes, scales, a, b, s, ids):
    """The sums and a bound of their error, in float64.  Each addition rounds
    once: n_in for the shared product and for x A^T, where the scale rounds once
    more; the three bf16 pieces of that leave 2^-24 and are summed in 3 rank
    additions (or rank, in one piece), and the two shares are added."""
    xd, w = x.double(), _unpack(codes, scales)
    n_in, rank = x.shape[1], a.shape[1]
    y, bound = xd @ w.t().contiguous(), n_in * U * (xd.abs() @ w.abs().t().contiguous())
    for i in range(a.shape[0]):
        rows = torch.nonzero(ids == i).flatten()
        if rows.numel() == 0:
            continue
        ai, bi, si = a[i].double().t().contiguous(), b[i].double().t().contiguous(), float(s[i])
        delta = si * (xd[rows] @ ai @ bi)
        mag = abs(si) * (xd[rows].abs() @ ai.abs() @ bi.abs())
        y[rows] += delta
        bound[rows] += (n_in + 3 * rank + 4) * U * mag + U * (y[rows].abs() + mag)
    return y, bound


def _close(name, got, ref, bound):
    assert torch.isfinite(got).all(), name
    lim = bound + STEP[got.dtype] * (ref.abs() + bound) + 1e-37
    worst = float(((got.double() - ref).abs() / lim).max())
    print(f"  {name}: worst error {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, name


def _ids(n_tok, n, kind, gen):
    if kind == "one":
        return torch.full((n_tok,), n - 1, dtype=torch.int32, device="cuda")
    if kind == "runs":      # packed prompts, some without
        at = torch.arange(n_tok, device="cuda") * 7 // max(n_tok, 1)
        return (torch.randint(-1, n, (7,), generator=gen, device="cuda")[at]).int()
    if kind == "each":
        return (torch.arange(n_tok, device="cuda") % n).int()
    return torch.randint(-3, n + 2, (n_tok,), generator=gen, device="cuda").int()   # "mixed", with ids outside


def _ws(nbytes):
    return torch.full((nbytes // 4,), float("nan"), device="cuda")


def _case(G, n_tok, n_in, n_out, rank, n, kind, out, pad_x=0, pad_y=0):
    gen = torch.Generator(device="cuda").manual_seed(n_tok + 3 * n_in + 5 * n_out + 7 * rank + 11 * n)
    xb = torch.full((n_tok, n_in + pad_x), float("nan"), dtype=BF, device="cuda")
    xb[:, :n_in] = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    x = xb[:, :n_in]
    codes, scales = _weights(n_out, n_in, gen)
    a, b, s = _adapters(n, rank, n_in, n_out, gen)
    ids = _ids(n_tok, n, kind, gen)
    yb = torch.full((n_tok + 2, n_out + pad_y), 7.0, dtype=out, device="cuda")
    y = yb[:n_tok, :n_out]
    y.fill_(float("nan"))
    ws = _ws(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank))
    G.mx_proj_lora(x, codes, scales, a, b, s, ids, y, workspace=ws)
    torch.cuda.synchronize()
    ref, bound = _reference(x, codes, scales, a, b, s, ids)
    _close(f"y {n_tok}x{n_in}x{n_out} rank {rank} {kind} {paths(n_tok, n_in, n_out)}", y, ref, bound)
    assert (yb[n_tok:] == 7.0).all() and (yb[:, n_out:] == 7.0).all()
    return x, codes, scales, a, b, s, ids, y


@pytest.mark.parametrize("kind", ["one", "runs", "each", "mixed"])
@pytest.mark.parametrize("n_tok,n_in,n_out,rank,n,out", [
    (1, 32, 1, 8, 1, F32), (1, 4096, 2048, 16, 3, BF), (3, 96, 70, 24, 2, BF), (4, 2048, 272, 8, 5, F32),
    (15, 160, 33, 128, 4, F32), (16, 1056, 1001, 16, 6, F32), (37, 1056, 1001, 40, 5, BF), (64, 2048, 1040, 16, 40, BF),
    (64, 4096, 64, 64, 64, F32), (100, 2048, 515, 32, 7, BF), (129, 64, 130, 16, 9, F32), (257, 288, 519, 72, 3, BF),
    (500, 1056, 1001, 24, 5, F32), (1000, 512, 2048, 16, 8, BF), (1500, 96, 264, 8, 100, F32), (2100, 2048, 768, 16, 4, BF),
])
def test_proj(G, n_tok, n_in, n_out, rank, n, out, kind):
    _case(G, n_tok, n_in, n_out, rank, n, kind, out)


@pytest.mark.parametrize("kind", ["one", "each", "mixed"])
@pytest.mark.parametrize("n_tok,n_in,n_out,rank", [
    (1, 4096, 8200, 16), (1, 4096, 47, 8), (1, 4128, 47, 16), (1, 2048, 4113, 32), (1, 2048, 1000, 24), (1, 2080, 99, 24),
    (1, 128, 16, 32), (1, 544, 33, 40), (2, 2048, 515, 16), (2, 1024, 8193, 32), (3, 1344, 100, 8), (3, 672, 515, 24),
    (4, 1024, 4100, 16), (4, 1056, 65, 16), (4, 512, 272, 32), (4, 128, 1, 8), (5, 128, 48, 16),
])
def test_proj_of_few_tokens(G, n_tok, n_in, n_out, rank, kind):
    """Both sides of what one launch takes."""
    _case(G, n_tok, n_in, n_out, rank, 4, kind, BF, pad_x=8)
    _case(G, n_tok, n_in, n_out, rank, 4, kind, F32)


@pytest.mark.parametrize("kind", ["each", "mixed"])
@pytest.mark.parametrize("n_tok,n_in,n_out,rank", [
    (64, 2048, 12352, 16), (33, 1056, 12301, 24), (64, 1056, 16370, 8), (700, 544, 1001, 16), (999, 1184, 515, 40),
    (300, 2048, 2048, 16), (193, 1056, 4090, 128), (97, 1056, 8180, 16), (255, 1056, 4080, 8),
])
def test_proj_in_shapes_of_64_tokens(G, n_tok, n_in, n_out, rank, kind):
    """And tokens without an adapter have the plain projection's bits."""
    assert [(p.tile, p.tokens) for p in plan(n_tok, n_in, n_out)] == [(0, 64)]
    x, codes, scales, _, _, _, ids, y = _case(G, n_tok, n_in, n_out, rank, 9, kind, BF, pad_x=8)
    plain = torch.empty_like(y)
    G.mx_proj(x, codes, scales, plain)
    off = (ids < 0) | (ids >= 9)
    assert torch.equal(y[off], plain[off])
    _case(G, n_tok, n_in, n_out, rank, 9, kind, F32)


@pytest.mark.parametrize("kind", ["runs", "mixed"])
@pytest.mark.parametrize("n_tok,n_in,n_out,want", TILE_CASES)
def test_proj_on_tiles(G, n_tok, n_in, n_out, want, kind):
    _case(G, n_tok, n_in, n_out, 16, 6, kind, BF)
    _case(G, n_tok, n_in, n_out, 40, 6, kind, F32)


@pytest.mark.parametrize("n_tok,n_out", [(1, 48), (3, 50), (33, 256), (300, 300), (600, 515)])
@pytest.mark.parametrize("pad_x,pad_y", [(8, 0), (0, 3), (64, 8)])
def test_proj_strides(G, n_tok, n_out, pad_x, pad_y):
    _case(G, n_tok, 160, n_out, 16, 3, "mixed", BF, pad_x, pad_y)
    _case(G, n_tok, 160, n_out, 8, 3, "mixed", F32, pad_x, pad_y)


@pytest.mark.parametrize("n_tok,n_in,n_out", [(3, 256, 300), (40, 256, 300), (64, 2048, 640), (300, 544, 700),
                                              (500, 1184, 12353), (700, 512, 8200)])
def test_tokens_do_not_depend_on_each_other(G, n_tok, n_in, n_out):
    """Without an adapter a token's row is that of mx_proj; a row does not change
    with the others' adapters, nor with infinities and NaN in them."""
    rank = 16
    x, codes, scales, a, b, s, ids, y = _case(G, n_tok, n_in, n_out, rank, 5, "mixed", BF)
    ws = _ws(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank))
    plain, again = torch.empty_like(y), torch.empty_like(y)
    G.mx_proj(x, codes, scales, plain)
    off = (ids < 0) | (ids >= 5)
    assert torch.equal(y[off], plain[off])
    gen = torch.Generator(device="cuda").manual_seed(1)
    keep = torch.rand(n_tok, generator=gen, device="cuda") < 0.5
    other = torch.where(keep, ids, torch.randint(-1, 5, (n_tok,), generator=gen, device="cuda").int())
    G.mx_proj_lora(x, codes, scales, a, b, s, other, again, workspace=ws)
    assert torch.equal(again[keep], y[keep])
    a, b, s = a.clone(), b.clone(), s.clone()
    a[1, 3, 5], b[2, n_out // 2, 7], b[3, :, 0], s[4] = float("nan"), float("inf"), float("-inf"), float("inf")
    G.mx_proj_lora(x, codes, scales, a, b, s, ids, again, workspace=ws)
    torch.cuda.synchronize()
    good = off | (ids == 0)
    assert torch.equal(again[good], y[good])
    assert torch.isnan(again[ids == 1]).all()
    assert not torch.isfinite(again[ids == 3]).any() and not torch.isfinite(again[ids == 4]).any()
    one = (ids == 2).nonzero().flatten()
    cols = torch.ones(n_out, dtype=torch.bool, device="cuda")
    cols[n_out // 2] = False
    assert torch.equal(again[one][:, cols], y[one][:, cols]) and not torch.isfinite(again[one][:, ~cols]).any()


def test_nan_tokens_and_infinite_tokens_stay_in_their_rows(G):
    for n_tok, n_in, n_out in ((3, 256, 300), (300, 544, 700)):
        x, codes, scales, a, b, s, ids, y = _case(G, n_tok, n_in, n_out, 16, 2, "one", F32)
        x = x.clone()
        x[1, 40], x[2, 41] = float("nan"), float("inf")
        again = torch.empty_like(y)
        G.mx_proj_lora(x, codes, scales, a, b, s, ids, again,
                       workspace=_ws(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, 16)))
        torch.cuda.synchronize()
        rest = [t for t in range(n_tok) if t not in (1, 2)]
        assert torch.isnan(again[1]).all() and not torch.isfinite(again[2]).any()
        assert torch.equal(again[rest], y[rest])


def _in_proj(G, n_tok, hidden, h_k, h_v, d, rank, n, kind, out, with_z):
    gen = torch.Generator(device="cuda").manual_seed(6000 + n_tok + hidden + d + rank)
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16 if out == BF else G.GDN_F32))
    c, v0 = h_k * d, h_v * d
    widths = [c, c, v0] + ([v0] if with_z else []) + [h_v, h_v]
    n_out = sum(widths)
    x = torch.randn(n_tok, hidden, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, hidden, gen)
    a, b, s = _adapters(n, rank, hidden, n_out, gen)
    ids = _ids(n_tok, n, kind, gen)
    full = lambda *sh, dt=out: torch.full(sh, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    bufs = {"q": full(n_tok, h_k, d), "k": full(n_tok, h_k, d), "v": full(n_tok, h_v, d),
            "z": full(n_tok, h_v, d) if with_z else None, "a": full(n_tok, h_v, dt=F32), "b": full(n_tok, h_v, dt=F32)}
    ws = _ws(pool.mx_in_proj_lora_workspace_bytes(n_tok, hidden, rank, with_z))
    pool.mx_in_proj_lora(x, codes, scales, a, b, s, ids, bufs["q"], bufs["k"], bufs["v"], bufs["a"], bufs["b"],
                         z=bufs["z"], workspace=ws)
    torch.cuda.synchronize()
    y, bound = _reference(x, codes, scales, a, b, s, ids)
    at = 0
    for name, wd in zip(("q", "k", "v") + (("z",) if with_z else ()) + ("a", "b"), widths):
        r, e = y[:, at:at + wd], bound[:, at:at + wd]
        at += wd
        if name in "ab":
            # the activations' slope is at most 1/4; exponential, sum and quotient round
            r = torch.sigmoid(-r if name == "a" else r)
            e = 0.25 * e + 8 * U * r
        _close(name, bufs[name].reshape(n_tok, wd), r, e)


@pytest.mark.parametrize("with_z", [True, False])
@pytest.mark.parametrize("n_tok,hidden,h_k,h_v,d,rank,n,kind,out", [
    (1, 2048, 16, 32, 128, 16, 2, "one", BF), (64, 2048, 16, 32, 128, 16, 40, "each", BF), (7, 96, 2, 2, 32, 8, 3, "mixed", F32),
    (70, 160, 1, 3, 64, 24, 4, "mixed", BF), (130, 256, 1, 1, 32, 16, 3, "runs", F32), (300, 1024, 2, 6, 64, 64, 3, "runs", BF),
    (700, 96, 2, 4, 64, 8, 9, "mixed", F32), (1100, 512, 4, 8, 128, 32, 5, "runs", BF), (1, 32, 1, 1, 32, 8, 1, "one", F32),
    (500, 544, 16, 32, 128, 16, 8, "runs", BF),
])
def test_in_proj(G, n_tok, hidden, h_k, h_v, d, rank, n, kind, out, with_z):
    _in_proj(G, n_tok, hidden, h_k, h_v, d, rank, n, kind, out, with_z)


def test_without_adapters_and_without_tokens(G):
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(20, 64, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(50, 64, gen)
    y, y2 = t(20, 50), t(20, 50)
    G.mx_proj(x, codes, scales, y)
    G.mx_proj_lora(x, codes, scales, t(0, 16, 64), None, None, None, y2)
    assert torch.equal(y, y2)
    G.mx_proj_lora(x[:0], codes, scales, t(1, 16, 64), t(1, 50, 16), t(1, dt=F32), t(0, dt=torch.int32), y2[:0])


@pytest.mark.parametrize("n_tok", [1, 40, 300, 1000])
def test_repeats_on_another_stream_and_in_a_graph(G, n_tok):
    n_in, n_out, rank = 512, 700, 16
    x, codes, scales, a, b, s, ids, _ = _case(G, n_tok, n_in, n_out, rank, 4, "mixed", BF)
    x = x.clone()
    y, y2 = (torch.empty(n_tok, n_out, dtype=BF, device="cuda") for _ in "ab")
    ws, ws2 = (_ws(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank)) for _ in "ab")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        G.mx_proj_lora(x, codes, scales, a, b, s, ids, y, workspace=ws)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in range(4):
        x.copy_(torch.randn(n_tok, n_in, generator=gen, device="cuda"))
        ids.copy_(torch.randint(-1, 4, (n_tok,), generator=gen, device="cuda"))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            G.mx_proj_lora(x, codes, scales, a, b, s, ids, y2, workspace=ws2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2), t


def test_refusals(G):
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [t(3, 64), u(10, 32), u(10, 2), t(2, 16, 64), t(2, 10, 16), t(2, dt=F32), i(3), t(3, 10)]
    ws = _ws(G.mx_proj_lora_workspace_bytes(3, 64, 10, 16))
    G.mx_proj_lora(*good, workspace=ws)
    for at, bad in ((0, t(3, 64, dt=F32)), (1, u(9, 32)), (3, t(2, 16, 96)), (3, t(2, 16, 64, dt=F32)), (3, None),
                    (4, t(2, 9, 16)), (4, t(2, 16, 10)), (4, None), (5, t(2)), (5, t(1, dt=F32)), (6, i(2)),
                    (6, i(3).float()), (6, i(3).cpu()), (7, t(2, 10)), (7, t(3, 10, dt=torch.float16))):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError):
            G.mx_proj_lora(*args, workspace=ws)
    with pytest.raises(G.GdnError):
        G.mx_proj_lora(*good)                       # no workspace
    with pytest.raises(G.GdnError):
        G.mx_proj_lora(*good[:3], t(2, 12, 64), t(2, 10, 12), *good[5:], workspace=ws)
    with pytest.raises(ValueError):
        G.mx_proj_lora(*good, workspace=ws.cpu())


@pytest.mark.parametrize("n_tok", [1, 40, 300])
@pytest.mark.parametrize("n_in,n_out,n,rank", [(128, 12352, 6000, 32), (16384, 48, 4200, 32)])
def test_adapters_past_2_31_elements(G, n_in, n_out, n, rank, n_tok):
    """The last of many adapters gives what it gives alone."""
    assert n * rank * max(n_in, n_out) > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, n_in, gen)
    a1, b1, s1 = _adapters(1, rank, n_in, n_out, gen)
    a, b, s = (torch.zeros(n, *t.shape[1:], dtype=t.dtype, device="cuda") for t in (a1, b1, s1))
    a[-1], b[-1], s[-1] = a1[0], b1[0], s1[0]
    y, alone = (torch.empty(n_tok, n_out, dtype=BF, device="cuda") for _ in "ab")
    ws = _ws(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank))
    ids = torch.full((n_tok,), n - 1, dtype=torch.int32, device="cuda")
    G.mx_proj_lora(x, codes, scales, a, b, s, ids, y, workspace=ws)
    G.mx_proj_lora(x, codes, scales, a1, b1, s1, torch.zeros_like(ids), alone, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, alone)

"""GPU: the 4-bit weight format and the projections with 4-bit weights,
against their definitions in float64."""
import pytest

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
    """The weights in float64 on the host, NaN where the scale byte is 255."""
    c, s = codes.cpu().long(), scales.cpu().long()
    idx = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)
    v = torch.where(idx >= 8, -LEVELS[idx & 7], LEVELS[idx & 7])
    scale = torch.where(s == 255, torch.nan, torch.ldexp(torch.ones((), dtype=torch.float64), (s - 127).double()))
    return v * scale.repeat_interleave(32, 1)


def _reference(w):
    """Codes' values and scale bytes by the definition, on the host in float64."""
    g = w.cpu().double().reshape(w.shape[0], -1, 32)
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(torch.isfinite(g), g, torch.zeros_like(g))
    top = g.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent.double() - 3, torch.zeros_like(top)).clamp(min=-127)
    v = (g * torch.ldexp(torch.ones((), dtype=torch.float64), -e).unsqueeze(-1)).abs()
    # to the nearest level, ties to the even code
    d = (v.unsqueeze(-1) - LEVELS).abs()
    near = d.amin(-1, keepdim=True)
    cand = (d == near)
    odd = torch.arange(8) % 2
    key = torch.where(cand, odd, 9)
    idx = key.argmin(-1)
    val = torch.copysign(LEVELS[idx], g) * torch.ldexp(torch.ones((), dtype=torch.float64), e).unsqueeze(-1)
    s = torch.where(bad, 255, (e + 127).long())
    val = torch.where(bad.unsqueeze(-1), torch.nan, val)
    return val.reshape(w.shape[0], -1), s


def _quantize(G, w):
    rows, cols = w.shape
    codes = torch.full((rows, cols // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 0xAA, dtype=torch.uint8, device="cuda")
    G.mx_quantize(w, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def _same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (16, 96), (7, 1056), (257, 2048), (1001, 160)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_and_back(G, rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    w = (torch.randn(rows, cols, generator=gen, device="cuda") *
         torch.exp(3 * torch.randn(rows, 1, generator=gen, device="cuda"))).to(dtype)
    codes, scales = _quantize(G, w)
    val, s = _reference(w)
    assert (scales.cpu().long() == s).all()
    assert _same(_unpack(codes, scales), val)
    for out in (BF, F32):
        back = torch.empty(rows, cols, dtype=out, device="cuda")
        G.mx_dequantize(codes, scales, back)
        torch.cuda.synchronize()
        assert _same(back.cpu().double(), val)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_edges(G, dtype):
    """Groups of zeros, ties, values that saturate, the smallest and largest
    exponents, subnormal weights, infinities and NaN."""
    w = torch.zeros(12, 64, device="cuda")
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], device="cuda")
    w[1, :8], w[1, 8:16] = ties, -ties
    w[2, 0], w[2, 1] = 7.9375, -7.0                 # past 6: both saturate
    w[3, :8] = ties * 2.0 ** -120
    w[4, :8] = ties * 2.0 ** 124
    w[5, 0] = 3.0e38
    w[6, 3] = 2.0 ** -126
    w[7, 5] = 2.0 ** -130                           # subnormal
    w[7, 6] = -(2.0 ** -128)
    w[8, 40] = float("inf")
    w[9, 0] = float("-inf")
    w[10, 33] = float("nan")
    w[11, 0] = -0.0
    w = w.to(dtype)
    codes, scales = _quantize(G, w)
    val, s = _reference(w)
    assert (scales.cpu().long() == s).all(), (scales.cpu(), s)
    assert _same(_unpack(codes, scales), val)
    back = torch.empty(12, 64, dtype=F32, device="cuda")
    G.mx_dequantize(codes, scales, back)
    assert _same(back.cpu().double(), val)
    assert torch.isnan(back[8, 32:]).all() and (back[8, :32] == 0).all()


def test_every_code_and_scale_reads_back(G):
    """All 16 codes under all 256 scale bytes, in fp32 and bf16."""
    codes = torch.zeros(256, 16, dtype=torch.uint8)
    for j in range(16):
        codes[:, j] = (j | ((15 - j) << 4))
    scales = torch.arange(256, dtype=torch.uint8).reshape(256, 1)
    for out in (F32, BF):
        back = torch.empty(256, 32, dtype=out, device="cuda")
        G.mx_dequantize(codes.cuda(), scales.cuda(), back)
        ref = _unpack(codes, scales)
        ref = torch.where(ref.abs() > torch.finfo(out).max, torch.copysign(torch.full_like(ref, torch.inf), ref), ref)
        assert _same(back.cpu().double(), ref)


def _weights(n_out, n_in, gen):
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 128, (n_out, n_in // 32), generator=gen, device="cuda").to(torch.uint8)
    return codes, scales


def _product(x, w):
    """x W^T and the sum of the products' magnitudes, float64 (fp64 products on the device)."""
    xd, wd = x.double(), w.cuda()
    return torch.mm(xd, wd.t().contiguous()), torch.mm(xd.abs(), wd.abs().t().contiguous())


def _close(name, got, ref, bound):
    assert torch.isfinite(got).all(), name
    lim = bound + STEP[got.dtype] * (ref.abs() + bound) + 1e-37
    worst = float(((got.double() - ref).abs() / lim).max())
    print(f"  {name}: worst error {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, name


def _proj(G, n_tok, n_in, n_out, out, pad_x=0, pad_y=0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(4000 + n_tok + 7 * n_in + 13 * n_out + seed)
    xb = torch.full((n_tok, n_in + pad_x), float("nan"), dtype=BF, device="cuda")
    xb[:, :n_in] = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, n_in, gen)
    # rows past the call's own hold NaN scales: reading them would show
    codes = torch.cat((codes, torch.full((8, n_in // 2), 0x77, dtype=torch.uint8, device="cuda")))
    scales = torch.cat((scales, torch.full((8, n_in // 32), 255, dtype=torch.uint8, device="cuda")))
    yb = torch.full((n_tok + 2, n_out + pad_y), 7.0, dtype=out, device="cuda")
    y = yb[:n_tok, :n_out]
    y.fill_(float("nan"))
    nb = G.mx_proj_workspace_bytes(n_tok, n_in, n_out)
    ws = torch.full((nb // 4,), float("nan"), device="cuda") if nb else None
    x = xb[:, :n_in]
    G.mx_proj(x, codes, scales, y, workspace=ws)
    torch.cuda.synchronize()
    ref, mag = _product(x, _unpack(codes[:n_out], scales[:n_out]))
    # every addition rounds once, in any order: n_in roundings of at most the products' magnitudes
    _close(f"y {n_tok}x{n_in}x{n_out}", y, ref, n_in * U * mag)
    assert (yb[n_tok:] == 7.0).all() and (yb[:, n_out:] == 7.0).all()
    return x, codes, scales, y, ws


@pytest.mark.parametrize("n_tok", [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("n_in,n_out,out", [(96, 70, BF), (2048, 272, F32), (4096, 64, BF), (1056, 1001, F32)])
def test_proj(G, n_tok, n_in, n_out, out):
    _proj(G, n_tok, n_in, n_out, out)


@pytest.mark.parametrize("n_tok,n_in,n_out,out", [
    (1, 32, 1, F32), (1, 32, 1, BF), (3, 64, 2, BF), (16, 128, 16, BF), (5, 8192, 33, F32), (40, 160, 15, BF),
    (1, 16384, 48, BF), (70, 12288, 130, BF), (64, 32, 4096, BF), (600, 2048, 1000, BF), (513, 96, 257, F32),
    (1000, 64, 520, BF), (1030, 1184, 515, F32), (2100, 2048, 768, BF), (4097, 224, 264, F32),
    (700, 2080, 300, BF), (777, 4096, 512, F32), (1, 2048, 12352, BF), (64, 4096, 2048, BF), (500, 2048, 2113, F32),
])
def test_proj_sizes(G, n_tok, n_in, n_out, out):
    _proj(G, n_tok, n_in, n_out, out)


@pytest.mark.parametrize("n_tok,n_out", [(1, 48), (3, 50), (33, 256), (90, 100), (300, 300), (600, 515)])
@pytest.mark.parametrize("pad_x,pad_y", [(8, 0), (0, 3), (64, 8)])
def test_proj_strides(G, n_tok, n_out, pad_x, pad_y):
    _proj(G, n_tok, 160, n_out, BF, pad_x, pad_y)
    _proj(G, n_tok, 160, n_out, F32, pad_x, pad_y)


@pytest.mark.parametrize("n_tok", [1, 20, 64, 200, 700])
def test_proj_nan_stays_in_its_row_and_channel(G, n_tok):
    """A group whose scale byte is 255 makes its own channel NaN, a token with
    a NaN its own row; everything else is untouched."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    n_in, n_out = 256, 300
    codes, scales = _weights(n_out, n_in, gen)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    good = torch.empty(n_tok, n_out, device="cuda")
    nb = G.mx_proj_workspace_bytes(n_tok, n_in, n_out)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
    G.mx_proj(x, codes, scales, good, workspace=ws)
    scales[17, 3] = 255
    x[n_tok - 1, 100] = float("nan")
    y = torch.empty_like(good)
    G.mx_proj(x, codes, scales, y, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isnan(y[:, 17]).all() and torch.isnan(y[n_tok - 1]).all()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[:, 17] = False
    keep[n_tok - 1] = False
    assert torch.equal(y[keep], good[keep])


@pytest.mark.parametrize("n_tok", [1, 37, 64, 200, 600])
def test_proj_repeats_bitwise_and_on_another_stream(G, n_tok):
    x, codes, scales, y, ws = _proj(G, n_tok, 2048, 640, F32)
    st = torch.cuda.Stream()
    y2, y3 = torch.empty_like(y), torch.empty_like(y)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        G.mx_proj(x, codes, scales, y2, workspace=ws)
    st.synchronize()
    G.mx_proj(x, codes, scales, y3, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)


def test_proj_refusals(G):
    b = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
    good = (t(3, 64), b(10, 32), b(10, 2), t(3, 10))
    G.mx_proj(*good)
    for i, bad in ((0, t(3, 64, dt=F32)), (0, t(2, 64)), (0, t(3, 128)[:, ::2]), (1, b(9, 32)), (2, b(9, 2)),
                   (1, t(10, 32)), (3, t(3, 10, dt=torch.float16)), (3, t(2, 10))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            G.mx_proj(*args)
    with pytest.raises(G.GdnError):
        G.mx_proj(t(3, 48), b(10, 24), b(10, 2), t(3, 10))
    with pytest.raises(G.GdnError):
        G.mx_proj(t(3, 68)[:, :64], *good[1:])
    G.mx_proj(t(0, 64), b(10, 32), b(10, 2), t(0, 10))


def _in_proj(G, n_tok, hidden, h_k, h_v, d, out, with_z, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(6000 + n_tok + hidden + d + seed)
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16 if out == BF else G.GDN_F32))
    c, v0 = h_k * d, h_v * d
    widths = [c, c, v0] + ([v0] if with_z else []) + [h_v, h_v]
    n_out = sum(widths)
    x = torch.randn(n_tok, hidden, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, hidden, gen)
    scales -= 2   # gates in the range where they move
    nan = float("nan")
    bufs = {"q": torch.full((n_tok, h_k, d), nan, dtype=out, device="cuda"),
            "k": torch.full((n_tok, h_k, d), nan, dtype=out, device="cuda"),
            "v": torch.full((n_tok, h_v, d), nan, dtype=out, device="cuda"),
            "z": torch.full((n_tok, h_v, d), nan, dtype=out, device="cuda") if with_z else None,
            "a": torch.full((n_tok, h_v), nan, device="cuda"), "b": torch.full((n_tok, h_v), nan, device="cuda")}
    nb = pool.mx_in_proj_workspace_bytes(n_tok, hidden, with_z)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda") if nb else None
    pool.mx_in_proj(x, codes, scales, bufs["q"], bufs["k"], bufs["v"], bufs["a"], bufs["b"], z=bufs["z"],
                    workspace=ws)
    torch.cuda.synchronize()
    y, mag = _product(x, _unpack(codes, scales))
    bound = hidden * U * mag
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
@pytest.mark.parametrize("n_tok,hidden,h_k,h_v,d,out", [
    (1, 2048, 16, 32, 128, BF), (64, 2048, 16, 32, 128, BF), (7, 96, 2, 2, 32, F32), (70, 160, 1, 3, 64, BF),
    (130, 256, 1, 1, 32, F32), (300, 1024, 2, 6, 64, BF), (700, 96, 2, 4, 64, F32), (600, 2048, 1, 2, 128, BF),
    (1100, 512, 4, 8, 128, BF), (1, 32, 1, 1, 32, F32),
])
def test_in_proj(G, n_tok, hidden, h_k, h_v, d, out, with_z):
    _in_proj(G, n_tok, hidden, h_k, h_v, d, out, with_z)


def test_in_proj_refusals(G):
    pool = G.Pool(G.make_desc(1, 1, 1, 2, 32, 32, 4, G.GDN_BF16))
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
    b = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    n = 4 * 32 + 2 * 32 + 4
    good = [t(3, 64), b(n, 32), b(n, 2), t(3, 1, 32), t(3, 1, 32), t(3, 2, 32), t(3, 2, dt=F32), t(3, 2, dt=F32)]
    z = t(3, 2, 32)
    pool.mx_in_proj(*good, z=z)
    pool.mx_in_proj(*good)            # without z fewer rows are read
    for i, bad in ((0, t(3, 64, dt=F32)), (1, b(n - 1, 32)), (2, b(n - 1, 2)), (3, t(2, 1, 32)), (5, t(3, 1, 32)),
                   (6, t(3, 2)), (7, t(3, 1, dt=F32))):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            pool.mx_in_proj(*args, z=z)
    with pytest.raises(ValueError):
        pool.mx_in_proj(*good, z=t(3, 1, 32))
    with pytest.raises(G.GdnError):
        pool.mx_in_proj(t(3, 48), *good[1:], z=z)

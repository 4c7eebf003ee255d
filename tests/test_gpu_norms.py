"""GPU: the block norm and the gated head norm against their formulas in
float64, with bounds counted from the roundings the kernels make."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24                     # one fp32 rounding
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
# A row's sum of squares: at most 32 terms one after the other in a lane, six
# steps across the wave, 16 waves; its square root halves the relative error,
# and the mean, eps, root, quotient and products add a few roundings more.
NORM = 40 * U


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _close(name, got, ref, bound):
    """|got - ref| within bound plus the rounding to got's own type."""
    assert torch.isfinite(got).all(), name
    err = (got.double() - ref).abs()
    lim = bound + STEP[got.dtype] * (ref.abs() + bound) + 1e-37
    worst = float((err / lim).max()) if err.numel() else 0.0
    print(f"  {name}: worst error {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, name


def _padded(shape, dtype, pad, gen, scale=1.0, fill=None):
    """A [rows, cols] view with `pad` more elements between rows, and its whole buffer."""
    rows, cols = shape
    buf = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
    view = buf[:, :cols]
    if fill is None:
        view.copy_(torch.randn(shape, generator=gen, device="cuda") * scale)
    else:
        view.fill_(fill)
    return view, buf


def _block_norm_case(G, n, h, io, res, add, post, pad=0, in_place=False, w_offset=1.0, res_scale=0.75,
                     eps=1e-6, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(1000 + 31 * n + h + seed)
    r, r_buf = _padded((n, h), res, pad, gen, scale=3.0 * scale)
    w = torch.randn(h, generator=gen, device="cuda") * 0.2
    x, x_buf = _padded((n, h), io, pad, gen, fill=float("nan"))
    kw = {}
    if add:
        y, y_buf = _padded((n, h), io, pad, gen, scale=scale)
        ro, ro_buf = (r, r_buf) if in_place else _padded((n, h), res, pad, gen, fill=float("nan"))
        kw = dict(y=y, residual_out=ro, res_scale=res_scale)
        if post:
            kw["w_post"] = 1.0 + 0.2 * torch.randn(h, generator=gen, device="cuda")
    r0 = r.double().clone()
    u = y.double().clone() if add else None
    if in_place and add:
        x, x_buf = y, y_buf
    G.block_norm(r, w, x, w_offset=w_offset, eps=eps, **kw)
    torch.cuda.synchronize()
    s, e = r0, torch.zeros_like(r0)
    if add:
        cu = 3 * U
        if post:
            u = kw["w_post"].double() * u / (u.square().mean(1, keepdim=True) + eps).sqrt()
            cu = NORM + 4 * U
        s = r0 + res_scale * u
        e = U * s.abs() + cu * (res_scale * u).abs()
        _close("residual_out", kw["residual_out"], s, e)
    inv = 1.0 / (s.square().mean(1, keepdim=True) + eps).sqrt()
    g = w_offset + w.double()
    ref = s * inv * g
    # the sum's own error moves the row's norm by at most its largest relative error
    rel = (e.square().mean(1, keepdim=True)).sqrt() * inv
    _close("x", x, ref, e * inv * g.abs() + (NORM + 2 * U + rel) * ref.abs() + 2 * U * (s * inv).abs())
    if pad:
        for b in {id(t): t for t in ([r_buf, x_buf] + ([y_buf, ro_buf] if add else []))}.values():
            assert (b[:, h:] == 7.0).all(), "padding between rows was written"


@pytest.mark.parametrize("n,h,io,res,add,post", [
    (1, 1, F32, F32, True, False), (3, 7, BF, F32, True, True), (1, 8, BF, BF, True, False),
    (2, 63, F32, BF, False, False), (5, 64, BF, BF, True, True), (1, 2048, BF, BF, True, False),
    (1, 2048, BF, BF, False, False), (33, 2048, BF, F32, True, True), (7, 2047, BF, BF, True, True),
    (4, 2049, F32, F32, True, False), (3, 2056, BF, F32, True, True), (2, 4095, BF, F32, True, False),
    (3, 4096, F32, F32, True, True), (2, 8192, BF, BF, True, True), (2, 8193, F32, BF, True, True),
    (2, 8200, BF, BF, True, False), (2, 16384, BF, F32, True, True), (1, 16383, F32, F32, True, True),
    (1000, 512, BF, BF, True, False), (2111, 96, BF, F32, True, True), (4100, 40, F32, F32, True, True),
])
def test_block_norm(G, n, h, io, res, add, post):
    _block_norm_case(G, n, h, io, res, add, post)


@pytest.mark.parametrize("h,pad", [(64, 8), (64, 3), (63, 1), (2048, 16), (2048, 5), (5000, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_norm_strides_and_in_place(G, h, pad, in_place):
    _block_norm_case(G, 6, h, BF, F32, True, True, pad=pad, in_place=in_place)
    _block_norm_case(G, 6, h, F32, F32, True, False, pad=pad, in_place=in_place)


def test_block_norm_rows_apart_from_each_other(G):
    """A row of zeros (its norm is 1/sqrt(eps)), one of tiny and one of huge
    values, and one with an infinity and a NaN, next to ordinary rows."""
    n, h = 8, 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = torch.randn(n, h, generator=gen, device="cuda")
    r[1] = 0.0
    r[2] *= 1e-18
    r[3] *= 1e17
    r[5, 7] = float("inf")
    r[6, 200] = float("nan")
    w = torch.ones(h, device="cuda")
    x = torch.empty_like(r)
    G.block_norm(r, w, x)
    torch.cuda.synchronize()
    good = [0, 1, 2, 3, 4, 7]
    rd = r[good].double()
    ref = rd / (rd.square().mean(1, keepdim=True) + 1e-6).sqrt()
    _close("finite rows", x[good], ref, NORM * ref.abs() + 1e-30)
    assert (x[1] == 0).all()
    assert torch.isnan(x[6]).all() and torch.isnan(x[5, 7]) and (x[5, :7] == 0).all()


def test_block_norm_alignment_of_the_first_element(G):
    """Operands whose first element is not 16-byte aligned take the element path."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    base = torch.randn(3 * 64 + 1, generator=gen, device="cuda").to(BF)
    r = base[1:].view(3, 64)
    w = torch.ones(64, device="cuda")
    x = torch.empty(3, 64, dtype=BF, device="cuda")
    G.block_norm(r, w, x)
    ref = r.double() / (r.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    _close("x", x, ref, (NORM + 2 * U) * ref.abs())


def _pool(G, h_v, d, io):
    return G.Pool(G.make_desc(1, 1, 1, h_v, d, d, 4, G.GDN_BF16 if io == BF else G.GDN_F32))


@pytest.mark.parametrize("n,h_v,d,io,out", [
    (1, 1, 32, BF, BF), (1, 32, 128, BF, BF), (3, 5, 64, F32, BF), (17, 3, 32, F32, F32),
    (64, 32, 128, BF, F32), (333, 7, 64, BF, BF), (129, 48, 128, F32, F32), (2000, 2, 32, BF, BF),
])
@pytest.mark.parametrize("strided", [False, True])
def test_gated_norm(G, n, h_v, d, io, out, strided):
    gen = torch.Generator(device="cuda").manual_seed(77 + n + d)
    pool = _pool(G, h_v, d, io)
    width, pad = h_v * d, 24 if strided else 0

    def make(dtype, scale):
        buf = torch.full((n, width + pad), 7.0, dtype=dtype, device="cuda")
        buf[:, :width] = (torch.randn(n, width, generator=gen, device="cuda") * scale).to(dtype)
        return buf, buf[:, :width].unflatten(1, (h_v, d))

    (_, o), (_, z), (out_buf, y) = make(io, 2.0), make(io, 3.0), make(out, 1.0)
    w = 1.0 + 0.2 * torch.randn(d, generator=gen, device="cuda")
    pool.gated_norm(o, z, w, y, eps=1e-5)
    torch.cuda.synchronize()
    od, zd = o.double(), z.double()
    ref = od / (od.square().mean(2, keepdim=True) + 1e-5).sqrt() * w.double() * zd * torch.sigmoid(zd)
    # the norm: 12 terms and steps, halved, and 6 roundings; the gate: the exponential's
    # argument carries |z| log2(e) roundings, its result and the quotient a few more
    _close("out", y, ref, (12 + 2 * zd.abs() + 8) * U * ref.abs())
    if strided:
        assert (out_buf[:, width:] == 7.0).all()


def test_gated_norm_edges(G):
    """Heads of zeros, gates far from zero on both sides, and a head with a
    NaN beside clean ones; out in place of o."""
    h_v, d = 4, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    pool = _pool(G, h_v, d, F32)
    o = torch.randn(3, h_v, d, generator=gen, device="cuda")
    z = torch.randn(3, h_v, d, generator=gen, device="cuda")
    o[0, 1] = 0.0
    z[1, 0, :8] = 200.0
    z[1, 0, 8:16] = -200.0
    o[2, 3, 5] = float("nan")
    w = torch.ones(d, device="cuda")
    od, zd = o.double(), z.double()
    ref = od / (od.square().mean(2, keepdim=True) + 1e-6).sqrt() * zd * torch.sigmoid(zd)
    pool.gated_norm(o, z, w, o)
    torch.cuda.synchronize()
    assert (o[0, 1] == 0).all()
    assert torch.isnan(o[2, 3]).all()
    clean = torch.ones(3, h_v, dtype=torch.bool, device="cuda")
    clean[2, 3] = False
    _close("out", o[clean], ref[clean], ((12 + 2 * zd.abs() + 8) * U * ref.abs())[clean])


def test_gated_norm_refusals(G):
    pool = _pool(G, 2, 32, BF)
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
    w = t(32, dt=F32)
    good = (t(3, 2, 32), t(3, 2, 32), w, t(3, 2, 32))
    pool.gated_norm(*good)
    for i, bad in ((0, t(3, 2, 32, dt=F32)), (1, t(2, 2, 32)), (1, t(3, 2, 64)), (2, w[:31]),
                   (3, t(3, 2, 32, dt=torch.float16)), (3, t(3, 3, 32)), (0, t(3, 2, 64)[:, :, ::2])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            pool.gated_norm(*args)
    with pytest.raises(G.GdnError):   # token stride not a multiple of 8
        pool.gated_norm(t(3, 68)[:, :64].unflatten(1, (2, 32)), *good[1:])
    with pytest.raises(G.GdnError):   # first element not 16-byte aligned
        pool.gated_norm(t(3 * 64 + 8).view(-1)[4:-4].view(3, 2, 32), *good[1:])
    with pytest.raises(G.GdnError):
        pool.gated_norm(*good, eps=-1.0)
    empty = t(0, 2, 32)
    pool.gated_norm(empty, empty, w, empty)


def test_block_norm_refusals(G):
    t = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")
    r, w, x = t(3, 64), t(64, dt=F32), t(3, 64)
    for args, kw in (
            ((r, w[:63], x), {}), ((r, w.bfloat16(), x), {}), ((r, w, t(3, 63)), {}), ((r, w, t(2, 64)), {}),
            ((r, w, x), {"y": t(3, 64)}), ((r, w, x), {"residual_out": t(3, 64)}), ((r, w, x), {"w_post": w}),
            ((r, w, x), {"y": t(3, 64, dt=F32), "residual_out": t(3, 64)}),
            ((r, w, x), {"y": t(3, 64), "residual_out": t(3, 64, dt=F32)}),
            ((t(3, 128)[:, ::2], w, x), {})):
        with pytest.raises(ValueError):
            G.block_norm(*args, **kw)
    with pytest.raises(G.GdnError):
        G.block_norm(t(1, 16385), t(16385, dt=F32), t(1, 16385))
    G.block_norm(t(0, 64), w, t(0, 64))

"""GPU: the projections with 4-bit weights where their kernels take different
paths: few tokens, tiles of both kinds, the 8-bit split of the tokens; values
of very different size in one group, infinities, NaN scales next to clean
rows, and operands past 2^31 elements."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# tokens, inputs, channels, results: one to four tokens, few, many with few
# channels, and tiles with and without the split; inputs end inside a pair of
# 64 and inside 64
PATHS = [(1, 2048, 300, BF), (4, 1056, 70, F32), (19, 2080, 300, BF), (300, 4096, 64, BF), (50, 64, 200, F32),
         (700, 544, 1500, BF), (700, 2080, 3000, BF), (2600, 1184, 2050, BF), (700, 544, 3000, F32),
         (5000, 96, 700, BF)]


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _weights(n_out, n_in, seed, lo=118, hi=128):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = torch.randint(lo, hi, (n_out, n_in // 32), generator=gen, device="cuda").to(torch.uint8)
    return codes, scales


def _decode(codes, scales):
    c, s = codes.long(), scales.long()
    idx = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)
    v = torch.where(idx >= 8, -1.0, 1.0).double() * LEVELS.to(c.device)[idx & 7]
    scale = torch.where(s == 255, torch.nan, torch.ldexp(torch.ones((), dtype=torch.float64, device=c.device),
                                                         (s - 127).double()))
    return v * scale.repeat_interleave(32, 1)


def _call(G, x, codes, scales, out):
    y = torch.full((x.shape[0], codes.shape[0]), 77.0, dtype=out, device="cuda")
    n = G.mx_proj_workspace_bytes(x.shape[0], x.shape[1], codes.shape[0])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    G.mx_proj(x, codes, scales, y, workspace=ws)
    torch.cuda.synchronize()
    return y


def _mm(a, b):
    return torch.mm(a, b.t().contiguous())


def _check(name, y, x, w):
    """n_in roundings of at most the products' magnitudes; the split leaves out
    at most 2^-22 of a group's largest value from each of its values."""
    xd, n_in = x.double(), x.shape[1]
    ref, mag = _mm(xd, w), _mm(xd.abs(), w.abs())
    top = xd.abs().reshape(x.shape[0], -1, 32).amax(-1).repeat_interleave(32, 1)
    bound = n_in * U * mag + 2.0 ** -22 * _mm(top, w.abs())
    lim = bound + STEP[y.dtype] * (ref.abs() + bound) + 1e-37
    worst = float(((y.double() - ref).abs() / lim).max())
    print(f"  {name}: worst error {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, name


@pytest.mark.parametrize("n_tok,n_in,n_out,out", PATHS)
def test_values_of_every_size(G, n_tok, n_in, n_out, out):
    """Tokens whose values differ by factors up to 2^24 inside a group, one of
    zeros, one of subnormal bf16 and one close to its largest values."""
    gen = torch.Generator(device="cuda").manual_seed(n_tok + n_in)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda")
    x *= torch.exp2(-24 * torch.rand(n_tok, n_in, generator=gen, device="cuda"))
    codes, scales = _weights(n_out, n_in, n_in)
    if n_tok > 3:
        x[1] = 0.0
        x[2] *= 2.0 ** -126
        x[3] = x[3].clamp(-2, 2) * 2.0 ** 125
    x = x.to(BF)
    w = _decode(codes, scales)
    y = _call(G, x, codes, scales, out)
    rows = torch.ones(n_tok, dtype=torch.bool, device="cuda")
    if n_tok > 3:
        assert (y[1] == 0).all()
        assert (y[2].double() - _mm(x[2:3].double(), w)[0]).abs().max() < 2.0 ** -126
        # products and sums past the largest value of either type become infinite in both
        rows[2] = rows[3] = False
        big = _mm(x[3:4].double() * 2.0 ** -40, w)[0]
        got = _call(G, (x[3:4].double() * 2.0 ** -40).to(BF).expand(n_tok, n_in).contiguous(), codes, scales, out)
        lim = n_in * U * _mm(x[3:4].double().abs() * 2.0 ** -40, w.abs())[0]
        assert ((got[0].double() - big).abs() <= lim + STEP[out] * (big.abs() + lim) + 2.0 ** 85 * 2.0 ** -22 * 2 *
                w.abs().sum(1)).all()
    _check("wide values", y[rows], x[rows], w)


@pytest.mark.parametrize("n_tok,n_in,n_out,out", PATHS)
def test_infinities_follow_the_products(G, n_tok, n_in, n_out, out):
    """A token with infinities has the products' infinities and NaN (an
    infinity times a zero weight, opposite infinities); one with a NaN has only
    NaN; the other tokens are what they are without them."""
    gen = torch.Generator(device="cuda").manual_seed(n_tok + n_out)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, n_in, n_out)
    clean = _call(G, x, codes, scales, out)
    bad = [0, n_tok // 2, n_tok - 1] if n_tok > 3 else [0]
    x[bad[0], n_in - 3] = float("inf")
    if n_tok > 3:
        x[bad[1], 5], x[bad[1], 7] = float("inf"), float("-inf")
        x[bad[2], 1], x[bad[2], 40] = float("nan"), float("inf")
    y = _call(G, x, codes, scales, out)
    # the definition, with a clean column sum kept apart: only the infinite products decide
    w = _decode(codes, scales)
    for t in bad:
        xt = x[t].double()
        special = torch.nonzero(~torch.isfinite(xt)).flatten()
        want = (xt[special].unsqueeze(0) * w[:, special]).sum(1)
        same = (torch.isnan(want) & torch.isnan(y[t])) | (want == y[t].double())
        assert bool(same.all()), t
    keep = torch.ones(n_tok, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("n_tok,n_in,n_out,out", PATHS)
def test_marked_groups_stay_in_their_channel(G, n_tok, n_in, n_out, out):
    """Scale byte 255 in the first and the last group of single channels."""
    gen = torch.Generator(device="cuda").manual_seed(n_tok)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, n_in, 3)
    clean = _call(G, x, codes, scales, out)
    marked = [0, 17, n_out // 2, n_out - 1]
    for i, c in enumerate(marked):
        scales[c, 0 if i % 2 else -1] = 255
    y = _call(G, x, codes, scales, out)
    keep = torch.ones(n_out, dtype=torch.bool, device="cuda")
    keep[marked] = False
    assert torch.isnan(y[:, marked]).all()
    assert torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("n_tok", [2, 40, 900])
def test_in_proj_gates_of_an_infinite_token(G, n_tok):
    """An infinite logit is a gate of 0 or 1; the rest of the call is untouched."""
    h_k, h_v, d, hidden = 2, 4, 64, 1024
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16))
    n_out = 2 * h_k * d + 2 * h_v * d + 2 * h_v
    codes, scales = _weights(n_out, hidden, 11, 112, 122)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n_tok, hidden, generator=gen, device="cuda").to(BF)

    def call():
        e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        r = dict(q=e(n_tok, h_k, d), k=e(n_tok, h_k, d), v=e(n_tok, h_v, d), a=e(n_tok, h_v, dt=F32),
                 b=e(n_tok, h_v, dt=F32), z=e(n_tok, h_v, d))
        n = pool.mx_in_proj_workspace_bytes(n_tok, hidden)
        pool.mx_in_proj(x, codes, scales, **r, workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        return r

    clean = call()
    x[1, 33] = float("inf")
    got = call()
    w = _decode(codes, scales)[:, 33] * float("inf")
    parts = torch.split(w, [h_k * d, h_k * d, h_v * d, h_v * d, h_v, h_v])
    for name, want in zip(("q", "k", "v", "z", "a", "b"), parts):
        if name in "ab":
            want = torch.sigmoid(-want if name == "a" else want)
        y = got[name].reshape(n_tok, -1).double()
        assert bool(((torch.isnan(want) & torch.isnan(y[1])) | (want == y[1])).all()), name
        rest = [t for t in range(n_tok) if t != 1]
        assert torch.equal(got[name][rest], clean[name][rest]), name


def test_outputs_past_2_31_elements(G):
    n_tok, n_in, n_out = 4_200_000, 64, 520
    x = torch.zeros(n_tok, n_in, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(300, n_in, generator=gen, device="cuda").to(BF)
    x[-300:] = last
    codes, scales = _weights(n_out, n_in, 5)
    y = _call(G, x, codes, scales, BF)
    _check("last tokens", y[-300:], last, _decode(codes, scales))
    assert (y[: n_tok - 300: 1009] == 0).all()


@pytest.mark.parametrize("n_tok", [1, 130])
def test_weights_past_2_31_bytes(G, n_tok):
    """Quantised here too: a matrix of more than 2^32 weights."""
    rows, cols = 70_000, 65_536
    src = torch.zeros(rows, cols, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    src[-100:] = torch.randn(100, cols, generator=gen, device="cuda").to(BF)
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    G.mx_quantize(src, codes, scales)
    back = torch.empty(rows, cols, dtype=BF, device="cuda")
    G.mx_dequantize(codes, scales, back)
    torch.cuda.synchronize()
    w = _decode(codes[-100:], scales[-100:])
    assert torch.equal(back[-100:].double(), w)
    # every weight lies within its group's step: the largest step is 2 of 4 .. 6, saturation 2 of 8
    step = torch.exp2(scales[-100:].double() - 127).repeat_interleave(32, 1)
    assert bool(((src[-100:].double() - w).abs() <= 2 * step).all())
    x = torch.randn(n_tok, cols, generator=gen, device="cuda").to(BF)
    y = _call(G, x, codes, scales, F32)
    _check("last channels", y[:, -100:], x, w)
    assert (y[:, : rows - 100] == 0).all()

"""GPU: what the projections with 4-bit weights hold their sums in.  Inputs are
chosen so that every partial sum, in any order, is a whole number of units
below 2^24: sums held in 32 bits then give the exact result, so it is compared
for equality, in fp32 as it is and in bf16 rounded once.  And on ordinary
inputs a bf16 result is the fp32 result of the same call, rounded."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# tokens, inputs, channels: one token, few, many into few channels, and many
# into many, with inputs that end inside 64 and inside 128 and odd widths
SIZES = [(1, 2048, 300), (4, 1056, 70), (64, 4096, 256), (200, 4096, 64), (50, 64, 200), (500, 2048, 2113),
         (700, 2080, 3000), (700, 544, 1500), (1000, 512, 2050), (2600, 1184, 2050), (3000, 512, 2050),
         (2000, 512, 8200), (700, 512, 8200)]


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _weights(n_out, n_in, gen, lo, hi):
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = torch.randint(lo, hi, (n_out, n_in // 32), generator=gen, device="cuda").to(torch.uint8)
    return codes, scales


def _decode(codes, scales):
    idx = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).long()
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=codes.device)
    return table[idx] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _call(G, x, codes, scales, out):
    y = torch.full((x.shape[0], codes.shape[0]), 77.0, dtype=out, device="cuda")
    n = G.mx_proj_workspace_bytes(x.shape[0], x.shape[1], codes.shape[0])
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if n else None
    G.mx_proj(x, codes, scales, y, workspace=ws)
    torch.cuda.synchronize()
    return y


def _whole(n_tok, n_in, gen):
    """Tokens of up to eight significant bits, whole multiples of 2^-4 up to 255."""
    m = torch.randint(-255, 256, (n_tok, n_in), generator=gen, device="cuda").double()
    x = m * torch.exp2(-torch.randint(0, 5, (n_tok, n_in), generator=gen, device="cuda").double())
    assert torch.equal(x.to(BF).double(), x)
    return x


def _exact(x, w, unit):
    """x W^T, exact: the sums of magnitudes stay below 2^24 units."""
    assert float(torch.mm(x.abs(), w.abs().t().contiguous()).max()) < 2 ** 24 * unit
    return torch.mm(x, w.t().contiguous())


def _count(y, want):
    bad = int((y.double() != want).sum())
    print(f"  {bad} of {y.numel()} results differ", flush=True)
    return bad


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_sums_in_32_bits(G, n_tok, n_in, n_out, out):
    gen = torch.Generator(device="cuda").manual_seed(n_tok + n_in)
    codes, scales = _weights(n_out, n_in, gen, 127, 128)
    x = _whole(n_tok, n_in, gen)
    want = _exact(x, _decode(codes, scales), 2.0 ** -5)
    assert _count(_call(G, x.to(BF), codes, scales, out), want.to(out).double()) == 0


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_small_values_beside_an_outlier(G, n_tok, n_in, n_out, out):
    """Each group of a token holds one value 2^16 above the others, where the
    weights are zero: it takes nothing from the others' products."""
    gen = torch.Generator(device="cuda").manual_seed(n_tok + n_out)
    codes, scales = _weights(n_out, n_in, gen, 127, 128)
    codes[:, 3::16] &= 0xF0                                  # weight 6 of every group
    x = _whole(n_tok, n_in, gen)
    x[:, 6::32] = 255.0 * 2 ** 16
    w = _decode(codes, scales)
    assert (w[:, 6::32] == 0).all()
    want = _exact(x, w, 2.0 ** -5)
    assert _count(_call(G, x.to(BF), codes, scales, out), want.to(out).double()) == 0


@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_bf16_is_the_rounded_fp32_result(G, n_tok, n_in, n_out):
    gen = torch.Generator(device="cuda").manual_seed(n_in + n_out)
    codes, scales = _weights(n_out, n_in, gen, 118, 128)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda")
    x[:, 5] *= 100.0                                         # a channel of outliers
    x = x.to(BF)
    full, half = _call(G, x, codes, scales, F32), _call(G, x, codes, scales, BF)
    assert _count(half, full.to(BF).double()) == 0


def test_in_proj_sums_in_32_bits(G):
    """Through the layer's in-projection: q, k, v and z."""
    h_k, h_v, d, hidden, n_tok = 4, 8, 128, 512, 1100
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16))
    gen = torch.Generator(device="cuda").manual_seed(12)
    widths = [h_k * d, h_k * d, h_v * d, h_v * d, h_v, h_v]
    codes, scales = _weights(sum(widths), hidden, gen, 127, 128)
    x = _whole(n_tok, hidden, gen)
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    r = dict(q=e(n_tok, h_k, d), k=e(n_tok, h_k, d), v=e(n_tok, h_v, d), a=e(n_tok, h_v, dt=F32),
             b=e(n_tok, h_v, dt=F32), z=e(n_tok, h_v, d))
    n = pool.mx_in_proj_workspace_bytes(n_tok, hidden)
    pool.mx_in_proj(x.to(BF), codes, scales, **r, workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    want = torch.split(_exact(x, _decode(codes, scales), 2.0 ** -5), widths, 1)
    for name, y in zip("qkvz", want):
        assert _count(r[name].reshape(n_tok, -1), y.to(BF).double()) == 0, name


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("scale", [127, 187])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_subnormal_tokens(G, n_tok, n_in, n_out, scale, out):
    """Tokens below the smallest normal bf16 value are multiplied as they are."""
    gen = torch.Generator(device="cuda").manual_seed(n_tok + scale)
    codes, scales = _weights(n_out, n_in, gen, scale, scale + 1)
    m = torch.randint(-127, 128, (n_tok, n_in), generator=gen, device="cuda").double()
    x = (m * 2.0 ** -133).to(BF)
    assert torch.equal(x.double(), m * 2.0 ** -133)
    want = _exact(m, _decode(codes, scales), 2.0 ** (scale - 128)) * 2.0 ** -133
    assert _count(_call(G, x, codes, scales, out), want.to(out).double()) == 0

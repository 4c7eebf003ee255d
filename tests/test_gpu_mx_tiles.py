"""GPU: the tile kernels of the projections with 4-bit weights, at sizes that
the launch rule is known to send there (tests/mx_plan.py): strides, marked
groups, infinities and NaN, repeats, a second stream, gates, and graphs, one of
them with the kernels' first use inside the capture.

Where values are compared for equality, inputs are such that every partial
sum, in any order, is a whole number of units below 2^24, so the fp32 sum is
exact."""
import importlib.util
import os
import subprocess
import sys

import pytest

from mx_plan import TILE_CASES, TILE_IN_PROJ, in_proj_channels, paths

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SIZES = [c[:3] for c in TILE_CASES]


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(n_out, n_in, gen, scale=127):
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    return codes, torch.full((n_out, n_in // 32), scale, dtype=torch.uint8, device="cuda")


def _decode(codes, scales):
    idx = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).long()
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float64, device=codes.device)
    return table[idx] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _whole(n_tok, n_in, gen):
    """Tokens of up to eight significant bits, whole multiples of 2^-4 up to 255."""
    m = torch.randint(-255, 256, (n_tok, n_in), generator=gen, device="cuda").double()
    return m * torch.exp2(-torch.randint(0, 5, (n_tok, n_in), generator=gen, device="cuda").double())


def _exact(x, w, unit):
    assert float(torch.mm(x.abs(), w.abs().t().contiguous()).max()) < 2 ** 24 * unit
    return torch.mm(x, w.t().contiguous())


def _same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("pad_x,pad_y", [(0, 0), (8, 0), (64, 8), (8, 3)])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_strides(G, n_tok, n_in, n_out, pad_x, pad_y, out):
    """Padding between the tokens' rows holds NaN and is not read, between the
    results' rows a mark that stays."""
    gen = _gen(n_tok + n_out + pad_x)
    codes, scales = _weights(n_out, n_in, gen)
    x = _whole(n_tok, n_in, gen)
    want = _exact(x, _decode(codes, scales), 2.0 ** -5).to(out)
    xb = torch.full((n_tok, n_in + pad_x), float("nan"), dtype=BF, device="cuda")
    xb[:, :n_in] = x.to(BF)
    yb = torch.full((n_tok + 2, n_out + pad_y), 7.0, dtype=out, device="cuda")
    yb[:n_tok, :n_out] = float("nan")
    # rows past the call's own hold NaN scales: reading them would show
    codes = torch.cat((codes, torch.full((8, n_in // 2), 0x77, dtype=torch.uint8, device="cuda")))
    scales = torch.cat((scales, torch.full((8, n_in // 32), 255, dtype=torch.uint8, device="cuda")))
    G.mx_proj(xb[:, :n_in], codes, scales, yb[:n_tok, :n_out])
    torch.cuda.synchronize()
    assert torch.equal(yb[:n_tok, :n_out], want)
    assert (yb[n_tok:] == 7.0).all() and (yb[:, n_out:] == 7.0).all()


@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_results_between_dwords(G, n_tok, n_in, n_out):
    """Results whose first element lies between dwords, and weights' scale
    bytes at an odd address."""
    gen = _gen(n_in)
    codes, scales = _weights(n_out, n_in, gen)
    x = _whole(n_tok, n_in, gen)
    want = _exact(x, _decode(codes, scales), 2.0 ** -5).to(BF)
    y = torch.empty(n_tok * n_out + 1, dtype=BF, device="cuda")[1:].view(n_tok, n_out)
    odd = torch.empty(scales.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(scales.shape)
    odd.copy_(scales)
    G.mx_proj(x.to(BF), codes, odd, y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_marked_groups_and_special_tokens(G, n_tok, n_in, n_out, out):
    """A scale byte of 255 makes its channel NaN, a NaN its token; infinities
    follow the products; everything else is what it is without them."""
    gen = _gen(n_out)
    codes, scales = _weights(n_out, n_in, gen)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    clean, y = (torch.empty(n_tok, n_out, dtype=out, device="cuda") for _ in "ab")
    G.mx_proj(x, codes, scales, clean)
    w = _decode(codes, scales)
    marked = [0, 17, n_out // 2, n_out - 1]
    for i, c in enumerate(marked):
        scales[c, 0 if i % 2 else -1] = 255
    special = [0, n_tok // 2, n_tok - 1]
    x[0, n_in - 3] = float("inf")
    x[n_tok // 2, 5], x[n_tok // 2, 7] = float("inf"), float("-inf")
    x[n_tok - 1, 1], x[n_tok - 1, 40] = float("nan"), float("inf")
    G.mx_proj(x, codes, scales, y)
    assert torch.isnan(y[:, marked]).all() and torch.isnan(y[n_tok - 1]).all()
    rest = torch.ones(n_out, dtype=torch.bool, device="cuda")
    rest[marked] = False
    for t in special[:2]:
        k = torch.nonzero(~torch.isfinite(x[t])).flatten()
        assert _same(y[t, rest].double(), (x[t, k].double() * w[:, k]).sum(1)[rest])
    rows = torch.ones(n_tok, dtype=torch.bool, device="cuda")
    rows[special] = False
    assert torch.equal(y[rows][:, rest], clean[rows][:, rest])


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("n_tok,n_in,n_out", SIZES)
def test_repeats_bitwise_and_on_another_stream(G, n_tok, n_in, n_out, out):
    gen = _gen(7)
    codes, scales = _weights(n_out, n_in, gen, 120)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    y = [torch.full((n_tok, n_out), float("nan"), dtype=out, device="cuda") for _ in range(4)]
    G.mx_proj(x, codes, scales, y[0])
    G.mx_proj(x, codes, scales, y[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        G.mx_proj(x, codes, scales, y[2])
    G.mx_proj(x, codes, scales, y[3], stream=st)
    st.synchronize()
    assert torch.isfinite(y[0]).all()
    for other in y[1:]:
        assert torch.equal(y[0], other)


@pytest.mark.parametrize("n_tok,hidden,h_k,h_v,d", [c[:5] for c in TILE_IN_PROJ])
def test_in_proj_outputs_and_gates(G, n_tok, hidden, h_k, h_v, d):
    """q, k, v and z exactly; the gates, of exact logits, to their activation's
    roundings; an infinite token's logits are gates of 0 or 1 (NaN where the
    weight is zero), and the other tokens are untouched."""
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16))
    gen = _gen(hidden)
    widths = [h_k * d, h_k * d, h_v * d, h_v * d, h_v, h_v]
    assert sum(widths) == in_proj_channels(h_k, h_v, d)
    codes, scales = _weights(sum(widths), hidden, gen)
    scales[-2 * h_v:] = 116                                  # logits in the range where gates move
    x = _whole(n_tok, hidden, gen)
    w = _decode(codes, scales)
    y = torch.split(torch.cat((_exact(x, w[:-2 * h_v], 2.0 ** -5), _exact(x, w[-2 * h_v:], 2.0 ** -16)), 1), widths, 1)
    x = x.to(BF)

    def call():
        e = lambda *s, dt=BF: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
        r = dict(q=e(n_tok, h_k, d), k=e(n_tok, h_k, d), v=e(n_tok, h_v, d), a=e(n_tok, h_v, dt=F32),
                 b=e(n_tok, h_v, dt=F32), z=e(n_tok, h_v, d))
        pool.mx_in_proj(x, codes, scales, **r)
        torch.cuda.synchronize()
        return {n: t.reshape(n_tok, -1) for n, t in r.items()}

    got = call()
    for name, want in zip("qkvz", y):
        assert torch.equal(got[name], want.to(BF)), name
    for name, logit in zip("ab", y[4:]):
        ref = torch.sigmoid(-logit if name == "a" else logit)
        # exponential (an ulp or two), sum and quotient
        worst = float(((got[name].double() - ref).abs() / (8 * U * ref + 1e-37)).max())
        print(f"  gate {name}: worst error {worst:.3f} of the bound", flush=True)
        assert worst <= 1.0
    t = n_tok // 2
    x[t, 33] = float("inf")
    after = call()
    inf = torch.split(w[:, 33] * float("inf"), widths)
    for name, want in zip("qkvzab", inf):
        if name in "ab":
            want = torch.sigmoid(-want if name == "a" else want)
        assert _same(after[name][t].double(), want), name
        keep = [i for i in range(n_tok) if i != t]
        assert torch.equal(after[name][keep], got[name][keep]), name


def test_a_captured_decode_step_takes_the_tiles(G):
    """1100 tokens a step through two blocks, replayed against eager steps."""
    n, hidden, h_k, h_v, d = 1100, 512, 4, 8, 128
    assert paths(n, hidden, in_proj_channels(h_k, h_v, d)) == ["tile128"]
    spec = importlib.util.spec_from_file_location("gdn_stack", os.path.join(ROOT, "examples", "gdn_stack.py"))
    E = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(E)
    a, b = (E.random_stack(2, hidden, h_k, h_v, d, n_slots=n, seed=9) for _ in "ab")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    r_in = torch.zeros(n, hidden, device="cuda")
    r_a, r_b = torch.empty_like(r_in), torch.empty_like(r_in)
    buf_a, buf_b = E.Buffers(a, n, 0), E.Buffers(b, n, 0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        r_a.copy_(r_in)
        a.decode(r_a, slots, buf_a)
    gen = _gen(n)
    for t in range(4):
        r_in.copy_(torch.randn(n, hidden, generator=gen, device="cuda"))
        graph.replay()
        r_b.copy_(r_in)
        b.decode(r_b, slots, buf_b)
        torch.cuda.synchronize()
        assert torch.equal(buf_a.x, buf_b.x) and torch.equal(r_a, r_b), f"replay {t}"
    assert torch.equal(a.pool.state, b.pool.state) and bool(torch.isfinite(buf_b.x).all())


FIRST_USE = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import gated_deltanet_state_layer_amd as G
g = torch.Generator(device="cuda").manual_seed(3)
calls = []
for n_tok, n_in, n_out, out in ((700, 512, 8200, torch.bfloat16), (700, 544, 1500, torch.float32)):
    x = torch.zeros(n_tok, n_in, dtype=torch.bfloat16, device="cuda")
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 128, (n_out, n_in // 32), generator=g, device="cuda").to(torch.uint8)
    y, eager = (torch.empty(n_tok, n_out, dtype=out, device="cuda") for _ in "ab")
    calls.append((x, codes, scales, y, eager))
torch.cuda.synchronize()
graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=side):
    for x, codes, scales, y, _ in calls:
        G.mx_proj(x, codes, scales, y)
for replay in range(4):
    for x, *_ in calls:
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    graph.replay()
    for x, codes, scales, y, eager in calls:
        G.mx_proj(x, codes, scales, eager)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and bool(torch.isfinite(y).all()) and bool((y != 0).any()), replay
print("replays equal")
"""


def test_first_use_inside_a_capture(G):
    """A process of its own, whose first call of the kernels is recorded."""
    assert paths(700, 512, 8200) == ["tile192", "strip"] and paths(700, 544, 1500) == ["tile128"]
    r = subprocess.run([sys.executable, "-c", FIRST_USE, ROOT], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "replays equal" in r.stdout, r.stdout + r.stderr

"""GPU: beam selection where scores of different beams are equal or nearly so, and
rows whose distribution is (almost) certain: the order, and scores to their rounding.

Scores are sums in 64 bits, rounded to 41 before they are compared.  What is exact on
the host here is exact by arithmetic: a row with one token left adds 0 to its beam."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NONE = -math.inf


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _select(G, x, scores, k, finished=None, eos=-1):
    r, w, v = x.shape
    parents, tokens = (torch.full((r, k), 99, dtype=torch.int32, device="cuda") for _ in "ab")
    out = torch.full((r, k), math.nan, device="cuda")
    fin = None if finished is None else torch.full((r, k), 9, dtype=torch.uint8, device="cuda")
    ws = torch.full((G.beam_select_workspace_bytes(r, w, v, k),), 255, dtype=torch.uint8, device="cuda")
    G.beam_select(x, scores.cuda(), parents, tokens, out, finished=finished, finished_out=fin, eos=eos, workspace=ws)
    torch.cuda.synchronize()
    return parents.cpu(), tokens.cpu(), out.cpu()


# short rows, rows of several stretches, and (512 rows of bf16) rows by the table
SIZES = [(250, 8, 600), (20, 8, 20011), (64, 8, 33001)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v", SIZES)
def test_one_token_left_keeps_the_score(G, r, w, v, dtype):
    """Beams of equal score whose rows have one token left each: all stay equal, bit
    for bit, so the lower beam comes first."""
    g = torch.Generator().manual_seed(v)
    x = torch.full((r, w, v), NONE, dtype=dtype, device="cuda")
    at = torch.randint(0, v, (r, w), generator=g)
    logit = torch.randn(r, w, generator=g) * 3 + 8
    logit[0] = 1.0e-5 * torch.randn(w, generator=g)
    logit[1] = -300.0 * torch.rand(w, generator=g)
    logit[2] = 1.0e6 * torch.randn(w, generator=g)
    logit[3], logit[4] = 0.0, torch.finfo(dtype).max
    x.scatter_(2, at[..., None].cuda(), logit[..., None].to(dtype).cuda())
    scores = (-8 * torch.rand(r, 1, generator=g)).expand(r, w).contiguous()
    scores[5], scores[6] = 0.0, -1.0e-6
    for k in (w, 3, 12):
        parents, tokens, out = _select(G, x, scores, k)
        n = min(k, w)
        assert (parents[:, :n] == torch.arange(n)).all() and (parents[:, n:] == -1).all(), k
        assert torch.equal(tokens[:, :n], at[:, :n].int()) and (tokens[:, n:] == -1).all(), k
        assert torch.equal(out[:, :n], scores[:, :n]) and (out[:, n:] == NONE).all(), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v", SIZES)
def test_one_token_left_beside_finished_beams(G, r, w, v, dtype):
    """As good as a finished beam of the same score: the lower beam comes first."""
    g = torch.Generator().manual_seed(v + 1)
    x = torch.full((r, w, v), NONE, dtype=dtype, device="cuda")
    at = torch.randint(0, v, (r, w), generator=g)
    x.scatter_(2, at[..., None].cuda(), (torch.randn(r, w, 1, generator=g) * 3 + 8).to(dtype).cuda())
    finished = torch.randint(0, 2, (r, w), generator=g).to(torch.uint8)
    scores = (-8 * torch.rand(r, 1, generator=g)).expand(r, w).contiguous()
    parents, tokens, out = _select(G, x, scores, w, finished.cuda(), 7)
    assert (parents == torch.arange(w)).all() and torch.equal(out, scores)
    assert torch.equal(tokens, torch.where(finished.bool(), 7, at.int()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v", SIZES)
def test_nearly_certain_rows(G, r, w, v, dtype):
    """One logit far above the rest: the best score is -log1p of what the rest adds.
    No probability is above 1."""
    g = torch.Generator().manual_seed(v + 2)
    x = torch.randn(r, w, v, generator=g).clamp(-4, 4).to(dtype)
    lead = torch.linspace(8, 60, r * w).view(r, w, 1)
    at = torch.randint(0, v, (r, w, 1), generator=g)
    x.scatter_(2, at, lead.to(dtype))
    rest = x.double().scatter(2, at, NONE)
    want = -torch.log1p(torch.exp(rest - x.double().gather(2, at)).sum(-1))
    for b in range(w):
        parents, tokens, out = _select(G, x[:, b:b + 1].cuda(), torch.zeros(r, 1), 1)
        got, ref = out[:, 0].double(), want[:, b]
        assert (got <= 0).all() and (parents == 0).all() and torch.equal(tokens[:, 0], at[:, b, 0].int())
        # rounded to fp32; a sum of v terms above 1 in fp64, each addition half a step
        lim = ref.abs() * (2.0 ** -24 + 2.0 ** -40) + v * 2.0 ** -53
        assert ((got - ref).abs() <= lim).all(), float(((got - ref).abs() / lim).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v", SIZES)
def test_shifted_rows_are_equal(G, r, w, v, dtype):
    """Rows that differ by a constant have equal distributions.  Logits are eighths
    below 32, exact in either type, so the definition gives equal scores; where that
    score is nearer than 2^-47 of itself (64 times what fp64 sums leave) to the border
    between two numbers of 41 bits, the request does not count."""
    g = torch.Generator().manual_seed(v + 3)
    levels = torch.randint(-96, 97, (r, 1, v), generator=g)
    levels[:, :, :8] = torch.arange(97, 105)   # the best ones, all different
    shift = 8 * torch.randint(-17, 18, (r, w, 1), generator=g)
    x = ((levels + shift) / 8.0).to(dtype)
    assert torch.equal(x.double() * 8, (levels + shift).double())
    row = levels[:, 0].double() / 8
    base = -8 * torch.rand(r, 1, generator=g).double()
    base = base.float().double()
    score = base + (row[:, :8] - row.amax(1, keepdim=True)) - torch.log(
        torch.exp(row - row.amax(1, keepdim=True)).sum(1, keepdim=True))
    frac, _ = torch.frexp(score.abs())
    border = ((frac * 2.0 ** 41 % 1.0) - 0.5).abs() * 2.0 ** -41 / frac
    clear = (border >= 2.0 ** -47).all(1)
    assert clear.float().mean() > 0.5
    k = min(64, 8 * w)
    parents, tokens, out = _select(G, x.cuda(), base.float().expand(r, w).contiguous(), k)
    assert torch.equal(parents[clear], (torch.arange(k) % w).int().expand(r, k)[clear])
    assert torch.equal(tokens[clear], (7 - torch.arange(k) // w).int().expand(r, k)[clear])
    assert torch.equal(out[clear][:, ::w], out[clear][:, w - 1::w])
    ref = score.flip(1)[:, torch.arange(k) // w]
    assert ((out.double() - ref).abs() <= ref.abs() * (2.0 ** -24 + 2.0 ** -40) + v * 2.0 ** -53).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v", SIZES)
def test_scores_equal_in_41_bits(G, r, w, v, dtype):
    """Every other beam has a second token that takes 2^-44.7 of the probability:
    in 41 bits that leaves the beam's score, a number of 24, as it was."""
    g = torch.Generator().manual_seed(v + 4)
    x = torch.full((r, w, v), NONE, dtype=dtype, device="cuda")
    best = torch.randint(0, 9, (r, w, 1), generator=g) / 4.0
    at = torch.randint(0, v // 2, (r, w, 1), generator=g)
    x.scatter_(2, at.cuda(), best.to(dtype).cuda())
    second = torch.where(torch.arange(w)[None, :, None] % 2 == 0, best - 31.0, NONE)
    assert torch.equal(second, second.to(dtype).float())
    x.scatter_(2, v // 2 + at.cuda(), second.to(dtype).cuda())
    scores = (16 * torch.rand(r, 1, generator=g) - 8).expand(r, w).contiguous()
    scores = torch.where(scores.abs() < 0.25, 1.0, scores)     # from 0.25 on, half a step of 41 bits is 2^-43 or more
    parents, tokens, out = _select(G, x, scores, w)
    assert (parents == torch.arange(w)).all() and torch.equal(tokens, at[..., 0].int())
    assert torch.equal(out, scores)


@pytest.mark.parametrize("base", [-8.123, -0.3, -100.0])
def test_scores_fall_where_they_lie_close(G, base):
    """64 beams whose scores lie around a border between two fp32 numbers, closer than
    2^-40 of their size: what comes out never rises."""
    base = float(torch.tensor(base))
    up = abs(base) * 2.0 ** -22
    for seed in range(8):
        g = torch.Generator().manual_seed(seed)
        # the second token takes a fraction of about `up` of the sum; neighbouring fp32 logits
        # change it by 1e-6 of that
        lead = math.log(1 / up)
        second = torch.full((64,), -lead)
        for i in range(1, 64):
            second[i] = torch.nextafter(second[i - 1], torch.tensor(-math.inf if seed % 2 else math.inf))
        second = second[torch.randperm(64, generator=g)] if seed > 3 else second
        x = torch.stack((torch.zeros(64), second), 1)[None]
        parents, _, out = _select(G, x.cuda(), torch.full((1, 64), base), 64)
        assert (out[:, :-1] >= out[:, 1:]).all(), seed
        exact = (base - torch.log1p(torch.exp(second.double())))[parents[0].long()]
        # 41 bits: half a step each, and what fp64 leaves
        assert (exact[:-1] - exact[1:] >= -abs(base) * (2.0 ** -40 + 2.0 ** -50)).all(), seed

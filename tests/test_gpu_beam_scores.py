"""GPU: beam selection where scores of different beams are equal or nearly so, and
rows whose distribution is (almost) certain: the order, and scores to their rounding.

Scores are sums in 64 bits.  What is exact on the host here is exact by arithmetic: a
row with one token left adds 0 to its beam."""
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

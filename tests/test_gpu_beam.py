"""GPU: beam selection against its definition in float64 on the host: parents
and tokens exactly, scores to their rounding."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
BIG = torch.finfo(F32).max


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _reference(logits, scores, finished, eos, k):
    """Entries (score, beam, logit, token) of one request, best first."""
    x = logits.cpu().double()
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=BIG)
    entries = []
    for b in range(x.shape[0]):
        base = float(scores[b])
        if not math.isfinite(base):
            continue
        if finished is not None and int(finished[b]):
            entries.append((base, b, 0.0, eos))
            continue
        row = x[b]
        if not bool((row > -math.inf).any()):
            continue
        top = float(row.max())          # apart from the logarithm: beside 1e38 that would be lost
        log_sum = math.log(float(torch.exp(row - top).sum()))
        kth = row.topk(min(k, row.numel())).values[-1]
        at = torch.nonzero((row >= kth) & (row > -math.inf)).flatten()
        best = sorted(((-float(row[t]), int(t)) for t in at))[:k]
        entries += [(base + ((-nx - top) - log_sum), b, -nx, t) for nx, t in best]
    return sorted(entries, key=lambda e: (-e[0], e[1], -e[2], e[3]))[:k]


def _check(G, logits, scores, k, finished=None, eos=-1, name=""):
    r, w, v = logits.shape
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    i32 = lambda: torch.full((r, k), 99, dtype=torch.int32, device="cuda")  # noqa: E731
    parents, tokens, out = i32(), i32(), torch.full((r, k), math.nan, device="cuda")
    fin_out = torch.full((r, k), 9, dtype=torch.uint8, device="cuda") if eos >= 0 else None
    ws = torch.full((G.beam_select_workspace_bytes(r, w, v, k) + 64,), 255, dtype=torch.uint8, device="cuda")
    G.beam_select(logits, dev(scores), parents, tokens, out, finished=dev(finished), finished_out=fin_out, eos=eos,
                  workspace=ws[:-64])
    torch.cuda.synchronize()
    assert (ws[-64:] == 255).all()
    for q in range(r):
        ref = _reference(logits[q], scores[q].tolist(), None if finished is None else finished[q], eos, k)
        pad = k - len(ref)
        where = f"{name} request {q}"
        assert parents[q].tolist() == [e[1] for e in ref] + [-1] * pad, where
        assert tokens[q].tolist() == [e[3] for e in ref] + [-1] * pad, where
        got = out[q].cpu().double()
        assert (got[len(ref):] == -math.inf).all(), where
        for g, e in zip(got.tolist(), ref):
            # a rounding to fp32; sums of v terms in fp64 and the exponential's 1.1e-12
            lim = 2.0 ** -24 * abs(e[0]) + v * 2.0 ** -53 + 2e-12 + 2.0 ** -50 * abs(e[2])
            assert g == e[0] or abs(g - e[0]) <= lim or (abs(e[0]) > BIG and math.isinf(g)), (where, g, e)
        if fin_out is not None:
            want = [int(e[3] == eos or (finished is not None and bool(finished[q][e[1]]))) for e in ref]
            assert fin_out[q].tolist() == want + [0] * pad, where


def _logits(gen, r, w, v, dtype, scale=2.5):
    return (torch.randn(r, w, v, generator=gen, device="cuda") * scale).to(dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,w,v,k", [
    (1, 1, 1, 1), (1, 1, 1, 4), (2, 3, 2, 6), (1, 4, 7, 64), (3, 2, 511, 5), (2, 2, 512, 2), (2, 3, 513, 8),
    (1, 4, 1000, 4), (2, 5, 4099, 10), (1, 64, 700, 64), (1, 16, 33000, 32), (2, 1, 50001, 1), (1, 2, 131072, 64),
    (70, 2, 1030, 3), (300, 4, 515, 4), (1, 9, 65537, 18),
])
def test_selection(G, r, w, v, k, dtype):
    gen = _gen(r + w + v + k)
    scores = -torch.rand(r, w, generator=torch.Generator().manual_seed(v)) * 8
    _check(G, _logits(gen, r, w, v, dtype), scores, k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [40, 1536, 20000])
def test_ties_go_to_the_lower_token_and_beam(G, v, dtype):
    """Few distinct logits, beams alike bit for bit."""
    gen = _gen(v)
    x = torch.randint(-3, 3, (2, 1, v), generator=gen, device="cuda").to(dtype)
    _check(G, x.expand(2, 6, v).contiguous(), torch.zeros(2, 6), 16, name="alike")
    _check(G, x.expand(2, 6, v).contiguous(), torch.zeros(2, 6), 64, name="alike, many")
    _check(G, torch.zeros(1, 3, v, dtype=dtype, device="cuda"), torch.tensor([[-1.0, -1.0, 0.0]]), 20, name="equal")
    y = torch.zeros(1, 2, v, dtype=dtype, device="cuda")
    y[0, 0, ::2] = -0.0
    z = -torch.rand(1, 2, v, device="cuda") - 0.1
    z[0, 0, 3:9] = 0.0
    z[0, 1, 5:33] = -0.0
    _check(G, z.to(dtype), torch.tensor([[0.0, -5.0]]), 24, name="zeros on top")
    _check(G, y, torch.tensor([[0.0, -5.0]]), 30, name="zeros of both signs")


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_equal_logits_far_apart_in_a_long_row(G, seed):
    """Equal bf16 logits among the best, from different stretches of a row."""
    gen = _gen(seed)
    x = _logits(gen, 32, 8, 40000, BF)
    _check(G, x, -torch.rand(32, 8, generator=torch.Generator().manual_seed(seed)) * 8, 16)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [33001, 70000])
def test_many_long_rows_of_every_kind(G, v, dtype):
    """Enough rows that a workgroup takes a long stretch: logits of many sizes,
    zeros, tiny ones, far ones early and late in a row, masks, infinities and NaN."""
    gen = _gen(v)
    x = _logits(gen, 66, 8, v, F32)
    x[0] *= 1.0e-6
    x[1] *= 2.0e-4
    x[2] *= 20.0
    x[3] *= 300.0
    x[4] -= 30.0
    x[5] -= 90.0
    x[6] += 70.0
    x[7, :, ::2] = 0.0
    x[8, :, 100:] = -0.0
    x[9, :, v - 3] = 64.0
    x[10, :, v - 3] = 700.0
    x[11, :, v // 2] = -700.0
    x[12, :, 5000:] = -math.inf
    x[13, :, :5000] = -math.inf
    x[14, :, 7::5] = math.nan
    x[15, :, v - 9] = math.inf
    x[16] = -math.inf
    x[17, :, ::3] = torch.finfo(dtype).min
    x[18] = -19.0 - x[18].abs()
    x[19] = -20.5 - x[19].abs()
    x[20, :, :20000] -= 1000.0
    x[21, :, 20000:] += 1000.0
    x[22] *= 1.0e30
    x[23] = 2.0 ** -13
    x[24] = -63.9
    x[25, :, 1:] = -64.0
    _check(G, x.to(dtype), -torch.rand(66, 8, generator=torch.Generator().manual_seed(v)) * 8, 8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("k", [1, 5, 64])
def test_rising_and_falling_rows(G, dtype, k):
    """Every element of a rising row beats those before it."""
    v = 5000
    up = torch.arange(v, device="cuda").float().mul(0.001)
    x = torch.stack((up, up.flip(0), torch.cat((up[::2], up[1::2]))))[None].to(dtype)
    _check(G, x, torch.tensor([[0.0, -0.5, -0.25]]), k)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_rows_infinities_and_nan(G, dtype):
    gen = _gen(4)
    v, low = 1200, torch.finfo(dtype).min
    x = _logits(gen, 1, 8, v, dtype)
    x[0, 0] = -math.inf                       # nothing left
    x[0, 1] = low                             # masked with the lowest value: all alike
    x[0, 2, 1:] = -math.inf                   # one token left
    x[0, 3, :600] = -math.inf                 # the first steps are empty
    x[0, 4, 5] = math.inf
    x[0, 4, 900] = math.inf
    x[0, 5, 10:20] = math.nan
    x[0, 6] = math.nan
    x[0, 7, :] = low
    x[0, 7, 1100] = 0.0
    scores = -torch.arange(8.0)[None]
    for k in (1, 3, 40, 64):
        _check(G, x, scores, k, name=f"k {k}")
        for b in range(8):
            _check(G, x[:, b:b + 1].contiguous(), scores[:, b:b + 1], k, name=f"beam {b} alone, k {k}")
    _check(G, torch.full((2, 3, v), -math.inf, dtype=dtype, device="cuda"), torch.zeros(2, 3), 4, name="none")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wide_values(G, dtype):
    """Logits that leave the exponential's range, also late in a row."""
    gen = _gen(5)
    x = _logits(gen, 2, 3, 9000, dtype)
    x[0, 0, 8000] = 1.0e4
    x[0, 1] *= 1.0e30
    x[0, 2, ::3] = -3.0e38
    x[1, 0] = x[1, 0] * 300.0
    x[1, 1] = torch.linspace(-2.0e4, 2.0e4, 9000, device="cuda").to(dtype)
    x[1, 2] = 1.0e-30
    _check(G, x, torch.tensor([[0.0, -1.0, -2.0], [-3.0, 5.0, 1.0e5]]), 12)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dead_and_finished_beams(G, dtype):
    gen = _gen(6)
    x = _logits(gen, 3, 4, 3001, dtype)
    scores = torch.tensor([[0.0, -math.inf, -math.inf, -math.inf], [-1.0, -2.0, math.nan, -0.5], [-math.inf] * 4])
    _check(G, x, scores, 4, name="first step")
    fin = torch.tensor([[0, 1, 1, 0], [1, 0, 1, 1], [1, 1, 0, 0]], dtype=torch.uint8)
    _check(G, x, scores, 7, fin, 2, name="some finished")
    _check(G, x, torch.zeros(3, 4), 7, torch.ones(3, 4, dtype=torch.uint8), 3000, name="all finished")
    x[:, :, 17] = 30.0
    _check(G, x, -torch.rand(3, 4), 8, fin, 17, name="eos chosen")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_and_unaligned_rows(G, dtype):
    gen = _gen(7)
    for v, pad in ((1000, 1), (1001, 6), (513, 15)):
        buf = torch.full((6 * (v + pad) + 1,), 1.0e9, dtype=dtype, device="cuda")   # what lies between the rows would win
        x = buf[1:].view(2, 3, v + pad)[:, :, :v]
        x.copy_(_logits(gen, 2, 3, v, dtype))
        _check(G, x, -torch.rand(2, 3), 9)


def test_close_scores_of_different_beams_are_ordered(G):
    """Scores a few 1e-9 apart, far below fp32's resolution."""
    gen = _gen(8)
    x = _logits(gen, 1, 1, 2000, F32, 1.0).expand(1, 5, 2000).contiguous()
    t = int(x[0, 0].argmax())
    for b, e in enumerate((3.0, 1.0, 2.0, 0.0, 4.0)):
        # moves the sum a little: another token, rare, gains e * 1e-9 of it
        x[0, b, 7 if t != 7 else 8] = math.log(1e-9 * (e + 1) * float(torch.logsumexp(x[0, 4].double(), 0).exp()))
    _check(G, x, torch.zeros(1, 5), 10)


def test_repeats_on_another_stream_and_in_a_graph(G):
    gen = _gen(9)
    r, w, v, k = 4, 3, 20011, 6
    x = torch.empty(r, w, v, dtype=BF, device="cuda")
    scores = torch.zeros(r, w, device="cuda")
    outs = [torch.empty(r, k, dtype=d, device="cuda") for d in (torch.int32, torch.int32, F32)]
    eager = [torch.empty_like(o) for o in outs]
    ws, ws2 = (torch.empty(G.beam_select_workspace_bytes(r, w, v, k), dtype=torch.uint8, device="cuda") for _ in "ab")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        G.beam_select(x, scores, *outs, workspace=ws)
    for t in range(4):
        x.copy_(_logits(gen, r, w, v, BF))
        scores.copy_(-torch.rand(r, w))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            G.beam_select(x, scores, *eager, workspace=ws2)
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), t


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_far_apart(G, dtype):
    """Two rows more than 2^31 elements from each other."""
    v, k, ld = 50001, 9, 2 ** 31 + 17
    buf = torch.empty(ld + v, dtype=dtype, device="cuda")
    x = buf.as_strided((2, 1, v), (ld, ld, 1))
    near = _logits(_gen(10), 2, 1, v, dtype).cuda()
    x.copy_(near)
    scores = torch.zeros(2, 1, device="cuda")
    ws = torch.empty(G.beam_select_workspace_bytes(2, 1, v, k), dtype=torch.uint8, device="cuda")
    got = []
    for logits in (x, near):
        outs = [torch.empty(2, k, dtype=d, device="cuda") for d in (torch.int32, torch.int32, F32)]
        G.beam_select(logits, scores, *outs, workspace=ws)
        got.append(outs)
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)

"""GPU: beam selection by the kernel with the table of exponentials, which takes
bf16 rows where each workgroup has eight steps or more: every number of results, rows
of one stretch and of several, beams without continuations, ties, unaligned rows."""
import math

import pytest

torch = pytest.importorskip("torch")
from test_gpu_beam import BF, G, _check, _gen, _logits  # noqa: E402,F401

pytestmark = pytest.mark.gpu
STEP = 8 * 64 * 8        # logits that a workgroup of eight waves takes in a step


def _stretches(rows, vocab):
    """Stretches of a row by the kernel with the table; 0 where another takes the call:
    512 workgroups in all, at most 64 to a row, eight steps or more to each."""
    steps = -(-vocab // STEP)
    want = max(1, min(64, steps, 512 // max(1, rows)))
    per = -(-steps // want)
    return -(-steps // per) if per >= 8 else 0


def _scores(r, w, seed):
    return -torch.rand(r, w, generator=torch.Generator().manual_seed(seed)) * 8


@pytest.mark.parametrize("k", [1, 2, 3, 16, 33, 64])
@pytest.mark.parametrize("r,w,v,stretches", [(64, 8, 33001, 1), (16, 8, 131072, 4), (2, 64, 118785, 4), (40, 4, 100000, 3),
                                             (1, 8, 2 ** 21 - 3, 64)])
def test_every_number_of_results(G, r, w, v, stretches, k):
    assert _stretches(r * w, v) == stretches
    _check(G, _logits(_gen(v + k), r, w, v, BF), _scores(r, w, v), k)


@pytest.mark.parametrize("r,w,v", [(64, 8, 33001), (16, 8, 131072)])
def test_finished_and_dead_beams(G, r, w, v):
    assert _stretches(r * w, v)
    g = torch.Generator().manual_seed(v)
    x, scores = _logits(_gen(v), r, w, v, BF), _scores(r, w, v)
    kind = torch.randint(0, 5, (r, w), generator=g)
    kind[0], kind[1], kind[2] = 1, 2, torch.arange(w) % 2
    scores[kind == 1] = -math.inf
    scores[kind == 3] = math.nan
    finished = ((kind == 2) | (torch.rand(r, w, generator=g) < 0.05)).to(torch.uint8)
    for k in (1, 16, 64):
        _check(G, x, scores, k, finished, 17, name=f"k {k}")


@pytest.mark.parametrize("r,w,v", [(64, 8, 33001), (16, 8, 131072), (128, 1, 118785)])
def test_ties_in_a_stretch_and_between_stretches(G, r, w, v):
    """Few distinct logits; in some rows one token of the best, first or last."""
    assert _stretches(r * w, v)
    x = torch.randint(-250, 4, (r, 1, v), generator=_gen(v), device="cuda").to(BF).expand(r, w, v).contiguous()
    x[0, :, v - 1], x[1, :, 0], x[2, :, v // 2] = 5.0, 5.0, 5.0
    x[3] = 0.0
    x[4, :, ::2] = -0.0
    for k in (1, 16, 64):
        _check(G, x, torch.zeros(r, w), k, name=f"k {k}")


@pytest.mark.parametrize("v,pad", [(33001, 1), (33000, 7), (40003, 6)])
def test_unaligned_rows(G, v, pad):
    r, w = 64, 8
    assert _stretches(r * w, v) == 1
    buf = torch.full((r * w * (v + pad) + 1,), 1.0e9, dtype=BF, device="cuda")   # what lies between the rows would win
    x = buf[1:].view(r, w, v + pad)[:, :, :v]
    x.copy_(_logits(_gen(v), r, w, v, BF))
    _check(G, x, _scores(r, w, v), 9)


@pytest.mark.parametrize("r,w,v", [(64, 8, 33001), (16, 8, 131072)])
def test_rows_that_leave_the_table(G, r, w, v):
    """Logits past the table's range early, late, in one wave or in one stretch; masks,
    infinities and NaN in the first step and behind it."""
    assert _stretches(r * w, v)
    x = _logits(_gen(v + 1), r, w, v, torch.float32)
    x[0, :, :STEP] = -math.inf
    x[1, :, 512:1024] = 100.0
    x[2, :, STEP + 600] = 64.0
    x[3, :, v - 1] = 63.75
    x[4, :, v // 2:] += 200.0
    x[5, :, :v // 2] -= 200.0
    x[6, :, 5:STEP - 5] = math.nan
    x[7, :, ::7] = math.inf
    x[8, :, STEP:] = -math.inf
    x[9, :, 1:] = -math.inf
    x[10, :, :v - 1] = -math.inf
    x[11] = torch.finfo(BF).min
    x[12, :, ::2] = torch.finfo(BF).min
    x[13] -= 25.0
    x[14, :, 64 * 8:] -= 25.0
    x[15] = x[15] * 1.0e-6
    for k in (1, 16, 64):
        _check(G, x.to(BF), _scores(r, w, v), k, name=f"k {k}")

"""GPU: adapters in the tile kernels of the projections with 4-bit weights, at every
way the rows of B take through LDS (beside the first blocks up to rank 64, into the
stages behind the main loop above), with many adapters to a tile and guard words
behind the workspace."""
import pytest

from mx_plan import TILE_CASES, TILE_IN_PROJ, in_proj_channels, paths, plan

torch = pytest.importorskip("torch")
from test_gpu_lora import BF, F32, G, STEP, U, _adapters, _close, _ids, _reference, _weights  # noqa: E402,F401

pytestmark = pytest.mark.gpu
GUARD = 4096


def _guarded(nbytes):
    """A workspace of NaN with guard bytes behind it."""
    buf = torch.full(((nbytes + GUARD) // 4,), float("nan"), device="cuda")
    assert nbytes % 4 == 0
    buf[nbytes // 4:] = 7.0
    return buf[:nbytes // 4], buf[nbytes // 4:]


def _run(G, n_tok, n_in, n_out, rank, n, kind, out):
    gen = torch.Generator(device="cuda").manual_seed(n_tok + 3 * n_in + 5 * n_out + 7 * rank + 11 * n)
    x = torch.randn(n_tok, n_in, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, n_in, gen)
    a, b, s = _adapters(n, rank, n_in, n_out, gen)
    ids = _ids(n_tok, n, kind, gen)
    y = torch.full((n_tok, n_out), float("nan"), dtype=out, device="cuda")
    ws, behind = _guarded(G.mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank))
    G.mx_proj_lora(x, codes, scales, a, b, s, ids, y, workspace=ws)
    torch.cuda.synchronize()
    ref, bound = _reference(x, codes, scales, a, b, s, ids)
    _close(f"y {n_tok}x{n_in}x{n_out} rank {rank} {kind} {paths(n_tok, n_in, n_out)}", y, ref, bound)
    assert (behind == 7.0).all()
    off = (ids < 0) | (ids >= n)
    if bool(off.any()):
        plain = torch.empty_like(y)
        G.mx_proj(x, codes, scales, plain)
        assert torch.equal(y[off], plain[off])


@pytest.mark.parametrize("rank", [8, 56, 64, 72, 120, 128])
@pytest.mark.parametrize("n_tok,n_in,n_out,want", TILE_CASES)
def test_every_rank_on_tiles(G, n_tok, n_in, n_out, want, rank):
    assert paths(n_tok, n_in, n_out) == want and plan(n_tok, n_in, n_out)[0].tile
    for out in (BF, F32):
        _run(G, n_tok, n_in, n_out, rank, 2, "one", out)
        _run(G, n_tok, n_in, n_out, rank, 5, "mixed", out)


@pytest.mark.parametrize("rank,n", [(8, 300), (16, 64), (40, 130), (128, 64)])
@pytest.mark.parametrize("n_tok,n_in,n_out", [(128, 2048, 12352), (200, 1056, 12352), (500, 1184, 12353)])
def test_many_adapters_to_a_tile(G, n_tok, n_in, n_out, rank, n):
    """A decode batch with an adapter each, more of them than tokens or fewer."""
    assert plan(n_tok, n_in, n_out)[0].tile
    _run(G, n_tok, n_in, n_out, rank, n, "each", BF)
    _run(G, n_tok, n_in, n_out, rank, n, "mixed", F32)


@pytest.mark.parametrize("rank", [64, 72, 128])
@pytest.mark.parametrize("n_tok,hidden,h_k,h_v,d,want", TILE_IN_PROJ)
def test_in_proj_of_high_ranks_on_tiles(G, n_tok, hidden, h_k, h_v, d, want, rank):
    n_out, n = in_proj_channels(h_k, h_v, d), 20
    assert paths(n_tok, hidden, n_out) == want
    gen = torch.Generator(device="cuda").manual_seed(n_tok + rank)
    pool = G.Pool(G.make_desc(1, 1, h_k, h_v, d, d, 4, G.GDN_BF16))
    x = torch.randn(n_tok, hidden, generator=gen, device="cuda").to(BF)
    codes, scales = _weights(n_out, hidden, gen)
    a, b, s = _adapters(n, rank, hidden, n_out, gen)
    ids = _ids(n_tok, n, "mixed", gen)
    full = lambda *sh, dt=BF: torch.full(sh, float("nan"), dtype=dt, device="cuda")  # noqa: E731
    outs = {"q": full(n_tok, h_k, d), "k": full(n_tok, h_k, d), "v": full(n_tok, h_v, d), "z": full(n_tok, h_v, d),
            "a": full(n_tok, h_v, dt=F32), "b": full(n_tok, h_v, dt=F32)}
    ws, behind = _guarded(pool.mx_in_proj_lora_workspace_bytes(n_tok, hidden, rank))
    pool.mx_in_proj_lora(x, codes, scales, a, b, s, ids, *(outs[o] for o in "qkvab"), z=outs["z"], workspace=ws)
    torch.cuda.synchronize()
    y, bound = _reference(x, codes, scales, a, b, s, ids)
    at = 0
    for name in "qkvzab":
        got = outs[name].reshape(n_tok, -1)
        r, e = y[:, at:at + got.shape[1]], bound[:, at:at + got.shape[1]]
        at += got.shape[1]
        if name in "ab":   # slope at most 1/4; exponential, sum and quotient round
            r = torch.sigmoid(-r if name == "a" else r)
            e = 0.25 * e + 8 * U * r
        _close(name, got, r, e)
    assert (behind == 7.0).all()


@pytest.mark.parametrize("rank", [8, 16, 128])
@pytest.mark.parametrize("n_tok,n_in,n_out", [(1, 4096, 2048), (5, 2048, 272), (48, 256, 300), (64, 2048, 12352),
                                              (700, 544, 1001)])
def test_the_workspace_is_enough_for_few_tokens(G, n_tok, n_in, n_out, rank):
    assert not plan(n_tok, n_in, n_out)[0].tile
    _run(G, n_tok, n_in, n_out, rank, 70, "each", BF)

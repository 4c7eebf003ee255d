"""The launches of the projections with 4-bit weights, on the host: they cover
the call, each channel once, and stay within what a launch may hold."""
import pytest

from mx_plan import TILE_CASES, TILE_IN_PROJ, fits, in_proj_channels, paths, plan

TOKENS = [1, 4, 5, 16, 17, 64, 129, 1000, 8192, 65537, (1 << 20) + 1, (1 << 24) + 3, 1 << 26, (1 << 27) - 1, 1 << 27,
          (1 << 27) + 1, 200_000_000, (1 << 28) - 65]
CHANNELS = [1, 15, 16, 17, 32, 33, 64, 65, 98, 128, 192, 1000, 12352, 65536, 1 << 20, (1 << 24) + 5, (1 << 27) + 1,
            (1 << 28) - 65]


@pytest.mark.parametrize("n_in", [32, 128, 256, 512, 2048, 1 << 20])
@pytest.mark.parametrize("n_tok", TOKENS)
def test_launches_cover_the_call_within_the_grid(n_tok, n_in):
    """Fewer than 2^32 threads (512 to a workgroup) each."""
    taken = 0
    for n_out in CHANNELS:
        if not fits(n_tok, n_out):
            continue
        taken += 1
        at = 0
        for p in plan(n_tok, n_in, n_out):
            assert p.c0 == at and p.c1 > at
            at = p.c1
            assert p.workgroups == -(-n_tok // p.tokens) * -(-(p.c1 - p.c0) // p.channels)
            assert 0 < p.workgroups * 512 < 1 << 32, (n_out, p)
        assert at == n_out
    assert taken or n_tok > (1 << 28) - 65


# The faster of both sides by measurement on the kernels as they are (bf16
# results): tokens, inputs, channels, the launches taken.  Left out are pairs
# within 6 % of each other.
@pytest.mark.parametrize("n_tok,n_in,n_out,want", [
    (96, 2048, 12352, ["skinny"]), (128, 2048, 12352, ["tile128"]), (160, 2048, 12352, ["tile128"]),
    (384, 2048, 12352, ["tile192"]), (500, 2048, 12352, ["tile192", "strip"]), (8192, 2048, 12352, ["tile192", "strip"]),
    (500, 4096, 2048, ["skinny"]), (1000, 4096, 2048, ["skinny"]), (1536, 4096, 2048, ["tile128"]),
    (500, 512, 2048, ["skinny"]), (1000, 512, 2048, ["tile128"]), (48, 128, 16384, ["tile128"]),
    (64, 128, 16384, ["tile128"]), (8192, 128, 16384, ["tile192"]),
])
def test_the_faster_kernels_are_taken(n_tok, n_in, n_out, want):
    assert paths(n_tok, n_in, n_out) == want


@pytest.mark.parametrize("n_tok,n_in,n_out,want", TILE_CASES)
def test_tile_cases_reach_the_tiles(n_tok, n_in, n_out, want):
    """The sizes that the GPU tests of the tile kernels rely on."""
    assert paths(n_tok, n_in, n_out) == want


@pytest.mark.parametrize("n_tok,hidden,h_k,h_v,d,want", TILE_IN_PROJ)
def test_tile_in_projections_reach_the_tiles(n_tok, hidden, h_k, h_v, d, want):
    assert paths(n_tok, hidden, in_proj_channels(h_k, h_v, d)) == want

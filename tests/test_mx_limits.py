"""Bounds and scratch sizes of the projections with 4-bit weights, on the host:
every launch of a call that is taken stays within the grid's limits."""
import ctypes

import pytest

pytest.importorskip("torch")
OK, UNSUPPORTED = 0, -2


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_state_layer_amd import binding
    return binding.load_library()


def _bytes(lib, n_tok, n_in, n_out):
    n = ctypes.c_size_t(123)
    return lib.gdn_mx_proj_workspace_bytes(n_tok, n_in, n_out, ctypes.byref(n)), n.value


@pytest.mark.parametrize("n_tok,n_out,status", [
    (0, 1, OK), (1, 1 << 27, OK), (1, 1 << 28, UNSUPPORTED), (1 << 27, 1, OK), (1 << 28, 1, UNSUPPORTED),
    (1 << 20, 1 << 14, UNSUPPORTED), (1 << 19, 1 << 14, OK), (1 << 62, 1, UNSUPPORTED),
])
def test_grid_bounds(lib, n_tok, n_out, status):
    assert _bytes(lib, n_tok, 512, n_out)[0] == status


def test_scratch_holds_the_split_or_nothing(lib):
    for n_tok in (0, 1, 4, 16, 64, 100, 500, 1000, 8192):
        for n_in in (32, 96, 480, 512, 544, 2048, 8192):
            for n_out in (1, 64, 2048, 12352):
                st, n = _bytes(lib, n_tok, n_in, n_out)
                pairs = (n_in + 127) // 128
                # hi and lo bytes of pairs of 64, four scale bytes a pair, a flag, rounded up to 256
                assert st == OK and (n == 0 or 0 <= n - n_tok * (pairs * 260 + 1) < 3 * 256)
                if n_tok <= 16 or n_in < 512:
                    assert n == 0

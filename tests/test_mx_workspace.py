"""Scratch of the projections with 4-bit weights, on the host: a workspace that
is enough for a call is enough for every call of fewer tokens, and a call's
size does not depend on whether its results are bf16."""
import ctypes

import pytest

pytest.importorskip("torch")


@pytest.mark.parametrize("n_in,n_out", [(8192, 1024), (2048, 12352), (4096, 2048), (512, 520)])
def test_scratch_grows_with_the_tokens(n_in, n_out):
    from gated_deltanet_state_layer_amd import binding
    lib = binding.load_library()
    n, most = ctypes.c_size_t(), 0
    for n_tok in range(0, 4200, 7):
        assert lib.gdn_mx_proj_workspace_bytes(n_tok, n_in, n_out, ctypes.byref(n)) == 0
        assert n.value >= most, n_tok
        most = n.value

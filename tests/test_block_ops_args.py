"""Refusals of the operators around the core (block norm, gated head norm,
4-bit weight format, projections with 4-bit weights), on the host: a bad
argument gives its status before anything is enqueued, and the binding refuses
tensors that do not fit before their pointers leave Python."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -4
NUL = None
A = 1 << 20          # never dereferenced: every call below is refused or empty


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_state_layer_amd import binding
    return binding.load_library()


NORM = dict(n_tok=2, hidden=64, io=1, res_t=0, y=A, ld_y=64, w_post=NUL, res_scale=1.0, res=A, ld_res=64,
            res_out=A, ld_ro=64, w_pre=A, w_offset=0.0, eps=1e-6, x=A, ld_x=64, stream=NUL)


@pytest.mark.parametrize("change,status", [
    ({"n_tok": -1}, INVALID), ({"hidden": 0}, INVALID), ({"hidden": 16385}, UNSUPPORTED),
    ({"io": 2}, INVALID), ({"res_t": -1}, INVALID), ({"eps": -1.0}, INVALID),
    ({"eps": float("nan")}, INVALID), ({"eps": float("inf")}, INVALID),
    ({"res_scale": float("inf")}, INVALID), ({"w_offset": float("nan")}, INVALID),
    ({"res": NUL}, INVALID), ({"w_pre": NUL}, INVALID), ({"x": NUL}, INVALID),
    ({"res_out": NUL}, INVALID), ({"y": NUL}, INVALID),
    ({"y": NUL, "res_out": NUL, "w_post": A}, INVALID),
    ({"ld_y": 63}, INVALID), ({"ld_res": 63}, INVALID), ({"ld_ro": 0}, INVALID), ({"ld_x": 63}, INVALID),
    ({"y": A + 1}, INVALID), ({"x": A + 1}, INVALID), ({"res": A + 2}, INVALID),
    ({"res_out": A + 2}, INVALID), ({"w_pre": A + 2}, INVALID), ({"w_post": A + 1}, INVALID),
    ({"n_tok": 0}, OK),
])
def test_block_norm_refusals(lib, change, status):
    assert lib.gdn_block_norm(*{**NORM, **change}.values()) == status


def test_gated_norm_refuses_a_null_pool(lib):
    assert lib.gdn_gated_norm(NUL, 1, A, 64, A, 64, A, 1e-6, 1, A, 64, NUL) == INVALID


@pytest.mark.parametrize("call", ["quantize", "dequantize"])
@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, INVALID), ({"cols": 0}, INVALID), ({"cols": 48}, UNSUPPORTED), ({"dtype": 5}, INVALID),
    ({"m": NUL}, INVALID), ({"codes": NUL}, INVALID), ({"scales": NUL}, INVALID),
    ({"m": A + 8}, INVALID), ({"codes": A + 4}, INVALID), ({"rows": 1 << 62}, INVALID), ({"rows": 0}, OK),
])
def test_mx_format_refusals(lib, call, change, status):
    p = {**dict(rows=4, cols=64, dtype=1, m=A, codes=A, scales=A), **change}
    if call == "quantize":
        st = lib.gdn_mx_quantize(p["rows"], p["cols"], p["dtype"], p["m"], p["codes"], p["scales"], NUL)
    else:
        st = lib.gdn_mx_dequantize(p["rows"], p["cols"], p["codes"], p["scales"], p["dtype"], p["m"], NUL)
    assert st == status


PROJ = dict(n_tok=2, n_in=64, n_out=10, x=A, ld_x=64, codes=A, scales=A, y_t=1, y=A, ld_y=10, ws=NUL,
            ws_bytes=0, stream=NUL)


@pytest.mark.parametrize("change,status", [
    ({"n_tok": -1}, INVALID), ({"n_in": 0}, INVALID), ({"n_in": 40}, UNSUPPORTED),
    ({"n_in": (1 << 20) + 32}, UNSUPPORTED), ({"n_out": 0}, INVALID), ({"n_out": 2 ** 31 - 1}, UNSUPPORTED),
    ({"n_tok": 1 << 40}, UNSUPPORTED), ({"y_t": 3}, INVALID),
    ({"x": NUL}, INVALID), ({"codes": NUL}, INVALID), ({"scales": NUL}, INVALID), ({"y": NUL}, INVALID),
    ({"x": A + 8}, INVALID), ({"codes": A + 8}, INVALID), ({"y": A + 1}, INVALID),
    ({"ld_x": 56}, INVALID), ({"ld_x": 68}, INVALID), ({"ld_x": 1 << 22}, UNSUPPORTED),
    ({"ld_y": 9}, INVALID), ({"ws": A + 8, "ws_bytes": 64}, INVALID), ({"n_tok": 0}, OK),
])
def test_mx_proj_refusals(lib, change, status):
    assert lib.gdn_mx_proj(*{**PROJ, **change}.values()) == status


def test_mx_proj_workspace(lib):
    n = ctypes.c_size_t(7)
    assert lib.gdn_mx_proj_workspace_bytes(4, 48, 8, ctypes.byref(n)) == UNSUPPORTED and n.value == 7
    assert lib.gdn_mx_proj_workspace_bytes(4, 64, 8, NUL) == INVALID
    for n_tok in (1, 16, 64, 65, 100, 128, 200, 256, 300, 511, 512, 1024, 4096, 8192):
        for n_in, n_out in ((2048, 2048), (4096, 2048), (2048, 12352), (32, 16)):
            assert lib.gdn_mx_proj_workspace_bytes(n_tok, n_in, n_out, ctypes.byref(n)) == OK
            if n.value:   # a call without the workspace it needs is refused
                p = {**PROJ, "n_tok": n_tok, "n_in": n_in, "n_out": n_out, "ld_x": n_in, "ld_y": n_out}
                assert lib.gdn_mx_proj(*{**p, "ws": NUL, "ws_bytes": n.value}.values()) == WORKSPACE
                assert lib.gdn_mx_proj(*{**p, "ws": A, "ws_bytes": n.value - 1}.values()) == WORKSPACE


def test_mx_in_proj_refuses_a_null_pool(lib):
    n = ctypes.c_size_t()
    assert lib.gdn_mx_in_proj_workspace_bytes(NUL, 1, 64, 1, ctypes.byref(n)) == INVALID
    assert lib.gdn_mx_in_proj(NUL, 1, 64, *([A] * 9), NUL, 0, NUL) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import gated_deltanet_state_layer_amd as G
    f = torch.zeros
    with pytest.raises(ValueError, match="residual: not a device tensor"):
        G.block_norm(f(2, 64), f(64), f(2, 64))
    with pytest.raises(ValueError, match="tokens, hidden"):
        G.block_norm(f(64), f(64), f(64))
    with pytest.raises(ValueError, match="dtype"):
        G.block_norm(f(2, 64).half(), f(64), f(2, 64))
    with pytest.raises(ValueError, match="not a device tensor"):
        G.mx_quantize(f(2, 64), f(2, 32).byte(), f(2, 2).byte())
    with pytest.raises(ValueError, match="dtype"):
        G.mx_dequantize(f(2, 32).byte(), f(2, 2).byte(), f(2, 64).half())
    with pytest.raises(ValueError, match="not a device tensor"):
        G.mx_proj(f(2, 64).bfloat16(), f(3, 32).byte(), f(3, 2).byte(), f(2, 3))
    with pytest.raises(ValueError, match="tokens, channels"):
        G.mx_proj(f(64).bfloat16(), f(3, 32).byte(), f(3, 2).byte(), f(3))

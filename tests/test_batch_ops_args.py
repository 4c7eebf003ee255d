"""Refusals of the operators for batches of many requests (maps, beam selection,
slot reordering, projections with adapters), on the host: a bad argument gives its
status before anything is enqueued, and the binding refuses tensors that do not
fit before their pointers leave Python."""
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


BEAM = dict(n_req=2, width=4, vocab=1000, n_out=4, dtype=1, logits=A, ld=1000, scores=A, finished=NUL, eos=2, parents=A,
            tokens=A, scores_out=A, finished_out=NUL, ws=A, ws_bytes=1 << 20, stream=NUL)


@pytest.mark.parametrize("change,status", [
    ({"n_req": -1}, INVALID), ({"width": 0}, INVALID), ({"width": 65}, UNSUPPORTED), ({"vocab": 0}, INVALID),
    ({"vocab": (1 << 30) + 1}, UNSUPPORTED), ({"n_out": 0}, INVALID), ({"n_out": 65}, UNSUPPORTED),
    ({"n_req": 1 << 20}, UNSUPPORTED), ({"dtype": 2}, INVALID), ({"ld": 999}, INVALID),
    ({"finished": A, "eos": -1}, INVALID), ({"logits": NUL}, INVALID), ({"scores": NUL}, INVALID),
    ({"parents": NUL}, INVALID), ({"tokens": NUL}, INVALID), ({"scores_out": NUL}, INVALID),
    ({"logits": A + 1}, INVALID), ({"scores": A + 2}, INVALID), ({"parents": A + 2}, INVALID),
    ({"tokens": A + 1}, INVALID), ({"scores_out": A + 2}, INVALID), ({"ws": NUL}, WORKSPACE),
    ({"ws_bytes": 100}, WORKSPACE), ({"ws": A + 8}, INVALID), ({"n_req": 0}, OK),
])
def test_beam_select_refusals(lib, change, status):
    assert lib.gdn_beam_select(*{**BEAM, **change}.values()) == status


def test_beam_select_workspace(lib):
    n = ctypes.c_size_t(7)
    assert lib.gdn_beam_select_workspace_bytes(1, 65, 10, 4, ctypes.byref(n)) == UNSUPPORTED and n.value == 7
    assert lib.gdn_beam_select_workspace_bytes(1, 4, 10, 4, NUL) == INVALID
    for r, w, v, k in ((1, 1, 1, 1), (1, 4, 32000, 4), (64, 8, 131072, 16), (16384, 64, 1 << 30, 64)):
        assert lib.gdn_beam_select_workspace_bytes(r, w, v, k, ctypes.byref(n)) == OK
        c = {**BEAM, "n_req": r, "width": w, "vocab": v, "n_out": k, "ld": v, "ws_bytes": n.value - 1}
        assert lib.gdn_beam_select(*c.values()) == WORKSPACE


def test_slot_reorder_and_batch_maps_refuse_a_null_pool(lib):
    assert lib.gdn_slot_reorder(NUL, 1, 2, A, A, A, NUL) == INVALID
    assert lib.gdn_batch_maps(NUL, 1, A, 8, A, *([NUL] * 4), NUL, 0, NUL, 0, NUL, 0, NUL, NUL, 0, NUL) == INVALID


LORA = dict(n_tok=2, n_in=64, n_out=10, x=A, ld_x=64, codes=A, scales=A, n=3, rank=16, a=A, b=A, scale=A, ids=A, y_t=1,
            y=A, ld_y=10, ws=A, ws_bytes=2 * 96, stream=NUL)


@pytest.mark.parametrize("change,status", [
    ({"n_tok": -1}, INVALID), ({"n_in": 40}, UNSUPPORTED), ({"n_out": 0}, INVALID), ({"y_t": 3}, INVALID),
    ({"n": -1}, INVALID), ({"rank": 0}, INVALID), ({"rank": 12}, UNSUPPORTED), ({"rank": 136}, UNSUPPORTED),
    ({"x": NUL}, INVALID), ({"codes": NUL}, INVALID), ({"scales": NUL}, INVALID), ({"y": NUL}, INVALID),
    ({"a": NUL}, INVALID), ({"b": NUL}, INVALID), ({"scale": NUL}, INVALID), ({"ids": NUL}, INVALID),
    ({"a": A + 8}, INVALID), ({"b": A + 8}, INVALID), ({"scale": A + 2}, INVALID), ({"ids": A + 1}, INVALID),
    ({"x": A + 8}, INVALID), ({"ld_x": 68}, INVALID), ({"ld_y": 9}, INVALID), ({"ws": NUL}, WORKSPACE),
    ({"ws_bytes": 2 * 96 - 1}, WORKSPACE), ({"ws": A + 8}, INVALID), ({"rank": 24}, WORKSPACE), ({"n_tok": 0}, OK),
    ({"n_tok": 0, "n": 0, "rank": 3}, OK),
])
def test_mx_proj_lora_refusals(lib, change, status):
    assert lib.gdn_mx_proj_lora(*{**LORA, **change}.values()) == status


def test_mx_lora_workspaces(lib):
    n = ctypes.c_size_t(7)
    assert lib.gdn_mx_proj_lora_workspace_bytes(4, 64, 8, 12, ctypes.byref(n)) == UNSUPPORTED and n.value == 7
    assert lib.gdn_mx_proj_lora_workspace_bytes(4, 64, 8, 16, NUL) == INVALID
    assert lib.gdn_mx_proj_lora_workspace_bytes(4, 64, 8, 24, ctypes.byref(n)) == OK and n.value == 4 * 2 * 96
    assert lib.gdn_mx_in_proj_lora_workspace_bytes(NUL, 4, 64, 16, 1, ctypes.byref(n)) == INVALID
    assert lib.gdn_mx_in_proj_lora(NUL, 1, 64, A, A, A, 1, 16, *([A] * 10), A, 64, NUL) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import gated_deltanet_state_layer_amd as G
    f = torch.zeros
    with pytest.raises(ValueError, match="not a device tensor"):
        G.beam_select(f(1, 2, 9), f(1, 2), f(1, 2).int(), f(1, 2).int(), f(1, 2))
    with pytest.raises(ValueError, match="requests, width, vocab"):
        G.beam_select(f(2, 9), f(1, 2), f(1, 2).int(), f(1, 2).int(), f(1, 2))
    with pytest.raises(ValueError, match="evenly spaced"):
        G.beam_select(f(2, 9, 2).transpose(1, 2), f(2, 2), f(2, 2).int(), f(2, 2).int(), f(2, 2))
    with pytest.raises(ValueError, match="not a device tensor"):
        G.mx_proj_lora(f(2, 64).bfloat16(), f(3, 32).byte(), f(3, 2).byte(), f(1, 8, 64).bfloat16(),
                       f(1, 3, 8).bfloat16(), f(1), f(2).int(), f(2, 3))
    pool = G.Pool.__new__(G.Pool)     # no GPU: only the checks run
    with pytest.raises(ValueError, match="requests, width"):
        pool.reorder(f(2, 3).int(), f(2, 4).int(), f(2, 3).int())
    with pytest.raises(ValueError, match="not a device tensor"):
        pool.reorder(f(2, 3).int(), f(2, 3).int(), f(2, 3).int())
    with pytest.raises(ValueError, match="needs adapter_ids"):
        pool.batch_maps(f(0).int(), f(1).int(), token_adapter=f(0).int())
    with pytest.raises(ValueError, match="not a device tensor"):
        pool.batch_maps(f(2).int(), f(3).int())


class Elsewhere(torch.Tensor):
    """Host memory that says it is on a device."""
    is_cuda = True
    on = 0

    def get_device(self):
        return self.on


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """Every tensor of a call is on the device where the library launches."""
    import gated_deltanet_state_layer_amd as G
    from gated_deltanet_state_layer_amd import binding
    monkeypatch.setattr(binding, "_current_device", lambda: 0)

    def calls_refuse(call, tensors):
        for wrong in tensors:
            args = {}
            for name, t in tensors.items():
                args[name] = t.clone().as_subclass(Elsewhere)
                args[name].on = int(name == wrong)
            with pytest.raises(ValueError, match=f"{wrong}: on .* but the current device"):
                call(**args)

    f = torch.zeros
    i, u, h = torch.int32, torch.uint8, torch.bfloat16
    calls_refuse(G.mx_proj_lora, dict(
        x=f(2, 64, dtype=h), codes=f(3, 32, dtype=u), scales=f(3, 2, dtype=u), lora_a=f(1, 8, 64, dtype=h),
        lora_b=f(1, 3, 8, dtype=h), lora_scale=f(1), token_adapter=f(2, dtype=i), out=f(2, 3), workspace=f(192, dtype=u)))
    calls_refuse(G.beam_select, dict(
        logits=f(1, 2, 9), scores=f(1, 2), parents=f(1, 2, dtype=i), tokens=f(1, 2, dtype=i), scores_out=f(1, 2),
        finished=f(1, 2, dtype=u), finished_out=f(1, 2, dtype=u), workspace=f(999, dtype=u)))
    pool = G.Pool.__new__(G.Pool)
    calls_refuse(pool.reorder, dict(slots=f(1, 2, dtype=i), parents=f(1, 2, dtype=i), slots_out=f(1, 2, dtype=i)))
    pool.desc = type("Desc", (), dict(h_v=1))
    pool._k_width = pool._v_width = 32
    pool.c_conv, pool.io_torch = 96, torch.float32
    calls_refuse(pool.mx_in_proj_lora, dict(
        x=f(2, 64, dtype=h), codes=f(130, 32, dtype=u), scales=f(130, 2, dtype=u), lora_a=f(1, 8, 64, dtype=h),
        lora_b=f(1, 130, 8, dtype=h), lora_scale=f(1), token_adapter=f(2, dtype=i), q=f(2, 32), k=f(2, 32),
        v=f(2, 32), a=f(2, 1), b=f(2, 1), z=f(2, 32), workspace=f(192, dtype=u)))
    maps = {n: f(4, dtype=i) for n in ("lens", "last_rows", "token_seq", "past", "token_pos", "adapter_ids",
                                       "token_adapter", "free_slots", "ckpt_slots")}
    maps.update(cu_seqlens=f(5, dtype=i), ckpt_offsets=f(5, dtype=i))
    calls_refuse(lambda **k: pool.batch_maps(ckpt_every=2, n_adapters=1, **k), maps)

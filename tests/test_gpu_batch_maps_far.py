"""GPU: the maps of a batch at the largest number of requests that a call takes,
2^31 - 1, whose last step of the scan ends past 32-bit integers."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
I32 = torch.int32


def test_as_many_requests_as_there_can_be():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    pool = G.Pool(G.make_desc(1, 1, 1, 1, 32, 32, 4))
    n, guard = 2 ** 31 - 1, 64
    # lengths other than 0, among them in the last two steps of any size up to 8192
    tokens = {0: 1, 70000: 2, n - 9000: 4, n - 4097: 1, n - 4096: 3, n - 4095: 2, n - 600: 5, n - 1: 6}
    lens = torch.zeros(n, dtype=I32, device="cuda")
    for j, t in tokens.items():
        lens[j] = t
    total = sum(tokens.values())
    buf = {name: torch.full((size + guard,), 77, dtype=I32, device="cuda")
           for name, size in dict(cu_seqlens=n + 1, ckpt_offsets=n + 1, token_seq=total + 5, token_pos=total + 5,
                                  ckpt_slots=20).items()}
    out = {name: b[:-guard] for name, b in buf.items()}
    pool.batch_maps(lens, ckpt_every=2, free_slots=torch.arange(100, 120, dtype=I32, device="cuda"), **out)
    torch.cuda.synchronize()
    assert pool.error() == 0
    for name, b in buf.items():
        assert (b[-guard:] == 77).all(), name
    at, rows, begin = 0, 0, 0
    for j, t in tokens.items():      # constant between the requests that have tokens
        assert bool((out["cu_seqlens"][begin:j + 1] == at).all()), j
        assert bool((out["ckpt_offsets"][begin:j + 1] == rows).all()), j
        assert out["token_seq"][at:at + t].tolist() == [j] * t
        assert out["token_pos"][at:at + t].tolist() == list(range(t))
        at, rows, begin = at + t, rows + t // 2, j + 1
    assert out["cu_seqlens"][n:].tolist() == [total] and out["ckpt_offsets"][n:].tolist() == [rows]
    assert out["token_seq"][total:].tolist() == out["token_pos"][total:].tolist() == [-1] * 5
    assert out["ckpt_slots"].tolist() == list(range(100, 100 + rows)) + [-1] * (20 - rows)

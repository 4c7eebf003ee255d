"""GPU: the maps of a batch from its requests' lengths, against their
definition, whole numbers exactly."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
GUARD = 77


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


@pytest.fixture(scope="module")
def pool(G):
    return G.Pool(G.make_desc(1, 1, 1, 1, 32, 32, 4))


def _reference(lens, room, past, ids, n_adapters, every, free, max_ckpt):
    cu, seq, pos, ad, off, at, used = [0], [], [], [], [0], 0, 0
    for j, n in enumerate(lens):
        n = min(max(n, 0), room - at)
        seq += [j] * n
        pos += [(past[j] if past else 0) + i for i in range(n)]
        if ids:
            ad += [ids[j] if 0 <= ids[j] < n_adapters else -1] * n
        at += n
        cu.append(at)
        if every:
            off.append(min(off[-1] + n // every, max_ckpt))
    pad = [-1] * (room - len(seq))
    last = [e - 1 if e > s else -1 for s, e in zip(cu, cu[1:])]
    out = {"cu_seqlens": cu, "last_rows": last, "token_seq": seq + pad, "token_pos": pos + pad}
    if ids:
        out["token_adapter"] = ad + pad
    if every:
        n = min(off[-1], len(free))
        out["ckpt_offsets"], out["ckpt_slots"] = off, free[:n] + [-1] * (max_ckpt - n)
    return out


def _check(G, pool, lens, room, past=None, ids=None, n_adapters=0, every=0, free=(), max_ckpt=0, shift=0, errors=0):
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ref = _reference(lens, room, past, ids, n_adapters, every, list(free), max_ckpt)
    bufs, out = {}, {}
    for name, v in ref.items():   # guard words around every output; `shift` words off 16-byte alignment
        bufs[name] = torch.full((len(v) + 16,), GUARD, dtype=torch.int32, device="cuda")
        out[name] = bufs[name][4 + shift: 4 + shift + len(v)]
    pool.batch_maps(dev(lens), past=None if past is None else dev(past), adapter_ids=None if ids is None else dev(ids),
                    n_adapters=n_adapters, ckpt_every=every, free_slots=dev(list(free)), **out)
    torch.cuda.synchronize()
    for name, v in ref.items():
        assert out[name].tolist() == v, name
        assert (bufs[name][:4 + shift] == GUARD).all() and (bufs[name][4 + shift + len(v):] == GUARD).all(), name
    assert pool.error() == errors


@pytest.mark.parametrize("n,most", [(1, 1), (1, 5000), (2, 3), (63, 1), (64, 40), (65, 2), (511, 9), (4095, 3), (4096, 1),
                                    (4097, 4), (9000, 2)])
@pytest.mark.parametrize("shift", [0, 1])
def test_maps(G, pool, n, most, shift):
    gen = torch.Generator().manual_seed(n + most)
    lens = torch.randint(0, most + 1, (n,), generator=gen).tolist()
    past = torch.randint(0, 10 ** 6, (n,), generator=gen).tolist()
    ids = torch.randint(-2, 6, (n,), generator=gen).tolist()
    total = sum(lens)
    for room in (total, total + 1, total + 2500):
        _check(G, pool, lens, room, past, ids, 6, shift=shift)
    _check(G, pool, lens, total + 3, None, None, 0, 2, range(100, 100 + total // 4), total // 2, shift=shift)


@pytest.mark.parametrize("every,n_free,max_ckpt", [(1, 0, 50), (16, 3, 9), (16, 100, 100), (7, 20, 4), (64, 8, 0)])
def test_checkpoint_tables(G, pool, every, n_free, max_ckpt):
    """Rows behind the last free slot and behind the last row are -1; rows past
    the table's end are dropped."""
    _check(G, pool, [5, 16, 0, 33, 64, 15], 140, [0, 16, 5, 0, 128, 1], None, 0, every, range(9, 9 + n_free), max_ckpt)


def test_empty_batches(G, pool):
    _check(G, pool, [], 0)
    _check(G, pool, [], 9)
    _check(G, pool, [0], 0, [3])
    _check(G, pool, [0] * 5000, 7, None, [1] * 5000, 2, 4, [1, 2], 3)
    cu = torch.full((3,), GUARD, dtype=torch.int32, device="cuda")
    pool.batch_maps(torch.tensor([4, 5], dtype=torch.int32, device="cuda"), cu)
    assert cu.tolist() == [0, 4, 9] and pool.error() == 0


def test_long_runs_of_empty_requests(G, pool):
    lens = [0] * 5000
    lens[0], lens[4095], lens[4096], lens[4999] = 3, 2, 1, 2049
    _check(G, pool, lens, 2100, list(range(5000)), [j % 3 for j in range(5000)], 3, 2, range(2000), 1030)


def test_tokens_past_the_room_are_dropped_and_reported(G, pool):
    _check(G, pool, [5, 6, 7], 13, [0, 1, 2], [0, 1, 0], 2, 3, [4, 5, 6, 7], 8, errors=2)
    _check(G, pool, [5, 6, 7], 11, [0, 1, 2], errors=2)
    _check(G, pool, [2 ** 31 - 1] * 5, 40, errors=2)
    _check(G, pool, [3, 2 ** 31 - 1, 2 ** 31 - 1, 5], 40, [1, 2, 3, 4], errors=2)
    # sums past 2^32 without maps of tokens
    cu = torch.empty(5, dtype=torch.int32, device="cuda")
    lens = torch.tensor([2 ** 31 - 1] * 4, dtype=torch.int32, device="cuda")
    pool.batch_maps(lens, cu, max_tokens=2 ** 31 - 2)
    assert cu.tolist() == [0] + [2 ** 31 - 2] * 4 and pool.error() == 2


def test_bad_lengths_and_adapters_are_reported(G, pool):
    _check(G, pool, [5, -6, 7], 13, [0, 1, 2], errors=2)
    _check(G, pool, [1, 2, 3], 6, None, [0, 2, 1], 2, errors=4)
    _check(G, pool, [1, 0, 3], 6, None, [0, 7, -9], 2, errors=4)


def test_graph_replays_follow_new_lengths(G, pool):
    n, room = 40, 3000
    i32 = lambda k: torch.full((k,), GUARD, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, past, ids, free = i32(n), i32(n), i32(n), torch.arange(500, 540, dtype=torch.int32, device="cuda")
    out = {"cu_seqlens": i32(n + 1), "last_rows": i32(n), "token_seq": i32(room), "token_pos": i32(room),
           "token_adapter": i32(room), "ckpt_offsets": i32(n + 1), "ckpt_slots": i32(64)}
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        pool.batch_maps(lens, past=past, adapter_ids=ids, n_adapters=4, ckpt_every=32, free_slots=free, **out)
    gen = torch.Generator().manual_seed(3)
    for t in range(4):
        new = [torch.randint(0, hi, (n,), generator=gen, dtype=torch.int32) for hi in (70, 1000, 4)]
        for d, v in zip((lens, past, ids), new):
            d.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        ref = _reference(new[0].tolist(), room, new[1].tolist(), new[2].tolist(), 4, 32, free.tolist(), 64)
        for name, v in ref.items():
            assert out[name].tolist() == v, (t, name)
    assert pool.error() == 0


def test_the_maps_feed_a_prefill_with_checkpoints(G):
    """Prompts packed by the maps, with checkpoints in the listed slots, leave what
    separate prefills of the same tokens leave."""
    desc = G.make_desc(12, 1, 2, 4, 64, 64, 4)
    a, b = G.Pool(desc), G.Pool(desc)
    gen = torch.Generator(device="cuda").manual_seed(5)
    lens, every, chunk = [40, 0, 75, 16], 32, 16
    n, t = len(lens), sum(lens)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = rnd(t, 2, 64).bfloat16(), rnd(t, 2, 64).bfloat16(), rnd(t, 4, 64).bfloat16()
    ga, gb, w = rnd(t, 4).sigmoid(), rnd(t, 4).sigmoid(), rnd(512, 4)
    out = {"cu_seqlens": i32([0] * (n + 1)), "token_seq": i32([0] * t), "ckpt_offsets": i32([0] * (n + 1)),
           "ckpt_slots": i32([0] * (t // every))}
    a.batch_maps(i32(lens), ckpt_every=every, free_slots=i32([9, 8]), **out)
    ws = torch.empty(a.prefill_workspace_bytes(n, t, chunk), dtype=torch.uint8, device="cuda")
    slots = i32([0, 1, 2, 3])
    o1, o2 = torch.empty(t, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(t, 4, 64, dtype=torch.bfloat16, device="cuda")
    a.prefill_ckpt(0, out["cu_seqlens"], slots, t, chunk, q, k, v, ga, gb, w, o1, every, out["ckpt_offsets"],
                   out["ckpt_slots"], workspace=ws)
    b.prefill(0, i32([0, 40, 40, 115, 131]), slots, t, chunk, q, k, v, ga, gb, w, o2, workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(a.state[:4], b.state[:4])
    # checkpoint rows: request 0 after 32 tokens into slot 9, request 2 after 32 into slot 8, its second has no slot
    assert out["ckpt_offsets"].tolist() == [0, 1, 1, 3, 3] and out["ckpt_slots"].tolist() == [9, 8, -1, -1]
    for slot, at in ((9, 0), (8, 40)):
        s = slice(at, at + 32)
        b.prefill(0, i32([0, 32]), i32([slot]), 32, chunk, q[s], k[s], v[s], ga[s], gb[s], w, o2, workspace=ws)
    assert torch.equal(a.state, b.state) and torch.equal(a.window, b.window)
    assert a.error() == 0 and b.error() == 0


def test_more_tokens_than_2_30(G, pool):
    a, b, room = 600_000_001, 600_000_006, 1_200_000_100
    lens = torch.tensor([a, 0, b], dtype=torch.int32, device="cuda")
    seq = torch.full((room + 1,), GUARD, dtype=torch.int32, device="cuda")
    cu = torch.empty(4, dtype=torch.int32, device="cuda")
    pool.batch_maps(lens, cu, token_seq=seq[:room])
    torch.cuda.synchronize()
    assert cu.tolist() == [0, a, a, a + b]
    assert (seq[:a] == 0).all() and (seq[a:a + b] == 2).all() and (seq[a + b:room] == -1).all() and int(seq[room]) == GUARD
    assert pool.error() == 0

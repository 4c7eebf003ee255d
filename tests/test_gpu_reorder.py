"""GPU: the reordering of beams' states in the pool, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    G.load_library()
    return G


def _place(slots, parents):
    """New slots and the copies (from, to), by the rule of the call."""
    w = len(slots)
    parents = [p if 0 <= p < w else -1 for p in parents]
    spare = [s for b, s in enumerate(slots) if b not in parents]
    out, copies, seen = [], [], set()
    for p in parents:
        if p >= 0 and p not in seen:
            out.append(slots[p])
        else:
            out.append(spare.pop(0))
            if p >= 0 and slots[p] >= 0 and out[-1] >= 0:
                copies.append((slots[p], out[-1]))
        seen.add(p)
    return out, copies


def _pool(G, n_slots, layers, h_k, h_v, d, io, ring, seed):
    pool = G.Pool(G.make_desc(n_slots, layers, h_k, h_v, d, d, 4, io, ring_len=ring))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pool.state.normal_(generator=gen)
    pool.window.copy_(torch.randn(pool.window.shape, generator=gen, device="cuda"))
    if ring:
        pool.ring_records.normal_(generator=gen)
        pool.ring_count.copy_(torch.randint(0, ring + 1, pool.ring_count.shape, generator=gen, device="cuda"))
    return pool


def _parts(pool):
    return [t for t in (pool.state, pool.window, pool.ring_count, pool.ring_records) if t is not None]


def _check(G, pool, slots, parents, in_place=False, errors=0):
    before = [t.clone() for t in _parts(pool)]
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    out = s if in_place else torch.full_like(s, -5)
    pool.reorder(s, torch.tensor(parents, dtype=torch.int32, device="cuda"), out)
    torch.cuda.synchronize()
    for r, (sl, pa) in enumerate(zip(slots, parents)):
        want, copies = _place(sl, pa)
        assert out[r].tolist() == want, r
        assert sorted(want) == sorted(sl)
        for src, dst in copies:
            if src < pool.desc.n_slots and dst < pool.desc.n_slots:
                for t in before:
                    t[dst] = t[src].clone()
    for t, ref in zip(_parts(pool), before):
        assert torch.equal(t, ref)      # the copies made, every other slot untouched
    assert pool.error() == errors


@pytest.mark.parametrize("layers,h_k,h_v,d,io,ring", [(1, 1, 1, 32, 1, 0), (3, 2, 4, 64, 0, 0), (2, 1, 3, 32, 1, 5),
                                                      (1, 2, 2, 128, 0, 0)])
@pytest.mark.parametrize("reqs,width", [(1, 1), (1, 2), (3, 4), (2, 7), (5, 16), (1, 33), (2, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder(G, layers, h_k, h_v, d, io, ring, reqs, width, in_place):
    n = reqs * width
    pool = _pool(G, n + 3, layers, h_k, h_v, d, io, ring, n)
    gen = torch.Generator().manual_seed(n + d)
    for kind in range(4):
        slots = torch.randperm(n + 3, generator=gen)[:n].view(reqs, width).tolist()
        lo, hi = ((0, width), (-2, width + 2), (0, max(1, width // 3)), (width - 1, width))[kind]
        _check(G, pool, slots, torch.randint(lo, hi, (reqs, width), generator=gen).tolist(), in_place)


def test_extremes(G):
    pool = _pool(G, 20, 2, 1, 2, 64, 1, 0, 1)
    slots = [list(range(8)), list(range(19, 11, -1))]
    _check(G, pool, slots, [list(range(8))] * 2)                 # every beam goes on: nothing is copied
    _check(G, pool, slots, [list(range(7, -1, -1))] * 2)         # a permutation: nothing is copied
    _check(G, pool, slots, [[0] * 8, [7] * 8])                   # one beam takes all
    _check(G, pool, slots, [[-1] * 8, [100] * 8])                # none goes on
    _check(G, pool, [[-1] * 8, slots[1]], [[0] * 8, [2] * 8])    # a padding request
    _check(G, pool, [[-1, 3, -1, 4, 5, 6, 7, 8], slots[1]], [[0, 0, 1, 1, 1, 2, 3, 3], [2] * 8])
    pool.reorder(*(torch.zeros(0, 4, dtype=torch.int32, device="cuda") for _ in range(3)))


def test_slots_outside_the_pool_are_skipped_and_reported(G):
    pool = _pool(G, 4, 1, 1, 1, 32, 1, 0, 2)
    _check(G, pool, [[0, 9, 1, 2]], [[0, 0, 2, 2]], errors=1)
    _check(G, pool, [[9, 0, 1, 2]], [[0, 0, 2, 2]], errors=1)
    _check(G, pool, [[9, 0, 1, 2]], [[0, 1, 2, 2]], errors=0)     # it is not copied


def test_validate_refuses_repeated_and_wrong_slots(G):
    pool = G.Pool(G.make_desc(4, 1, 1, 1, 32, 32, 4, flags=G.GDN_VALIDATE))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = i32([[0, 0]])
    for bad in ([[1, 1]], [[0, 4]]):
        with pytest.raises(G.GdnError) as e:
            pool.reorder(i32(bad), i32([[0, 0]]), out)
        assert e.value.status == -3
    pool.reorder(i32([[-1, -1]]), i32([[0, 0]]), out)
    assert out.tolist() == [[-1, -1]]


def test_graph_replays_in_place(G):
    """Replays go on from the table that the one before left."""
    pool, twin = (_pool(G, 24, 2, 1, 2, 64, 1, 4, 9) for _ in range(2))
    slots = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
    parents = torch.zeros_like(slots)
    other = slots.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        pool.reorder(slots, parents, slots)
    gen = torch.Generator().manual_seed(1)
    for t in range(4):
        p = torch.randint(0, 8, (3, 8), generator=gen, dtype=torch.int32)
        parents.copy_(p)
        graph.replay()
        nxt = torch.empty_like(other)
        twin.reorder(other, p.cuda(), nxt)
        other = nxt
        torch.cuda.synchronize()
        assert torch.equal(slots, other), t
        for x, y in zip(_parts(pool), _parts(twin)):
            assert torch.equal(x, y), t


def test_slots_past_4_gib(G):
    """Copies among the last slots of a pool of 2^32 state bytes and more."""
    pool = G.Pool(G.make_desc(2100, 1, 16, 32, 128, 128, 4))
    assert pool.state.numel() * 4 > 2 ** 32
    for slot in (2, 2098, 2099):
        pool.state[slot] = slot
        pool.window[slot] = slot
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = i32([[2099, 2, 2098]])
    pool.reorder(slots, i32([[0, 0, 1]]), slots)
    torch.cuda.synchronize()
    assert slots.tolist() == [[2099, 2098, 2]]
    for slot, held in ((2, 2), (2098, 2099), (2099, 2099)):
        assert (pool.state[slot] == held).all() and (pool.window[slot] == pool.window[held]).all()

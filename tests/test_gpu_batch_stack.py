"""GPU: the operators for batches of many requests together, as
examples/gdn_stack.py runs them: prompts of different lengths with and without
adapters, packed by the batch's maps, then beam search over the slots, against
the same steps in float64 (the oracle for the core), and a captured step against
the eager one."""
import importlib.util
import os

import numpy as np
import pytest

import gdn_synth as syn
from gpu_util import TOL_BF16, host, say
from oracle import gdn_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("gdn_stack", os.path.join(ROOT, "examples", "gdn_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _weights(packed):
    codes, scales = (t.cpu().numpy().astype(np.int64) for t in packed)
    idx = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    return np.where(idx >= 8, -1.0, 1.0) * LEVELS[idx & 7] * np.repeat(2.0 ** (scales - 127), 32, 1)


def _norm(x, eps):
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def _project(x, packed, lora, adapter):
    y = x @ _weights(packed).T
    a, b, s = (host(t) for t in lora)
    for t, i in enumerate(adapter):
        if i >= 0:
            y[t] += s[i] * (b[i] @ (a[i] @ x[t]))
    return y


def _reference(stack, r, adapter, core, s):
    """All blocks in float64, rounded to bf16 where the calls store bf16."""
    y = np.zeros_like(r)
    for i, w in enumerate(stack.layers):
        r = r + y
        x = syn.bf16_round(_norm(r, stack.eps) * (1.0 + host(w.w_norm)))
        p = _project(x, w.w_in, w.lora_in, adapter)
        c, v0 = s.h_k * s.d_k, s.h_v * s.d_v
        q, k, v, z, ya, yb = np.split(p, np.cumsum([c, c, v0, v0, s.h_v]), -1)
        n = r.shape[0]
        o = core(i, q.reshape(n, s.h_k, -1), k.reshape(n, s.h_k, -1), v.reshape(n, s.h_v, -1),
                 1.0 / (1.0 + np.exp(ya)), 1.0 / (1.0 + np.exp(-yb)), host(w.conv_w))
        g = syn.bf16_round(_norm(o, stack.eps) * host(w.w_head) * O.silu(z.reshape(n, s.h_v, -1)))
        y = syn.bf16_round(_project(g.reshape(n, -1), w.w_out, w.lora_out, adapter))
    return syn.bf16_round(_norm(r + y, stack.eps) * (1.0 + host(stack.w_final)))


def _same(name, got, ref):
    """Both sides round the same values to bf16; a value near the border may
    fall to either side, which the following steps carry on."""
    rms = np.sqrt(np.mean(ref * ref))
    err = float(np.abs(got - ref).max() / rms)
    say(f"  {name}: {err:.2e} of the rms")
    assert err <= TOL_BF16 + 2.0 ** -8 * np.abs(ref).max() / rms, name


def _best(logits, scores, done, eos, k):
    """Entries (score, beam, token), by the definition, from the logits as they are."""
    entries = []
    for b, (row, base) in enumerate(zip(logits, scores)):
        if not np.isfinite(base):
            continue
        if done[b]:
            entries.append((base, b, eos))
            continue
        c = base + ((row - row.max()) - np.log(np.exp(row - row.max()).sum()))
        entries += [(c[t], b, int(t)) for t in np.argsort(-c, kind="stable")[:k]]
    return sorted(entries, key=lambda e: (-e[0], e[1], e[2]))[:k]


def test_prompts_adapters_and_beams_follow_the_definition(E):
    """fp32 io between the calls: prompts of 5, 1 and 70 tokens, adapters 1, none
    and 0, then four steps of three beams each."""
    import gated_deltanet_state_layer_amd as G
    s = syn.Shapes(2, 4, 32, 32, 4)
    hidden, n_layers, vocab, w, eos = 96, 2, 50, 3, 7
    stack = E.random_stack(n_layers, hidden, s.h_k, s.h_v, s.d_k, s.conv_k, n_slots=9, io=G.GDN_F32, seed=5, adapters=2,
                           rank=8)
    pool = O.OraclePool(9, n_layers, s)
    gen = torch.Generator(device="cuda").manual_seed(6)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, ids = [[2, 0, 3], [1, 8, 4], [7, 5, 6]], [1, -1, 0]
    batch = E.Batch(stack.pool, i32([5, 1, 70]), i32(ids), 2)
    adapter = [1] * 5 + [-1] + [0] * 70
    assert batch.cu.tolist() == [0, 5, 6, 76] and batch.last.tolist() == [4, 5, 75] and batch.adapter.tolist() == adapter
    r = torch.randn(76, hidden, generator=gen, device="cuda")
    first = np.array([sl[0] for sl in slots], np.int32)
    ref = _reference(stack, host(r), adapter,
                     lambda i, q, k, v, a, b, cw: pool.prefill(i, np.array([0, 5, 6, 76]), first, q, k, v, a, b, cw), s)
    buf = E.Buffers(stack, 76, 3)
    buf.adapter.copy_(batch.adapter)
    x = stack.prefill(r, batch.cu, i32(first.tolist()), buf)
    torch.cuda.synchronize()
    _same("prompts", host(x), ref)

    embed = torch.randn(vocab, hidden, generator=gen, device="cuda")
    head = E.pack(torch.randn(vocab, hidden, generator=gen, device="cuda") * hidden ** -0.5 * 3.0)
    beams = E.Beams(stack, embed, head, i32(slots), eos)
    beams.buf.adapter.copy_(i32(np.repeat(ids, w).tolist()))
    beams.start()
    x = x[batch.last.long()].repeat_interleave(w, 0)
    table = [list(sl) for sl in slots]
    for t in range(5):
        scores, done = host(beams.scores), beams.done.cpu().numpy()
        if t > 0:
            r_in = host(beams.r)
            flat = np.array(table, np.int32).reshape(-1)
            ref = _reference(stack, r_in, np.repeat(ids, w),
                             lambda i, q, k, v, a, b, cw: pool.decode(i, flat, q, k, v, a, b, cw), s)
            x = stack.decode(beams.r, beams.slots.view(-1), beams.buf)
            torch.cuda.synchronize()
            _same(f"step {t}, hidden states", host(x), ref)
        before = stack.pool.state.clone(), stack.pool.window.clone()
        beams.select(x)
        torch.cuda.synchronize()
        logits = host(beams.logits).reshape(3, w, vocab)
        for q in range(3):
            best = _best(logits[q], scores[q], done[q], eos, w)
            assert beams.parents[q].tolist() == [e[1] for e in best], (t, q)
            assert beams.tokens[q].tolist() == [e[2] for e in best], (t, q)
            # a rounding to fp32 of sums whose fp64 error is far below it
            assert np.allclose(host(beams.scores[q]), [e[0] for e in best], rtol=2.0 ** -24 * 1.01, atol=1e-12)
            assert beams.done[q].tolist() == [int(bool(done[q][e[1]]) or e[2] == eos) for e in best]
            # the states of the beams continued, wherever the table says they are: bit for
            # bit on the GPU, and the oracle's the same way
            new = beams.slots[q].tolist()
            assert sorted(new) == sorted(table[q])
            for e, j in zip(best, new):
                assert torch.equal(stack.pool.state[j], before[0][table[q][e[1]]])
                assert torch.equal(stack.pool.window[j], before[1][table[q][e[1]]])
            for part in (pool.S, pool.X):
                kept = [part[table[q][e[1]]].copy() for e in best]
                for j, old in zip(new, kept):
                    part[j] = old
            table[q] = new
    assert stack.pool.error() == 0


@pytest.mark.parametrize("n,w", [(1, 4), (3, 3), (20, 4), (200, 4)])
def test_captured_beam_steps_equal_eager_ones(E, n, w):
    """200 requests of four beams take the tile kernels."""
    hidden, vocab = 512, 1000

    def make():
        stack = E.random_stack(2, hidden, 4, 8, 64, n_slots=n * w, seed=9, adapters=3, rank=16)
        gen = torch.Generator(device="cuda").manual_seed(2)
        embed = torch.randn(vocab, hidden, generator=gen, device="cuda")
        head = E.pack(torch.randn(vocab, hidden, generator=gen, device="cuda") * 0.1)
        beams = E.Beams(stack, embed, head, torch.arange(n * w, dtype=torch.int32, device="cuda").view(n, w), eos=3)
        beams.buf.adapter.copy_(torch.arange(n * w, device="cuda") // w % 4 - 1)
        beams.start()
        return beams, torch.randn(n * w, hidden, generator=gen, device="cuda").bfloat16()

    (a, x), (b, _) = make(), make()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        a.step()
    a.select(x)
    b.select(x)
    for t in range(5):
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        for name in ("slots", "parents", "tokens", "scores", "done", "r"):
            assert torch.equal(getattr(a, name), getattr(b, name)), (t, name)
    assert torch.equal(a.stack.pool.state, b.stack.pool.state) and torch.equal(a.stack.pool.window, b.stack.pool.window)
    assert a.stack.pool.error() == 0 and bool(torch.isfinite(a.scores).all())


def test_two_graphs_share_a_workspace():
    """A projection with adapters in one graph, a selection in another, both with
    the same scratch memory, replayed in turn."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_deltanet_state_layer_amd as G
    gen = torch.Generator(device="cuda").manual_seed(12)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    t, n_in, n_out, rank, r, w, v, k = 300, 512, 700, 24, 4, 5, 30011, 8
    x, y, want = (rnd(t, c).to(torch.bfloat16) for c in (n_in, n_out, n_out))
    codes = torch.randint(0, 256, (n_out, n_in // 2), generator=gen, device="cuda").to(torch.uint8)
    scales = torch.randint(118, 124, (n_out, n_in // 32), generator=gen, device="cuda").to(torch.uint8)
    a, b, s = rnd(3, rank, n_in).to(torch.bfloat16), rnd(3, n_out, rank).to(torch.bfloat16), rnd(3)
    ids = (torch.arange(t, device="cuda") % 4).int()
    logits, scores = rnd(r, w, v), -torch.rand(r, w, generator=gen, device="cuda")
    outs, expect = ([torch.empty(r, k, dtype=d, device="cuda") for d in (torch.int32, torch.int32, torch.float32)]
                    for _ in "ab")
    size = max(G.mx_proj_lora_workspace_bytes(t, n_in, n_out, rank), G.beam_select_workspace_bytes(r, w, v, k))
    ws, own = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in "ab")
    proj, select, side = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(proj, stream=side):
        G.mx_proj_lora(x, codes, scales, a, b, s, ids, y, workspace=ws)
    with torch.cuda.graph(select, stream=side):
        G.beam_select(logits, scores, *outs, workspace=ws)
    for step in range(5):
        x.copy_(rnd(t, n_in))
        logits.copy_(rnd(r, w, v))
        for graph in (proj, select) if step % 2 else (select, proj):
            graph.replay()
        G.mx_proj_lora(x, codes, scales, a, b, s, ids, want, workspace=own)
        G.beam_select(logits, scores, *expect, workspace=own)
        torch.cuda.synchronize()
        assert torch.equal(y, want), step
        for got, ref in zip(outs, expect):
            assert torch.equal(got, ref), step

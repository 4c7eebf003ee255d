"""GPU: the operators around the core together with it, as examples/gdn_stack.py
runs them, against the same steps in float64 (the oracle for the core), and a
decode step recorded into a graph against the eager one."""
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


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("gdn_stack", os.path.join(ROOT, "examples", "gdn_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _weights(packed):
    codes, scales = (t.cpu().numpy().astype(np.int64) for t in packed)
    idx = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    return np.where(idx >= 8, -1.0, 1.0) * LEVELS[idx & 7] * np.repeat(2.0 ** (scales - 127), 32, 1)


def _norm(x, eps):
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def _reference(stack, r, core, s):
    """All blocks in float64, rounded to bf16 where the calls store bf16."""
    y = np.zeros_like(r)
    for i, w in enumerate(stack.layers):
        r = r + y
        x = syn.bf16_round(_norm(r, stack.eps) * (1.0 + host(w.w_norm)))
        p = x @ _weights(w.w_in).T
        c, v0 = s.h_k * s.d_k, s.h_v * s.d_v
        q, k, v, z, ya, yb = np.split(p, np.cumsum([c, c, v0, v0, s.h_v]), -1)
        a, b = 1.0 / (1.0 + np.exp(ya)), 1.0 / (1.0 + np.exp(-yb))
        n = r.shape[0]
        o = core(i, q.reshape(n, s.h_k, -1), k.reshape(n, s.h_k, -1), v.reshape(n, s.h_v, -1), a, b,
                 host(w.conv_w))
        z = z.reshape(n, s.h_v, -1)
        g = syn.bf16_round(_norm(o, stack.eps) * host(w.w_head) * O.silu(z))
        y = syn.bf16_round(g.reshape(n, -1) @ _weights(w.w_out).T)
    r = r + y
    return syn.bf16_round(_norm(r, stack.eps) * (1.0 + host(stack.w_final))), r


def _same(name, got, ref):
    """Both sides round the same values to bf16; a value near the border may
    fall to either side, which the following steps carry on."""
    rms = np.sqrt(np.mean(ref * ref))
    err = float(np.abs(got - ref).max() / rms)
    say(f"  {name}: {err:.2e} of the rms")
    assert err <= TOL_BF16 + 2.0 ** -8 * np.abs(ref).max() / rms, name


def test_prompts_and_decoded_tokens_follow_the_definition(E):
    """fp32 io between the calls: prompts of 5, 1 and 70 tokens, then three
    decoded tokens of two of them."""
    import gated_deltanet_state_layer_amd as G
    s = syn.Shapes(2, 4, 32, 32, 4)
    hidden, n_layers = 96, 2
    stack = E.random_stack(n_layers, hidden, s.h_k, s.h_v, s.d_k, s.conv_k, n_slots=4, io=G.GDN_F32, seed=5)
    pool = O.OraclePool(4, n_layers, s)
    gen = torch.Generator(device="cuda").manual_seed(6)
    cu, slots = np.array([0, 5, 6, 76], np.int32), np.array([2, 0, 3], np.int32)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    r = torch.randn(76, hidden, generator=gen, device="cuda")
    ref_x, ref_r = _reference(stack, host(r), lambda i, q, k, v, a, b, w: pool.prefill(i, cu, slots, q, k, v, a, b, w), s)
    x = stack.prefill(r, dev(cu), dev(slots), E.Buffers(stack, 76, 3))
    torch.cuda.synchronize()
    _same("prompt, hidden states", host(x), ref_x)
    _same("prompt, residual", host(r), ref_r)
    buf, slots = E.Buffers(stack, 2, 0), np.array([3, 2], np.int32)
    for t in range(3):
        r = torch.randn(2, hidden, generator=gen, device="cuda")
        ref_x, ref_r = _reference(stack, host(r), lambda i, q, k, v, a, b, w: pool.decode(i, slots, q, k, v, a, b, w), s)
        x = stack.decode(r, dev(slots), buf)
        torch.cuda.synchronize()
        _same(f"token {t}, hidden states", host(x), ref_x)
        _same(f"token {t}, residual", host(r), ref_r)
    assert stack.pool.error() == 0


@pytest.mark.parametrize("n", [1, 8, 70])
def test_graph_replayed_steps_equal_eager_ones(E, n):
    """70 tokens a step take the tile kernel with its workspace."""
    make = lambda: E.random_stack(2, 512, 4, 8, 64, n_slots=n, seed=9)  # noqa: E731
    a, b = make(), make()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    r_in = torch.zeros(n, 512, device="cuda")
    r_a, r_b = torch.empty_like(r_in), torch.empty_like(r_in)
    buf_a, buf_b = E.Buffers(a, n, 0), E.Buffers(b, n, 0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        r_a.copy_(r_in)
        a.decode(r_a, slots, buf_a)
    gen = torch.Generator(device="cuda").manual_seed(n)
    for t in range(5):
        r_in.copy_(torch.randn(n, 512, generator=gen, device="cuda"))
        graph.replay()
        r_b.copy_(r_in)
        b.decode(r_b, slots, buf_b)
        torch.cuda.synchronize()
        assert torch.equal(buf_a.x, buf_b.x) and torch.equal(r_a, r_b), f"replay {t}"
    assert torch.equal(a.pool.state, b.pool.state) and bool(torch.isfinite(buf_b.x).all())

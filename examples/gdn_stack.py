"""A stack of Gated DeltaNet blocks with 4-bit weights, from the residual
stream in to the normed hidden states out, on the calls of the library:

    x, r   = block_norm(r, y)          residual add and norm in front of a block
    q .. b = mx_in_proj(x)             q, k, v, the gate z and the gates a, b
    o      = decode / prefill          the layer core over the slot pool
    g      = gated_norm(o, z)          per-head norm times silu(z)
    y      = mx_proj(g)                out-projection back to the hidden size

and one more block_norm behind the last block.  Run as a program, it loads
random weights, serves a batch of prompts and decodes some tokens from a
captured graph, and prints the times:

    python examples/gdn_stack.py [--layers 4] [--requests 8] [--prompt 1000] [--steps 32]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_state_layer_amd as G  # noqa: E402

CHUNK = 64


class Layer:
    """One block's weights: 4-bit projections, conv taps and norm vectors."""

    def __init__(self, w_norm, w_in, conv_w, w_head, w_out):
        self.w_norm, self.conv_w, self.w_head = w_norm, conv_w, w_head
        self.w_in, self.w_out = self._pack(w_in), self._pack(w_out)

    @staticmethod
    def _pack(w):
        rows, cols = w.shape
        codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=w.device)
        scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=w.device)
        return G.mx_quantize(w.contiguous(), codes, scales)


class Buffers:
    """What a pass over n_tok tokens writes, and its scratch memory: kept from
    call to call of the same size, so that a pass allocates nothing."""

    def __init__(self, stack, n_tok, n_seq):
        p, d = stack.pool, stack.pool.desc
        io = p.io_torch

        def empty(*shape, dtype=io):
            return torch.empty(shape, dtype=dtype, device="cuda")

        hk, hv = (n_tok, d.h_k, d.d_k), (n_tok, d.h_v, d.d_v)
        self.x, self.y = empty(n_tok, stack.hidden, dtype=torch.bfloat16), \
            empty(n_tok, stack.hidden, dtype=torch.bfloat16)
        self.q, self.k, self.v, self.z, self.o = empty(*hk), empty(*hk), empty(*hv), empty(*hv), empty(*hv)
        self.a, self.b = (empty(n_tok, d.h_v, dtype=torch.float32) for _ in "ab")
        self.g = empty(*hv, dtype=torch.bfloat16)
        need = max(p.mx_in_proj_workspace_bytes(n_tok, stack.hidden),
                   G.mx_proj_workspace_bytes(n_tok, d.h_v * d.d_v, stack.hidden),
                   p.prefill_workspace_bytes(n_seq, n_tok, CHUNK) if n_seq else 0)
        self.ws = empty(max(need, 256), dtype=torch.uint8)


class Stack:
    def __init__(self, layers, w_final, hidden, desc, eps=1e-6):
        self.layers, self.w_final, self.hidden, self.eps = layers, w_final, hidden, eps
        self.pool = G.Pool(desc)

    def _blocks(self, r, buf, core):
        """The residual stream r [tokens, hidden] (updated in place) through all
        blocks; returns the normed hidden states (buf.x)."""
        p, y = self.pool, None
        for i, w in enumerate(self.layers):
            G.block_norm(r, w.w_norm, buf.x, y=y, residual_out=None if y is None else r, w_offset=1.0,
                         eps=self.eps)
            p.mx_in_proj(buf.x, *w.w_in, buf.q, buf.k, buf.v, buf.a, buf.b, z=buf.z, workspace=buf.ws)
            core(i, w, buf)
            p.gated_norm(buf.o, buf.z, w.w_head, buf.g, eps=self.eps)
            y = G.mx_proj(buf.g.flatten(1), *w.w_out, buf.y, workspace=buf.ws)
        return G.block_norm(r, self.w_final, buf.x, y=y, residual_out=r, w_offset=1.0, eps=self.eps)

    def prefill(self, r, cu_seqlens, slots, buf):
        """Prompts packed one behind the other, sequence j on slot slots[j]."""
        def core(i, w, b):
            self.pool.prefill(i, cu_seqlens, slots, r.shape[0], CHUNK, b.q, b.k, b.v, b.a, b.b, w.conv_w, b.o,
                              b.ws)
        return self._blocks(r, buf, core)

    def decode(self, r, slots, buf):
        """One token for each listed slot."""
        def core(i, w, b):
            self.pool.decode(i, slots, b.q, b.k, b.v, b.a, b.b, w.conv_w, b.o)
        return self._blocks(r, buf, core)


def random_layer(hidden, h_k, h_v, d, conv_k, gen):
    n = lambda *s, scale=1.0: torch.randn(s, generator=gen, device="cuda") * scale  # noqa: E731
    channels = 2 * h_k * d + 2 * h_v * d + 2 * h_v
    return Layer(n(hidden, scale=0.1), n(channels, hidden, scale=hidden ** -0.5),
                 n(2 * h_k * d + h_v * d, conv_k, scale=conv_k ** -0.5), 1.0 + n(d, scale=0.1),
                 n(hidden, h_v * d, scale=(h_v * d) ** -0.5))


def random_stack(n_layers, hidden, h_k, h_v, d, conv_k=4, n_slots=8, io=G.GDN_BF16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layers = [random_layer(hidden, h_k, h_v, d, conv_k, gen) for _ in range(n_layers)]
    w_final = torch.randn(hidden, generator=gen, device="cuda") * 0.1
    return Stack(layers, w_final, hidden, G.make_desc(n_slots, n_layers, h_k, h_v, d, d, conv_k, io))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    hidden, n = 2048, a.requests
    stack = random_stack(a.layers, hidden, 16, 32, 128, n_slots=n)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda") * a.prompt
    r = torch.randn(n * a.prompt, hidden, device="cuda")
    buf = Buffers(stack, n * a.prompt, n)
    for name in ("first prefill", "prefill"):
        stack.pool.reset(slots)
        torch.cuda.synchronize()
        t = time.perf_counter()
        x = stack.prefill(r.clone(), cu, slots, buf)
        torch.cuda.synchronize()
        print(f"{name} of {n} x {a.prompt} tokens: {(time.perf_counter() - t) * 1e3:.2f} ms", flush=True)

    step_r, step = torch.empty(n, hidden, device="cuda"), Buffers(stack, n, 0)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        stack.decode(step_r, slots, step)
    x = x.view(n, a.prompt, hidden)[:, -1].float()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        step_r.copy_(x)          # stands for sampling and embedding the next token
        graph.replay()
        x = step.x.float()
    torch.cuda.synchronize()
    print(f"decode step of {n} requests, {a.layers} layers: "
          f"{(time.perf_counter() - t) / a.steps * 1e6:.1f} us", flush=True)
    assert stack.pool.error() == 0 and bool(torch.isfinite(x).all())


if __name__ == "__main__":
    main()

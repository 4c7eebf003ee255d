"""A stack of Gated DeltaNet blocks with 4-bit weights, from the residual
stream in to the normed hidden states out, on the calls of the library:

    x, r   = block_norm(r, y)          residual add and norm in front of a block
    q .. b = mx_in_proj(x)             q, k, v, the gate z and the gates a, b
    o      = decode / prefill          the layer core over the slot pool
    g      = gated_norm(o, z)          per-head norm times silu(z)
    y      = mx_proj(g)                out-projection back to the hidden size

and one more block_norm behind the last block.  With adapters, the projections
are those with a low-rank adapter per token.  Run as a program, it loads random
weights, serves a batch of prompts of different lengths and decodes some tokens
from a captured graph, with --beams by beam search, and prints the times:

    python examples/gdn_stack.py [--layers 4] [--requests 8] [--prompt 1000] [--steps 32]
                                 [--adapters 0] [--rank 16] [--beams 1] [--vocab 32000]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_state_layer_amd as G  # noqa: E402

CHUNK = 64


def pack(w):
    """A matrix in 4 bits: codes and scales."""
    rows, cols = w.shape
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device=w.device)
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=w.device)
    return G.mx_quantize(w.contiguous(), codes, scales)


class Layer:
    """One block's weights: 4-bit projections, conv taps and norm vectors, and the
    adapters of both projections (A, B and scale each), if there are any."""

    def __init__(self, w_norm, w_in, conv_w, w_head, w_out, lora_in=None, lora_out=None):
        self.w_norm, self.conv_w, self.w_head = w_norm, conv_w, w_head
        self.w_in, self.w_out = pack(w_in), pack(w_out)
        self.lora_in, self.lora_out = lora_in, lora_out


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
        lora = stack.layers[0].lora_in
        if lora is not None:
            rank = lora[0].shape[1]
            need = max(need, p.mx_in_proj_lora_workspace_bytes(n_tok, stack.hidden, rank),
                       G.mx_proj_lora_workspace_bytes(n_tok, d.h_v * d.d_v, stack.hidden, rank))
        self.ws = empty(max(need, 256), dtype=torch.uint8)
        self.adapter = torch.full((n_tok,), -1, dtype=torch.int32, device="cuda")   # of each token


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
            if w.lora_in is None:
                p.mx_in_proj(buf.x, *w.w_in, buf.q, buf.k, buf.v, buf.a, buf.b, z=buf.z, workspace=buf.ws)
            else:
                p.mx_in_proj_lora(buf.x, *w.w_in, *w.lora_in, buf.adapter, buf.q, buf.k, buf.v, buf.a, buf.b,
                                  z=buf.z, workspace=buf.ws)
            core(i, w, buf)
            p.gated_norm(buf.o, buf.z, w.w_head, buf.g, eps=self.eps)
            if w.lora_out is None:
                y = G.mx_proj(buf.g.flatten(1), *w.w_out, buf.y, workspace=buf.ws)
            else:
                y = G.mx_proj_lora(buf.g.flatten(1), *w.w_out, *w.lora_out, buf.adapter, buf.y, workspace=buf.ws)
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


class Beams:
    """Beam search over a stack's slots: request r's beam b on slot slots[r, b].
    `embed` gives a token's residual, `head` (packed) the logits."""

    def __init__(self, stack, embed, head, slots, eos):
        self.stack, self.embed, self.head, self.slots, self.eos = stack, embed, head, slots, eos
        (n, w), vocab = slots.shape, embed.shape[0]

        def empty(*shape, dtype=torch.int32):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.parents, self.tokens = empty(n, w), empty(n, w)
        self.scores, self.next_scores = empty(n, w, dtype=torch.float32), empty(n, w, dtype=torch.float32)
        self.done, self.next_done = empty(n, w, dtype=torch.uint8), empty(n, w, dtype=torch.uint8)
        self.logits = empty(n * w, vocab, dtype=torch.bfloat16)
        self.ws = empty(G.beam_select_workspace_bytes(n, w, vocab, w), dtype=torch.uint8)
        self.r, self.buf = empty(n * w, stack.hidden, dtype=torch.float32), Buffers(stack, n * w, 0)

    def start(self):
        """Only the first beam of each request has something to continue."""
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0.0
        self.done.zero_()

    def select(self, x):
        """From the beams' hidden states to their best continuations, the states
        of the beams continued and the next tokens' residuals."""
        n, w = self.slots.shape
        G.mx_proj(x, *self.head, self.logits)
        G.beam_select(self.logits.view(n, w, -1), self.scores, self.parents, self.tokens, self.next_scores,
                      finished=self.done, finished_out=self.next_done, eos=self.eos, workspace=self.ws)
        self.scores.copy_(self.next_scores)
        self.done.copy_(self.next_done)
        self.stack.pool.reorder(self.slots, self.parents, self.slots)
        torch.index_select(self.embed, 0, self.tokens.view(-1).clamp(min=0), out=self.r)

    def step(self):
        """One token of every beam, and the choice of the next."""
        self.select(self.stack.decode(self.r, self.slots.view(-1), self.buf))


def random_lora(n, rank, n_in, n_out, gen):
    a = torch.randn(n, rank, n_in, generator=gen, device="cuda") * n_in ** -0.5
    b = torch.randn(n, n_out, rank, generator=gen, device="cuda") * (0.25 * rank ** -0.5)
    return a.bfloat16(), b.bfloat16(), torch.ones(n, device="cuda")


def random_layer(hidden, h_k, h_v, d, conv_k, gen, adapters=0, rank=16):
    n = lambda *s, scale=1.0: torch.randn(s, generator=gen, device="cuda") * scale  # noqa: E731
    channels = 2 * h_k * d + 2 * h_v * d + 2 * h_v
    layer = Layer(n(hidden, scale=0.1), n(channels, hidden, scale=hidden ** -0.5),
                  n(2 * h_k * d + h_v * d, conv_k, scale=conv_k ** -0.5), 1.0 + n(d, scale=0.1),
                  n(hidden, h_v * d, scale=(h_v * d) ** -0.5))
    if adapters:
        layer.lora_in = random_lora(adapters, rank, hidden, channels, gen)
        layer.lora_out = random_lora(adapters, rank, h_v * d, hidden, gen)
    return layer


def random_stack(n_layers, hidden, h_k, h_v, d, conv_k=4, n_slots=8, io=G.GDN_BF16, seed=0, adapters=0, rank=16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layers = [random_layer(hidden, h_k, h_v, d, conv_k, gen, adapters, rank) for _ in range(n_layers)]
    w_final = torch.randn(hidden, generator=gen, device="cuda") * 0.1
    return Stack(layers, w_final, hidden, G.make_desc(n_slots, n_layers, h_k, h_v, d, d, conv_k, io))


class Batch:
    """A batch of prompts: its maps, made on the GPU from the lengths."""

    def __init__(self, pool, lens, adapter_ids, adapters):
        n, t = lens.numel(), int(lens.sum())
        i32 = lambda k: torch.empty(k, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu, self.last, self.adapter = i32(n + 1), i32(n), i32(t)
        pool.batch_maps(lens, self.cu, last_rows=self.last, adapter_ids=adapter_ids, n_adapters=adapters,
                        token_adapter=self.adapter)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--adapters", type=int, default=0)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--beams", type=int, default=1)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    hidden, n, w = 2048, a.requests, a.beams
    stack = random_stack(a.layers, hidden, 16, 32, 128, n_slots=n * w, adapters=a.adapters, rank=a.rank)
    slots = torch.arange(n * w, dtype=torch.int32, device="cuda").view(n, w)
    first = slots[:, 0].contiguous()       # prompts go to the first beams' slots
    lens = torch.arange(n, dtype=torch.int32, device="cuda") % 7 - 3 + a.prompt
    # adapters in turn, every last request without
    ids = torch.arange(n, dtype=torch.int32, device="cuda") % (a.adapters + 1)
    ids = torch.where(ids == a.adapters, -1, ids)
    batch = Batch(stack.pool, lens, ids, a.adapters)
    t_all = int(batch.cu[-1])
    r = torch.randn(t_all, hidden, device="cuda")
    buf = Buffers(stack, t_all, n)
    buf.adapter.copy_(batch.adapter)
    for name in ("first prefill", "prefill"):
        stack.pool.reset(slots.view(-1))
        torch.cuda.synchronize()
        t = time.perf_counter()
        x = stack.prefill(r.clone(), batch.cu, first, buf)
        torch.cuda.synchronize()
        print(f"{name} of {n} prompts, {t_all} tokens: {(time.perf_counter() - t) * 1e3:.2f} ms", flush=True)
    x = x[batch.last.long()]

    gen = torch.Generator(device="cuda").manual_seed(1)
    embed = torch.randn(a.vocab, hidden, generator=gen, device="cuda")
    head = pack(torch.randn(a.vocab, hidden, generator=gen, device="cuda") * hidden ** -0.5)
    beams = Beams(stack, embed, head, slots, eos=0)
    beams.buf.adapter.copy_(ids.repeat_interleave(w))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        beams.step()
    beams.start()
    beams.select(x.repeat_interleave(w, 0))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    print(f"decode step of {n} requests with {w} beams, {a.layers} layers, {a.adapters} adapters: "
          f"{(time.perf_counter() - t) / a.steps * 1e6:.1f} us", flush=True)
    assert stack.pool.error() == 0 and bool(torch.isfinite(beams.scores).all())


if __name__ == "__main__":
    main()

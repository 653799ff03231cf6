"""The attention half of one layer, as a serving engine runs it: q/k/v group ->
K/V cache -> attention -> o_proj, for a system prompt, the chats that share it,
and the steps in which each of them gets its next token.

    python examples/serve_attention.py

Weights and activations are synthetic, and q and k go to attention as the group gives
them: a model that normalises or rotates them does so in between, before ``cache_append``.
``Layer`` is the layer, ``serve`` the
life of a small batch; it returns what each step computed.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exl3_trellis_quantized_rot_gb300 as tfx  # noqa: E402
import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, BITS = 1024, 8, 2, 256, 4


def weight(seed: int, K: int, N: int, member: int = 0, max_rows: int = 1024) -> tfx.Weight:
    up = lambda a, t: torch.from_numpy(np.ascontiguousarray(a).view(t)).cuda()  # noqa: E731
    # sign vectors scaled so that outputs have about the inputs' size
    svh = (synth.svh(seed, N, member).astype(np.float32) / (1.1547 * K ** 0.5)).astype(np.float16)
    w = tfx.Weight(up(synth.codes(seed, K, N, BITS, member), np.int32), up(synth.suh(seed, K, member), np.int16),
                   up(svh, np.int16), K, N, BITS)
    tfx.reserve(w, max_rows)
    return w


class Layer:
    def __init__(self, slots: int, pages: int, page_size: int, width: int):
        self.qkv = [weight(1, HIDDEN, n * DIM, m) for m, n in enumerate((HEADS, KV_HEADS, KV_HEADS))]
        self.o = weight(2, HEADS * DIM, HIDDEN)
        shape = (1, pages, page_size, KV_HEADS, DIM)
        # pages are never read past what a sequence holds: what they contain before does not matter
        self.cache = tfx.Cache(torch.empty(shape, dtype=torch.float16, device="cuda"),
                               torch.empty(shape, dtype=torch.float16, device="cuda"), slots, width)
        tfx.cache_reserve(self.cache, max_batch=slots, heads=HEADS)

    def project(self, x, seqs, offsets):
        """q of the rows x; their k and v join the cache, rows offsets[i]:offsets[i+1] as sequence seqs[i]'s next tokens."""
        q, k, v = (y.unflatten(1, (-1, DIM)) for y in tfx.group(self.qkv, x))
        tfx.cache_extend(self.cache, seqs, offsets)  # once a step; append once a layer
        tfx.cache_append(self.cache, 0, k, v)
        return q, k, v

    def prompt(self, x, slot: int):
        """A whole prompt into an empty slot."""
        ends = torch.tensor([0, x.shape[0]], dtype=torch.int32)
        q, k, v = self.project(x, torch.tensor([slot], dtype=torch.int32, device="cuda"), ends.cuda())
        a = tfx.attn_prompt(q, k, v, ends)
        return q, a, tfx.linear(self.o, a.flatten(1))

    def step(self, x, seqs, shared: int):
        """One new token a sequence; the first `shared` tokens are the same in all."""
        q, _, _ = self.project(x, seqs, torch.arange(len(seqs) + 1, dtype=torch.int32, device="cuda"))
        a = tfx.attn_decode(self.cache, 0, q, seqs, shared=shared)
        return q, a, tfx.linear(self.o, a.flatten(1))


def serve(system: int = 300, chats: int = 8, steps: int = 3, page_size: int = 32):
    """A system prompt, `chats` forks of it, some steps, then half of them end and the pool is compacted."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rows = lambda n: torch.randn((n, HIDDEN), generator=g, device="cuda").half()  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    width = (system + 4 * steps) // page_size + 2
    layer = Layer(slots=chats + 1, pages=width + 3 * chats, page_size=page_size, width=width)
    told = [("prompt", layer.prompt(rows(system), 0), [0])]
    live = list(range(1, chats + 1))
    tfx.cache_fork(layer.cache, ints(*[0] * chats), ints(*live))
    for _ in range(steps):
        told.append(("step", layer.step(rows(len(live)), ints(*live), system), list(live)))
    tfx.cache_free(layer.cache, ints(*live[::2]))
    tfx.cache_compact(layer.cache)
    live = live[1::2]
    for _ in range(steps):
        told.append(("step", layer.step(rows(len(live)), ints(*live), system), list(live)))
    return layer, told


def main() -> None:
    layer, told = serve()
    for kind, (_, a, y), live in told:
        print(f"{kind:7s} sequences {live}: attention {tuple(a.shape)}, layer output rms {float(y.float().square().mean().sqrt()):.3f}")
    c = layer.cache
    print(f"tokens held {c.lens.tolist()}, pages in use {int((c.refs > 0).sum())} of {c.s.pages}, status {c.status()}")


if __name__ == "__main__":
    main()

"""A decode loop with a budgeted paged cache beside the sparse indexer.

One attention layer of a served model, for a batch of sequences: the prompt's chunk is rotated and appended to the
paged K/V cache, attended, and its attention weight added up per entry; then single tokens follow, and whenever a
sequence's cache has grown past the budget the entries of least weight are evicted in place. The indexer of a sparse
layer runs in the same loop on its own keys: rotated (the second half of each head), quantised and appended to its
FP4 cache, scored, its best positions selected.

    python examples/budgeted_decode.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import long_context_decode_lightning_gb300 as hsi  # noqa: E402


@dataclass
class Config:
    batch: int = 4
    prompt: int = 700        # tokens of the longest prompt; the others are shorter
    steps: int = 200         # decode steps
    budget: int = 512        # entries a cache is cut back to ...
    slack: int = 64          # ... when it holds this many more
    sink: int = 4
    recent: int = 64
    q_heads: int = 32
    kv_heads: int = 8
    dim: int = 128
    page: int = 16
    k: int = 64              # positions the indexer selects
    seed: int = 0


class Layer:
    """The layer's caches and the buffers of a step; every call is enqueued on the current stream."""

    def __init__(self, c: Config, dev="cuda"):
        self.c, B = c, c.batch
        self.gen = torch.Generator(device=dev).manual_seed(c.seed)
        self.prompts = [c.prompt - 37 * b for b in range(B)]
        self.room = max(c.prompt, c.budget + c.slack) + 1      # entries a sequence's pages hold
        pages = -(-self.room // c.page)
        shape = (B * pages, c.page, c.kv_heads, c.dim)
        order = torch.randperm(B * pages, generator=torch.Generator().manual_seed(c.seed))
        self.table = order.view(B, pages).to(torch.int32).to(dev)
        self.kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.kv = hsi.PagedKV(torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                              torch.zeros(shape, dtype=torch.bfloat16, device=dev), self.table, self.kv_len)
        self.acc = torch.zeros(B, c.kv_heads, self.room, device=dev)
        self.keep = torch.empty(B, c.kv_heads, c.budget, dtype=torch.int32, device=dev)
        self.new_len = torch.empty(B, dtype=torch.int32, device=dev)
        self.steps, self.gain = hsi.rope_steps(c.dim, device=dev)
        self.lens = [0] * B                                    # the host's copy of kv_len: it sizes the launches
        self.tokens = 0                                        # positions handed out so far, beyond the prompts'
        # the indexer: 32 heads of 128, the upper half rotated
        self.half, _ = hsi.rope_steps(64, device=dev)
        total = c.prompt + c.steps
        self.recs = hsi.n_records(total)
        self.k_rec = torch.zeros(B * self.recs * hsi.MX_REC_BYTES, dtype=torch.uint8, device=dev)
        self.k_off = torch.arange(B, dtype=torch.int64, device=dev) * self.recs
        self.n_vis = torch.zeros(B, dtype=torch.int32, device=dev)
        self.cap = torch.full((B,), total, dtype=torch.int32, device=dev)
        self.signs = [1 if (i * 2654435761 >> 7) & 1 else -1 for i in range(128)]
        self.total = total

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.kv_len.device).to(torch.bfloat16)

    def attend(self, new: list[int], positions: torch.Tensor):
        """The new tokens of every sequence through the attention layer; returns q, out, lse, q_start."""
        c, dev = self.c, self.kv_len.device
        T, at = sum(new), [0]
        for m in new:
            at.append(at[-1] + m)
        self.lens = [n + m for n, m in zip(self.lens, new)]
        q_start = torch.tensor(at, dtype=torch.int32, device=dev)
        self.kv_len += q_start[1:] - q_start[:-1]
        q, k, v = self.normal(T, c.q_heads, c.dim), self.normal(T, c.kv_heads, c.dim), self.normal(T, c.kv_heads, c.dim)
        hsi.paged_append(self.kv, k, v, q_start, positions=positions, steps=self.steps, gain=self.gain, q=q, q_out=q)
        out, lse = torch.empty_like(q), torch.empty(T, c.q_heads, device=dev)
        scale, longest = c.dim ** -0.5, max(self.lens)
        hsi.paged_attention(self.kv, q, q_start, max(new), longest, scale, out, lse=lse)
        hsi.attention_weights(self.kv, q, lse, q_start, max(new), longest, scale, self.acc, self.acc)
        return q, out, lse, q_start

    def evict(self) -> bool:
        """Cut caches past the budget back to it, in place."""
        c = self.c
        if max(self.lens) < c.budget + c.slack:
            return False
        hsi.evict_select(self.acc, self.kv_len, max(self.lens), c.budget, self.keep, self.new_len, sink=c.sink,
                         recent=c.recent, acc_out=self.acc)
        hsi.paged_compact(self.kv, self.keep, self.new_len)
        self.kv_len.copy_(self.new_len)
        self.lens = [min(n, c.budget) for n in self.lens]
        return True

    def index(self, positions: torch.Tensor):
        """One token of the indexer: its key into the FP4 cache, its queries scored against it; the best positions."""
        c, dev = self.c, self.kv_len.device
        B = c.batch
        k_x, q_x = self.normal(B, 1, 128), self.normal(B, 32, 128)
        w = torch.randn(B, 32, generator=self.gen, device=dev) / 32 ** 0.5
        hsi.rope(k_x, positions, self.half, k_x, rot_offset=64, interleaved=True)
        hsi.rope(q_x, positions, self.half, q_x, rot_offset=64, interleaved=True)
        q_rec = torch.empty(B * 4 * hsi.MX_REC_BYTES, dtype=torch.uint8, device=dev)
        hsi.quantize_mxfp4(q_x, B, 32, self.signs, q_rec)
        hsi.append_token(k_x, self.signs, None, self.k_rec, self.k_off, self.n_vis, self.cap, B, fmt=hsi.FMT_MXFP4)
        scores = torch.empty(B, self.total, device=dev)
        idx = torch.empty(B, c.k, dtype=torch.int32, device=dev)
        val = torch.empty(B, c.k, device=dev)
        hsi.full_layer(q_rec, None, w, self.k_rec, None, self.k_off, self.n_vis, B, self.total, scores, c.k, idx, val,
                       fmt=hsi.FMT_MXFP4)
        return idx

    def prompt(self):
        dev = self.kv_len.device
        pos = torch.cat([torch.arange(n, dtype=torch.int32, device=dev) for n in self.prompts])
        return self.attend(self.prompts, pos)

    def step(self):
        """One token a sequence; returns the attention's and the indexer's results."""
        dev = self.kv_len.device
        pos = torch.tensor([n + self.tokens for n in self.prompts], dtype=torch.int32, device=dev)
        self.tokens += 1
        self.evict()
        return self.attend([1] * self.c.batch, pos), self.index(pos)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    c = Config(steps=ap.parse_args().steps)
    hsi.build()
    hsi.device_check()
    layer = Layer(c)
    layer.prompt()
    print("after the prompt:", layer.kv_len.tolist())
    for i in range(c.steps):
        (_, out, _, _), idx = layer.step()
    torch.cuda.synchronize()
    assert hsi.device_error() == 0
    print(f"after {c.steps} steps: {layer.kv_len.tolist()} entries, out {tuple(out.shape)}, indexer top-{c.k} {tuple(idx.shape)}")
    print("weight gathered by the first entries:", [round(v, 1) for v in layer.acc[0, 0, :4].tolist()])


if __name__ == "__main__":
    main()

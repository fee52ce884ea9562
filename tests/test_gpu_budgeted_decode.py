"""examples/budgeted_decode.py: the rotary positions, the paged cache, its attention, weights and eviction, and the
indexer, run together for a prompt and a run of tokens, with the attention layer followed in 64 bits."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from paged_cases import DEV, within

import long_context_decode_lightning_gb300 as hsi

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hsi.build()
    hsi.device_check()
    spec = importlib.util.spec_from_file_location("budgeted_decode", os.path.join(ROOT, "examples", "budgeted_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["budgeted_decode"] = mod
    spec.loader.exec_module(mod)
    return mod


def _entries(layer, b):
    """K and V of sequence b's cache [entries, heads, dim] as they lie in the pages."""
    c, n = layer.c, int(layer.kv_len[b])
    pages = layer.table[b, :-(-n // c.page)].long()
    return [t[pages].flatten(0, 1)[:n].double() for t in (layer.kv.k, layer.kv.v)]


@pytest.mark.parametrize("kw", [dict(), dict(batch=3, prompt=260, budget=96, slack=8, sink=1, recent=16, q_heads=14,
                                             kv_heads=2, dim=64, page=8, steps=40)])
def test_the_loop(example, kw):
    c = example.Config(**{"steps": 90, **kw})
    layer = example.Layer(c)
    acc = torch.zeros_like(layer.acc, dtype=torch.float64)
    evictions = 0

    def check(q, out, lse, q_start, new):
        scale, group = c.dim ** -0.5, c.q_heads // c.kv_heads
        for b in range(c.batch):
            K, V = _entries(layer, b)
            m, n, at = new[b], K.shape[0], int(q_start[b])
            seen = torch.ones(m, n, dtype=torch.bool, device=DEV).tril(n - m)
            for h in range(c.q_heads):
                g = h // group
                s = torch.where(seen, q[at:at + m, h].double() @ K[:, g].T * scale, -torch.inf)
                p = torch.softmax(s, 1)
                # bf16: P and the result are rounded once each (2^-8), the scores' error is far below
                within(out[at:at + m, h], p @ V[:, g], 2.0 ** -8 * ((p @ V[:, g]).abs() + 1.01 * (p @ V[:, g].abs())))
                acc[b, g, :n] += p.sum(0)
        # sums of exp(score - lse), each within some 2^-17 of itself; they pile up over the steps
        within(layer.acc, acc, 2.0 ** -15 * acc + 1e-12, "weights")

    check(*layer.prompt(), layer.prompts)
    for i in range(c.steps):
        lens, before, was = list(layer.lens), acc.clone(), layer.acc.clone()
        (q, out, lse, q_start), idx = layer.step()
        if max(lens) >= c.budget + c.slack:
            evictions += 1
            for b in range(c.batch):
                n = min(lens[b], c.budget)
                for g in range(c.kv_heads):
                    kept = layer.keep[b, g, :n].long()
                    assert bool((kept[1:] > kept[:-1]).all()) and int(kept[-1]) == lens[b] - 1
                    dropped = torch.ones(lens[b], dtype=torch.bool, device=DEV)
                    dropped[kept] = False
                    if bool(dropped.any()):  # nothing dropped weighs more than what was kept for its weight
                        free = kept[(kept >= c.sink) & (kept < lens[b] - c.recent)]
                        assert float(was[b, g, :lens[b]][dropped].max()) <= float(was[b, g, free].min())
                    acc[b, g] = 0
                    acc[b, g, :n] = before[b, g, kept]
        check(q, out, lse, q_start, [1] * c.batch)
        assert bool((idx.max(1).values == 0).all()) if i == 0 else bool((idx.max(1).values <= i).all())
    assert evictions >= 1 and max(layer.lens) < c.budget + c.slack + 1
    assert hsi.device_error() == 0

"""The .aligned barriers of the paged-cache kernels, by reading: each stands in a helper that brings the warp's lanes
together first, and no kernel writes one of its own."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "long_context_decode_lightning_gb300", "csrc")
BARRIER = re.compile(r'"(?:barrier\.cluster\.arrive[^"]*|bar\.sync|barrier\.sync)[^"]*"')


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_barriers_come_after_syncwarp():
    text = _source("ptx.cuh")
    found = list(BARRIER.finditer(text))
    assert len(found) >= 2
    for m in found:
        body = text[text.rindex("{", 0, text.rindex("asm volatile", 0, m.start())):m.start()]
        assert "__syncwarp();" in body, m.group()


def test_paged_kernels_use_the_helpers():
    for name in ("attend.cuh", "attend_chunk.cuh", "weights.cuh", "evict.cuh", "rope.cuh", "paged.cuh"):
        assert not BARRIER.search(_source(name)), name

"""Rotary positions and the paged cache without a GPU: the steps of every scaling against their formulas, and
the host-side refusals (validation fails before a pointer is used)."""
import ctypes
import math
import shutil

import pytest
import torch

import long_context_decode_lightning_gb300 as hsi

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not on PATH")


@pytest.fixture(scope="module")
def L():
    hsi.build()
    return hsi.lib()


def _inv_freq(rot, base, scaling, f, length, fast, slow):
    if scaling == "ntk":
        base *= f ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        inv = [v / f for v in inv]
    if scaling == "yarn":
        lo, hi = (rot * math.log(length / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (fast, slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        out = []
        for i, v in enumerate(inv):
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(v * (1 - r) + v / f * r)
        inv = out
    return inv


@needs_nvcc
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base,f,length", [(64, 10000.0, 8.0, 4096), (128, 500000.0, 40.0, 65536), (32, 10000.0, 1.0, 2048)])
def test_rope_steps(L, scaling, rot, base, f, length):
    steps, gain = hsi.rope_steps(rot, base, scaling, f, length, device="cpu")
    want = [round(v / (2 * math.pi) * 2.0 ** 64) for v in _inv_freq(rot, base, scaling, f, length, 32.0, 1.0)]
    for got, w in zip(steps.tolist(), want):
        assert abs(got - w) <= w * 2.0 ** -48  # two libraries' pow
    assert gain == pytest.approx(0.1 * math.log(f) + 1.0 if scaling == "yarn" else 1.0, rel=1e-6)


@needs_nvcc
def test_rope_refusals(L):
    fake = 1 << 20
    s, g = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    steps = lambda *a: L.hsi_rope_steps(*a, s, ctypes.byref(g))  # noqa: E731
    assert steps(64, 10000.0, 0, 0.0, 0.0, 0.0, 0.0) == 0
    assert steps(63, 10000.0, 0, 1.0, 0.0, 0.0, 0.0) == -1
    assert steps(64, 1.0, 0, 1.0, 0.0, 0.0, 0.0) == -1
    assert steps(64, math.nan, 0, 1.0, 0.0, 0.0, 0.0) == -1
    assert steps(64, 10000.0, 4, 1.0, 0.0, 0.0, 0.0) == -1
    assert steps(64, 10000.0, 1, 0.5, 0.0, 0.0, 0.0) == -1
    assert steps(2, 10000.0, 2, 2.0, 0.0, 0.0, 0.0) == -1
    assert steps(64, 10000.0, 3, 2.0, 0.0, 32.0, 1.0) == -1
    assert steps(64, 10000.0, 3, 2.0, 4096.0, 1.0, 32.0) == -1

    def rope(x=fake, y=fake * 2, dt=0, T=4, H=2, D=64, pos=fake, st=fake, rot=64, off=0, gain=1.0, xs=(128, 64), ys=(128, 64)):
        return L.hsi_rope(x, *xs, dt, T, H, D, pos, st, rot, off, 0, gain, 0, y, *ys, None)

    assert rope(x=None) == -1 and rope(y=None) == -1 and rope(pos=None) == -1 and rope(st=None) == -1
    assert rope(dt=3) == -1 and rope(T=0) == -1 and rope(H=0) == -1
    assert rope(rot=63) == -1 and rope(rot=66) == -1 and rope(off=2) == -1 and rope(off=-2, rot=32) == -1
    assert rope(gain=math.nan) == -1
    assert rope(x=fake + 1) == -1
    assert rope(y=fake, ys=(256, 64)) == -1  # in place needs the same strides
    assert rope(ys=(32, 64)) == -1 and rope(ys=(128, 32)) == -1  # results over each other


def _cache(**kw):
    a = dict(k=1 << 20, v=1 << 21, page_stride=16 * 128, token_stride=128, head_stride=64, n_pages=10, table=1 << 20,
             ld_table=4, kv_len=1 << 20, B=2, heads=2, dim=64, page_size=16, dtype=0)
    a.update(kw)
    return ctypes.byref(hsi._PagedKV(**a))


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(kv_len=None), -1), (dict(B=0), -1),
              (dict(heads=0), -1), (dict(n_pages=0), -1), (dict(ld_table=0), -1), (dict(k=(1 << 20) + 8), -1),
              (dict(page_stride=16 * 128 + 4), -1), (dict(token_stride=60), -1), (dict(head_stride=32), -1),
              (dict(page_stride=-128), -1), (dict(dtype=3), -1), (dict(dtype=2), -2), (dict(dim=96), -2),
              (dict(page_size=24), -2), (dict(page_size=4), -2), (dict(page_size=8192), -2), (dict(page_size=0), -1)]


@needs_nvcc
@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(L, kw, status):
    f, c = 1 << 20, _cache(**kw)
    assert L.hsi_paged_append(c, f, 128, 64, f, 128, 64, f, 3, None, None, 0, 0, 0, 1.0, None, 0, 0, 0, None, 0, 0, None) == status
    assert L.hsi_paged_attention(c, f, 256, 64, 4, f, 3, 3, 60, 0.1, 1, 2 * f, 256, 64, None, f, 1 << 40, None) == status
    assert L.hsi_attention_weights(c, f, 256, 64, 4, f, f, 3, 3, 60, 0.1, 1, 1.0, None, 0, f, 64, None) == status
    assert L.hsi_paged_compact(c, f, 32, f, 32, f, 4, None) == status


@needs_nvcc
def test_refusals(L):
    f, c = 1 << 20, _cache()
    assert L.hsi_paged_append(None, f, 128, 64, f, 128, 64, f, 3, None, None, 0, 0, 0, 1.0, None, 0, 0, 0, None, 0, 0, None) == -1

    def append(k=f, ks=(128, 64), T=3, pos=f, st=f, rot=64, off=0, q=None, qh=4, qo=None):
        return L.hsi_paged_append(c, k, *ks, f, 128, 64, f, T, pos, st, rot, off, 0, 1.0, q, 256, 64, qh, qo, 256, 64, None)

    assert append(k=None) == -1 and append(k=f + 8) == -1 and append(ks=(132, 64)) == -1 and append(T=0) == -1
    assert append(pos=None) == -1 and append(rot=65) == -1 and append(rot=128) == -1
    assert append(rot=8) == -2 and append(rot=32, off=4) == -2
    assert append(q=f, qo=None) == -1 and append(q=f, qo=2 * f, qh=0) == -1 and append(q=f, qo=2 * f, st=None) == -1

    def attend(q=f, qs=(256, 64), Hq=4, st=f, T=3, mq=3, mkv=60, scale=0.1, out=2 * f, os=(256, 64), ws=f, n=1 << 40):
        return L.hsi_paged_attention(c, q, *qs, Hq, st, T, mq, mkv, scale, 1, out, *os, None, ws, n, None)

    assert attend(q=None) == -1 and attend(q=f + 8) == -1 and attend(qs=(257, 64)) == -1 and attend(Hq=3) == -1
    assert attend(Hq=0) == -1 and attend(st=None) == -1 and attend(T=0) == -1 and attend(mq=0) == -1
    assert attend(mkv=0) == -1 and attend(scale=math.nan) == -1 and attend(out=None) == -1 and attend(out=f) == -1
    assert attend(os=(32, 64)) == -1 and attend(os=(256, 32)) == -1
    assert attend(ws=None) == -5 and attend(ws=f + 16) == -5 and attend(n=8) == -5

    def weights(lse=f, ai=None, la=0, ao=f, lo=60, decay=1.0):
        return L.hsi_attention_weights(c, f, 256, 64, 4, lse, f, 3, 3, 60, 0.1, 1, decay, ai, la, ao, lo, None)

    assert weights(lse=None) == -1 and weights(ao=None) == -1 and weights(lo=59) == -1
    assert weights(ai=f, la=59) == -1 and weights(decay=math.nan) == -1

    def select(acc=f, ld=100, kl=f, B=1, H=1, n=100, budget=50, sink=0, recent=0, keep=f, lk=50, nl=f, ao=None, lo=0):
        return L.hsi_evict_select(acc, ld, kl, B, H, n, budget, sink, recent, keep, lk, nl, ao, lo, None)

    assert select(acc=None) == -1 and select(kl=None) == -1 and select(keep=None) == -1 and select(nl=None) == -1
    assert select(ld=99) == -1 and select(B=0) == -1 and select(H=0) == -1 and select(n=0) == -1 and select(budget=0) == -1
    assert select(sink=-1) == -1 and select(sink=30, recent=21) == -1 and select(lk=49) == -1
    assert select(ao=2 * f, lo=49) == -1
    assert select(n=1 << 19, ld=1 << 19, ao=f, lo=1 << 19) == -2  # in place past the clusters' shared memory

    def compact(keep=f, lk=32, nl=f, budget=32, dst=f, ld=4):
        return L.hsi_paged_compact(c, keep, lk, nl, budget, dst, ld, None)

    assert compact(keep=None) == -1 and compact(nl=None) == -1 and compact(dst=None) == -1 and compact(budget=0) == -1
    assert compact(lk=31) == -1 and compact(ld=1) == -1


def test_binding_checks_before_the_library():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        hsi.PagedKV(k, k, torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        hsi.PagedKV(k, k, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        hsi.PagedKV(k, k.half(), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        hsi.rope_steps(64, scaling="other", device="cpu")

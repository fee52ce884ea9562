"""Rotary positions and the paged cache on the GPU (through the C ABI) against plain forms in 64 bits: every
type, head layout, page size and length where the kernels take another path, with NaN in every place of the
pages that holds no entry."""
import math

import numpy as np
import pytest
import torch

from paged_cases import DEV, UNIT, Case, within

import long_context_decode_lightning_gb300 as hsi

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hsi.build()
    hsi.device_check()
    yield
    assert hsi.device_error() == 0


# ------------------------------------------------------------------- rotation --

def _rotate64(x, pos, steps, gain, off, pairs, inverse):
    """The definition, in 64 bits: the phase in Python integers."""
    rot = 2 * len(steps)
    y = x.double().cpu()
    p = [[(int(a) * (int(s) % (1 << 64))) % (1 << 64) for s in steps.tolist()] for a in pos.tolist()]
    a = torch.tensor([[v * (2 * math.pi / 2 ** 64) for v in r] for r in p], dtype=torch.float64)[:, None, :]
    c, s = gain * a.cos(), gain * a.sin() * (-1 if inverse else 1)
    i = torch.arange(rot // 2)
    m, n = (off + 2 * i, off + 2 * i + 1) if pairs else (off + i, off + rot // 2 + i)
    u, v = y[..., m].clone(), y[..., n].clone()
    y[..., m], y[..., n] = u * c - v * s, u * s + v * c
    # angle: pi 2^-24 from the fp32 phase, sincospi and the two products a few 2^-24 each; the store's rounding
    size = torch.zeros_like(y)
    size[..., m] = size[..., n] = gain * (u.abs() + v.abs())
    return y.to(DEV), (size * 10 * 2.0 ** -24).to(DEV)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H,D,rot,off,pairs,top", [
    (1, 1, 64, 64, 0, True, 10), (64, 32, 128, 64, 64, True, 1 << 20), (33, 5, 128, 128, 0, False, 131072),
    (7, 3, 96, 32, 64, False, 1 << 30), (257, 2, 64, 32, 0, False, 5000), (5, 1, 256, 256, 0, True, 1 << 20),
    (3, 2, 50, 6, 3, False, 999), (4, 3, 41, 10, 7, True, 77),  # dims and offsets of no vector
    (700, 4, 128, 96, 32, True, 40000)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dtype, T, H, D, rot, off, pairs, top, inverse):
    g = torch.Generator(device=DEV).manual_seed(T * 1000 + D)
    x = torch.randn(T, H, D, generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, top, (T,), generator=g, device=DEV, dtype=torch.int32)
    pos[0] = -3  # a negative position turns backwards
    steps, gain = hsi.rope_steps(rot, scaling="yarn", factor=4.0, original_len=4096)
    out = torch.full_like(x, math.nan)
    hsi.rope(x, pos, steps, out, rot_offset=off, interleaved=pairs, gain=gain, inverse=inverse)
    want, tol = _rotate64(x, pos, steps, gain, off, pairs, inverse)
    within(out, want, tol + want.abs() * UNIT[dtype], "rope")
    kept = torch.ones(D, dtype=torch.bool)
    kept[off:off + rot] = False
    assert torch.equal(out[..., kept], x[..., kept])
    y = x.clone()  # in place: bit for bit the same
    hsi.rope(y, pos, steps, y, rot_offset=off, interleaved=pairs, gain=gain, inverse=inverse)
    assert torch.equal(y, out)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_strided_and_unaligned(dtype):
    """Heads of a fused projection, a transposed output, and rows that start off 16 bytes."""
    T, H, D = 19, 4, 64
    steps, gain = hsi.rope_steps(D)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 991
    fused = torch.randn(T, 3 * H, D + 1, device=DEV).to(dtype)
    for x in (fused[:, H:2 * H, :D], fused[:, H:2 * H, 1:], fused[:, ::3, :D]):
        out = torch.full((H, T, D), math.nan, dtype=dtype, device=DEV).transpose(0, 1)
        hsi.rope(x, pos, steps, out, gain=gain)
        want, tol = _rotate64(x, pos, steps, gain, 0, False, False)
        within(out, want, tol + want.abs() * UNIT[dtype], "rope")


def test_rope_gradient():
    """The inverse is the gradient: against central differences of sum(w * rope(x)) (linear: exact but for
    rounding), and <R x, y> = <x, R^T y>."""
    T, H, D, rot, off = 3, 2, 64, 32, 16
    steps, gain = hsi.rope_steps(rot, scaling="yarn", factor=8.0, original_len=2048)
    pos = torch.tensor([0, 5, 70001], dtype=torch.int32, device=DEV)
    x, w = torch.randn(T, H, D, device=DEV), torch.randn(T, H, D, device=DEV)
    out, grad = torch.empty_like(x), torch.empty_like(x)
    for pairs in (True, False):
        kw = dict(rot_offset=off, interleaved=pairs, gain=gain)
        hsi.rope(w, pos, steps, grad, inverse=True, **kw)

        def f(z):
            hsi.rope(z.contiguous(), pos, steps, out, **kw)
            return float((out.double() * w.double()).sum())

        for t, h, d in [(0, 0, 16), (1, 1, 47), (2, 0, 31), (2, 1, 0), (1, 0, 20)]:
            e = torch.zeros_like(x)
            e[t, h, d] = 0.5
            # f sums 384 fp32 values of size below 4 |w|: rounding below 384 * 16 * 2^-23
            assert abs((f(x + e) - f(x - e)) - float(grad[t, h, d])) < 384 * 16 * 2.0 ** -23
        assert abs(f(x) - float((x.double() * grad.double()).sum())) < 384 * 16 * 2.0 ** -23


# --------------------------------------------------------------------- append --

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("layout", ["NHD", "HND", "KV"])
@pytest.mark.parametrize("kv_lens,q_lens,page,D", [
    ([1], [1], 8, 64), ([17, 300, 64], [1, 1, 1], 16, 128), ([40, 33, 129, 7], [40, 0, 100, 7], 32, 64),
    ([1000, 513], [513, 2], 64, 128)])
def test_append(dtype, layout, kv_lens, q_lens, page, D):
    c = Case(3, kv_lens, q_lens, 6, 2, D, page, dtype, layout)
    before_k, before_v = c.k.clone(), c.v.clone()
    T = c.T
    k_new, v_new = (torch.randn(T, 2, D, device=DEV).to(dtype) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (T,), device=DEV, dtype=torch.int32)
    for pairs in (True, False):
        steps, gain = hsi.rope_steps(D if pairs else 32, scaling="ntk", factor=4.0)
        off = 0 if pairs else 16
        q_out = torch.full_like(c.q, math.nan)
        hsi.paged_append(c.kv, k_new, v_new, c.q_start, positions=pos, steps=steps, rot_offset=off, interleaved=pairs,
                         gain=gain, q=c.q, q_out=q_out)
        assert hsi.device_error() == 0
        # rotated exactly as the plain rotation does
        k_rot, q_rot = torch.empty_like(k_new), torch.empty_like(c.q)
        hsi.rope(k_new, pos, steps, k_rot, rot_offset=off, interleaved=pairs, gain=gain)
        hsi.rope(c.q, pos, steps, q_rot, rot_offset=off, interleaved=pairs, gain=gain)
        want_k, want_v = before_k.clone(), before_v.clone()
        t = 0
        for b in range(c.B):
            for i in range(q_lens[b]):
                e = kv_lens[b] - q_lens[b] + i
                p = int(c.table[b, e // page])
                want_k[p, e % page], want_v[p, e % page] = k_rot[t], v_new[t]
                t += 1
        assert torch.equal(q_out, q_rot)
        for got, want in ((c.k, want_k), (c.v, want_v)):
            assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))
    hsi.paged_append(c.kv, k_new, v_new, c.q_start)  # no rotation
    want_k = before_k.clone()
    t = 0
    for b in range(c.B):
        for i in range(q_lens[b]):
            e = kv_lens[b] - q_lens[b] + i
            want_k[int(c.table[b, e // page]), e % page] = k_new[t]
            t += 1
    assert torch.equal(c.k.contiguous().view(torch.int16), want_k.contiguous().view(torch.int16))


def test_append_leaves_out_what_has_no_place():
    c = Case(5, [20, 3], [2, 4], 2, 1, 64, 8, BF)  # sequence 1: four new tokens but three entries
    k = torch.randn(9, 1, 64, device=DEV).to(BF)  # tokens 6 .. 8 belong to nobody
    before = c.k.clone()
    hsi.paged_append(c.kv, k, k, c.q_start)
    assert hsi.device_error() == -6  # the first of the four
    want = before
    want[int(c.table[0, 2]), 2], want[int(c.table[0, 2]), 3] = k[0], k[1]
    for i in range(3):
        want[int(c.table[1, 0]), i] = k[3 + i]
    assert torch.equal(c.k.view(torch.int16), want.view(torch.int16))
    c.table[0, 2] = c.k.shape[0]  # a page that does not exist
    hsi.paged_append(c.kv, k, k, torch.tensor([0, 2, 2], dtype=torch.int32, device=DEV))
    assert hsi.device_error() == -6
    assert torch.equal(c.k.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------ attention --

SHAPES = [
    # kv_lens, q_lens, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 8),
    ([777, 400, 5], [1, 1, 1], 16, 2, 64, 16),
    ([0, 130, 64, 63, 65], [1, 1, 0, 1, 2], 8, 2, 128, 64),
    ([4097, 1], [1, 1], 32, 8, 128, 128),
    ([2000, 1999], [5, 3], 32, 4, 128, 32),
    ([300, 20, 128], [300, 20, 1], 7, 1, 128, 16),
    ([513, 900], [129, 257], 6, 2, 64, 32),
    ([1300], [1000], 4, 4, 128, 256),
    ([10, 3], [4, 9], 6, 3, 64, 8),  # more new tokens than entries: rows that see nothing
    ([1500, 700], [33, 16], 24, 2, 128, 64),
    ([2300], [384], 16, 2, 64, 64),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv_lens,q_lens,Hq,Hkv,D,page", SHAPES)
def test_attention_and_weights(dtype, causal, kv_lens, q_lens, Hq, Hkv, D, page):
    c = Case(len(kv_lens) * 100 + D, kv_lens, q_lens, Hq, Hkv, D, page, dtype)
    scale = D ** -0.5
    out = torch.full_like(c.q, math.nan)
    lse = torch.full((c.T, Hq), math.nan, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, scale, out, lse=lse, causal=causal)
    assert hsi.device_error() == 0
    want, want_lse, tol, tol_lse = c.attention(scale, causal)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    acc = torch.rand(c.B, Hkv, c.max_kv + 3, device=DEV)
    new = torch.full_like(acc, -5.0)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, scale, acc, new, decay=0.9, causal=causal)
    assert hsi.device_error() == 0
    w, wt = c.weights(scale, causal, lse, 0.9, acc)
    for b, n in enumerate(kv_lens):
        assert bool((new[b, :, n:] == -5.0).all())
        for g in range(Hkv):
            within(new[b, g, :n], w[b][g], wt[b][g], f"weights {b} {g}")
    # in place, and from nothing
    again = acc.clone()
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, scale, again, again, decay=0.9, causal=causal)
    none = torch.zeros_like(acc)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, scale, None, none, causal=causal)
    w0, wt0 = c.weights(scale, causal, lse, 1.0, None)
    for b, n in enumerate(kv_lens):
        assert torch.equal(again[b, :, :n], new[b, :, :n])
        for g in range(Hkv):
            within(none[b, g, :n], w0[b][g], wt0[b][g], f"weights from nothing {b} {g}")


@pytest.mark.parametrize("layout", ["HND", "KV"])
@pytest.mark.parametrize("kv_lens,q_lens,group", [([700, 90], [1, 1], 4), ([700, 390], [150, 70], 4)])
def test_attention_layouts_strides_streams(layout, kv_lens, q_lens, group):
    """Other page layouts, q as heads of a fused projection, out transposed, on a stream of its own."""
    c = Case(11, kv_lens, q_lens, 2 * group, 2, 64, 16, BF, layout)
    fused = torch.randn(c.T, 4 * group, 64, device=DEV).to(BF)
    fused[:, group:3 * group] = c.q
    q = fused[:, group:3 * group]
    out = torch.full((2 * group, c.T, 64), math.nan, dtype=BF, device=DEV).transpose(0, 1)
    lse = torch.empty(c.T, 2 * group, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = hsi.paged_attention_workspace(c.kv, q, c.max_q, c.max_kv)
        hsi.paged_attention(c.kv, q, c.q_start, c.max_q, c.max_kv, 0.125, out, lse=lse, ws=ws)
        acc = torch.zeros(2, 2, c.max_kv, device=DEV)
        hsi.attention_weights(c.kv, q, lse, c.q_start, c.max_q, c.max_kv, 0.125, None, acc)
    s.synchronize()
    assert hsi.device_error() == 0
    want, want_lse, tol, tol_lse = c.attention(0.125, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    w, wt = c.weights(0.125, True, lse, 1.0, None)
    for b, n in enumerate(kv_lens):
        for g in range(2):
            within(acc[b, g, :n], w[b][g], wt[b][g], "weights")


@pytest.mark.parametrize("Hq,Hkv,kv_lens,q_lens", [(130, 1, [300, 90], [3, 2]), (256, 2, [140], [1]), (96, 1, [500], [5])])
def test_attention_of_wide_groups(Hq, Hkv, kv_lens, q_lens):
    """Groups past the 128 rows of a tile, and groups that leave part of one empty."""
    c = Case(43, kv_lens, q_lens, Hq, Hkv, 64, 32, BF)
    out, lse = torch.full_like(c.q, math.nan), torch.empty(c.T, Hq, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.125, out, lse=lse)
    want, want_lse, tol, tol_lse = c.attention(0.125, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    acc = torch.zeros(c.B, Hkv, c.max_kv, device=DEV)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, 0.125, None, acc)
    w, wt = c.weights(0.125, True, lse, 1.0, None)
    for b, n in enumerate(kv_lens):
        for g in range(Hkv):
            within(acc[b, g, :n], w[b][g], wt[b][g], "weights")


@pytest.mark.parametrize("m", [1, 40])
def test_attention_of_broadcast_queries(m):
    """One query row expanded over heads and tokens (strides of 0)."""
    c = Case(47, [333, 64], [m, m], 4, 2, 64, 16, BF)
    q = c.q[:1, :1].expand(c.T, 4, 64)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 4, device=DEV)
    hsi.paged_attention(c.kv, q, c.q_start, c.max_q, c.max_kv, 0.125, out, lse=lse)
    c.q = q.contiguous()
    want, want_lse, tol, tol_lse = c.attention(0.125, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    acc = torch.zeros(c.B, 2, c.max_kv, device=DEV)
    hsi.attention_weights(c.kv, q, lse, c.q_start, c.max_q, c.max_kv, 0.125, None, acc)
    w, wt = c.weights(0.125, True, lse, 1.0, None)
    for b, n in enumerate(c.kv_lens):
        for g in range(2):
            within(acc[b, g, :n], w[b][g], wt[b][g], "weights")


@pytest.mark.parametrize("m", [1, 3])
@pytest.mark.parametrize("B,longest", [(40, 900), (70, 5000), (300, 40)])
def test_attention_of_many_sequences(m, B, longest):
    """More sequences than a warp has lanes, of lengths from none on: the line, and the short form."""
    lens = [(i * 7919) % (longest + 1) for i in range(B)]
    lens = [max(n, m) if i % 5 else n for i, n in enumerate(lens)]
    new = [m if n else 0 for n in lens]
    c = Case(53, lens, new, 4, 2, 64, 32, BF)
    out, lse = torch.full_like(c.q, math.nan), torch.empty(c.T, 4, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.125, out, lse=lse)
    assert hsi.device_error() == 0
    want, want_lse, tol, tol_lse = c.attention(0.125, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    acc = torch.zeros(c.B, 2, c.max_kv, device=DEV)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, 0.125, None, acc)
    w, wt = c.weights(0.125, True, lse, 1.0, None)
    for b in range(0, B, 9):
        within(acc[b, 1, :lens[b]], w[b][1], wt[b][1], "weights")


@pytest.mark.parametrize("q_lens", [[1, 1], [200, 140]])
def test_attention_of_a_cache_past_32_bit_offsets(q_lens):
    """The sequences' pages lie behind 2^31 elements of K."""
    page, D, H = 64, 128, 2
    c = Case(13, [900, 333], q_lens, 4, H, D, page, BF, first_page=(1 << 31) // (page * D * H) + 1, spare=1)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 4, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, out, lse=lse)
    want, want_lse, tol, tol_lse = c.attention(0.1, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    acc = torch.zeros(2, H, c.max_kv, device=DEV)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, 0.1, None, acc)
    w, wt = c.weights(0.1, True, lse, 1.0, None)
    for g in range(H):
        within(acc[0, g, :900], w[0][g], wt[0][g], "weights")
    k_new = torch.randn(c.T, H, D, device=DEV).to(BF)
    hsi.paged_append(c.kv, k_new, k_new, c.q_start)
    e = 900 - q_lens[0]
    assert torch.equal(c.k[int(c.table[0, e // page]), e % page], k_new[0])
    assert hsi.device_error() == 0


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [90, 300, 17]])
def test_attention_large_scores_and_repeatability(q_lens):
    """Scores that jump by hundreds (the running maximum moves at most tiles), a negative scale, and the same
    bits from every call."""
    c = Case(17, [1000, 800, 70], q_lens, 8, 2, 128, 32, BF, q_scale=30.0)
    for scale in (1.0, -0.4, 0.0):
        outs = []
        for _ in range(3):
            out, lse = torch.empty_like(c.q), torch.empty(c.T, 8, device=DEV)
            hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, scale, out, lse=lse)
            acc = torch.zeros(3, 2, 1000, device=DEV)
            hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, scale, None, acc)
            outs.append((out, lse, acc))
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
        want, want_lse, tol, tol_lse = c.attention(scale, True)
        within(outs[0][0], want, tol, "out")
        within(outs[0][1], want_lse, tol_lse, "lse")


@pytest.mark.parametrize("q_lens", [[1, 1], [150, 3]])
def test_attention_with_bad_lengths_and_pages(q_lens):
    """A page id of no page reads as zeros, a length past the bound is clamped: both are reported, no result is
    touched outside its place, other sequences keep theirs."""
    c = Case(19, [500, 400], q_lens, 4, 2, 64, 16, BF)
    good, bad = torch.empty_like(c.q), torch.empty_like(c.q)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, good)
    assert hsi.device_error() == 0
    c.table[0, 3] = -1
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, bad)
    assert hsi.device_error() == -6
    assert torch.equal(bad[q_lens[0]:], good[q_lens[0]:]) and bool(torch.isfinite(bad).all())
    c.table[0, 3] = c.table[0, 2]
    want, _, tol, _ = c.attention(0.1, True)
    c.kv_len[1] = 1 << 20
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, 400, 0.1, bad)
    assert hsi.device_error() == -6
    within(bad[q_lens[0]:], want[q_lens[0]:], tol[q_lens[0]:], "clamped")
    start = c.q_start.clone()
    start[1] = -4
    hsi.paged_attention(c.kv, c.q, start, c.max_q, c.max_kv, 0.1, bad)
    assert hsi.device_error() == -6


@pytest.mark.parametrize("q_lens", [[1, 1], [64, 200]])
def test_attention_in_a_graph_over_growing_lengths(q_lens):
    c = Case(23, [600, 512], q_lens, 8, 2, 128, 64, BF)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 8, device=DEV)
    ws = hsi.paged_attention_workspace(c.kv, c.q, c.max_q, c.max_kv)
    full = c.kv_len.clone()

    def step():
        hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.09, out, lse=lse, ws=ws)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([300, 201], [600, 512], [200, 256]):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        short = Case(23, [600, 512], q_lens, 8, 2, 128, 64, BF)
        short.kv_lens, short.K, short.V = lens, [k[:n] for k, n in zip(short.K, lens)], [v[:n] for v, n in zip(short.V, lens)]
        want, want_lse, tol, tol_lse = short.attention(0.09, True)
        within(out, want, tol, "out")
        within(lse, want_lse, tol_lse, "lse")
    c.kv_len.copy_(full)
    assert hsi.device_error() == 0


# ------------------------------------------------------------------- eviction --

def _kept(acc, n, budget, sink, recent):
    """Indices by (protected, weight desc, index asc), ascending."""
    if n <= budget:
        return np.arange(n)
    a = acc[:n].astype(np.float64).copy()
    a[:sink] = np.inf
    if recent:
        a[max(0, n - recent):n] = np.inf
    prot = np.zeros(n, bool)
    prot[:sink] = True
    if recent:
        prot[max(0, n - recent):] = True
    order = sorted(range(n), key=lambda i: (not prot[i], -a[i], i))
    return np.sort(np.array(order[:budget]))


@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([1], 1, 0, 0), ([5, 0, 9], 4, 1, 1), ([1025, 512, 100], 512, 4, 64), ([8192, 8191, 8193], 4000, 0, 0),
    ([20000, 16385], 9999, 4, 1000), ([70000], 1, 0, 1), ([40000, 70001], 65000, 7, 0), ([131072], 100000, 0, 8),
    ([300], 200, 200, 0), ([300], 200, 0, 200), ([300], 301, 3, 3)])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "extreme"])
def test_evict_select(lens, budget, sink, recent, kind):
    H, B, ld = 2, len(lens), max(lens) + 5
    rng = np.random.default_rng(budget + len(kind))
    acc = rng.random((B, H, ld)).astype(np.float32)
    if kind == "ties":
        acc = np.floor(acc ** 4 * 16).astype(np.float32) / 8
    elif kind == "equal":
        acc[:] = 0.25
    elif kind == "extreme":
        acc = (np.sign(acc - 0.5) * np.exp((acc - 0.5) * 170)).astype(np.float32)
        acc[..., ::7], acc[..., 1::11], acc[..., 2::13] = np.inf, -0.0, 0.0
        acc[..., 3::17] = -np.inf
    t = torch.from_numpy(acc).to(DEV)
    kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    keep = torch.full((B, H, budget + 3), -9, dtype=torch.int32, device=DEV)
    new_len = torch.empty(B, dtype=torch.int32, device=DEV)
    out = torch.full((B, H, budget + 2), 7.0, device=DEV)
    hsi.evict_select(t, kv_len, max(lens), budget, keep, new_len, sink=sink, recent=recent, acc_out=out)
    assert hsi.device_error() == 0
    assert new_len.tolist() == [min(n, budget) for n in lens]
    k, o = keep.cpu().numpy(), out.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(H):
            want = _kept(acc[b, h], n, budget, sink, recent)
            m = len(want)
            assert np.array_equal(k[b, h, :m], want)
            assert (k[b, h, m:budget] == -1).all() and (k[b, h, budget:] == -9).all()
            assert np.array_equal(o[b, h, :m].view(np.int32), acc[b, h][want].view(np.int32))
            assert (o[b, h, m:budget] == 0).all() and (o[b, h, budget:] == 7).all()
    if ld >= budget:  # in place: the kept weights in front, zeros behind them
        hsi.evict_select(t, kv_len, max(lens), budget, keep, new_len, sink=sink, recent=recent, acc_out=t)
        got = t.cpu().numpy()
        for b, n in enumerate(lens):
            m = min(n, budget)
            assert np.array_equal(got[b, :, :m].view(np.int32), o[b, :, :m].view(np.int32))
            assert (got[b, :, m:max(lens)] == 0).all()


@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, 0xFFC00000, 0xFFFFFFFF])
@pytest.mark.parametrize("n,budget", [(700, 300), (40000, 20000)])
def test_evict_select_with_nans(bits, n, budget):
    """NaNs rank as numbers past +inf or -inf; the budget is kept exactly, nothing is written outside it."""
    rng = np.random.default_rng(bits % 1000 + n)
    acc = rng.random(n).astype(np.float32)
    bad = np.flatnonzero(rng.random(n) < 0.3)
    acc.view(np.uint32)[bad] = bits
    t = torch.from_numpy(acc).view(1, 1, n).to(DEV)
    keep = torch.full((1, 1, budget + 64), -9, dtype=torch.int32, device=DEV)
    new_len = torch.empty(1, dtype=torch.int32, device=DEV)
    hsi.evict_select(t, torch.tensor([n], dtype=torch.int32, device=DEV), n, budget, keep, new_len, sink=3, recent=10)
    assert hsi.device_error() == 0 and int(new_len) == budget
    rank = acc.copy()
    rank[bad] = np.inf if bits < 1 << 31 else -1.0
    k = keep.cpu().numpy()[0, 0]
    assert np.array_equal(k[:budget], _kept(rank, n, budget, 3, 10)) and (k[budget:] == -9).all()


def test_evict_select_of_rows_past_the_shared_memory():
    n, budget = 500_000, 123_457
    rng = np.random.default_rng(3)
    acc = np.floor(rng.random((1, 1, n)) ** 3 * 30000).astype(np.float32)
    t = torch.from_numpy(acc).to(DEV)
    kv_len = torch.tensor([n], dtype=torch.int32, device=DEV)
    keep = torch.empty(1, 1, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(1, dtype=torch.int32, device=DEV)
    out = torch.empty(1, 1, budget, device=DEV)
    hsi.evict_select(t, kv_len, n, budget, keep, new_len, sink=4, recent=100, acc_out=out)
    assert hsi.device_error() == 0
    want = _kept(acc[0, 0], n, budget, 4, 100)
    assert np.array_equal(keep.cpu().numpy()[0, 0], want)
    assert np.array_equal(out.cpu().numpy()[0, 0], acc[0, 0][want])
    with pytest.raises(hsi.HsiError) as e:
        hsi.evict_select(t, kv_len, n, budget, keep, new_len, acc_out=t)
    assert e.value.status == -2


@pytest.mark.parametrize("lens,budget,page,D,Hkv,layout", [
    ([100, 40, 0], 50, 8, 64, 3, "NHD"), ([2000, 1700], 1111, 16, 128, 2, "HND"), ([3000], 2999, 64, 64, 1, "KV"),
    ([5000, 600], 513, 256, 128, 2, "NHD")])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(lens, budget, page, D, Hkv, layout, in_place):
    need = -(-budget // page)
    c = Case(29, lens, [0] * len(lens), Hkv, Hkv, D, page, BF, layout, spare=need * len(lens))
    acc = torch.rand(c.B, Hkv, max(lens), device=DEV)
    keep = torch.empty(c.B, Hkv, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(c.B, dtype=torch.int32, device=DEV)
    hsi.evict_select(acc, c.kv_len, max(lens), budget, keep, new_len, sink=2, recent=5)
    if in_place:
        dst = c.table
    else:
        used = set(c.table[(c.table >= 0) & (c.table < c.k.shape[0])].tolist())
        free = [p for p in range(c.k.shape[0]) if p not in used]
        dst = torch.tensor(free[:need * c.B], dtype=torch.int32, device=DEV).view(c.B, need)
    before = c.k.clone(), c.v.clone()
    hsi.paged_compact(c.kv, keep, new_len, None if in_place else dst)
    assert hsi.device_error() == 0
    for pages, was, src in ((c.k, before[0], c.K), (c.v, before[1], c.V)):
        want = was.clone()
        for b in range(c.B):
            for h in range(Hkv):
                for i, e in enumerate(keep[b, h, :int(new_len[b])].tolist()):
                    want[int(dst[b, i // page]), i % page, h] = src[b][e, h]
        assert torch.equal(pages.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


@pytest.mark.parametrize("lens,budget,D,Hkv", [([60000], 50000, 64, 1), ([40000, 33000], 30001, 128, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact_of_long_sequences(lens, budget, D, Hkv, in_place):
    page, B = 64, len(lens)
    need = -(-budget // page)
    c = Case(59, lens, [0] * B, Hkv, Hkv, D, page, BF, spare=need * B)
    acc = torch.rand(B, Hkv, max(lens), device=DEV)
    keep = torch.empty(B, Hkv, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(B, dtype=torch.int32, device=DEV)
    hsi.evict_select(acc, c.kv_len, max(lens), budget, keep, new_len)
    dst = c.table
    if not in_place:
        used = set(c.table[(c.table >= 0) & (c.table < c.k.shape[0])].tolist())
        free = [p for p in range(c.k.shape[0]) if p not in used]
        dst = torch.tensor(free[:need * B], dtype=torch.int32, device=DEV).view(B, need)
    want = [c.k.clone(), c.v.clone()]
    for pages, src in zip(want, (c.K, c.V)):
        for b in range(B):
            n = int(new_len[b])
            i = torch.arange(n, device=DEV)
            for h in range(Hkv):
                pages[dst[b, i // page].long(), i % page, h] = src[b][keep[b, h, :n].long(), h]
    hsi.paged_compact(c.kv, keep, new_len, None if in_place else dst)
    assert hsi.device_error() == 0
    for pages, w in zip((c.k, c.v), want):
        assert torch.equal(pages.view(torch.int16), w.view(torch.int16))


def test_compact_skips_what_is_wrong():
    c = Case(31, [100], [0], 1, 1, 64, 16, BF)
    before = c.k.clone()
    keep = torch.tensor([[[0, 100, 1 << 30, -1]]], dtype=torch.int32, device=DEV)
    hsi.paged_compact(c.kv, keep, torch.tensor([4], dtype=torch.int32, device=DEV))
    assert hsi.device_error() == -6
    assert torch.equal(c.k.view(torch.int16), before.view(torch.int16))


# ------------------------------------------------------------------ refusals --

# short form, line, chunk kernels; few entries for many rows (clusters share the weights' units)
@pytest.mark.parametrize("kv_lens,q_lens", [([900, 500], [1, 1]), ([20000, 12000], [1, 1]), ([3000, 1000], [150, 90]),
                                            ([300], [300])])
def test_wait_that_runs_out_is_reported(kv_lens, q_lens):
    """A copy that is never made: the waits for it end, the status says so, and the next calls are right."""
    c = Case(37, kv_lens, q_lens, 8, 2, 128, 16, BF)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 8, device=DEV)
    acc = torch.zeros(c.B, 2, c.max_kv, device=DEV)

    def attend():
        hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, out, lse=lse)

    def weights():
        hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, 0.1, None, acc)

    attend()
    assert hsi.device_error() == 0
    for call in (attend, weights):
        try:
            hsi.debug_set(hsi.DEBUG_WAIT_LIMIT_NS, 20_000_000)
            hsi.debug_set(hsi.DEBUG_SKIP_FIRST_COPY, 1)
            call()
            assert hsi.device_error() == -4
        finally:
            hsi.debug_set(hsi.DEBUG_SKIP_FIRST_COPY, 0)
            hsi.debug_set(hsi.DEBUG_WAIT_LIMIT_NS, 1_000_000_000)
    attend()
    weights()
    assert hsi.device_error() == 0
    want, want_lse, tol, tol_lse = c.attention(0.1, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    w, wt = c.weights(0.1, True, lse, 1.0, None)
    for b, n in enumerate(kv_lens):
        for g in range(2):
            within(acc[b, g, :n], w[b][g], wt[b][g], "weights")


def test_refusals():
    c = Case(41, [100], [3], 4, 2, 64, 16, BF)
    out = torch.empty_like(c.q)

    def status(fn):
        with pytest.raises(hsi.HsiError) as e:
            fn()
        return e.value.status

    ws = hsi.paged_attention_workspace(c.kv, c.q, 3, 100)
    assert status(lambda: hsi.paged_attention(c.kv, c.q, c.q_start, 3, 100, 0.1, out, ws=ws[:ws.numel() // 2])) == -5
    assert status(lambda: hsi.paged_attention(c.kv, c.q, c.q_start, 0, 100, 0.1, out, ws=ws)) == -1
    assert status(lambda: hsi.paged_attention(c.kv, c.q, c.q_start, 3, 100, math.nan, out, ws=ws)) == -1
    assert status(lambda: hsi.paged_attention(c.kv, c.q, c.q_start, 3, 100, 0.1, c.q, ws=ws)) == -1
    with pytest.raises(ValueError):
        hsi.paged_attention(c.kv, c.q.half(), c.q_start, 3, 100, 0.1, out)
    with pytest.raises(ValueError):
        hsi.paged_attention(c.kv, c.q, c.q_start.long(), 3, 100, 0.1, out)
    with pytest.raises(ValueError):
        hsi.PagedKV(c.k, c.v[:, ::2], c.table, c.kv_len)
    odd = torch.zeros(4, 24, 2, 64, dtype=BF, device=DEV)  # pages of 24 entries
    kv = hsi.PagedKV(odd, odd.clone(), c.table, c.kv_len)
    assert status(lambda: hsi.paged_attention(kv, c.q, c.q_start, 3, 100, 0.1, out)) == -2
    wide = torch.zeros(4, 16, 2, 96, dtype=BF, device=DEV)
    kv = hsi.PagedKV(wide, wide.clone(), c.table, c.kv_len)
    q96 = torch.zeros(3, 4, 96, dtype=BF, device=DEV)
    assert status(lambda: hsi.paged_attention(kv, q96, c.q_start, 3, 100, 0.1, torch.empty_like(q96))) == -2
    acc = torch.zeros(1, 2, 99, device=DEV)
    lse = torch.zeros(3, 4, device=DEV)
    assert status(lambda: hsi.attention_weights(c.kv, c.q, lse, c.q_start, 3, 100, 0.1, None, acc)) == -1

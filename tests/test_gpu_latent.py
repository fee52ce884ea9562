"""The latent cache against plain forms in 64 bits: append in every format, reading back, and attention with and
without lists, at the lengths, heads, pages and masks where they can go wrong."""
import math

import pytest
import torch

from latent_cases import BF16, DEV, FORMATS, FP4, FP8, FP16, UNIT, Latent, decode, encode, within, x_type

import long_context_decode_lightning_gb300 as hsi

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hsi.build()
    hsi.device_check()
    yield
    assert hsi.device_error() == 0


# --------------------------------------------------------------------- append --

@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("page,gap", [(0, 0), (1, 0), (16, 1), (64, 0)])
@pytest.mark.parametrize("kv_lens,q_lens", [([1], [1]), ([70, 5, 300], [1, 1, 1]), ([130, 64, 9, 33], [130, 7, 0, 33])])
def test_append_as_the_format_keeps_them(fmt, dim, page, gap, kv_lens, q_lens):
    c = Latent(1, kv_lens, q_lens, 1, fmt, dim, page, gap=gap)
    x = torch.cat([c.x[b][n - m:] for b, (n, m) in enumerate(zip(kv_lens, q_lens))])
    for b, (n, m) in enumerate(zip(kv_lens, q_lens)):  # what the new entries hold before does not matter
        for e in range(n - m, n):
            c.data[c.place(b, e)] = 1
    before = c.data.clone()
    wide = torch.zeros(x.shape[0], dim + 24, dtype=x.dtype, device=DEV)
    wide[:, :dim] = x
    hsi.latent_append(c.cache, wide[:, :dim], c.q_start)
    assert hsi.device_error() == 0
    for b, (n, m) in enumerate(zip(kv_lens, q_lens)):
        for e in range(n - m, n):
            assert torch.equal(c.data[c.place(b, e)], c.kept[b][e]), (b, e)
            c.data[c.place(b, e)] = before[c.place(b, e)]
    assert torch.equal(c.data.view(torch.uint8), before.view(torch.uint8))  # and nothing else


def _rows_of_edges(fmt, dim):
    """Values next to the borders of the formats: zeros, ties, the smallest and largest numbers, every exponent."""
    g = torch.Generator(device=DEV).manual_seed(5)
    rows = [torch.zeros(dim, device=DEV), torch.full((dim,), -0.0, device=DEV)]
    for e in list(range(-133, -110, 3)) + [-20, -7, 0, 9, 50, 110, 119, 126]:
        for m in (1.0, 1.75, 1.7578125, 1.5):
            r = torch.rand(dim, generator=g, device=DEV) * 2 - 1
            r[::16] = 1.0
            rows.append(r.double().mul(m * 2.0 ** e).float())
    steps = torch.arange(dim, device=DEV) % 64
    for e in (-118, -3, 0, 7):  # multiples of half a step of E4M3 at every binade: ties
        rows.append((torch.where(steps % 2 == 0, 448.0, 0.0) * (steps % 16 == 0) + (2 * steps + 1) * 2.0 ** -10)
                    .double().mul(2.0 ** e).float())
        rows.append(((steps % 17) * 0.25).double().mul(2.0 ** e).float())  # halves of E2M1
    x = torch.stack(rows)
    return x.clamp(-60000, 60000).half() if fmt == FP16 else x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt,dim", [(FP8, 576), (FP8, 512), (FP4, 512)])
def test_append_and_read_back_at_the_formats_borders(fmt, dim):
    x = _rows_of_edges(fmt, dim)
    n = x.shape[0]
    c = Latent(2, [n], [n], 1, fmt, dim, 0)
    hsi.latent_append(c.cache, x, c.q_start)
    want = encode(fmt, x)
    at = int(c.offsets[0])
    off = (c.data[at:at + n] != want).nonzero()
    assert not off.numel(), [(r, i, x[r, i].item(), int(c.data[at + r, i]), int(want[r, i])) for r, i in off[:5].tolist()]
    if fmt == FP4:  # the library's own main-KV entry
        kv = torch.zeros(n, 288, dtype=torch.uint8, device=DEV)
        hsi.quantize_mainkv(x, kv)
        assert torch.equal(kv, want)
    back = torch.empty(n, dim, dtype=torch.bfloat16, device=DEV)
    hsi.latent_read(c.cache, back, c.q_start)
    assert hsi.device_error() == 0
    assert torch.equal(back.double(), decode(fmt, dim, want))  # every value is exact


@pytest.mark.parametrize("fmt", [FP8, FP4])
def test_append_reports_what_is_not_finite(fmt):
    for bad in (math.inf, -math.inf, math.nan):
        c = Latent(3, [20], [3], 1, fmt, 512, 16)
        x = torch.randn(3, 512, device=DEV).bfloat16()
        x[1, 77] = bad
        hsi.latent_append(c.cache, x, c.q_start)
        assert hsi.device_error() == -6
        for i in (0, 2):
            assert torch.equal(c.data[c.place(0, 17 + i)], encode(fmt, x[i:i + 1])[0])


def _rotated(x, pos, rot, off, pairs, gain):
    """fp64 rotation and its error bound: the angle's cosine and sine are off by less than 2^-21 (an fp32 phase of at
    most pi, and sincospif), and each of the two products and their sum rounds once in fp32. In fp16 numbers below 2^-14
    are 2^-24 apart, so that their rounding is off by up to 2^-25 however small they are."""
    y, tol = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    half = rot // 2
    for i in range(half):
        a = pos.double() * 10000.0 ** (-2.0 * i / rot)
        m, n = (off + 2 * i, off + 2 * i + 1) if pairs else (off + i, off + half + i)
        u, v = x[:, m].double(), x[:, n].double()
        y[:, m], y[:, n] = gain * (u * a.cos() - v * a.sin()), gain * (u * a.sin() + v * a.cos())
        tol[:, m] = tol[:, n] = gain * (u.abs() + v.abs()) * 2.0 ** -20 + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    return y, tol


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("rot,off,pairs", [(64, None, True), (64, None, False), (32, 8, False), (16, 480, True),
                                           (512, 0, False)])
def test_append_rotates(fmt, dim, rot, off, pairs):
    c = Latent(4, [40, 100000 if fmt == FP8 and rot == 64 else 77], [7, 13], 1, fmt, dim, 16)
    x = torch.randn(20, dim, device=DEV).to(x_type(fmt))
    pos = torch.randint(-5, 1 << 20, (20,), device=DEV, dtype=torch.int32)
    steps, _ = hsi.rope_steps(rot, 10000.0)
    gain = 1.25
    hsi.latent_append(c.cache, x, c.q_start, positions=pos, steps=steps, rot_offset=off, interleaved=pairs, gain=gain)
    assert hsi.device_error() == 0
    got = torch.stack([c.data[c.place(b, n - m + i)] for b, (n, m) in enumerate(zip(c.kv_lens, c.q_lens))
                       for i in range(m)])
    # as hsi.rope turns them, then kept as they are
    y = x.view(20, 1, dim).clone()
    hsi.rope(y, pos, steps, y, rot_offset=dim - rot if off is None else off, interleaved=pairs, gain=gain)
    y = y.view(20, dim)
    want, tol = _rotated(x, pos, rot, dim - rot if off is None else off, pairs, gain)
    within(y, want, tol + UNIT[x.dtype] * (want.abs() + tol), "rope")
    if fmt in (BF16, FP16):
        within(got, want, tol + UNIT[x.dtype] * (want.abs() + tol), "entries")
    else:
        assert torch.equal(got, encode(fmt, y))


@pytest.mark.parametrize("start", [[0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [6, 4, 2, 0]])
def test_append_reports_a_wrong_q_start(start):
    c = Latent(5, [30, 30, 30], [2, 2, 2], 1, BF16, 512, 16)
    before = c.data.clone()
    x = torch.ones(6, 512, device=DEV).bfloat16()
    hsi.latent_append(c.cache, x, torch.tensor(start, dtype=torch.int32, device=DEV))
    assert hsi.device_error() == -6
    ok = {(0, 4, 2, 6): [], (-1, 2, 4, 6): [(1, 28), (1, 29), (2, 28), (2, 29)],
          (0, 2, 4, 7): [(0, 28), (0, 29), (1, 28), (1, 29)], (6, 4, 2, 0): []}[tuple(start)]
    changed = {(b, e) for b in range(3) for e in range(30) if not torch.equal(c.data[c.place(b, e)], before[c.place(b, e)])}
    assert changed <= set(ok) | {(0, 26), (0, 27), (0, 28), (0, 29), (2, 26), (2, 27), (2, 28), (2, 29)}
    assert set(ok) <= changed


def test_append_leaves_out_what_has_no_place():
    c = Latent(6, [20, 20, 20], [3, 3, 3], 1, FP8, 576, 16, table_pad=0)
    x = torch.randn(12, 576, device=DEV).bfloat16()
    before = c.data.clone()
    c.kv_len.copy_(torch.tensor([2, 34, 20], dtype=torch.int32))  # before the start, past the table
    c.table[2, 1] = 1 << 20                                       # no such page
    hsi.latent_append(c.cache, x, c.q_start)                      # (tokens 9 .. 11 belong to no sequence)
    assert hsi.device_error() == -6
    want = before.clone()
    for tok, (b, e) in {1: (0, 0), 2: (0, 1), 3: (1, 31)}.items():
        want[c.place(b, e)] = encode(FP8, x[tok:tok + 1])[0]
    assert torch.equal(c.data, want)
    c = Latent(6, [20, 20], [1, 1], 1, FP8, 576, 0)
    before = c.data.clone()
    c.offsets.copy_(torch.tensor([-1, c.data.shape[0] - 19]))
    hsi.latent_append(c.cache, x[:2], c.q_start)
    assert hsi.device_error() == -6
    assert torch.equal(c.data, before)


# ----------------------------------------------------------------------- read --

@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("page,gap", [(0, 1), (1, 0), (32, 0)])
def test_read(fmt, dim, page, gap):
    lens = [70, 1, 0, 131]
    c = Latent(11, lens, [1, 1, 0, 3], 1, fmt, dim, page, gap=gap)
    # whole sequences, into rows further apart, with rows outside every one left as they were
    start = torch.tensor([2, 72, 73, 73, 204], dtype=torch.int32, device=DEV)
    wide = torch.full((210, dim + 8), -7.0, dtype=x_type(fmt), device=DEV)
    hsi.latent_read(c.cache, wide[:, :dim], start)
    want = torch.full((210, dim), -7.0, dtype=torch.float64, device=DEV)
    want[2:204] = torch.cat(c.values)
    assert torch.equal(wide[:, :dim].double(), want) and bool((wide[:, dim:] == -7).all())
    # parts of sequences
    out = torch.full((12, dim), -7.0, dtype=x_type(fmt), device=DEV)
    start = torch.tensor([0, 5, 6, 6, 11], dtype=torch.int32, device=DEV)
    hsi.latent_read(c.cache, out, start, first=torch.tensor([65, 0, 0, 60], dtype=torch.int32, device=DEV))
    assert torch.equal(out[:11].double(), torch.cat((c.values[0][65:], c.values[1], c.values[3][60:65])))
    assert bool((out[11] == -7).all())
    # lists
    idx = c.lists(12, 37, causal=True, holes=0.3)
    got = torch.full((5, 37, dim), -7.0, dtype=x_type(fmt), device=DEV)
    hsi.latent_read(c.cache, got, c.q_start, idx=idx)
    assert hsi.device_error() == 0
    for t, b in enumerate([0, 1, 3, 3, 3]):
        want = torch.where((idx[t] >= 0)[:, None], c.values[b][idx[t].clamp(min=0).long()], 0.0)
        assert torch.equal(got[t].double(), want), t


@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP8, 576), (FP4, 512)])
def test_read_reports_entries_that_are_not_there(fmt, dim):
    c = Latent(13, [40, 9], [1, 1], 1, fmt, dim, 16)
    out = torch.full((6, dim), -7.0, dtype=x_type(fmt), device=DEV)
    start = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    hsi.latent_read(c.cache, out, start, first=torch.tensor([38, -1], dtype=torch.int32, device=DEV))
    assert hsi.device_error() == -6
    z = torch.zeros(1, dim, dtype=torch.float64, device=DEV)
    assert torch.equal(out.double(), torch.cat((c.values[0][38:40], z, z, c.values[1][:2])))
    idx = torch.tensor([[0, 40, -1], [9, 8, 1 << 30]], dtype=torch.int32, device=DEV)
    got = torch.full((2, 3, dim), -7.0, dtype=x_type(fmt), device=DEV)
    hsi.latent_read(c.cache, got, c.q_start, idx=idx)
    assert hsi.device_error() == -6
    assert torch.equal(got.double(), torch.stack((torch.cat((c.values[0][:1], z, z)), torch.cat((z, c.values[1][8:9], z)))))
    c.table[0, 2] = -1  # a page that is not there
    hsi.latent_read(c.cache, out[:3], torch.tensor([0, 3, 3], dtype=torch.int32, device=DEV),
                    first=torch.tensor([31, 0], dtype=torch.int32, device=DEV))
    assert hsi.device_error() == -6
    assert torch.equal(out[:3].double(), torch.cat((c.values[0][31:32], z, z)))


def test_read_past_32_bit_offsets():
    """A contiguous cache of more than 2^31 bytes and values."""
    n = (1 << 31) // 512 + 1000
    data = torch.zeros(n, 512, dtype=torch.bfloat16, device=DEV)
    x = torch.randn(300, 512, device=DEV).bfloat16()
    data[-300:] = x
    cache = hsi.LatentCache(data, torch.tensor([n], dtype=torch.int32, device=DEV),
                            offsets=torch.zeros(1, dtype=torch.int64, device=DEV))
    out = torch.empty(300, 512, dtype=torch.bfloat16, device=DEV)
    start = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    hsi.latent_read(cache, out, start, first=torch.tensor([n - 300], dtype=torch.int32, device=DEV))
    assert torch.equal(out, x)
    hsi.latent_append(cache, x.flip(0).contiguous(), start)
    hsi.latent_read(cache, out, start, first=torch.tensor([n - 300], dtype=torch.int32, device=DEV))
    assert hsi.device_error() == 0 and torch.equal(out, x.flip(0))


# ------------------------------------------------------------------ attention --

SHAPES = [  # kv_lens, q_lens, heads, page
    ([1], [1], 1, 16),
    ([64, 65, 63, 0], [1, 1, 1, 0], 16, 16),
    ([300, 0, 129, 7], [1, 1, 3, 7], 5, 64),
    ([2500, 700], [1, 1], 128, 64),
    ([1000, 130, 20000], [1, 1, 1], 64, 0),
    ([700, 90], [150, 70], 16, 32),
    ([333, 128, 200], [65, 128, 1], 40, 1),
    ([450], [31], 130, 256),
    ([192, 260], [64, 3], 96, 0),
]


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv_lens,q_lens,H,page", SHAPES)
def test_attention(fmt, dim, causal, kv_lens, q_lens, H, page):
    if causal and any(n < m for n, m in zip(kv_lens, q_lens)):
        kv_lens = [max(n, m) for n, m in zip(kv_lens, q_lens)]
    Latent(21, kv_lens, q_lens, H, fmt, dim, page).check(SCALE, causal)


@pytest.mark.parametrize("fmt,dim", FORMATS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("k", [1, 64, 100, 513])
@pytest.mark.parametrize("kv_lens,q_lens,H,page", [([900, 90, 64], [1, 3, 1], 64, 16), ([450, 1], [40, 1], 16, 0),
                                                   ([700, 33], [2, 1], 128, 64), ([333, 200, 9], [9, 0, 1], 37, 1)])
def test_attention_over_lists(fmt, dim, causal, k, kv_lens, q_lens, H, page):
    c = Latent(22, kv_lens, q_lens, H, fmt, dim, page)
    c.check(SCALE, causal, idx=c.lists(23, k, causal))


@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP16, 512), (FP8, 576), (FP4, 512)])
@pytest.mark.parametrize("kv_lens,q_lens,H,k", [
    ([2000, 300], [170, 40], 64, 0), ([900], [900], 20, 0), ([3000, 100], [130, 60], 48, 130), ([500, 40], [90, 17], 128, 65),
    ([9000], [1], 64, 0), ([5000, 100, 3000, 0, 64, 65], [1, 1, 1, 0, 1, 1], 16, 0), ([300] * 20, [1] * 20, 128, 0),
    ([4000, 90], [2, 1], 128, 1000), ([700] * 100, [1] * 100, 16, 300)])
def test_attention_of_units_in_runs_and_clusters(fmt, dim, kv_lens, q_lens, H, k):
    """More units than SMs, one unit for all of them, clusters of every size, lists of several tiles."""
    c = Latent(49, kv_lens, q_lens, H, fmt, dim, 64)
    c.check(SCALE, True, idx=c.lists(50, k, True) if k else None)


def test_attention_over_odd_lists():
    """Lists that are empty, that hold one entry in their last place, or the same entry many times; rows apart."""
    c = Latent(24, [500, 80], [3, 2], 24, BF16, 576, 16)
    wide = torch.full((5, 300), 1 << 30, dtype=torch.int32, device=DEV)
    idx = wide[:, :200]
    idx.fill_(-1)
    idx[1, 199] = 321
    idx[2, ::3] = 7
    idx[3, 64:128] = torch.arange(64, dtype=torch.int32, device=DEV)
    c.check(SCALE, True, idx=idx)


def test_attention_over_lists_reports_what_a_token_does_not_see():
    c = Latent(25, [100, 50], [2, 1], 16, BF16, 512, 16)
    idx = c.lists(26, 40, True, holes=0)
    good = idx.clone()
    idx[0, 5], idx[1, 39], idx[2, 0] = 99, 100, 1 << 30  # the next token, past the length, far past it
    good[0, 5] = good[1, 39] = good[2, 0] = -1
    hsi.latent_attention(c.cache, c.q, c.q_start, 2, 100, SCALE, c.out, lse=c.lse, idx=idx)
    assert hsi.device_error() == -6
    out, lse, tol, tol_lse = c.attention(SCALE, True, good)
    within(c.out, out, tol)
    within(c.lse, lse, tol_lse)


@pytest.mark.parametrize("q_lens,k", [([1, 1], 0), ([90, 33], 0), ([2, 1], 70)])
def test_attention_strides_streams_and_rows_outside(q_lens, k):
    """Strided q, out and entries, another stream, no lse, rows behind the last sequence, two runs alike."""
    c = Latent(27, [700, 390], q_lens, 20, FP16, 576, 16, gap=1)
    T = c.T
    q = torch.zeros(T + 3, 23, 600, dtype=torch.float16, device=DEV)[:, 1:21, :576]
    q[:T] = c.q
    out = torch.full((T + 3, 22, 520), -5.0, dtype=torch.float16, device=DEV)
    lse = torch.full((T + 3, 20), -5.0, device=DEV)
    idx = None
    if k:
        idx = torch.full((T + 3, k), 1 << 30, dtype=torch.int32, device=DEV)
        idx[:T] = c.lists(28, k, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hsi.latent_attention(c.cache, q, c.q_start, c.max_q, c.max_kv, SCALE, out[:, 2:, :512], lse=lse, idx=idx, stream=s)
    s.synchronize()
    assert hsi.device_error() == 0
    want, wl, tol, tol_lse = c.attention(SCALE, True, None if idx is None else idx[:T])
    within(out[:T, 2:, :512], want, tol)
    within(lse[:T], wl, tol_lse)
    assert bool((out[T:] == -5).all()) and bool((out[:, :2] == -5).all()) and bool((out[..., 512:] == -5).all())
    assert bool((lse[T:] == -5).all())
    again = torch.full_like(out, -5.0)
    hsi.latent_attention(c.cache, q, c.q_start, c.max_q, c.max_kv, SCALE, again[:, 2:, :512], idx=idx)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_attention_of_broadcast_queries():
    c = Latent(29, [300, 200], [3, 1], 32, BF16, 576, 16)
    c.q = c.q[:1, :1].expand(4, 32, 576)
    c.check(SCALE)


@pytest.mark.parametrize("scale", [0.0, -SCALE, 3.0])
@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP16, 512), (FP4, 512)])
def test_attention_at_every_scale(scale, fmt, dim):
    for q_lens, k in (([1, 1], 0), ([40, 9], 0), ([2, 1], 130)):
        c = Latent(30, [900, 300], q_lens, 48, fmt, dim, 64)
        c.check(scale, True, idx=c.lists(31, k, True) if k else None)


@pytest.mark.parametrize("B,longest", [(40, 900), (70, 3000), (300, 40)])
def test_attention_of_many_sequences(B, longest):
    g = torch.Generator().manual_seed(B)
    lens = [int(v) for v in torch.randint(0, longest + 1, (B,), generator=g)]
    new = [min(n, int(v)) for n, v in zip(lens, torch.randint(0, 4, (B,), generator=g))]
    c = Latent(32, lens, new, 16, BF16, 512, 16)
    c.check(SCALE)
    c.check(SCALE, idx=c.lists(33, 33, True))


@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP8, 576)])
def test_attention_of_a_cache_past_32_bit_offsets(fmt, dim):
    page = 64
    first = (1 << 32) // (page * (dim + 80 if fmt == FP8 else 2 * dim)) + 5
    c = Latent(34, [500, 130], [1, 3], 64, fmt, dim, page, first_page=first)
    c.check(SCALE)
    c.check(SCALE, idx=c.lists(35, 90, True))


def test_attention_with_bad_lengths_and_pages():
    """Reported, what can be read is read, and nothing outside the cache is."""
    for k in (0, 50):
        c = Latent(36, [200, 100, 90], [1, 1, 1], 16, BF16, 576, 16, table_pad=0)
        idx = c.lists(37, k, True, holes=0) if k else None
        args = (c.q, c.q_start, 1, 200, SCALE, c.out)
        c.kv_len[1] = -4
        c.table[2, 2] = 1 << 29
        hsi.latent_attention(c.cache, *args, lse=c.lse, idx=idx)
        assert hsi.device_error() == -6
        assert bool((c.lse[1] == -math.inf).all()) and bool((c.out[1] == 0).all())
        out, lse, tol, tol_lse = c.attention(SCALE, True, idx)
        within(c.out[0], out[0], tol[0])
        c.kv_len[1] = 100
        c.kv_len[0] = 100000  # past the table: clamped to what it lists
        hsi.latent_attention(c.cache, *args, lse=c.lse, idx=idx)
        assert hsi.device_error() == -6
        within(c.out[1], out[1], tol[1])


def test_attention_many_small_weights_are_not_lost():
    """One entry far above many equal ones: the sum of what is small is not."""
    for fmt in (BF16, FP16):
        n = 20000
        c = Latent(38, [n], [1], 16, fmt, 512, 64)
        e = torch.zeros(n, 512, dtype=x_type(fmt), device=DEV)
        e[:, 1] = 1.0
        e[5000, 0] = 1.0
        e[5000, 1] = 0.0
        c.values = [e.double()]
        for i in range(0, n, 64):
            c.data[int(c.table[0, i // 64]), :min(64, n - i)] = e[i:i + 64]
        c.q = torch.zeros_like(c.q)
        c.q[..., 0] = 16.0
        c.check(1.0)


@pytest.mark.parametrize("fmt", [BF16, FP16])
@pytest.mark.parametrize("q_lens,k", [([1, 1], 0), ([40, 9], 0), ([3, 2], 500)])
def test_attention_whose_maxima_keep_growing(fmt, q_lens, k):
    """Some heads' scores rise from tile to tile by far more than the sums take without being rescaled, others fall."""
    c = Latent(43, [1500, 700], q_lens, 24, fmt, 512, 64)
    for b, n in enumerate(c.kv_lens):
        c.x[b][:, 0] = (torch.arange(n, device=DEV) // 64) * 2.0
        c.values[b] = c.x[b].double()
        for e in range(0, n, 64):
            c.data[int(c.table[b, e // 64]), :min(64, n - e)] = c.x[b][e:e + 64]
    c.q[:, :, 0] = torch.tensor([12.0, -12.0, 0.0, 3.0, 24.0, 1.0], device=DEV).repeat(4)
    c.check(1.0, True, idx=c.lists(44, k, True).sort(1).values if k else None)


def test_attention_of_more_new_tokens_than_entries():
    """Rows that see nothing beside rows that do: zeros and -inf."""
    for H in (16, 64, 100):
        c = Latent(45, [1, 0, 70, 2], [3, 2, 90, 2], H, BF16, 576, 16)
        c.check(SCALE)
        assert bool((c.out[:2] == 0).all()) and bool((c.lse[:2] == -math.inf).all())
        c.check(SCALE, idx=c.lists(46, 9, True))


@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP8, 576), (FP4, 512)])
@pytest.mark.parametrize("kv_lens,q_lens,k", [([900, 500], [1, 1], 0), ([20000, 12000], [1, 1], 0), ([600], [90], 0),
                                              ([700, 90], [2, 3], 200)])
def test_wait_that_runs_out_is_reported(fmt, dim, kv_lens, q_lens, k):
    """A copy that is never made: the waits for it end, the status says so, and the next call is right."""
    c = Latent(47, kv_lens, q_lens, 32, fmt, dim, 16)
    idx = c.lists(48, k, True) if k else None
    c.check(SCALE, idx=idx)
    try:
        hsi.debug_set(hsi.DEBUG_WAIT_LIMIT_NS, 20_000_000)
        hsi.debug_set(hsi.DEBUG_SKIP_FIRST_COPY, 1)
        hsi.latent_attention(c.cache, c.q, c.q_start, c.max_q, c.max_kv, SCALE, c.out, lse=c.lse, idx=idx)
        assert hsi.device_error() == -4
    finally:
        hsi.debug_set(hsi.DEBUG_SKIP_FIRST_COPY, 0)
        hsi.debug_set(hsi.DEBUG_WAIT_LIMIT_NS, 1_000_000_000)
    c.check(SCALE, idx=idx)


def test_attention_on_two_streams_at_once():
    """Calls with a workspace each, side by side."""
    cases = [Latent(50 + i, [3000, 900], [1, 1], 64, fmt, 576, 64) for i, fmt in enumerate([BF16, FP8])]
    streams = [torch.cuda.Stream() for _ in cases]
    work = [hsi.latent_attention_workspace(c.cache, c.q, 1, 3000) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, ws in zip(cases, streams, work):
            hsi.latent_attention(c.cache, c.q, c.q_start, 1, 3000, SCALE, c.out, lse=c.lse, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert hsi.device_error() == 0
    for c in cases:
        out, lse, tol, tol_lse = c.attention(SCALE, True)
        within(c.out, out, tol)
        within(c.lse, lse, tol_lse)


@pytest.mark.parametrize("q_lens,k", [([1, 1], 0), ([33, 2], 0), ([2, 1], 70)])
def test_nan_query_gives_nan(q_lens, k):
    c = Latent(39, [600, 300], q_lens, 16, BF16, 576, 64)
    idx = c.lists(40, k, True) if k else None
    c.q[0, 3, 100] = math.nan
    hsi.latent_attention(c.cache, c.q, c.q_start, c.max_q, c.max_kv, SCALE, c.out, lse=c.lse, idx=idx)
    assert hsi.device_error() == 0
    bad = torch.zeros_like(c.lse, dtype=torch.bool)
    bad[0, 3] = True
    assert torch.equal(torch.isnan(c.lse), bad)
    assert torch.equal(torch.isnan(c.out).any(-1), bad) and torch.equal(torch.isnan(c.out).all(-1), bad)


@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP8, 576)])
def test_calls_in_a_graph_over_growing_lengths(fmt, dim):
    """Append, attention and reading back as a decode loop replays them."""
    lens = [130, 60, 1]
    c = Latent(41, [n + 8 for n in lens], [1, 1, 1], 64, fmt, dim, 16)
    grow = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c.kv_len.copy_(grow)
    x = torch.zeros(3, dim, dtype=torch.bfloat16, device=DEV)
    back = torch.zeros(3, dim, dtype=torch.bfloat16, device=DEV)
    last = torch.zeros(3, dtype=torch.int32, device=DEV)
    ws = hsi.latent_attention_workspace(c.cache, c.q, 1, 200)

    def step():
        c.kv_len.add_(1)
        hsi.latent_append(c.cache, x, c.q_start)
        hsi.latent_attention(c.cache, c.q, c.q_start, 1, 200, SCALE, c.out, lse=c.lse, ws=ws)
        torch.sub(c.kv_len, 1, out=last)
        hsi.latent_read(c.cache, back, c.q_start, first=last)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.kv_len.copy_(grow)
    for i in range(8):
        x.copy_(torch.randn(3, dim, device=DEV))
        graph.replay()
        assert hsi.device_error() == 0
        kept = encode(fmt, x)
        for b in range(3):
            e = lens[b] + i
            assert torch.equal(c.data[c.place(b, e)], kept[b])
            c.values[b][e] = decode(fmt, dim, kept[b:b + 1])[0]
        c.kv_lens = [n + i + 1 for n in lens]
        values, c.values = c.values, [v[:n] for v, n in zip(c.values, c.kv_lens)]
        out, lse, tol, tol_lse = c.attention(SCALE, True)
        c.values = values
        within(c.out, out, tol)
        within(c.lse, lse, tol_lse)
        assert torch.equal(back.double(), decode(fmt, dim, kept))


def test_main_kv_after_the_indexer_s_selection():
    """The library's main KV read in place: what gather_mainkv gives for a selection, and the attention over it."""
    B, n, k = 3, 700, 64
    x = torch.randn(B * n, 512, device=DEV).bfloat16()
    kv = torch.zeros(B * n, 288, dtype=torch.uint8, device=DEV)
    hsi.quantize_mainkv(x, kv)
    off = torch.arange(B, dtype=torch.int64, device=DEV) * n
    vis = torch.tensor([n, 500, 30], dtype=torch.int32, device=DEV)
    scores = torch.randn(B, n, device=DEV)
    idx, val = torch.empty(B, k, dtype=torch.int32, device=DEV), torch.empty(B, k, device=DEV)
    hsi.topk(scores, vis, B, n, k, idx, val)
    rows = torch.empty(B, k, 512, dtype=torch.bfloat16, device=DEV)
    hsi.gather_mainkv(kv, off, vis, idx, k, B, rows)
    cache = hsi.LatentCache(kv, vis, offsets=off, fmt=FP4, dim=512)
    start = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    back = torch.full_like(rows, -1.0)
    hsi.latent_read(cache, back, start, idx=idx)
    assert torch.equal(back, rows)
    q = torch.randn(B, 64, 512, device=DEV).bfloat16()
    out, lse = torch.empty(B, 64, 512, dtype=torch.bfloat16, device=DEV), torch.empty(B, 64, device=DEV)
    hsi.latent_attention(cache, q, start, 1, n, SCALE, out, lse=lse, idx=idx)
    assert hsi.device_error() == 0
    c = Latent(42, [n, 500, 30], [1, 1, 1], 64, FP4, 512, 0)
    c.values = [decode(FP4, 512, kv[b * n:(b + 1) * n]) for b in range(B)]
    want, wl, tol, tol_lse = c.attention(SCALE, True, idx, q=q)
    within(out, want, tol)
    within(lse, wl, tol_lse)

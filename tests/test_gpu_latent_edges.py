"""The latent cache at the edges of its formats, strides and starts, against plain forms in 64 bits."""
import copy
import math

import pytest
import torch

from latent_cases import BF16, DEV, E4M3, FP4, FP8, Latent, nearest, two, within, x_type

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


# ------------------------------------------------- FP8 entries of the largest numbers --

def _largest(dim):
    """Rows whose groups of 64 reach the largest bf16 numbers, 224 to 255 times 2^120, of both signs."""
    g = torch.Generator(device=DEV).manual_seed(61)
    rows = []
    for top in (224, 225, 232, 239, 240, 244, 247, 248, 249, 252, 255):
        for sign in (1.0, -1.0):
            r = (torch.rand(dim, generator=g, device=DEV, dtype=torch.float64) * 2 - 1) * top
            r[::64] = sign * top
            r[5::64] = -sign * top
            r[64:128] *= 2.0 ** -20  # a group of other numbers beside them
            rows.append(r * 2.0 ** 120)
    x = torch.stack(rows)
    x = x.float().bfloat16()
    assert bool(torch.isfinite(x).all())
    return x


def _kept(x):
    """The entry's codes as values, by its definition: e the smallest in [-118, 120] by which the largest of the 64 is at
    most 448, the nearest E4M3 number to x / 2^e, at e = 120 of those up to 240 (256 times 2^120 is past bf16)."""
    codes = x.shape[1] - 64
    d, out, es = x.double(), x.double(), []
    for g in range(0, codes, 64):
        v = d[:, g:g + 64]
        e = torch.full((x.shape[0],), -118, device=DEV)
        for k in range(-118, 120):
            e = torch.where(v.abs().amax(1) > 448.0 * 2.0 ** k, k + 1, e)
        a = v.abs() * two(-e)[:, None]
        table = torch.tensor(E4M3, dtype=torch.float64, device=DEV)
        small = [t for t in E4M3 if t <= 240]
        near = torch.where((e == 120)[:, None], table[nearest(a, small)], table[nearest(a, E4M3)])
        out[:, g:g + 64] = torch.sign(v) * near * two(e)[:, None]
        es.append(e)
    return out, torch.stack(es, 1)


@pytest.mark.parametrize("dim", [512, 576])
def test_fp8_entries_of_the_largest_numbers_read_back_finite(dim):
    x = _largest(dim)
    n = x.shape[0]
    c = Latent(62, [n], [n], 1, FP8, dim, 0)
    hsi.latent_append(c.cache, x, c.q_start)
    back = torch.empty(n, dim, dtype=torch.bfloat16, device=DEV)
    hsi.latent_read(c.cache, back, c.q_start)
    assert hsi.device_error() == 0
    want, e = _kept(x)
    assert int(e.max()) == 120 and int((e == 119).sum()) > 0  # both sides of the border
    at, codes = int(c.offsets[0]), dim - 64
    assert torch.equal(c.data[at:at + n, codes + 128:codes + 128 + codes // 64].long(), e + 127)
    assert torch.equal(back.double(), want)  # finite, and every value is exact
    # at most half a step of E4M3 off, 2^-4 of the value, or of its smallest codes (2^-10 of 2^e)
    off = (back.double() - x.double()).abs()[:, :codes]
    assert bool((off <= x.double().abs()[:, :codes] / 16 + (two(e) * 2.0 ** -10).repeat_interleave(64, 1)).all())


@pytest.mark.parametrize("dim", [512, 576])
def test_attention_over_one_entry_of_the_largest_numbers_is_that_entry(dim):
    x = _largest(dim)
    n = x.shape[0]
    c = Latent(63, [1] * n, [1] * n, 16, FP8, dim, 16)
    hsi.latent_append(c.cache, x, c.q_start)
    c.q.zero_()
    hsi.latent_attention(c.cache, c.q, c.q_start, 1, 1, SCALE, c.out, lse=c.lse)
    assert hsi.device_error() == 0
    assert torch.equal(c.out.double(), _kept(x)[0][:, None, :512].expand(n, 16, 512))
    assert bool((c.lse == 0).all())


# ------------------------------------------------------------- wrong starts of sequences --

STARTS = [[0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [6, 4, 2, 0], [0, 2, 1 << 30, 6], [0, 6, 0, 6]]
FORMS = [(BF16, 576), (FP8, 576), (FP4, 512)]


def owners(start, T):
    """The sequence of each token, from the definition: b where start[b] <= t < start[b+1], where start does not descend
    around t (the sequences that end at or before t are the first b) and b does not leave [0, T]; or -1."""
    B, out = len(start) - 1, []
    for t in range(T):
        ended = [b for b in range(B) if start[b + 1] <= t]
        b = len(ended)
        good = ended == list(range(b)) and b < B and 0 <= start[b] <= t and start[b + 1] <= T
        out.append(b if good else -1)
    return out


def only(c, b, toks, past):
    """Sequence b's tokens of a case, as a case whose new tokens they are (past: of the sequence's tokens, the last one's end)."""
    s = copy.copy(c)
    s.kv_lens, s.q_lens, s.values, s.T = [c.kv_lens[b] - (past - toks[-1] - 1)], [len(toks)], [c.values[b]], len(toks)
    return s


@pytest.mark.parametrize("fmt,dim", FORMS)
@pytest.mark.parametrize("start", STARTS)
def test_read_reports_a_wrong_start(fmt, dim, start):
    c = Latent(71, [300, 280, 260], [2, 2, 2], 1, fmt, dim, 16)
    bounds = torch.tensor(start, dtype=torch.int32, device=DEV)
    first = torch.tensor([10, 20, 30], dtype=torch.int32, device=DEV)
    own = owners(start, 6)
    out = torch.full((6, dim), -7.0, dtype=x_type(fmt), device=DEV)
    hsi.latent_read(c.cache, out, bounds, first=first)
    assert hsi.device_error() == -6
    for t, b in enumerate(own):
        want = c.values[b][10 * (b + 1) + t - start[b]] if b >= 0 else torch.full((dim,), -7.0, device=DEV).double()
        assert torch.equal(out[t].double(), want), t
    idx = torch.randint(0, 250, (6, 70), device=DEV, dtype=torch.int32)
    got = torch.full((6, 70, dim), -7.0, dtype=x_type(fmt), device=DEV)
    hsi.latent_read(c.cache, got, bounds, idx=idx)
    assert hsi.device_error() == -6
    for t, b in enumerate(own):
        assert torch.equal(got[t].double(), c.values[b][idx[t].long()] if b >= 0 else got[t].double() * 0 - 7), t


@pytest.mark.parametrize("fmt,dim", FORMS)
@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("lens", [[40, 50, 60], [300, 280, 260], [9000, 5000, 7000]])  # units whole, in runs, joined
@pytest.mark.parametrize("start", STARTS)
def test_attention_reports_a_wrong_start(fmt, dim, H, lens, start):
    """With lists, tokens around which the starts descend and those of a sequence that leaves the call's tokens are left
    alone. Without, a sequence that leaves them is, and every row is where the starts descend."""
    c = Latent(72, lens, [2, 2, 2], H, fmt, dim, 64)
    bounds = torch.tensor(start, dtype=torch.int32, device=DEV)
    falls = any(a > b for a, b in zip(start, start[1:]))
    idx = torch.randint(0, 35, (6, 70), device=DEV, dtype=torch.int32)
    for lists in (None, idx):
        own = [-1] * 6 if falls and lists is None else owners(start, 6)
        c.out.fill_(-3.0)
        c.lse.fill_(-3.0)
        hsi.latent_attention(c.cache, c.q, bounds, 6, max(lens), SCALE, c.out, lse=c.lse, idx=lists)
        assert hsi.device_error() == -6
        for b in range(3):
            toks = [t for t in range(6) if own[t] == b]
            if not toks:
                continue
            out, lse, tol, tol_lse = only(c, b, toks, start[b + 1]).attention(
                SCALE, True, None if lists is None else lists[toks], q=c.q[toks])
            within(c.out[toks], out, tol, "out")
            within(c.lse[toks], lse, tol_lse, "lse")
        left = [t for t in range(6) if own[t] < 0]
        assert bool((c.out[left] == -3).all()) and bool((c.lse[left] == -3).all())


@pytest.mark.parametrize("longest", [30, 700])
@pytest.mark.parametrize("at", [1, 32, 33, 64, 70])
def test_attention_looks_at_the_starts_of_many_sequences(longest, at):
    c = Latent(76, [longest - b % 20 for b in range(70)], [1] * 70, 16, BF16, 512, 16)
    bounds = c.q_start.clone()
    bounds[at] = at - 2  # before the start of the sequence that it ends
    hsi.latent_attention(c.cache, c.q, bounds, 3, longest, SCALE, c.out, lse=c.lse)
    assert hsi.device_error() == -6
    assert bool((c.out == -3).all()) and bool((c.lse == -3).all())
    c.check(SCALE)


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("lens", [[40, 50, 60], [3000, 2800, 2600]])
def test_attention_of_more_new_tokens_than_the_bound(H, lens):
    """Without lists such a sequence is left alone and reported; with lists the bound is not looked at."""
    c = Latent(73, lens, [2, 5, 1], H, BF16, 576, 64)
    idx = c.lists(74, 70, True)
    hsi.latent_attention(c.cache, c.q, c.q_start, 2, max(lens), SCALE, c.out, lse=c.lse)
    assert hsi.device_error() == -6
    out, lse, tol, tol_lse = c.attention(SCALE, True)
    rows = [0, 1, 7]
    within(c.out[rows], out[rows], tol[rows], "out")
    within(c.lse[rows], lse[rows], tol_lse[rows], "lse")
    assert bool((c.out[2:7] == -3).all()) and bool((c.lse[2:7] == -3).all())
    hsi.latent_attention(c.cache, c.q, c.q_start, 2, max(lens), SCALE, c.out, lse=c.lse, idx=idx)
    assert hsi.device_error() == 0
    out, lse, tol, tol_lse = c.attention(SCALE, True, idx)
    within(c.out, out, tol, "out")
    within(c.lse, lse, tol_lse, "lse")


# ----------------------------------------------------------------------- strides of one row --

@pytest.mark.parametrize("fmt,dim", [(BF16, 576), (FP8, 512)])
def test_strides_that_no_second_row_uses_are_not_looked_at(fmt, dim):
    """One token, one head: what lies between rows does not matter where there is one."""
    c = Latent(75, [90], [1], 1, fmt, dim, 16)
    x = torch.randn(2, dim + 3, device=DEV).bfloat16()[:1, :dim]
    assert x.stride(0) % 8
    before = c.data.clone()
    hsi.latent_append(c.cache, x, c.q_start)
    at = c.place(0, 89)
    dense = torch.zeros_like(c.data)
    dense.copy_(before)
    kept = c.data[at].clone()
    c.data.copy_(before)
    hsi.latent_append(c.cache, x.contiguous(), c.q_start)
    assert torch.equal(kept, c.data[at])
    out = torch.full((2, dim + 3), -7.0, dtype=torch.bfloat16, device=DEV)
    hsi.latent_read(c.cache, out[:1, :dim], c.q_start, first=torch.tensor([89], dtype=torch.int32, device=DEV))
    plain = torch.empty(1, dim, dtype=torch.bfloat16, device=DEV)
    hsi.latent_read(c.cache, plain, c.q_start, first=torch.tensor([89], dtype=torch.int32, device=DEV))
    assert torch.equal(out[:1, :dim], plain) and bool((out[1] == -7).all()) and bool((out[0, dim:] == -7).all())
    odd = torch.full((1, 3 * dim + 4), -7.0, dtype=torch.bfloat16, device=DEV).as_strided((1, 3, dim), (3 * dim + 4, dim, 1))
    idx = torch.tensor([[5, -1, 7]], dtype=torch.int32, device=DEV)
    even = torch.empty(1, 3, dim, dtype=torch.bfloat16, device=DEV)
    hsi.latent_read(c.cache, odd, c.q_start, idx=idx)
    hsi.latent_read(c.cache, even, c.q_start, idx=idx)
    assert torch.equal(odd, even)
    want = torch.empty(1, 1, 512, dtype=torch.bfloat16, device=DEV)
    hsi.latent_attention(c.cache, c.q, c.q_start, 1, 90, SCALE, want)
    q = torch.zeros(2, dim + 4, dtype=torch.bfloat16, device=DEV)
    q[0, :dim] = c.q[0, 0]
    got = torch.full((2, 517), -7.0, dtype=torch.bfloat16, device=DEV)
    hsi.latent_attention(c.cache, q.as_strided((1, 1, dim), (dim + 4, dim + 3, 1)), c.q_start, 1, 90, SCALE,
                         got.as_strided((1, 1, 512), (515, 517, 1)))
    assert hsi.device_error() == 0
    assert torch.equal(got[0, :512], want[0, 0]) and bool((got[0, 512:] == -7).all()) and bool((got[1] == -7).all())

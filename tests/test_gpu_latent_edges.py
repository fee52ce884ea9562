"""The latent cache at the edges of its formats, strides and starts, against plain forms in 64 bits."""
import math

import pytest
import torch

from latent_cases import BF16, DEV, E4M3, FP8, Latent, nearest, two

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

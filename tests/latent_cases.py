"""Shared set-up of the latent-cache tests: caches with poisoned unused places and plain forms in 64 bits."""
import math

import numpy as np
import torch

import long_context_decode_lightning_gb300 as hsi
from paged_cases import DEV, UNIT, within  # noqa: F401

BF16, FP16, FP8, FP4 = hsi.LATENT_BF16, hsi.LATENT_FP16, hsi.LATENT_FP8, hsi.LATENT_FP4
FORMATS = [(BF16, 576), (FP16, 576), (FP8, 576), (BF16, 512), (FP8, 512), (FP4, 512)]
V = 512


def two(e):
    """2^e of whole numbers, exactly, in fp64."""
    return torch.tensor([math.ldexp(1.0, k) for k in range(-130, 130)], dtype=torch.float64, device=e.device)[e.long() + 130]


def x_type(fmt):
    return torch.float16 if fmt == FP16 else torch.bfloat16


def _fields(ebits, mbits, bias):
    """Values of the non-negative codes of a small floating-point type."""
    return [math.ldexp(m, 1 - bias - mbits) if e == 0 else math.ldexp((1 << mbits) + m, e - bias - mbits)
            for e in range(1 << ebits) for m in range(1 << mbits)]


E4M3, E2M1 = _fields(4, 3, 7)[:127], _fields(2, 1, 1)


def nearest(a, values):
    """The index of the value nearest to a >= 0, ties to the even one, the largest for anything above."""
    v = torch.tensor(values, dtype=torch.float64, device=a.device)
    mid = (v[1:] + v[:-1]) / 2
    lo, hi = torch.searchsorted(mid, a.contiguous()), torch.searchsorted(mid, a.contiguous(), right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def encode(fmt, x):
    """Rows of 16-bit values as the cache keeps them."""
    if fmt in (BF16, FP16):
        return x.clone()
    rows, dim = x.shape
    d = x.double()
    sign = torch.signbit(d).to(torch.uint8)
    if fmt == FP8:
        codes = dim - 64
        out = torch.zeros(rows, dim + 80, dtype=torch.uint8, device=x.device)
        for g in range(codes // 64):
            v = d[:, 64 * g:64 * g + 64]
            top = v.abs().amax(1)
            e = torch.full((rows,), 120, dtype=torch.int64, device=x.device)
            for k in range(120, -119, -1):  # the smallest that holds the largest value
                e = torch.where(top <= 448.0 * 2.0 ** k, k, e)
            c = nearest(v.abs() * two(-e)[:, None], E4M3).to(torch.uint8)
            out[:, 64 * g:64 * g + 64] = c + 128 * sign[:, 64 * g:64 * g + 64]
            out[:, codes + 128 + g] = (e + 127).to(torch.uint8)
        out[:, codes:codes + 128] = x[:, codes:].contiguous().view(torch.uint8)
        return out
    out = torch.zeros(rows, 288, dtype=torch.uint8, device=x.device)
    for g in range(32):
        v = d[:, 16 * g:16 * g + 16]
        sb = nearest(v.abs().amax(1) / 6, E4M3)
        s = torch.tensor(E4M3, dtype=torch.float64, device=x.device)[sb][:, None]
        c = nearest(torch.where(s > 0, v.abs() / s, 0.0), E2M1)
        c = torch.where(s > 0, c + 8 * sign[:, 16 * g:16 * g + 16], 0).to(torch.uint8)
        out[:, 8 * g:8 * g + 8] = c[:, 0::2] + 16 * c[:, 1::2]
        out[:, 256 + g] = sb.to(torch.uint8)
    return out


def decode(fmt, dim, e):
    """Entries as fp64 values."""
    if fmt in (BF16, FP16):
        return e.double()
    e4m3 = torch.tensor(E4M3 + [480.0], dtype=torch.float64, device=e.device)
    e4m3 = torch.cat((e4m3, -e4m3))
    if fmt == FP8:
        codes = dim - 64
        s = two(e[:, codes + 128:codes + 128 + codes // 64].long() - 127)
        tail = e[:, codes:codes + 128].contiguous().view(torch.bfloat16).double()
        return torch.cat((e4m3[e[:, :codes].long()] * s.repeat_interleave(64, 1), tail), 1)
    e2m1 = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=e.device)
    c = torch.stack((e[:, :256] & 15, e[:, :256] >> 4), -1).flatten(1).long()
    return e2m1[c] * e4m3[e[:, 256:].long()].repeat_interleave(16, 1)


class Latent:
    """B sequences of kv_lens entries, the last q_lens of them new, in pages (page > 0) or one run a sequence. Every
    place that holds no entry is NaN (bytes: 0xFF), every table slot past a sequence's pages names no page."""

    def __init__(self, seed, kv_lens, q_lens, H, fmt, dim, page, q_scale=1.5, spare=3, table_pad=2, gap=0, first_page=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv_lens, self.q_lens, self.H, self.fmt, self.dim, self.page = list(kv_lens), list(q_lens), H, fmt, dim, page
        self.B, self.T = len(kv_lens), int(sum(q_lens))
        dt = x_type(fmt)
        self.x = [torch.randn(n, dim, generator=g, device=DEV).to(dt) for n in kv_lens]
        self.kept = [encode(fmt, x) for x in self.x]
        self.values = [decode(fmt, dim, e) for e in self.kept]
        width = dim if fmt in (BF16, FP16) else self.kept[0].shape[1]

        def poisoned(*shape):
            if fmt in (BF16, FP16):
                return torch.full(shape, math.nan, dtype=dt, device=DEV)
            return torch.full(shape, 0xFF, dtype=torch.uint8, device=DEV)

        pad = 8 if gap and fmt in (BF16, FP16) else 16 if gap else 0  # entries further apart than their bytes
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device=DEV)
        if page:
            used = [-(-n // page) for n in kv_lens]
            per = max(1, max(used)) + table_pad
            ids = first_page + torch.randperm(sum(used) + spare, generator=torch.Generator().manual_seed(seed))
            self.data = poisoned(first_page + sum(used) + spare, page, width + pad)[..., :width]
            table = torch.full((self.B, per), -7, dtype=torch.int32)
            table[:, 1::2] = 1 << 30
            at = 0
            for b, n in enumerate(kv_lens):
                table[b, :used[b]] = ids[at:at + used[b]].int()
                at += used[b]
                for i in range(used[b]):
                    rows = self.kept[b][i * page:(i + 1) * page]
                    self.data[int(table[b, i]), :rows.shape[0]] = rows
            self.table, self.offsets = table.to(DEV), None
        else:
            starts = [spare + 5 * b + sum(kv_lens[:b]) for b in range(self.B)]
            self.data = poisoned(starts[-1] + kv_lens[-1] + spare, width + pad)[..., :width]
            for b, n in enumerate(kv_lens):
                self.data[starts[b]:starts[b] + n] = self.kept[b]
            self.table, self.offsets = None, torch.tensor(starts, dtype=torch.int64, device=DEV)
        self.q = (torch.randn(max(self.T, 1), H, dim, generator=g, device=DEV) * q_scale).to(dt)
        self.cache = hsi.LatentCache(self.data, self.kv_len, table=self.table, offsets=self.offsets, fmt=fmt, dim=dim)
        self.max_q, self.max_kv = max(1, max(q_lens)), max(1, max(kv_lens))
        self.out = torch.full((max(self.T, 1), H, V), -3.0, dtype=dt, device=DEV)
        self.lse = torch.full((max(self.T, 1), H), -3.0, device=DEV)

    def place(self, b, e):
        """The entry's place in data, as an index."""
        if self.page:
            return int(self.table[b, e // self.page]), e % self.page
        return (int(self.offsets[b]) + e,)

    def lists(self, seed, k, causal, holes=0.1):
        """k distinct entries that each token sees, in no order, some of the places -1 (all of them where it sees none)."""
        g = torch.Generator(device=DEV).manual_seed(seed)
        rows = []
        for b, (n, m) in enumerate(zip(self.kv_lens, self.q_lens)):
            for i in range(m):
                seen = max(0, n - m + i + 1) if causal else n
                e = torch.full((k,), -1, dtype=torch.int32, device=DEV)
                pick = torch.randperm(seen, generator=g, device=DEV)[:k].int()
                e[:pick.numel()] = pick
                if holes:
                    e[torch.rand(k, generator=g, device=DEV) < holes] = -1
                rows.append(e)
        return torch.stack(rows)

    def attention(self, scale, causal, idx=None, q=None):
        """out, lse and the error bounds of each, all fp64.

        A score is a sum of dim products in fp32: off by at most dim 2^-23 of the sum of their sizes, E below. p is
        rounded once to 16 bits (fp16: 2^-25 absolute below its normal range, p <= 1 where it is rounded and the sum of
        p is at least 1), the result once more: u (|out| + sum p |v| / sum p) + 2 E sum p |v| / sum p. A p below fp32's
        smallest normal number, 2^-126 where the row's largest is 1, may count as 0, and so may such a result: with
        values that are 0 in the row's large entries (FP4 has many) nothing else is left of a dim, which is then
        off by up to 2^-126 max |v| for each entry and once more for itself."""
        q = self.q if q is None else q
        u = UNIT[q.dtype]
        out = torch.zeros(self.T, self.H, V, dtype=torch.float64, device=DEV)
        lse = torch.full((self.T, self.H), -math.inf, dtype=torch.float64, device=DEV)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        t = 0
        for b, (n, m) in enumerate(zip(self.kv_lens, self.q_lens)):
            for i in range(m):
                seen = max(0, n - m + i + 1) if causal else n
                kv = self.values[b][:seen] if idx is None else self.values[b][idx[t][idx[t] >= 0].long()]
                if kv.shape[0]:
                    Q, val = q[t].double(), kv[:, :V]
                    s = Q @ kv.T * scale
                    E = (Q.abs() @ kv.abs().T * abs(scale)).amax(1) * self.dim * 2.0 ** -23 + 2.0 ** -18
                    p = torch.softmax(s, 1)
                    out[t], lse[t] = p @ val, torch.logsumexp(s, 1)
                    size = p @ val.abs()
                    tol[t] = u * (out[t].abs() + size) + 2 * E[:, None] * size + \
                        (kv.shape[0] * val.abs().max() + 1) * 2.0 ** -126 + \
                        (kv.shape[0] * 2.0 ** -25 * val.abs().max() if q.dtype == torch.float16 else 0.0)
                    tol_lse[t] = E + lse[t].abs() * 2.0 ** -22
                t += 1
        return out, lse, tol, tol_lse

    def check(self, scale, causal=True, idx=None, **kw):
        hsi.latent_attention(self.cache, self.q, self.q_start, self.max_q, self.max_kv, scale, self.out, lse=self.lse,
                             idx=idx, causal=causal, **kw)
        assert hsi.device_error() == 0
        out, lse, tol, tol_lse = self.attention(scale, causal, idx)
        within(self.out[:self.T], out, tol, "out")
        within(self.lse[:self.T], lse, tol_lse, "lse")

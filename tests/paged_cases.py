"""Shared set-up of the paged-cache tests: caches with poisoned unused places and plain forms in 64 bits."""
import math

import numpy as np
import torch

import long_context_decode_lightning_gb300 as hsi

DEV = "cuda"
# unit roundoff of a store in each type
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


class Case:
    """B sequences of kv_lens entries, the last q_lens of them new. Every place of the pages that holds no
    entry is NaN, every table slot past a sequence's pages names no page."""

    def __init__(self, seed, kv_lens, q_lens, Hq, Hkv, D, page, dtype, layout="NHD", q_scale=2.0, spare=3, table_pad=2,
                 first_page=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.kv_lens, self.q_lens = list(kv_lens), list(q_lens)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.B = len(kv_lens)
        per = max(1, -(-max(kv_lens) // page)) + table_pad
        used = [-(-n // page) for n in kv_lens]
        n_pages = first_page + sum(used) + spare
        shape = {"NHD": (n_pages, page, Hkv, D), "HND": (n_pages, Hkv, page, D), "KV": (n_pages, 2, page, Hkv, D)}[layout]
        if layout == "KV":  # both tensors in one allocation
            kv = torch.full(shape, math.nan, dtype=dtype, device=DEV)
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device=DEV) for _ in range(2))
            if layout == "HND":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        ids = first_page + torch.randperm(sum(used) + spare, generator=torch.Generator().manual_seed(seed))
        table = torch.full((self.B, per), -7, dtype=torch.int32)
        table[:, 1::2] = 1 << 30
        at = 0
        self.K, self.V = [], []
        for b, n in enumerate(kv_lens):
            table[b, :used[b]] = ids[at:at + used[b]].int()
            at += used[b]
            for pages, keep in ((self.k, self.K), (self.v, self.V)):
                x = torch.randn(n, Hkv, D, generator=g, device=DEV).to(dtype)
                keep.append(x)
                for i in range(used[b]):
                    rows = x[i * page:(i + 1) * page]
                    pages[int(table[b, i]), :rows.shape[0]] = rows
        self.table = table.to(DEV)
        self.kv_len = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device=DEV)
        self.T = int(sum(q_lens))
        self.q = (torch.randn(max(self.T, 1), Hq, D, generator=g, device=DEV) * q_scale).to(dtype)
        self.kv = hsi.PagedKV(self.k, self.v, self.table, self.kv_len)
        self.max_q, self.max_kv = max(1, max(q_lens)), max(1, max(kv_lens))

    def rows(self, b, causal):
        """Scores' mask of sequence b: [new tokens, entries]."""
        m, n = self.q_lens[b], self.kv_lens[b]
        seen = torch.ones(m, n, dtype=torch.bool, device=DEV)
        return seen.tril(n - m) if causal else seen

    def attention(self, scale, causal, q=None):
        """out, lse, and the error bounds of each, all fp64.

        A score is a sum of D products in fp32: off by at most D 2^-23 of the sum of their sizes, E below. p is
        rounded once to the cache's type (fp16: 2^-25 absolute below its normal range, p <= 1 where it is rounded and
        the sum of p is at least 1), the result once more: u (|out| + sum p |v| / sum p) + 2 E sum p |v| / sum p."""
        q = self.q if q is None else q
        u = UNIT[self.dtype]
        out = torch.zeros(self.T, self.Hq, self.D, dtype=torch.float64, device=DEV)
        lse = torch.full((self.T, self.Hq), -math.inf, dtype=torch.float64, device=DEV)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        group, at = self.Hq // self.Hkv, 0
        for b in range(self.B):
            m, n = self.q_lens[b], self.kv_lens[b]
            if m and n:
                seen = self.rows(b, causal)
                for h in range(self.Hq):
                    K, V = self.K[b][:, h // group].double(), self.V[b][:, h // group].double()
                    Q = q[at:at + m, h].double()
                    s = torch.where(seen, Q @ K.T * scale, -math.inf)
                    live = seen.any(1)
                    E = (Q.abs() @ K.abs().T * abs(scale)).amax(1) * self.D * 2.0 ** -23 + 2.0 ** -18
                    p = torch.nan_to_num(torch.softmax(s, 1))
                    out[at:at + m, h] = p @ V
                    lse[at:at + m, h] = torch.logsumexp(s, 1)
                    size = p @ V.abs()
                    tol[at:at + m, h] = u * ((p @ V).abs() + size) + 2 * E[:, None] * size + \
                        (n * 2.0 ** -25 * V.abs().max() if self.dtype == torch.float16 else 0.0)
                    tol_lse[at:at + m, h] = torch.where(live, E + lse[at:at + m, h].abs() * 2.0 ** -22, 0.0)
            at += m
        return out, lse, tol, tol_lse

    def weights(self, scale, causal, lse, decay, acc):
        """acc after the call and its error bound: every p off by E (above) and by the rounding of
        scale q.k - lse in base 2, the sum by 2^-22 of its size."""
        want = [[None] * self.Hkv for _ in range(self.B)]
        tol = [[None] * self.Hkv for _ in range(self.B)]
        group, at = self.Hq // self.Hkv, 0
        for b in range(self.B):
            m, n = self.q_lens[b], self.kv_lens[b]
            for g in range(self.Hkv):
                x = decay * acc[b, g, :n].double() if acc is not None else torch.zeros(n, dtype=torch.float64, device=DEV)
                t = x.abs() * 2.0 ** -22
                for h in range(g * group, (g + 1) * group):
                    if not m or not n:
                        continue
                    Q, K = self.q[at:at + m, h].double(), self.K[b][:, g].double()
                    L = lse[at:at + m, h].double()[:, None]
                    p = torch.where(self.rows(b, causal), torch.exp(Q @ K.T * scale - L), 0.0)
                    p = torch.where(L == -math.inf, 0.0, p)
                    E = Q.abs() @ K.abs().T * abs(scale) * (self.D * 2.0 ** -23 + 2.0 ** -22) + \
                        torch.nan_to_num(L.abs(), posinf=0.0) * 2.0 ** -22 + 2.0 ** -20
                    x = x + p.sum(0)
                    t = t + (p * E).sum(0)
                want[b][g], tol[b][g] = x, t
            at += m
        return want, tol


def within(got, want, tol, what=""):
    d = (got.double() - want).abs()
    same = got.double() == want  # infinities
    bad = ~(same | (d <= tol))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off, worst {float(torch.where(same, 0.0, d - tol).max()):.3g} past its bound"

"""The paged-cache calls where they are easily wrong: NaN that comes in with the inputs, weights far below a row's
largest, positions and counts near the ends of their ranges, views, streams, and every path of a move in place."""
import math

import pytest
import torch

from paged_cases import DEV, UNIT, Case, within

import long_context_decode_lightning_gb300 as hsi

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hsi.build()
    hsi.device_check()
    yield
    assert hsi.device_error() == 0


# -------------------------------------------------------------------- streams --

class _Calls:
    """In the library's place: takes every call, asks for a megabyte of scratch, and knows the addresses it was given."""

    def __init__(self):
        self.args = []

    def __getattr__(self, name):
        def call(*args):
            if name in ("hsi_workspace_size", "hsi_paged_attention_ws"):
                return 1 << 20
            self.args.append([a for a in args if isinstance(a, int)])
            return 0
        return call


def test_scratch_that_a_call_makes_belongs_to_its_stream(monkeypatch):
    """Without a workspace the wrappers make one and drop it at return, while its kernels may still wait: its memory
    may go back to the given stream only, never to the current one."""
    c = Case(61, [100], [1], 4, 2, 64, 16, BF)
    out, lib, s = torch.empty_like(c.q), _Calls(), torch.cuda.Stream()
    x, i = torch.zeros(64, 128, device=DEV), torch.zeros(64, 128, dtype=torch.int32, device=DEV)
    monkeypatch.setattr(hsi, "_lib", lib)
    calls = [
        lambda: hsi.paged_attention(c.kv, c.q, c.q_start, 1, 100, 0.1, out, stream=s),
        lambda: hsi.quantize_nvfp4(x, 1, 64, [1] * 128, x, x, stream=s),
        lambda: hsi.topk(x, i, 64, 128, 8, i, x, stream=s),
        lambda: hsi.candidate_pool(i, 64, 128, i, i, i, scores=x, stream=s),
        lambda: hsi.full_layer(x, x, x, x, x, x, i, 64, 128, x, 8, i, x, stream=s),
        lambda: hsi.prefill_layer(x, x, x, x, x, x, i, 64, 128, x, 8, i, x, stream=s),
        lambda: hsi.reindex_layer(x, x, x, x, x, x, i, i, i, i, 64, x, 8, i, x, stream=s),
        lambda: hsi.calib_read(x, stream=s),
        lambda: hsi.calib_mma(128, 1, stream=s),
    ]
    mine = {t.data_ptr() for t in (x, i, out, c.q, c.q_start)}
    for n, call in enumerate(calls):
        lib.args.clear()
        call()
        segments = torch.cuda.memory_snapshot()
        made = [(a, g["stream"]) for a in lib.args[0] if a not in mine for g in segments
                if g["address"] <= a < g["address"] + g["total_size"]]
        assert len(made) == 1 and made[0][1] == s.cuda_stream, f"call {n}: {made}"


# --------------------------------------------------------------------- views --

@pytest.mark.parametrize("q_lens", [[1, 1], [1, 40]])
def test_lengths_past_a_sliced_table(q_lens):
    """What stands behind a slice of a wider table is not its own: a length that reaches there is clamped and reported."""
    c = Case(63, [100, 90], q_lens, 4, 2, 64, 16, BF)
    width = 6  # 96 entries; the columns behind name no page
    kv = hsi.PagedKV(c.k, c.v, c.table[:, :width], c.kv_len)
    out = torch.empty_like(c.q)
    hsi.paged_attention(kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, out)
    assert hsi.device_error() == -6
    want, _, tol, _ = c.attention(0.1, True)
    within(out[1:], want[1:], tol[1:], "the other sequence")
    short = Case(63, [100, 90], q_lens, 4, 2, 64, 16, BF)
    short.kv_lens[0], short.K[0], short.V[0] = 96, short.K[0][:96], short.V[0][:96]
    want, _, tol, _ = short.attention(0.1, True)
    within(out[:1], want[:1], tol[:1], "clamped")
    k_new = torch.randn(c.T, 2, 64, device=DEV).to(BF)
    hsi.paged_append(kv, k_new, k_new, c.q_start)
    assert hsi.device_error() == -6
    for i in range(q_lens[1]):
        e = 90 - q_lens[1] + i
        assert torch.equal(c.k[int(c.table[1, e // 16]), e % 16], k_new[1 + i])


# -------------------------------------------------------------------------- NaN --

# a cluster a unit; the line with units cut and whole; one unit over many runs; chunks cut, whole and both
NAN_SHAPES = [([700, 90], [1, 1], 8, 2), ([4000] * 3, [2, 1, 1], 8, 2), ([40 + i % 7 for i in range(300)], [1] * 300, 4, 2),
              ([20000], [1], 4, 1), ([300, 200, 128], [150, 120, 100], 8, 4), ([20000], [40], 4, 1), ([128] * 40, [60] * 40, 8, 4),
              ([1300], [700], 8, 8)]


def _attend(c):
    out, lse = torch.full_like(c.q, 5.0), torch.full((c.T, c.Hq), 5.0, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, out, lse=lse)
    acc = torch.zeros(c.B, c.Hkv, c.max_kv, device=DEV)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, 0.1, None, acc)
    assert hsi.device_error() == 0
    return out, lse, acc


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("kv_lens,q_lens,Hq,Hkv", NAN_SHAPES)
def test_nan_query_gives_nan(dtype, kv_lens, q_lens, Hq, Hkv):
    """A row whose every score is NaN is no row that sees nothing: out and lse are NaN, and so are its weights."""
    c = Case(67, kv_lens, q_lens, Hq, Hkv, 64, 16, dtype)
    was, was_lse, was_acc = _attend(c)
    row, head, b = c.T - 1, Hq - 1, c.B - 1
    c.q[row, head, 3] = math.nan
    out, lse, acc = _attend(c)
    assert bool(out[row, head].isnan().all()) and bool(lse[row, head].isnan())
    assert bool(acc[b, Hkv - 1, :kv_lens[b]].isnan().all())
    out[row, head], lse[row, head], acc[b, Hkv - 1] = was[row, head], was_lse[row, head], was_acc[b, Hkv - 1]
    assert torch.equal(out, was) and torch.equal(lse, was_lse) and torch.equal(acc, was_acc)


@pytest.mark.parametrize("kv_lens,q_lens,Hq,Hkv", NAN_SHAPES)
def test_nan_key_reaches_the_rows_that_see_it(kv_lens, q_lens, Hq, Hkv):
    """A NaN in the last sequence's last key: its last row's alone (causal), or, a few entries earlier, some rows'."""
    c = Case(71, kv_lens, q_lens, Hq, Hkv, 64, 16, BF)
    was, was_lse, _ = _attend(c)
    n, m, group = kv_lens[-1], q_lens[-1], Hq // Hkv
    rows = min(m, 3)  # the last `rows` tokens see entry n - rows
    e = n - rows
    c.k[int(c.table[-1, e // 16]), e % 16, Hkv - 1, 5] = math.nan
    out, lse, _ = _attend(c)
    assert bool(out[c.T - rows:, Hq - group:].isnan().all()) and bool(lse[c.T - rows:, Hq - group:].isnan().all())
    out[c.T - rows:, Hq - group:], lse[c.T - rows:, Hq - group:] = was[c.T - rows:, Hq - group:], was_lse[c.T - rows:, Hq - group:]
    assert torch.equal(out, was) and torch.equal(lse, was_lse)


# --------------------------------------------------------------- small weights --

@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,m", [(131072, 1), (5000, 1), (1000, 1), (131072, 30), (5000, 100)])
def test_many_small_weights_are_not_lost(dtype, n, m):
    """One entry of weight 1 and value 0, all others of weight 2^-25.1 and value 1: the output is what the small ones
    hold together. p is rounded to the cache's type, relative to itself (u) and, in fp16, by no more than half the
    smallest fp16 number, 2^-25, where the row's largest p stands at 2^7 at least; the result is rounded once more."""
    D = 64
    c = Case(73, [n], [m], 2, 1, D, 64, dtype)
    c.q.zero_()
    c.q[..., 0] = 4.0
    live = c.table[0, :-(-n // 64)].long()
    c.k[live] = 0.0
    c.v[live] = 1.0
    c.k[live[0], 0, 0, 0] = 25.1 * math.log(2.0) / 4.0
    c.v[live[0], 0] = 0.0
    top = 4.0 * float(c.k[live[0], 0, 0, 0])
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 2, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, m, n, 1.0, out, lse=lse)
    assert hsi.device_error() == 0
    seen = torch.arange(n - m + 1, n + 1, device=DEV, dtype=torch.float64)
    small = (seen - 1) * math.exp(-top)
    want = (small / (1 + small))[:, None, None].expand(m, 2, D)
    # the exponent, 25 in base 2, and ex2: below 2^-16 of a p; fp16: 2^-25 * 2^-7 absolute each
    tol = want * (2 * UNIT[dtype] + 2.0 ** -16) + (n * 2.0 ** -32 if dtype == HF else 0.0)
    within(out, want, tol, "out")
    within(lse, (top + torch.log1p(small))[:, None].expand(m, 2), torch.full_like(want[..., 0], 2.0 ** -16), "lse")


@pytest.mark.parametrize("kv_lens,q_lens", [([900, 300], [1, 1]), ([30000], [2]), ([700, 400], [300, 90]), ([9000], [30])])
def test_fp16_values_as_large_as_the_type(kv_lens, q_lens):
    """Equal scores over values near the largest fp16 number: sums are fp32, the result is an average."""
    c = Case(79, kv_lens, q_lens, 4, 2, 64, 16, HF)
    c.q.zero_()
    for v in c.V:
        v.copy_(torch.where(v > 0, 60000.0, 65504.0).to(HF))
    for b, n in enumerate(kv_lens):
        for i in range(-(-n // 16)):
            rows = c.V[b][i * 16:(i + 1) * 16]
            c.v[int(c.table[b, i]), :rows.shape[0]] = rows
    out = torch.empty_like(c.q)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, 0.1, out)
    want, _, tol, _ = c.attention(0.1, True)
    within(out, want, tol, "out")


# ------------------------------------------------------------ far and many entries --

@pytest.mark.parametrize("causal", [True, False])
def test_weights_past_31_bits_of_rows_times_entries(causal):
    """64 query heads of one KV head over 33.6 million entries (one page, listed again and again): entries times heads
    pass 2^31, and every entry's weight is that of its place in the page."""
    D, page, n, Hq = 64, 4096, 33_600_003, 64
    g = torch.Generator(device=DEV).manual_seed(83)
    k = torch.randn(1, page, 1, D, generator=g, device=DEV).to(BF)
    table = torch.zeros(1, -(-n // page), dtype=torch.int32, device=DEV)
    kv = hsi.PagedKV(k, k, table, torch.tensor([n], dtype=torch.int32, device=DEV))
    q = torch.randn(1, Hq, D, generator=g, device=DEV).to(BF)
    lse = torch.rand(1, Hq, generator=g, device=DEV) + 3.0
    acc = torch.full((1, 1, n), -1.0, device=DEV)
    hsi.attention_weights(kv, q, lse, torch.tensor([0, 1], dtype=torch.int32, device=DEV), 1, n, 0.125, None, acc, causal=causal)
    assert hsi.device_error() == 0
    Q, K = q[0].double(), k[0, :, 0].double()
    p = torch.exp(Q @ K.T * 0.125 - lse[0].double()[:, None])
    # p off by the score's error (D products in fp32) and the rounding of its exponent in base 2; the sum by 2^-22
    E = Q.abs() @ K.abs().T * 0.125 * (D * 2.0 ** -23 + 2.0 ** -22) + lse[0].double()[:, None] * 2.0 ** -22 + 2.0 ** -20
    want, tol = p.sum(0), (p * E).sum(0) + p.sum(0) * 2.0 ** -22
    whole = n // page * page
    rows = acc[0, 0, :whole].view(-1, page)
    assert bool((rows == rows[0]).all())
    within(rows[0], want, tol, "weights")
    assert torch.equal(acc[0, 0, whole:], rows[0, :n - whole])


def test_wide_bounds_of_a_mixed_batch():
    """A chunk of 2048 tokens, single tokens and none in one call, under a bound of a million entries a sequence."""
    page, D, lens, new = 64, 64, [2300, 40, 700] + [100] * 29, [2048, 1, 0] + [1] * 29
    c = Case(101, lens, new, 32, 8, D, page, BF, table_pad=(1 << 20) // page)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 32, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, 2048, 1 << 20, 0.125, out, lse=lse)
    acc = torch.zeros(c.B, 8, 1 << 20, device=DEV)
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, 2048, 1 << 20, 0.125, None, acc)
    assert hsi.device_error() == 0
    want, want_lse, tol, tol_lse = c.attention(0.125, True)
    within(out, want, tol, "out")
    within(lse, want_lse, tol_lse, "lse")
    w, wt = c.weights(0.125, True, lse, 1.0, None)
    for b, n in enumerate(lens):
        assert not bool(acc[b, :, n:].any())
        for g in range(0, 8, 5):
            within(acc[b, g, :n], w[b][g], wt[b][g], "weights")


# --------------------------------------------------------------------- q_start --

@pytest.mark.parametrize("start", [[0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7], [6, 4, 2, 0]])
@pytest.mark.parametrize("more", [0, 37])  # up to 32 sequences a warp's lanes look at once
def test_append_reports_a_wrong_q_start(start, more):
    """A q_start that descends or leaves the call's tokens is reported; tokens of two sequences or of one that leaves the
    call's are left alone, the others written where the call's other users look for them."""
    lens, T = [20, 30, 10] + [5] * more, 6
    c = Case(89, lens, [2, 2, 2] + [0] * more, 2, 1, 64, 8, BF)
    k = torch.randn(T, 1, 64, device=DEV).to(BF)
    want = c.k.clone(), c.v.clone()
    start = start + [start[-1]] * more
    steps, gain = hsi.rope_steps(64)
    q, q_out = c.q[:T].clone(), torch.full((T, 2, 64), 7.0, dtype=BF, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    k_rot, q_rot, want_q = torch.empty_like(k), torch.empty_like(q), q_out.clone()
    hsi.rope(k, pos, steps, k_rot, gain=gain)
    hsi.rope(q, pos, steps, q_rot, gain=gain)
    for t in range(T):
        owners = [b for b in range(3) if 0 <= start[b] <= t < start[b + 1] <= T]
        if len(owners) != 1:
            continue
        b = owners[0]
        e = lens[b] - start[b + 1] + t
        page, at = int(c.table[b, e // 8]), e % 8
        want[0][page, at], want[1][page, at], want_q[t] = k_rot[t], k[t], q_rot[t]
    hsi.paged_append(c.kv, k, k, torch.tensor(start, dtype=torch.int32, device=DEV), positions=pos, steps=steps, gain=gain,
                     q=q, q_out=q_out)
    assert hsi.device_error() == -6
    for now, w in zip((c.k, c.v), want):
        assert torch.equal(now.view(torch.int16), w.view(torch.int16))
    assert torch.equal(q_out, want_q)


@pytest.mark.parametrize("n_extra", [0, 1])
def test_append_past_a_sequence_s_pages(n_extra):
    """A length past what the table's row lists: tokens that still have a place go there, the others nowhere (not onto
    the entries that end the row), and it is reported."""
    c = Case(91, [32, 20], [3, 1], 2, 1, 64, 8, BF, table_pad=0)  # rows of four pages, 32 entries
    c.kv_len[0] = 32 + n_extra
    k = torch.randn(4, 1, 64, device=DEV).to(BF)
    want = c.k.clone()
    for i in range(3):
        e = 32 + n_extra - 3 + i
        if e < 32:
            want[int(c.table[0, e // 8]), e % 8] = k[i]
    want[int(c.table[1, 2]), 3] = k[3]
    hsi.paged_append(c.kv, k, k, c.q_start)
    assert hsi.device_error() == (-6 if n_extra else 0)
    assert torch.equal(c.k.view(torch.int16), want.view(torch.int16))


# -------------------------------------------------------------- moved caches --

def test_attention_after_a_move_to_other_pages():
    """The kept entries on their new pages, under their new table and lengths, and a second move, in place there."""
    lens, budget, page, D = [500, 300], 200, 16, 64
    need = -(-budget // page)
    c = Case(103, lens, [1, 1], 4, 2, D, page, BF, spare=2 * need)
    used = set(c.table[(c.table >= 0) & (c.table < c.k.shape[0])].tolist())
    free = [p for p in range(c.k.shape[0]) if p not in used]
    dst = torch.tensor(free[:2 * need], dtype=torch.int32, device=DEV).view(2, need)
    for move, n in ((dst, budget), (None, 90)):
        acc = torch.rand(2, 2, max(c.kv_lens), device=DEV)
        keep = torch.empty(2, 2, n, dtype=torch.int32, device=DEV)
        new_len = torch.empty(2, dtype=torch.int32, device=DEV)
        hsi.evict_select(acc, c.kv.kv_len, max(c.kv_lens), n, keep, new_len, recent=1)
        hsi.paged_compact(c.kv, keep, new_len, move)
        if move is not None:
            c.kv.table = move
        c.kv.kv_len = new_len
        c.kv_lens = [n, n]
        for x in (c.K, c.V):
            for b in range(2):
                x[b] = torch.stack([x[b][keep[b, g].long(), g] for g in range(2)], 1)
        out = torch.empty_like(c.q)
        hsi.paged_attention(c.kv, c.q, c.q_start, 1, n, 0.125, out)
        assert hsi.device_error() == 0
        want, _, tol, _ = c.attention(0.125, True)
        within(out, want, tol, "out")


# ------------------------------------------------- paths that nothing else takes --

@pytest.mark.parametrize("page,D,layout", [(16, 64, "NHD"), (64, 128, "HND")])
def test_compact_in_place_of_a_batch(page, D, layout):
    """Eight sequences of eight heads: blocks for every SM, clusters of eight and more than one turn, in place."""
    lens, budget, H = [6000, 5991, 5003, 4000, 3999, 17, 0, 5555], 4000, 8
    c = Case(97, lens, [0] * 8, H, H, D, page, BF, layout)
    acc = torch.rand(8, H, max(lens), device=DEV)
    keep = torch.empty(8, H, budget, dtype=torch.int32, device=DEV)
    new_len = torch.empty(8, dtype=torch.int32, device=DEV)
    hsi.evict_select(acc, c.kv_len, max(lens), budget, keep, new_len, sink=4, recent=100)
    want = [c.k.clone(), c.v.clone()]
    for pages, src in zip(want, (c.K, c.V)):
        for b, n in enumerate(new_len.tolist()):
            i = torch.arange(n, device=DEV)
            for h in range(H):
                pages[c.table[b, i // page].long(), i % page, h] = src[b][keep[b, h, :n].long(), h]
    hsi.paged_compact(c.kv, keep, new_len)
    assert hsi.device_error() == 0
    for pages, w in zip((c.k, c.v), want):
        assert torch.equal(pages.contiguous().view(torch.int16), w.contiguous().view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [1.0, 0.1, -0.4, 0.0])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [90, 300, 17]])
def test_weights_of_large_scores_at_every_scale(dtype, scale, q_lens):
    """Weights under scores of hundreds, negative and zero scales. p = exp(x) with x off by E: p off by p (e^E - 1)."""
    c = Case(17, [1000, 800, 70], q_lens, 8, 2, 128, 32, dtype, q_scale=30.0)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 8, device=DEV)
    hsi.paged_attention(c.kv, c.q, c.q_start, c.max_q, c.max_kv, scale, out, lse=lse)
    want_out, want_lse, tol_out, tol_lse = c.attention(scale, True)
    within(out, want_out, tol_out, "out")
    within(lse, want_lse, tol_lse, "lse")
    old = torch.rand(3, 2, 1000, device=DEV)
    acc = old.clone()
    hsi.attention_weights(c.kv, c.q, lse, c.q_start, c.max_q, c.max_kv, scale, acc, acc, decay=0.5)
    assert hsi.device_error() == 0
    at = 0
    for b, (n, m) in enumerate(zip(c.kv_lens, c.q_lens)):
        for g in range(2):
            want = 0.5 * old[b, g, :n].double()
            tol = want * 2.0 ** -22
            for h in range(4 * g, 4 * g + 4):
                Q, K, L = c.q[at:at + m, h].double(), c.K[b][:, g].double(), lse[at:at + m, h].double()[:, None]
                p = torch.where(c.rows(b, True), torch.exp(Q @ K.T * scale - L), 0.0)
                E = Q.abs() @ K.abs().T * abs(scale) * (128 * 2.0 ** -23 + 2.0 ** -22) + L.abs() * 2.0 ** -22 + 2.0 ** -20
                want, tol = want + p.sum(0), tol + (p * (torch.expm1(E) + 2.0 ** -22)).sum(0)
            within(acc[b, g, :n], want, tol, f"weights {b} {g}")
        at += m

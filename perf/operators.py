"""Timed cases of the paged-cache operators: rotary positions, the append to a paged cache, attention over it,
the accumulated attention weight of its entries and the eviction by that weight.

Every operator is here in its plain form (elementary torch operations in fp32) and as the calls a user makes
of the library. A paged cache holds K and V as [pages, page size, KV heads, D]; the entries of sequence b are
listed by its row of the page table, and its last new tokens are the last entries of its length.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases --

def listed():
    return [
        # the rotary half of the indexer's 32 query heads, one decode step of 64 sequences, contexts to 1M
        dict(name="rope, one step", op="rope", T=64, H=32, D=128, rot=64, off=64, pairs=True, dtype="bf16",
             scaling="yarn", back=False, top=1 << 20),
        # the gradient of a prompt's queries, 8192 tokens, whole head, halves layout
        dict(name="rope, prompt gradient", op="rope", T=8192, H=32, D=128, rot=128, off=0, pairs=False, dtype="fp32",
             scaling="none", back=True, top=131072),
        # one token of 64 sequences: q rotated, k rotated into its page, v copied
        dict(name="append, one token", op="append", B=64, q=1, n=1024, Hq=32, Hkv=8, D=128, page=16, dtype="bf16",
             pairs=False),
        # four prompts of different lengths, 64-wide heads
        dict(name="append, ragged prompts", op="append", B=4, q=2049, n=4099, Hq=32, Hkv=8, D=64, page=32,
             dtype="fp16", pairs=True),
        # three short conversations, one token each: latency
        dict(name="attend, one token short", op="attend", B=3, q=1, n=777, Hq=16, Hkv=2, D=64, page=16, dtype="fp16",
             causal=True),
        # sixteen long sequences, one token each: the cache is read once
        dict(name="attend, one token long", op="attend", B=16, q=1, n=65536, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", causal=True),
        # chunks of four prompts of odd lengths, seven query heads to a KV head
        dict(name="attend, ragged chunks", op="attend", B=4, q=1001, n=5003, Hq=28, Hkv=4, D=128, page=32,
             dtype="bf16", causal=True),
        # the last 2048 tokens of a 32768-token prompt
        dict(name="attend, long chunk", op="attend", B=1, q=2048, n=32768, Hq=32, Hkv=8, D=128, page=64, dtype="bf16",
             causal=True),
        # the weights a decode step adds to sixteen sequences' entries
        dict(name="weights, one token", op="weights", B=16, q=1, n=32768, Hq=32, Hkv=8, D=128, page=64, dtype="bf16",
             causal=True),
        # the weights a prompt's chunks add
        dict(name="weights, chunks", op="weights", B=2, q=1024, n=16384, Hq=32, Hkv=8, D=128, page=32, dtype="bf16",
             causal=True),
        # two short sequences over their budget
        dict(name="evict, short", op="evict", B=2, n=1025, keep=512, sink=4, recent=64, Hkv=2, D=64, page=16,
             dtype="fp16"),
        # eight sequences of 16384 entries back to 8192
        dict(name="evict, half of 16384", op="evict", B=8, n=16384, keep=8192, sink=4, recent=512, Hkv=8, D=128,
             page=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "weights", "evict"])
    D, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "fp16"])
    page, Hkv, group = rng.choice([8, 16, 32, 64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        rot = rng.choice([D, D, D // 2, 32])
        H = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, min(16384, (1 << 25) // (H * D))))
        return dict(op=op, T=T, H=H, D=D, rot=rot, off=rng.choice([0, D - rot]), pairs=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    back=rng.random() < 0.4, top=_log(rng, 64, 1 << 20))
    if op == "append":
        B = _log(rng, 1, 128)
        q = rng.choice([1, _log(rng, 1, max(1, 8192 // B))])
        return dict(op=op, B=B, q=q, n=q + _log(rng, 1, 1024), Hq=Hkv * group, Hkv=Hkv, D=D, page=page, dtype=dtype,
                    pairs=rng.random() < 0.5)
    if op == "evict":
        n = _log(rng, 64, 131072)
        B = _log(rng, 1, max(1, min(16, (1 << 27) // (n * Hkv * D))))
        return dict(op=op, B=B, n=n, keep=max(16, int(n * rng.uniform(0.2, 1.1))), sink=rng.choice([0, 1, 4]),
                    recent=rng.choice([0, 1, 8]), Hkv=Hkv, D=D, page=page, dtype=dtype)
    q = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 1024)])
    n = q + _log(rng, 1, 32768)
    cap = (1 << 29) if op == "attend" else (1 << 28)  # values of the plain form's score matrix
    while Hkv * group * q * n > cap:
        n = q + max(1, (n - q) // 2)
        q = max(1, q // 2)
    B = _log(rng, 1, max(1, min(32, cap // (Hkv * group * q * n), (1 << 28) // (n * Hkv * D))))
    return dict(op=op, B=B, q=q, n=n, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, dtype=dtype,
                causal=rng.random() < 0.8)


# ------------------------------------------------- lengths, frequencies, inputs --

def _lengths(c):
    """Entries and new tokens of each sequence: from the full lengths down towards half of them."""
    B = c["B"]
    new = [max(1, c.get("q", 1) - b * c.get("q", 1) // (2 * B)) for b in range(B)]
    return [max(new[b], c["n"] - b * c["n"] // (2 * B)) for b in range(B)], new


def _inv_freq(rot, scaling):
    """Radians a position and the gain of each scaling: contexts of 8 x 32768 from a model of 32768."""
    base, f, length = 10000.0, 8.0, 32768
    if scaling == "ntk":
        base *= f ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        inv = [v / f for v in inv]
    if scaling == "yarn":
        def at(turns):
            return rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        inv = [v * (1 - r) + v / f * r for v, r in zip(inv, ramp)]
    return inv, 0.1 * math.log(f) + 1.0 if scaling == "yarn" else 1.0


def _steps(inv):
    """Turns a position in units of 2^-64, as a plan that a program keeps."""
    steps = [round(v / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for v in inv]
    return torch.tensor([s - (1 << 64) if s >= 1 << 63 else s for s in steps], dtype=torch.int64, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(c, gen, more=0):
    """Pages in random order, `more` further ones for each sequence's other table."""
    lens, new = _lengths(c)
    per = -(-c["n"] // c["page"])
    extra = -(-more // c["page"])
    total = c["B"] * (per + extra)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    s = dict(c=c, table=order[:c["B"] * per].view(c["B"], per), kv_len=_ints(lens), lens=lens, new=new)
    for name in "kv":
        s[name] = torch.randn(total, c["page"], c["Hkv"], c["D"], generator=gen, device="cuda", dtype=DT[c["dtype"]])
    if more:
        s["other"] = order[c["B"] * per:].view(c["B"], extra)
    if "q" in c:
        at = [0]
        for t in new:
            at.append(at[-1] + t)
        s["q_start"], s["T"] = _ints(at), at[-1]
        # new token -> its sequence and its entry
        seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), torch.tensor(new, device="cuda"))
        s["seq"] = seq
        s["entry"] = (torch.arange(at[-1], device="cuda") - s["q_start"].long()[seq]
                      + (s["kv_len"] - _ints(new)).long()[seq])
    return s


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, dtype=None, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype or DT[c["dtype"]])

    op = c["op"]
    if op == "rope":
        inv, gain = _inv_freq(c["rot"], c["scaling"])
        x = normal(c["T"], c["H"], c["D"])
        return dict(c=c, x=x, out=torch.zeros_like(x), steps=_steps(inv), gain=gain,
                    pos=torch.randint(0, c["top"], (c["T"],), generator=gen, device="cuda", dtype=torch.int32))
    s = _cache(c, gen, c.get("keep", 0))
    if op == "append":
        inv, gain = _inv_freq(c["D"], "none")
        s.update(steps=_steps(inv), gain=gain, q=normal(s["T"], c["Hq"], c["D"]),
                 k_new=normal(s["T"], c["Hkv"], c["D"]), v_new=normal(s["T"], c["Hkv"], c["D"]))
        s["q_out"], s["pos"] = torch.zeros_like(s["q"]), s["entry"].to(torch.int32)
    elif op == "evict":
        # weights as they pile up: a few large ones, many small, equal ones among them
        w = torch.rand(c["B"], c["Hkv"], c["n"], generator=gen, device="cuda").pow_(6).mul_(4096).floor_().div_(512)
        s.update(acc=w, acc_out=torch.zeros(c["B"], c["Hkv"], c["keep"], device="cuda"),
                 keep=torch.full((c["B"], c["Hkv"], c["keep"]), -1, dtype=torch.int32, device="cuda"),
                 new_len=torch.zeros(c["B"], dtype=torch.int32, device="cuda"))
    else:
        s["q"] = normal(s["T"], c["Hq"], c["D"], scale=2.0)
        s["scale"] = 1.0 / math.sqrt(c["D"])
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["T"], c["Hq"], device="cuda")
        if op == "weights":
            s["acc"] = torch.rand(c["B"], c["Hkv"], c["n"], generator=gen, device="cuda")
            s["acc_out"] = torch.zeros_like(s["acc"])
            s["decay"] = 0.95
            s["lse"] = _plain_lse(s)
    return s


# ------------------------------------------------------------------ plain forms --

def _plain_rotate(x, pos, steps, gain, rot, off, pairs, back):
    """x [T, H, D] -> fp32. The phase wraps in 64-bit integers, so far positions lose nothing."""
    phase = (pos.long()[:, None] * steps[None, :]).float() * (2 * math.pi / 2.0 ** 64)
    cos, sin = (phase.cos() * gain)[:, None, :], (phase.sin() * gain)[:, None, :]
    if back:
        sin = -sin
    y = x.float().clone()
    r = y[..., off:off + rot]
    u, v = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = u * cos - v * sin, u * sin + v * cos
    y[..., off:off + rot] = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return y


def _plain_entries(s, pages):
    """[B, n, Hkv, D] in fp32, zero past each sequence's length."""
    c = s["c"]
    x = pages[s["table"].long()].flatten(1, 2)[:, :c["n"]].float()
    live = torch.arange(c["n"], device="cuda")[None, :] < s["kv_len"][:, None]
    return torch.where(live[:, :, None, None], x, 0.0)


def _plain_scores(s):
    """scale q.k of the padded rows [B, Hkv, group, q, n], -inf where a row does not see an entry."""
    c = s["c"]
    B, n, Hkv, D = c["B"], c["n"], c["Hkv"], c["D"]
    t = torch.arange(c["q"], device="cuda")
    new = s["q_start"][1:] - s["q_start"][:-1]
    row = (s["q_start"][:-1, None] + t).clamp(max=s["T"] - 1).long()
    q = s["q"][row].float().view(B, c["q"], Hkv, c["Hq"] // Hkv, D).permute(0, 2, 3, 1, 4)
    k = _plain_entries(s, s["k"]).permute(0, 2, 3, 1)
    x = torch.matmul(q.reshape(B, Hkv, -1, D) * s["scale"], k).view(B, Hkv, c["Hq"] // Hkv, c["q"], n)
    last = (s["kv_len"] - new)[:, None] + t + 1 if c["causal"] else s["kv_len"][:, None].expand(B, c["q"])
    last = torch.where(t < new[:, None], torch.minimum(last, s["kv_len"][:, None]), 0)
    x.masked_fill_(torch.arange(n, device="cuda") >= last[:, None, None, :, None], -math.inf)
    return x


def _plain_rows(s, x):
    """[B, Hkv, group, q, ...] -> the rows of the new tokens [T, Hq, ...]."""
    x = x.movedim(3, 1).flatten(2, 3)
    return x[s["seq"], torch.arange(s["T"], device="cuda") - s["q_start"].long()[s["seq"]]]


def _plain_softmax(s):
    x = _plain_scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return x, total, _plain_rows(s, (total.log() + top)[..., 0])


def _plain_lse(s):
    return _plain_softmax(s)[2].contiguous()


def _plain_attend(s):
    x, total, lse = _plain_softmax(s)
    v = _plain_entries(s, s["v"]).transpose(1, 2)
    o = torch.matmul(x.flatten(2, 3), v).view(*x.shape[:4], -1)
    o = torch.where(total > 0, o / total, 0.0)
    return {"out": _plain_rows(s, o).to(s["q"].dtype), "lse": lse}


def _plain_weights(s):
    c = s["c"]
    x = _plain_scores(s)
    t = torch.arange(c["q"], device="cuda")
    row = (s["q_start"][:-1, None] + t).clamp(max=s["T"] - 1).long()
    lse = s["lse"][row].view(c["B"], c["q"], c["Hkv"], -1).permute(0, 2, 3, 1)
    p = x.sub_(lse[..., None]).exp_().sum((2, 3))
    live = torch.arange(c["n"], device="cuda") < s["kv_len"][:, None]
    s["acc_out"].copy_(torch.where(live[:, None, :], s["acc"] * s["decay"] + p, s["acc_out"]))
    return {"acc": s["acc_out"]}


def _plain_append(s):
    c = s["c"]
    rot = (s["pos"], s["steps"], s["gain"], c["D"], 0, c["pairs"], False)
    s["q_out"].copy_(_plain_rotate(s["q"], *rot))
    page, at = s["table"][s["seq"], s["entry"] // c["page"]].long(), s["entry"] % c["page"]
    s["k"][page, at] = _plain_rotate(s["k_new"], *rot).to(s["k"].dtype)
    s["v"][page, at] = s["v_new"]
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_evict(s):
    c = s["c"]
    B, n, keep = c["B"], c["n"], c["keep"]
    i = torch.arange(n, device="cuda")
    length = s["kv_len"][:, None, None]
    w = torch.where((i < c["sink"]) | (i >= length - c["recent"]), math.inf, s["acc"])
    w = torch.where(i < length, w, -math.inf)
    first = w.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    slot = torch.arange(keep, device="cuda")
    new_len = s["kv_len"].clamp(max=keep)
    if first.shape[-1] < keep:
        first = torch.nn.functional.pad(first, (0, keep - first.shape[-1]), value=n)
    live = slot < new_len[:, None, None]
    first = torch.where(live, first, n).sort(-1).values
    s["keep"].copy_(torch.where(live, first, -1))
    s["new_len"].copy_(new_len)
    at = first.clamp(max=n - 1)
    s["acc_out"].copy_(torch.where(live, s["acc"].gather(-1, at), 0.0))
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(c["Hkv"], device="cuda")[None, :, None].expand(B, -1, keep)
    src, dst = s["table"][b, at // c["page"]].long(), s["other"][b, slot // c["page"]].expand(-1, c["Hkv"], -1).long()
    place = (slot % c["page"]).expand(B, c["Hkv"], -1)
    for pages in (s["k"], s["v"]):
        pages[dst[live.expand_as(dst)], place[live.expand_as(dst)], h[live.expand_as(dst)]] = \
            pages[src, at % c["page"], h][live.expand_as(dst)]
    return {"keep": s["keep"], "new_len": s["new_len"], "acc": s["acc_out"], "k": s["k"], "v": s["v"]}


def _plain(s):
    c = s["c"]
    if c["op"] == "rope":
        y = _plain_rotate(s["x"], s["pos"], s["steps"], s["gain"], c["rot"], c["off"], c["pairs"], c["back"])
        return {"out": y.to(s["x"].dtype)}
    return {"append": _plain_append, "attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict}[
        c["op"]](s)


# ------------------------------------------------------------- the library's calls --

def _library(s):
    import long_context_decode_lightning_gb300 as hsi
    c = s["c"]
    op = c["op"]
    if op == "rope":
        hsi.rope(s["x"], s["pos"], s["steps"], s["out"], rot_offset=c["off"], interleaved=c["pairs"], gain=s["gain"],
                 inverse=c["back"])
        return {"out": s["out"]}
    if "kv" not in s:  # the handle a program keeps for its cache
        s["kv"] = hsi.PagedKV(s["k"], s["v"], s["table"], s["kv_len"])
    if op == "append":
        hsi.paged_append(s["kv"], s["k_new"], s["v_new"], s["q_start"], c["q"], positions=s["pos"], steps=s["steps"],
                         interleaved=c["pairs"], gain=s["gain"], q=s["q"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if op == "attend":
        if "ws" not in s:
            s["ws"] = hsi.paged_attention_workspace(s["kv"], s["q"], c["q"], c["n"])
        hsi.paged_attention(s["kv"], s["q"], s["q_start"], c["q"], c["n"], s["scale"], s["out"], lse=s["lse"],
                            causal=c["causal"], ws=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        hsi.attention_weights(s["kv"], s["q"], s["lse"], s["q_start"], c["q"], c["n"], s["scale"], s["acc"],
                              s["acc_out"], decay=s["decay"], causal=c["causal"])
        return {"acc": s["acc_out"]}
    hsi.evict_select(s["acc"], s["kv_len"], c["n"], c["keep"], s["keep"], s["new_len"], sink=c["sink"],
                     recent=c["recent"], acc_out=s["acc_out"])
    hsi.paged_compact(s["kv"], s["keep"], s["new_len"], s["other"])
    return {"keep": s["keep"], "new_len": s["new_len"], "acc": s["acc_out"], "k": s["k"], "v": s["v"]}


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------- floors and 64 bits --

def work(c):
    es = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rope":
        return {"bytes": 2 * c["T"] * c["H"] * c["D"] * es + 4 * c["T"] + 4 * c["rot"],
                "flops": 3 * c["T"] * c["H"] * c["rot"]}
    lens, new = _lengths(c)
    if c["op"] == "append":
        return {"bytes": sum(new) * (2 * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * es + 4),
                "flops": 3 * sum(new) * (c["Hq"] + c["Hkv"]) * c["D"]}
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens) * c["Hkv"]
        return {"bytes": 4 * sum(lens) * c["Hkv"] + kept * (4 * c["D"] * es + 8), "flops": 2 * sum(lens) * c["Hkv"]}
    seen = sum(m * n - m * (m - 1) // 2 if c["causal"] else m * n for n, m in zip(lens, new)) * c["Hq"]
    rows, entries = sum(new) * c["Hq"], sum(lens) * c["Hkv"]
    if c["op"] == "attend":
        return {"bytes": 2 * entries * c["D"] * es + rows * (2 * c["D"] * es + 4), "flops": 4 * c["D"] * seen}
    return {"bytes": entries * (c["D"] * es + 8) + rows * (c["D"] * es + 4), "flops": 2 * c["D"] * seen}


def _exact_rotate(x, pos, inv, gain, off, pairs, back):
    """Pair by pair in fp64, from the frequencies themselves."""
    y = x.double()
    half = len(inv)
    for i in range(half):
        a = pos.double() * inv[i]
        co, si = gain * torch.cos(a)[:, None], gain * torch.sin(a)[:, None] * (-1.0 if back else 1.0)
        m, n = (off + 2 * i, off + 2 * i + 1) if pairs else (off + i, off + half + i)
        u, v = x[..., m].double(), x[..., n].double()
        y[..., m], y[..., n] = co * u - si * v, co * v + si * u
    return y


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "rope":
        inv, gain = _inv_freq(c["rot"], c["scaling"])
        return {"out": _exact_rotate(s["x"], s["pos"], inv, gain, c["off"], c["pairs"], c["back"])}
    if op == "append":
        inv, gain = _inv_freq(c["D"], "none")
        k, v = s["k"].double(), s["v"].double()
        k_new = _exact_rotate(s["k_new"], s["pos"], inv, gain, 0, c["pairs"], False)
        for t, (b, e) in enumerate(zip(s["seq"].tolist(), s["entry"].tolist())):
            page = s["table"][b, e // c["page"]].long()
            k[page, e % c["page"]], v[page, e % c["page"]] = k_new[t], s["v_new"][t].double()
        return {"q": _exact_rotate(s["q"], s["pos"], inv, gain, 0, c["pairs"], False), "k": k, "v": v}
    if op == "evict":
        return None  # whole numbers and copies: nothing is computed
    lens, new = s["lens"], s["new"]
    group = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["T"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    acc = s["acc_out"].double() if op == "weights" else None
    at = 0
    for b in range(c["B"]):
        n, m = lens[b], new[b]
        pages = s["table"][b, :-(-n // c["page"])].long()
        seen = torch.ones(m, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = seen.tril(n - m)
        for g in range(c["Hkv"]):
            k = s["k"][pages, :, g].flatten(0, 1)[:n].double()
            if acc is not None:
                acc[b, g, :n] = s["acc"][b, g, :n].double() * s["decay"]
            else:
                v = s["v"][pages, :, g].flatten(0, 1)[:n].double()
            for h in range(g * group, (g + 1) * group):
                x = (s["q"][at:at + m, h].double() @ k.T) * s["scale"]
                if acc is not None:
                    p = torch.exp(x - s["lse"][at:at + m, h].double()[:, None])
                    acc[b, g, :n] += torch.where(seen, p, 0.0).sum(0)
                else:
                    x = torch.where(seen, x, -math.inf)
                    lse[at:at + m, h] = torch.logsumexp(x, -1)
                    out[at:at + m, h] = torch.nan_to_num(torch.softmax(x, -1)) @ v
        at += m
    return {"acc": acc} if acc is not None else {"out": out, "lse": lse}

"""The latent cache without a GPU: the host-side refusals of the C calls and of the binding (validation fails before a
pointer is used)."""
import ctypes
import shutil

import pytest
import torch
from test_warp_barriers import BARRIER, _source

import long_context_decode_lightning_gb300 as hsi

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None, reason="nvcc not on PATH")
F = 1 << 20  # an address that nothing reads


@pytest.fixture(scope="module")
def L():
    hsi.build()
    return hsi.lib()


def cache(**kw):
    f = dict(data=F, page_stride=64 * 1152, token_stride=1152, n_pages=100, table=F, ld_table=32, offsets=None, kv_len=F,
             B=4, dim=576, page_size=64, format=hsi.LATENT_BF16, table_width=0)
    f.update(kw)
    return hsi._LatentCache(**f)


def append(L, c, x=F, xt=576, q_start=F, T=4, pos=None, steps=None, rot=0, off=0, gain=1.0):
    return L.hsi_latent_append(ctypes.byref(c) if c else None, x, xt, q_start, T, pos, steps, rot, off, 1, gain, None)


def read(L, c, start=F, T=4, first=None, idx=None, ld=0, k=0, out=F, ot=576):
    return L.hsi_latent_read(ctypes.byref(c) if c else None, start, T, first, idx, ld, k, out, ot, None)


def attend(L, c, q=F, qt=16 * 576, qh=576, H=16, q_start=F, T=4, max_q=1, max_kv=2000, idx=None, ld=0, k=0, scale=0.1,
           out=2 * F, ot=16 * 512, oh=512, ws=F, ws_bytes=1 << 40):
    return L.hsi_latent_attention(ctypes.byref(c) if c else None, q, qt, qh, H, q_start, T, max_q, max_kv, idx, ld, k,
                                  scale, 1, out, ot, oh, None, ws, ws_bytes, None)


CALLS = [append, read, attend]


def test_entry_bytes(L):
    size = L.hsi_latent_entry_bytes
    assert [size(f, 576) for f in range(4)] == [1152, 1152, 656, 0]
    assert [size(f, 512) for f in range(4)] == [1024, 1024, 592, 288]
    assert size(4, 512) == size(-1, 512) == size(0, 128) == 0


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("status,kw", [
    (-1, dict(data=None)), (-1, dict(data=F + 8)), (-1, dict(kv_len=None)), (-1, dict(B=0)), (-1, dict(n_pages=0)),
    (-1, dict(format=4)), (-1, dict(format=-1)), (-2, dict(dim=128)), (-2, dict(dim=640)),
    (-2, dict(format=hsi.LATENT_FP4)), (-2, dict(B=65536)),
    (-1, dict(token_stride=1136)), (-1, dict(token_stride=1160)), (-1, dict(token_stride=1 << 40)),
    (-1, dict(token_stride=-1152)), (-1, dict(page_stride=1136)), (-1, dict(page_stride=64 * 1152 + 8)),
    (-1, dict(page_size=0)), (-2, dict(page_size=48)), (-2, dict(page_size=1 << 17)),
    (-1, dict(ld_table=0)), (-1, dict(table_width=33)), (-1, dict(table_width=-1)), (-1, dict(n_pages=(1 << 31) - 1)),
    (-1, dict(table=None)), (-1, dict(table=None, offsets=F + 4)),
])
def test_wrong_caches(L, call, status, kw):
    assert call(L, cache(**kw)) == status


@pytest.mark.parametrize("call", CALLS)
def test_no_cache(L, call):
    assert call(L, None) == -1


@pytest.mark.parametrize("status,kw", [
    (-1, dict(x=None)), (-1, dict(x=F + 8)), (-1, dict(xt=580)), (-1, dict(xt=-576)), (-1, dict(q_start=None)),
    (-1, dict(T=0)), (-1, dict(T=1 << 31)), (-1, dict(steps=F, rot=64)), (-1, dict(steps=F + 4, pos=F, rot=64)),
    (-1, dict(steps=F, pos=F, rot=63)), (-1, dict(steps=F, pos=F, rot=64, off=520)),
    (-1, dict(steps=F, pos=F, rot=64, off=-8)), (-2, dict(steps=F, pos=F, rot=24)),
    (-2, dict(steps=F, pos=F, rot=64, off=4)), (-1, dict(steps=F, pos=F, rot=64, gain=float("nan"))),
])
def test_wrong_appends(L, status, kw):
    assert append(L, cache(), **kw) == status


@pytest.mark.parametrize("status,kw", [
    (-1, dict(start=None)), (-1, dict(T=0)), (-1, dict(T=1 << 31)), (-1, dict(out=None)), (-1, dict(out=F + 2)),
    (-1, dict(ot=568)), (-1, dict(ot=580)), (-1, dict(idx=F, ld=10, k=0)), (-1, dict(idx=F, ld=9, k=10, ot=5760)),
    (-1, dict(idx=F + 2, ld=10, k=10, ot=5760)), (-1, dict(idx=F, ld=10, k=10, ot=5752)),
    (-1, dict(idx=F, ld=10, k=10, ot=5760, first=F)), (-2, dict(idx=F, ld=1 << 30, k=1 << 30, ot=1 << 45, T=1 << 20)),
])
def test_wrong_reads(L, status, kw):
    assert read(L, cache(), **kw) == status


@pytest.mark.parametrize("status,kw", [
    (-1, dict(q=None)), (-1, dict(q=F + 8)), (-1, dict(qt=577)), (-1, dict(qh=-8)), (-1, dict(q_start=None)),
    (-1, dict(T=0)), (-1, dict(T=1 << 31)), (-1, dict(H=0)), (-1, dict(max_q=0)), (-1, dict(max_kv=0)),
    (-1, dict(max_kv=1 << 31)), (-1, dict(scale=float("nan"))), (-1, dict(out=None)), (-1, dict(out=F)),
    (-1, dict(ot=504)), (-1, dict(oh=504)), (-1, dict(oh=516)), (-1, dict(idx=F, ld=4, k=5)), (-1, dict(idx=F, ld=4, k=0)),
    (-1, dict(idx=F + 1, ld=4, k=4)), (-5, dict(ws=None)), (-5, dict(ws_bytes=0)), (-5, dict(ws=F + 128)),
    (-2, dict(H=65536)),
])
def test_wrong_attentions(L, status, kw):
    assert attend(L, cache(), **kw) == status


def test_a_list_of_no_entries_is_not_the_want_of_lists(L):
    """k without idx (the address of an empty tensor is NULL): refused, not attention over everything."""
    assert attend(L, cache(), idx=None, k=5) == -1
    assert attend(L, cache(), idx=None, ld=5, k=5) == -1
    assert read(L, cache(), idx=None, ld=5, k=5, ot=5 * 576) == -1


def test_lengths_that_31_bits_cannot_count(L):
    wide = cache(table=None, offsets=F, n_pages=(1 << 31) + 5)
    assert attend(L, wide, max_kv=(1 << 31) - 1) == -2


@pytest.mark.parametrize("k", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 4096])
def test_lists_that_31_bits_cannot_count(L, k):
    """The kernels round k up to whole tiles in 32 bits; refused before the workspace is looked at."""
    assert attend(L, cache(), idx=F, ld=k, k=k, T=1, ws=None) == -2
    assert attend(L, cache(), idx=F, ld=1 << 40, k=k, T=1, ws=None) == -2


def test_the_longest_lists_are_counted(L):
    assert attend(L, cache(), idx=F, ld=(1 << 31) - 1, k=(1 << 31) - 4097, T=1, ws=None) == -5  # (but for the workspace)


def test_strides_that_no_second_row_uses(L):
    """Of one token or head they are not looked at (calls that a later check refuses); of two they are."""
    turn = dict(steps=F, pos=F, rot=24)
    assert append(L, cache(), xt=580, T=1, **turn) == append(L, cache(), xt=-8, T=1, **turn) == -2
    assert append(L, cache(), xt=580, T=2, **turn) == -1
    one = dict(T=1, H=1, ws=None)
    assert attend(L, cache(), qt=577, qh=-3, ot=7, oh=-1, **one) == -5
    assert attend(L, cache(), qh=577, **dict(one, H=2)) == attend(L, cache(), oh=513, **dict(one, H=2)) == -1
    assert attend(L, cache(), qt=577, **dict(one, T=2)) == attend(L, cache(), ot=513, **dict(one, T=2)) == -1
    assert attend(L, cache(), q=F + 8, **one) == attend(L, cache(), out=F + 8, **one) == -1


def test_kernels_use_the_barrier_helpers():
    for name in ("latent.cuh", "latent_attend.cuh"):
        assert not BARRIER.search(_source(name)), name


# ------------------------------------------------------------------ the binding --

class _Gpu(torch.Tensor):
    """A CPU tensor that says it is on the GPU: refusals need no more."""
    is_cuda = True


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Gpu)


def made(**kw):
    f = dict(data=gpu(10, 16, 576), kv_len=gpu(2, dtype=torch.int32), table=gpu(2, 4, dtype=torch.int32))
    f.update(kw)
    return hsi.LatentCache(**f)


def test_the_binding_makes_caches(L):
    c = made()
    assert (c.fmt, c.dim, c.B, c.c.token_stride, c.c.page_stride, c.c.n_pages) == (hsi.LATENT_BF16, 576, 2, 1152, 18432, 10)
    c = made(data=gpu(10, 16, 656, dtype=torch.uint8), fmt=hsi.LATENT_FP8, dim=576)
    assert (c.c.token_stride, c.x_dtype) == (656, torch.bfloat16)
    c = made(data=gpu(300, 288, dtype=torch.uint8), fmt=hsi.LATENT_FP4, dim=512, table=None,
             offsets=gpu(2, dtype=torch.int64))
    assert (c.c.token_stride, c.c.n_pages, c.c.table, c.table) == (288, 300, None, None)
    wide = gpu(2, 9, dtype=torch.int32)
    c = made(table=wide[:, :4])
    assert (c.c.ld_table, c.c.table_width) == (9, 4)
    other = gpu(2, 3, dtype=torch.int32)
    c.table = other
    assert (c.c.table, c.c.ld_table, c.table is other) == (other.data_ptr(), 3, True)


@pytest.mark.parametrize("kw", [
    dict(data=gpu(10, 16, 576, dtype=torch.float32)), dict(data=gpu(10, 16, 576), fmt=hsi.LATENT_FP16),
    dict(data=gpu(10, 16, 576), dim=512), dict(data=gpu(10, 16, 656, dtype=torch.uint8)),
    dict(data=gpu(10, 16, 656, dtype=torch.uint8), fmt=hsi.LATENT_FP8),
    dict(data=gpu(10, 16, 640, dtype=torch.uint8), fmt=hsi.LATENT_FP8, dim=576),
    dict(data=gpu(10, 16, 656, dtype=torch.uint8), fmt=hsi.LATENT_BF16, dim=576),
    dict(table=None), dict(offsets=gpu(2, dtype=torch.int64)), dict(data=gpu(160, 576)),
    dict(table=None, offsets=gpu(2, dtype=torch.int64)), dict(data=gpu(10, 16, 1152)[..., ::2]),
    dict(table=gpu(2, 4, dtype=torch.int64)), dict(table=gpu(8, dtype=torch.int32)),
    dict(kv_len=gpu(3, dtype=torch.int32)), dict(data=torch.zeros(10, 16, 576, dtype=torch.bfloat16)),
    dict(data=gpu(160, 576), table=None, offsets=gpu(2, dtype=torch.int32)),
])
def test_the_binding_refuses_caches(L, kw):
    with pytest.raises(ValueError):
        made(**kw)


def test_the_binding_refuses_calls(L):
    c, i32 = made(), dict(dtype=torch.int32)
    q_start, q, out = gpu(3, **i32), gpu(4, 8, 576), gpu(4, 8, 512)
    bad = [
        lambda: hsi.latent_append(c, gpu(4, 512), q_start),
        lambda: hsi.latent_append(c, gpu(4, 576, dtype=torch.float16), q_start),
        lambda: hsi.latent_append(c, gpu(4, 1, 576), q_start),
        lambda: hsi.latent_append(c, gpu(576, 4).T, q_start),
        lambda: hsi.latent_append(c, gpu(4, 576), gpu(2, **i32)),
        lambda: hsi.latent_append(c, gpu(4, 576), q_start, positions=gpu(3, **i32), steps=gpu(32, dtype=torch.int64)),
        lambda: hsi.latent_append(c, gpu(4, 576), q_start, positions=gpu(4, **i32), steps=gpu(32, **i32)),
        lambda: hsi.latent_read(c, gpu(4, 512), q_start),
        lambda: hsi.latent_read(c, gpu(4, 576, dtype=torch.float16), q_start),
        lambda: hsi.latent_read(c, gpu(4, 3, 576), q_start),
        lambda: hsi.latent_read(c, gpu(4, 576), q_start, idx=gpu(4, 3, **i32)),
        lambda: hsi.latent_read(c, gpu(4, 3, 576), q_start, idx=gpu(4, 4, **i32)),
        lambda: hsi.latent_read(c, gpu(4, 3, 600)[..., :576], q_start, idx=gpu(4, 3, **i32)),
        lambda: hsi.latent_read(c, gpu(4, 576), q_start, first=gpu(3, **i32)),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, gpu(4, 8, 576)),
        lambda: hsi.latent_attention(c, gpu(4, 8, 512), q_start, 1, 64, 0.1, out),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, gpu(4, 8, 512, dtype=torch.float16)),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, out, idx=gpu(3, 5, **i32)),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, out, idx=gpu(4, 5, dtype=torch.int64)),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, out, idx=gpu(4, 10, **i32)[:, ::2]),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, out, ws=torch.zeros(8)),
        lambda: hsi.latent_attention(c, q, q_start, 1, 64, 0.1, out, lse=gpu(4, 8), ws=gpu(8)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was taken")


def test_scratch_that_a_call_makes_belongs_to_its_stream(L, monkeypatch):
    """Without a workspace the wrapper makes one on the given stream, and hands the kernel that stream."""
    class Stream:
        cuda_stream = 77

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, args))
                return 4096 if name.endswith("_ws") else 0
            return call

    calls, made_for, s, c = [], [], Stream(), made()
    monkeypatch.setattr(hsi, "_lib", Lib())
    monkeypatch.setattr(hsi, "_scratch", lambda n, device, stream: made_for.append((n, stream)) or gpu(n, dtype=torch.uint8))
    hsi.latent_attention(c, gpu(4, 8, 576), gpu(3, dtype=torch.int32), 1, 64, 0.1, gpu(4, 8, 512), stream=s)
    assert made_for == [(4096, s)]
    assert [name for name, _ in calls] == ["hsi_latent_attention_ws", "hsi_latent_attention"] and calls[-1][1][-1] == 77


@pytest.mark.parametrize("idx", [gpu(4, 0, dtype=torch.int32), gpu(4, 7, dtype=torch.int32)[:, :0]])
def test_the_binding_refuses_lists_of_no_entries(L, monkeypatch, idx):
    """Such a tensor has no address, which the library would take for a call without lists."""
    class Lib:
        def __getattr__(self, name):
            return lambda *args: called.append(name) or 0

    c, q_start, called = made(), gpu(3, dtype=torch.int32), []
    monkeypatch.setattr(hsi, "_lib", Lib())
    with pytest.raises(ValueError, match="idx"):
        hsi.latent_attention(c, gpu(4, 8, 576), q_start, 1, 64, 0.1, gpu(4, 8, 512), idx=idx, ws=gpu(8))
    with pytest.raises(ValueError, match="idx"):
        hsi.latent_read(c, gpu(4, 0, 576), q_start, idx=idx)
    assert not called


def test_the_binding_refuses_a_table_of_no_pages(L):
    """Such a tensor has no address, by which a paged cache would count as one that may be given offsets."""
    for none in (gpu(2, 0, dtype=torch.int32), gpu(2, 4, dtype=torch.int32)[:, :0]):
        with pytest.raises(ValueError, match="table"):
            made(table=none)
        c = made()
        kept = c.table
        with pytest.raises(ValueError, match="table"):
            c.table = none
        assert c.table is kept and c.c.table == kept.data_ptr()


def test_lists_of_one_entry_may_lie_apart(L):
    """Of one entry a row, the distance between a row's entries does not matter; of two it does."""
    wide = gpu(4, 6, dtype=torch.int32)
    one, two = wide[:, ::7], wide[:, ::3]
    assert one.shape == (4, 1) and hsi._lists(one, 4) == (wide.data_ptr(), 6, 1)
    col = wide.view(24)[:4].view(1, 4).T
    assert col.stride() == (1, 4) and hsi._lists(col, 4) == (wide.data_ptr(), 1, 1)
    with pytest.raises(ValueError, match="idx"):
        hsi._lists(two, 4)

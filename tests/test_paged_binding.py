"""The paged-cache calls of the binding without a GPU: views that are narrower than a call's bounds, handles whose
tensors change, and the arguments that reach the library (a recorder stands in its place)."""
import types

import pytest
import torch

import long_context_decode_lightning_gb300 as hsi


class OnGpu(torch.Tensor):
    """A tensor that says it lies on the GPU; nothing here reads one."""
    is_cuda = True


class Recorder:
    """In the library's place: takes every call and keeps its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def ints(*shape):
    return gpu(*shape, dtype=torch.int32)


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(hsi, "_lib", r)
    return r


STREAM = types.SimpleNamespace(cuda_stream=0)
B, H, PAGE, PAGES = 2, 2, 16, 4


def cache(table=None):
    k = gpu(8, PAGE, H, 64, dtype=torch.bfloat16)
    return hsi.PagedKV(k, k, ints(B, PAGES) if table is None else table, ints(B))


def weights(kv, acc_in, acc_out, max_kv):
    q = gpu(B, 4, 64, dtype=torch.bfloat16)
    hsi.attention_weights(kv, q, gpu(B, 4), ints(B + 1), 1, max_kv, 0.1, acc_in, acc_out, stream=STREAM)


def select(acc, max_len, budget, acc_out=None):
    hsi.evict_select(acc, ints(B), max_len, budget, ints(B, H, budget), ints(B), acc_out=acc_out, stream=STREAM)


def refused(lib, call, *args):
    with pytest.raises(hsi.HsiError) as e:
        call(*args)
    assert e.value.status == -1 and not lib.calls


@pytest.mark.parametrize("cut", [slice(0, 40), slice(24, 64)])  # rows of 64, 40 of them in the view
def test_views_narrower_than_a_bound_are_refused(lib, cut):
    """Their rows stand 64 apart, but the places past the view's 40 are not the call's to read or write."""
    wide, view, kv = gpu(B, H, 64), gpu(B, H, 64)[:, :, cut], cache()
    refused(lib, weights, kv, None, view, 41)
    refused(lib, weights, kv, view, wide, 64)
    refused(lib, select, view, 41, 8)
    refused(lib, select, wide, 64, 41, view)
    refused(lib, select, view, 64, 8, view)
    weights(kv, view, view, 40)
    select(view, 40, 40, view)
    assert [c[0] for c in lib.calls] == ["hsi_attention_weights", "hsi_evict_select"]
    assert lib.calls[0][1][-2] == 64 and lib.calls[1][1][1] == 64  # the rows' distances


def test_weights_need_no_more_than_the_table_holds(lib):
    """A bound past the table is the table's: 64 entries."""
    weights(cache(), None, gpu(B, H, 64), 1 << 20)
    lib.calls.clear()
    refused(lib, weights, cache(), None, gpu(B, H, 63), 1 << 20)


def test_table_views_keep_their_width(lib):
    """Rows of a sliced table stand further apart than the pages that they list."""
    table = ints(B, 2 * PAGES)
    kv = cache(table[:, :PAGES])
    assert (kv.c.ld_table, kv.c.table_width) == (2 * PAGES, PAGES)
    assert (cache().c.ld_table, cache().c.table_width) == (PAGES, PAGES)
    keep = ints(B, H, PAGES * PAGE)
    hsi.paged_compact(kv, keep, ints(B), table[:, PAGES:], stream=STREAM)
    assert lib.calls.pop()[1][-2] == 2 * PAGES
    refused(lib, lambda: hsi.paged_compact(kv, keep, ints(B), table[:, PAGES + 1:], stream=STREAM))
    refused(lib, lambda: hsi.paged_compact(kv, ints(B, H, PAGES * PAGE + 1), ints(B), stream=STREAM))
    weights(kv, None, gpu(B, H, PAGES * PAGE), 1 << 20)
    lib.calls.clear()
    refused(lib, weights, kv, None, gpu(B, H, PAGES * PAGE - 1), 1 << 20)


def test_the_library_refuses_a_wrong_table_width():
    """(validation fails before a pointer is used)"""
    import ctypes
    import shutil
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not on PATH")
    hsi.build()
    f = 1 << 20

    def compact(width, ld=4, budget=32):
        kv = hsi._PagedKV(f, 2 * f, 16 * 128, 128, 64, 10, f, ld, f, 2, 2, 64, 16, 0, width)
        return hsi.lib().hsi_paged_compact(ctypes.byref(kv), f, 64, f, budget, f, ld, None)

    assert compact(-1) == -1 and compact(5) == -1
    assert compact(1) == -1  # in place: 32 places in one page of 16


def test_wide_bounds_of_mixed_batches():
    """Bounds of a batch in which one sequence brings a chunk and one may hold a million entries: what the kernels can
    count is not refused (validation goes on to the scratch, or to the lse, that is missing here), what they cannot is."""
    import ctypes
    import shutil
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not on PATH")
    hsi.build()
    L, f = hsi.lib(), 1 << 20

    def status(B, heads, q_heads, max_q, max_kv, T, token_stride=64 * 1024, fn="attention"):
        kv = hsi._PagedKV(f, 2 * f, 64 * 64 * 8, 512, 64, 1 << 20, f, 1 << 26, f, B, heads, 64, 64, 0)
        args = (ctypes.byref(kv), f, token_stride, 64, q_heads)
        if fn == "attention":
            return L.hsi_paged_attention(*args, f, T, max_q, max_kv, 0.1, 1, 4 * f, 64 * 1024, 64, None, None, 0, None)
        return L.hsi_attention_weights(*args, None, f, T, max_q, max_kv, 0.1, 1, 1.0, None, 0, f, max_kv, None)

    for fn, passed in (("attention", -5), ("weights", -1)):
        assert status(32, 8, 32, 2048, 1 << 20, 4096, fn=fn) == passed
        assert status(256, 8, 32, 2048, 1 << 17, 4096, fn=fn) == passed
        assert status(256, 8, 32, 1, 1 << 20, 256, fn=fn) == passed
        assert status(1, 8, 32, 1, (1 << 31) - 1, 1, fn=fn) == -2  # entries rounded up to tiles would pass 2^31
        assert status(1, 1, 64, 1 << 26, 64, 1 << 26, token_stride=0, fn=fn) == -2  # 2^32 rows of a KV head
    assert status(65535, 8, 32, 1 << 20, 1 << 20, 1 << 20) == -2


def test_a_cache_follows_its_tensors(lib):
    """After a move to other pages the caller sets table and kv_len: the library sees the new ones, and a move in place
    is one of the library's own table."""
    kv, dst, new_len = cache(), ints(B, PAGES + 1), ints(B)
    kv.table, kv.kv_len = dst, new_len
    assert (kv.c.table, kv.c.ld_table, kv.c.table_width) == (dst.data_ptr(), PAGES + 1, PAGES + 1)
    assert kv.c.kv_len == new_len.data_ptr() and kv.table is dst and kv.kv_len is new_len
    hsi.paged_compact(kv, ints(B, H, 8), ints(B), stream=STREAM)
    assert lib.calls[0][1][-3] == kv.c.table
    for wrong in (ints(B + 1, PAGES), ints(PAGES), gpu(B, PAGES), torch.zeros(B, PAGES, dtype=torch.int32)):
        with pytest.raises(ValueError):
            kv.table = wrong
    for wrong in (ints(B + 1), ints(B, 1), torch.zeros(B, dtype=torch.int32)):
        with pytest.raises(ValueError):
            kv.kv_len = wrong
    assert kv.table is dst and kv.kv_len is new_len and kv.c.table == dst.data_ptr()
    for name in ("k", "v"):
        with pytest.raises(AttributeError):
            setattr(kv, name, gpu(8, PAGE, H, 64, dtype=torch.bfloat16))


def test_in_place_needs_the_same_rows():
    """The same buffer read and written at other rows' distances, and lengths written over the lengths that are read:
    the host sees both. (A single row has no distance.)"""
    import ctypes
    import shutil
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not on PATH")
    hsi.build()
    L, f = hsi.lib(), 1 << 20

    def select(new_len=2 * f, acc_out=f, ld_out=100, B=2, heads=1):
        return L.hsi_evict_select(f, 100, f, B, heads, 100, 50, 0, 0, f, 50, new_len, acc_out, ld_out, None)

    assert select(new_len=f) == -1 and select(new_len=f, acc_out=None) == -1
    assert select(ld_out=120) == -1 and select(ld_out=50) == -1 and select(ld_out=50, B=1, heads=2) == -1
    kv = hsi._PagedKV(f, 2 * f, 16 * 128, 128, 64, 10, f, 4, f, 2, 2, 64, 16, 0)

    def weights(la, lo):
        return L.hsi_attention_weights(ctypes.byref(kv), f, 256, 64, 4, f, f, 3, 3, 60, 0.1, 1, 1.0, f, la, f, lo, None)

    assert weights(60, 61) == -1 and weights(100, 60) == -1
    assert L.hsi_paged_compact(ctypes.byref(kv), f, 32, f, 32, f, 5, None) == -1


def test_sizes_that_32_bits_cannot_count():
    """Places up to a turn past the budget, and a token's vectors, pass 2^31: refused before a pointer is used."""
    import ctypes
    import shutil
    if shutil.which("nvcc") is None:
        pytest.skip("nvcc not on PATH")
    hsi.build()
    L, f, most = hsi.lib(), 1 << 20, (1 << 31) - 1
    kv = ctypes.byref(hsi._PagedKV(f, 2 * f, 4096 * 128, 128, 64, 10, f, 1 << 20, f, 2, 2, 64, 4096, 0))
    for dst, ld in ((f, 1 << 20), (2 * f, 1 << 19)):
        assert L.hsi_paged_compact(kv, f, most, f, most, dst, ld, None) == -2
    heads = (1 << 25) + 1
    assert L.hsi_paged_append(kv, f, 128, 64, f, 128, 64, f, 1, f, f, 64, 0, 0, 1.0, f, 64 * heads, 64, heads, 2 * f,
                              64 * heads, 64, None) == -1

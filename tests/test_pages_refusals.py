"""What the paged cache and its attention refuse on the host, without a GPU: the C calls by
themselves, and the binding's checks of types, shapes and devices."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")

from tree_indexed_sparse_build_b200 import zha  # noqa: E402

F = ctypes.c_float


def _desc(**kw):
    d = dict(kv_heads=2, head_dim=64, page_tokens=16, num_pages=10, max_seqs=4, max_seq_pages=5, kv_dtype=zha.ZHA_BF16)
    d.update(kw)
    return zha.zha_pages_desc(**d)


def test_workspace_size():
    # a 64-word header, eight arrays of max_seqs, five of num_pages, the bitmap and the table
    assert zha.zha_pages_workspace_bytes(_desc()) == 256 * (1 + 8 + 5 + 1 + 1)
    assert zha.zha_pages_workspace_bytes(_desc(max_seqs=100, max_seq_pages=1000)) == 256 + 8 * 512 + 5 * 256 + 256 + 400128


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=96), 3), (dict(page_tokens=4), 3), (dict(page_tokens=24), 3), (dict(page_tokens=512), 3),
    (dict(page_tokens=0), 1), (dict(num_pages=0), 1), (dict(max_seqs=0), 1), (dict(max_seqs=65536), 1),
    (dict(max_seq_pages=0), 1), (dict(kv_heads=0), 1), (dict(kv_dtype=2), 1), (dict(num_pages=2 ** 30), 3),
    (dict(max_seq_pages=2 ** 27), 3), (dict(max_seqs=65535, max_seq_pages=2 ** 15), 3)])
def test_bad_geometry(bad, status):
    d = _desc(**bad)
    assert zha.zha_pages_workspace_bytes(d) == 0
    h = ctypes.c_void_p(1)
    assert zha.lib().zha_pages_init(ctypes.byref(d), ctypes.c_void_p(0x10000), 1 << 40, None, ctypes.byref(h)) == status
    assert h.value is None


def test_bad_workspace():
    h, d, lib = ctypes.c_void_p(), _desc(), zha.lib()
    need = zha.zha_pages_workspace_bytes(d)
    assert lib.zha_pages_init(ctypes.byref(d), None, need, None, ctypes.byref(h)) == zha.ZHA_ERR_INVALID_ARG
    assert lib.zha_pages_init(ctypes.byref(d), ctypes.c_void_p(0x10080), need, None, ctypes.byref(h)) == \
        zha.ZHA_ERR_INVALID_ARG
    assert lib.zha_pages_init(ctypes.byref(d), ctypes.c_void_p(0x10000), need - 1, None, ctypes.byref(h)) == \
        zha.ZHA_ERR_INVALID_ARG
    assert lib.zha_pages_init(ctypes.byref(d), ctypes.c_void_p(0x10000), need, None, None) == zha.ZHA_ERR_INVALID_ARG


def test_null_handles():
    lib, p = zha.lib(), ctypes.c_void_p(0x1000)
    bad = zha.ZHA_ERR_INVALID_ARG
    assert lib.zha_pages_destroy(None) == bad
    assert lib.zha_pages_load(None, p, p, None) == bad
    assert lib.zha_pages_append(None, p, p, p, 1, p, p, 1, None, None) == bad
    assert lib.zha_pages_fork(None, p, p, p, p, 1, None) == bad
    assert lib.zha_pages_copy(None, p, p, None, p, p, p, p, 1, None) == bad
    assert lib.zha_pages_free(None, p, 1, None) == bad
    assert lib.zha_pages_compact(None, p, p, None, None) == bad
    assert lib.zha_pages_gather(None, p, p, p, 1, p, p, 8, None) == bad
    assert lib.zha_pages_check(None, None) == bad
    assert lib.zha_pages_get_desc(None, None) == bad
    assert lib.zha_pages_set_wait_limit(None, 0) == bad
    assert lib.zha_prefix_attn_decode(None, p, 1, 1, 2, 1, p, p, p, 0, 0, 0, F(1.0), p, 1, p, 1 << 20, None) == bad
    assert lib.zha_prefix_attn_scratch_bytes(None, 1, 2, 1, 0) == 0
    assert lib.zha_pages_device(None) == -1 and lib.zha_pages_launch_count(None) == -1
    assert not lib.zha_pages_table(None) and not lib.zha_pages_lens(None) and not lib.zha_pages_refs(None)


# The binding's checks, with a fixed geometry in place of a handle's.
H = object()


@pytest.fixture(autouse=True)
def fake(monkeypatch):
    monkeypatch.setattr(zha, "zha_pages_get_desc", lambda h: _desc())
    monkeypatch.setattr(zha, "zha_pages_device", lambda h: 0)


def _pool(dtype=torch.bfloat16, n=10 * 2 * 16 * 64):
    return torch.zeros(n, dtype=dtype)


def _s(n=1, dtype=torch.int32):
    return torch.zeros(n, dtype=dtype)


def _new(n=1, T=3, dtype=torch.bfloat16, heads=2, d=64):
    return torch.zeros((n, heads, T, d), dtype=dtype)


def test_pools_of_another_size_or_type():
    for K, V, what in ((_pool(torch.float32), _pool(), "K: dtype"), (_pool(n=64), _pool(), "K: 64"),
                       (_pool(), _pool(n=64), "V: 64")):
        for call in (lambda: zha.zha_pages_append(H, K, V, _s(), _new(), _new()),
                     lambda: zha.zha_pages_fork(H, K, V, _s(), _s()),
                     lambda: zha.zha_pages_copy(H, _pool(), _pool(), H, K, V, _s(), _s()),
                     lambda: zha.zha_pages_compact(H, K, V),
                     lambda: zha.zha_pages_gather(H, K, V, _s(), _new(), _new()),
                     lambda: zha.zha_prefix_attn_decode(H, _new(), K, V, _s(), 0, 0, False, 0.1, _new(), _s())):
            with pytest.raises(ValueError, match=what):
                call()
    with pytest.raises(ValueError, match="K_from: 64"):
        zha.zha_pages_copy(H, _pool(n=64), _pool(), H, _pool(), _pool(), _s(), _s())


def test_lists():
    K = V = _pool()
    with pytest.raises(ValueError, match="seqs: dtype torch.int64"):
        zha.zha_pages_append(H, K, V, _s(dtype=torch.int64), _new(), _new())
    with pytest.raises(ValueError, match="counts: 2 elements"):
        zha.zha_pages_append(H, K, V, _s(), _new(), _new(), _s(2))
    with pytest.raises(ValueError, match="dst: 1 elements, expected 2"):
        zha.zha_pages_fork(H, K, V, _s(2), _s(1))
    with pytest.raises(ValueError, match="src: dtype"):
        zha.zha_pages_copy(H, K, V, H, K, V, _s(dtype=torch.int16), _s())
    with pytest.raises(ValueError, match="seqs: dtype"):
        zha.zha_pages_free(H, _s(dtype=torch.int64))
    with pytest.raises(ValueError, match="seqs: 2 elements"):
        zha.zha_prefix_attn_decode(H, _new(), K, V, _s(2), 0, 0, False, 0.1, _new(), _s())
    with pytest.raises(ValueError, match="table: 3 elements"):
        zha.zha_pages_load(H, _s(3), _s(4))
    with pytest.raises(ValueError, match="lens: 3 elements"):
        zha.zha_pages_load(H, _s(20), _s(3))
    with pytest.raises(ValueError, match="live: 2 elements"):
        zha.zha_pages_compact(H, K, V, _s(2))


def test_rows():
    K = V = _pool()
    for bad in (_new(n=2), _new(heads=1), _new(d=128), _new(dtype=torch.float32), torch.zeros(6, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="K_new"):
            zha.zha_pages_append(H, K, V, _s(), bad, _new())
        with pytest.raises(ValueError, match="K_out"):
            zha.zha_pages_gather(H, K, V, _s(), bad, _new())
    with pytest.raises(ValueError, match="V_new"):
        zha.zha_pages_append(H, K, V, _s(), _new(T=3), _new(T=4))
    with pytest.raises(ValueError, match="Q: shape"):
        zha.zha_prefix_attn_decode(H, _new(d=128), K, V, _s(), 0, 0, False, 0.1, _new(), _s())
    with pytest.raises(ValueError, match="Q: dtype torch.float16"):
        zha.zha_prefix_attn_decode(H, _new(dtype=torch.float16), K, V, _s(), 0, 0, False, 0.1, _new(), _s())
    with pytest.raises(ValueError, match="O: 4 elements"):
        zha.zha_prefix_attn_decode(H, _new(), K, V, _s(), 0, 0, False, 0.1, torch.zeros(4), _s())


def test_what_fits_reaches_the_device_check():
    K = V = _pool()
    for call in (lambda: zha.zha_pages_append(H, K, V, _s(), _new(), _new(), _s()),
                 lambda: zha.zha_pages_fork(H, K, V, _s(), _s()),
                 lambda: zha.zha_pages_load(H, _s(20), _s(4)),
                 lambda: zha.zha_pages_gather(H, K, V, _s(), _new(), _new()),
                 lambda: zha.zha_prefix_attn_decode(H, _new(), K, V, _s(), 0, 0, False, 0.1, _new(), _s())):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def _handle(**kw):
    """Memory that looks like a handle of this geometry on a device that is not there (all of its other
    fields are 148): for what a call answers before it asks the device."""
    d = _desc(**kw)
    h = (ctypes.c_int * 256)(*[148] * 256)
    ctypes.memmove(h, ctypes.byref(d), ctypes.sizeof(d))
    assert zha.lib().zha_pages_device(h) == 148
    return h


@pytest.mark.parametrize("geometry,q_heads,nq,batches", [
    # (32-key tiles of fp32 queries pass 31 bits between the two batches, 128-key tiles of bf16 queries do not)
    (dict(kv_heads=32, head_dim=128, page_tokens=256, num_pages=4, max_seqs=1, max_seq_pages=65536), 32, 1, (127, 128)),
    (dict(kv_heads=8, head_dim=128, page_tokens=64, num_pages=4, max_seqs=1, max_seq_pages=16384), 64, 512, (15, 128))])
def test_scratch_of_a_call_that_only_some_types_fit(geometry, q_heads, nq, batches):
    size = zha.lib().zha_prefix_attn_scratch_bytes
    h = _handle(**geometry)
    few, many = (size(h, b, q_heads, nq, 0) for b in batches)
    # a row's maximum, sum and head_dim values, for every row at least
    assert many >= batches[1] * q_heads * nq * (geometry["head_dim"] + 2) * 4 and few >= many * batches[0] // batches[1] // 2
    assert size(h, 2 ** 20 + 1, q_heads, nq, 0) == 0 and size(h, 1, q_heads, 2 ** 20 + 1, 0) == 0


def test_calls_with_another_device_current():
    # .. than the handle's, or none at all: refused before anything is launched, copied or read
    lib, p, h, g = zha.lib(), ctypes.c_void_p(0x1000), _handle(), _handle()
    bad = zha.ZHA_ERR_INVALID_ARG
    assert lib.zha_pages_load(h, p, p, None) == bad
    assert lib.zha_pages_append(h, p, p, p, 1, p, p, 1, None, None) == bad
    assert lib.zha_pages_fork(h, p, p, p, p, 1, None) == bad
    assert lib.zha_pages_copy(g, p, p, h, p, p, p, p, 1, None) == bad
    assert lib.zha_pages_free(h, p, 1, None) == bad
    assert lib.zha_pages_compact(h, p, p, None, None) == bad
    assert lib.zha_pages_gather(h, p, p, p, 1, p, p, 8, None) == bad
    assert lib.zha_prefix_attn_decode(h, p, 1, 1, 2, 1, p, p, p, 0, 0, 0, F(1.0), p, 1, p, 1 << 20, None) == bad
    # (the default stream is the current device's: a check on it would not wait for the cache's work)
    assert lib.zha_pages_check(h, None) == bad


def test_pools_that_a_copy_reads(monkeypatch):
    # the pools that are named are the ones that are read, and another cache's have to be named
    calls = []
    monkeypatch.setattr(zha, "zha_pages_copy", lambda *a: calls.append(a))
    pages, other = (object.__new__(zha.Pages) for _ in range(2))
    pages.handle, other.handle = None, None
    K, V, A, B, s = (object() for _ in range(5))
    pages.copy(K, V, s, s)
    pages.copy(K, V, s, s, K_from=A, V_from=B)
    pages.copy(K, V, s, s, source=other, K_from=A, V_from=B)
    assert [c[1:3] for c in calls] == [(K, V), (A, B), (A, B)]
    for kw in (dict(source=other), dict(source=other, K_from=A), dict(K_from=A), dict(V_from=B)):
        with pytest.raises(ValueError, match="K_from and V_from"):
            pages.copy(K, V, s, s, **kw)
    assert len(calls) == 3

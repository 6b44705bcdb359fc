"""What the 4-bit cache's binding refuses before anything is launched."""
import numpy as np
import pytest
import torch

import speculative_decoding_tree_bit_gb300 as sdv
from speculative_decoding_tree_bit_gb300 import _build


@pytest.fixture(scope="module")
def M():
    _build.build()
    sdv.lib()
    from speculative_decoding_tree_bit_gb300 import model
    return model


def rows16(n, heads, dim=128):
    return torch.zeros(n, heads, dim, dtype=torch.bfloat16)


def test_slopes_and_starts_too_short_are_refused(M):
    """They are read by query head and by request."""
    c = M.KV4Cache(np.zeros((3, 1)), 1, 2, 128, 64, device="cpu")
    rows, q, lse = M.RequestRows([0, 1, 2, 4], device="cpu"), rows16(4, 8), torch.zeros(4, 8)
    for score, what in ((M.KV4Score(slopes=torch.zeros(7)), "slopes"), (M.KV4Score(slopes=torch.zeros(0)), "slopes"),
                        (M.KV4Score(start=torch.zeros(2, dtype=torch.int32)), "start")):
        with pytest.raises(ValueError, match=what):
            c.attend(q, rows, score=score)
        with pytest.raises(ValueError, match=what):
            c.observe(q, lse, rows, score=score)


def test_tensors_off_the_caches_gpu_are_refused(M):
    """Their pointers mean nothing to the kernels."""
    def cache(index):
        c = M.KV4Cache(np.zeros((2, 1)), 1, 2, 128, 64, device="cpu")
        c._index = index
        return c
    gpu = cache(0)  # stands for a cache on GPU 0; everything below lies on the CPU
    rows = M.RequestRows([0, 1, 3], device="cpu")
    with pytest.raises(ValueError, match="rows is on cpu"):
        gpu.read(rows)
    rows.index = 0
    k, q, lse, w = rows16(3, 2), rows16(3, 4), torch.zeros(3, 4), torch.zeros(2, 2, 64)
    i32, i64, f32 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    with pytest.raises(ValueError, match="k is on cpu"):
        gpu.append(k, k, rows)
    with pytest.raises(ValueError, match="q is on cpu"):
        gpu.attend(q, rows)
    with pytest.raises(ValueError, match="q is on cpu"):
        gpu.observe(q, lse, rows)
    with pytest.raises(ValueError, match="dst is on cpu"):
        gpu.evict(cache(0), 16)
    with pytest.raises(ValueError, match="at is on cpu"):
        gpu.read(rows, at=i32)
    # each optional tensor, with the ones before it taken as they are
    here, M._here = M._here, lambda t, index, what: here(t, index, what) if what == off else None
    try:
        for off, call in (("v", lambda: gpu.append(k, k, rows)), ("src", lambda: gpu.append(k, k, rows, src=i32)),
                          ("count", lambda: gpu.append(k, k, rows, count=i32)), ("pos", lambda: gpu.append(k, k, rows, pos=i32)),
                          ("at", lambda: gpu.append(k, k, rows, at=i32)), ("k", lambda: gpu.attend(q, rows, k, k)),
                          ("v", lambda: gpu.attend(q, rows, k, k)), ("out", lambda: gpu.attend(q, rows, out=q)),
                          ("lse", lambda: gpu.attend(q, rows, lse=lse)), ("anc", lambda: gpu.attend(q, rows, anc=i64)),
                          ("pos", lambda: gpu.attend(q, rows, pos=i32)),
                          ("slopes", lambda: gpu.attend(q, rows, score=M.KV4Score(slopes=torch.zeros(4)))),
                          ("start", lambda: gpu.attend(q, rows, score=M.KV4Score(start=i32))),
                          ("lse", lambda: gpu.observe(q, lse, rows)), ("out", lambda: gpu.observe(q, lse, rows, out=w)),
                          ("pos", lambda: gpu.observe(q, lse, rows, pos=i32)),
                          ("row_weight", lambda: gpu.observe(q, lse, rows, row_weight=f32))):
            with pytest.raises(ValueError, match=f"^{off} is on cpu, the cache on cuda:0"):
                call()
    finally:
        M._here = here


def test_a_cache_on_the_cpu_launches_nothing(M):
    c, d = (M.KV4Cache(np.zeros((1, 1)), 1, 2, 128, 64, device="cpu") for _ in range(2))
    rows = M.RequestRows([0, 2], device="cpu")
    k, q = rows16(2, 2), rows16(2, 4)
    for call in (lambda: c.append(k, k, rows), lambda: c.read(rows), lambda: c.attend(q, rows),
                 lambda: c.observe(q, torch.zeros(2, 4), rows), lambda: c.evict(d, 16)):
        with pytest.raises(ValueError, match="lies on the CPU"):
            call()


def test_the_workspace_is_made_on_the_calls_stream(M, monkeypatch):
    """... where its zeroing comes before the kernel, not on the current one;
    and not kept when a capture only records that zeroing."""
    import contextlib
    entered = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: (entered.append(s), contextlib.nullcontext())[1])
    c = M.KV4Cache(np.zeros((1, 1)), 1, 2, 128, 64, device="cpu")
    size = lambda n: n  # noqa: E731
    a = c._workspace("attn", "other", size, 5000)
    assert entered == ["other"] and a[2] >= 5000 and int(a[3][:M.KV4_TICKET_BYTES].sum()) == 0
    assert c._workspace("attn", "other", size, 5000) is a and entered == ["other"]
    assert c._workspace("attn", None, size, 4500)[1] == a[1]  # large enough already
    real = M.torch.empty
    class Captured(torch.Tensor):
        is_cuda = True
    monkeypatch.setattr(M.torch, "empty", lambda *s, **k: real(*s, **k).as_subclass(Captured))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    b = c._workspace("attn", None, size, 9000)
    assert c._workspace("attn", None, size, 9000) is not b
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    d = c._workspace("attn", None, size, 9000)
    assert d[1] not in (a[1],) and c._workspace("attn", None, size, 9000) is d


def test_calls_without_rows_take_null_arrays(M):
    """As an empty tensor's pointer is."""
    import ctypes
    ptr, L = 4096, sdv.lib()
    c, cu = sdv.KV4(ptr, ptr, ptr, 8, 64, 2, 128, ptr, 4, ptr), np.array([0, 0, 0], np.int32)
    b, h = ctypes.byref(c), cu.ctypes.data
    assert L.sd_kv4_append(b, None, None, 256, 0, ptr, h, 2, None, None, None, None, None, None) == 0
    assert L.sd_kv4_read(b, ptr, h, 2, None, None, None, None, None) == 0
    assert L.sd_kv4_attn(b, None, 512, 4, ptr, h, 2, None, None, 0, None, None, None, 0, None, None, ptr, 1 << 24, None,
                         None) == 0

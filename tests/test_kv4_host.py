"""The 4-bit cache without a GPU: refusals of the C entry points and of the
binding, sizes, and the 64-bit definition the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as ref
import speculative_decoding_tree_bit_gb300 as sdv
from speculative_decoding_tree_bit_gb300 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sdv.lib()


PTR = 4096  # never dereferenced: every call below is refused on the host


def _cache(**kw):
    c = sdv.KV4(PTR, PTR, PTR, 8, 64, 2, 128, PTR, 4, PTR)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _cu(*v):
    return np.array(v, np.int32)


CACHE_FAULTS = [(dict(blocks=0), 1), (dict(pos=0), 1), (dict(weight=0), 1), (dict(page_table=0), 1),
                (dict(ctx_len=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(n_kv_heads=0), 1),
                (dict(head_dim=96), 2), (dict(page_size=16), 2), (dict(page_size=48), 2), (dict(blocks=PTR + 8), 1),
                (dict(pos=PTR + 4), 1), (dict(max_pages=1 << 26), 2)]


def test_group_bytes(L):
    assert [L.sd_kv4_group_bytes(d) for d in (64, 128, 96, 0)] == [2304, 4352, 0, 0]


@pytest.mark.parametrize("fault,code", CACHE_FAULTS)
def test_a_bad_cache_is_refused_everywhere(L, fault, code):
    c, ok = _cache(**fault), _cache(pos=2 * PTR, weight=2 * PTR, ctx_len=2 * PTR)
    cu = _cu(0, 3)
    h = cu.ctypes.data
    b = ctypes.byref
    ws = 1 << 24
    assert L.sd_kv4_append(b(c), PTR, PTR, 256, 3, PTR, h, 1, None, None, None, None, None, None) == code
    assert L.sd_kv4_read(b(c), PTR, h, 1, None, PTR, PTR, None, None) == code
    assert L.sd_kv4_attn(b(c), PTR, 512, 4, PTR, h, 1, None, None, 0, None, None, None, 0, PTR, None, PTR, ws, None,
                         None) == code
    assert L.sd_kv4_observe(b(c), PTR, 512, 4, PTR, PTR, h, 1, None, None, None, 0, 1.0, PTR, None, None) == code
    assert L.sd_kv4_evict(b(c), b(ok), 1, 64, 0, 0, PTR, ws, None, None) == code
    assert L.sd_kv4_evict(b(ok), b(c), 1, 64, 0, 0, PTR, ws, None, None) == code
    assert L.sd_last_error()


def test_append_and_read_refusals(L):
    c, cu = _cache(), _cu(0, 3)
    def call(k=PTR, v=PTR, stride=256, n_src=3, cu_d=PTR, off=cu, R=1, src=None):
        return L.sd_kv4_append(ctypes.byref(c), k, v, stride, n_src, cu_d, off.ctypes.data if off is not None else None,
                               R, src, None, None, None, None, None)
    assert call(k=None) == 1 and call(v=None) == 1 and call(k=PTR + 2) == 1 and call(v=PTR + 8) == 1
    assert call(stride=255) == 1 and call(stride=257) == 1 and call(stride=200) == 1
    assert call(n_src=2) == 1 and call(n_src=-1, src=PTR) == 1
    assert call(cu_d=None) == 1 and call(off=None) == 1 and call(R=0) == 1 and call(R=1 << 17) == 1
    assert call(off=_cu(1, 3)) == 1 and call(off=_cu(0, 3, 2), R=2) == 1
    assert call(off=_cu(0, 0), n_src=0) == 0  # no rows: nothing is launched
    def rd(k=PTR, v=PTR, off=cu):
        return L.sd_kv4_read(ctypes.byref(c), PTR, off.ctypes.data, 1, None, k, v, None, None)
    assert rd(k=None) == 1 and rd(v=PTR + 2) == 1 and rd(off=_cu(0, 0)) == 0


def test_attention_refusals(L):
    c, cu = _cache(), _cu(0, 3)
    ws = L.sd_kv4_attn_workspace(1, 3, 4, 2, 128)
    assert ws > 0
    def call(q=PTR, stride=512, hq=4, off=cu, k=None, v=None, kvs=0, score=None, max_ctx=0, out=PTR, w=PTR, n=None):
        return L.sd_kv4_attn(ctypes.byref(c), q, stride, hq, PTR, off.ctypes.data, off.size - 1, k, v, kvs, None, None,
                             ctypes.byref(score) if score else None, max_ctx, out, None, w, ws if n is None else n,
                             None, None)
    assert call(q=None) == 1 and call(q=PTR + 4) == 1 and call(stride=511) == 1 and call(stride=516) == 1
    assert call(hq=3) == 1 and call(hq=0) == 1 and call(hq=34, stride=34 * 128) == 2
    assert call(off=_cu(0, 65)) == 2 and call(max_ctx=-1) == 1
    assert call(k=PTR) == 1 and call(v=PTR) == 1
    assert call(k=PTR, v=PTR, kvs=128) == 1 and call(k=PTR, v=PTR + 2, kvs=256) == 1
    assert call(out=None) == 1 and call(out=PTR + 8) == 1
    assert call(w=None) == 1 and call(w=PTR + 128) == 1 and call(n=ws - 1) == 9
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(scale=-0.5),
                dict(window=-1)):
        s = sdv.KV4ScoreArgs(0.0, 0.0, None, 0, None)
        for key, val in bad.items():
            setattr(s, key, val)
        assert call(score=s) == 1, bad
    assert call(off=_cu(0, 0)) == 0
    assert L.sd_kv4_attn_workspace(1, 3, 5, 2, 128) == 0 and L.sd_kv4_attn_workspace(0, 3, 4, 2, 128) == 0
    def obs(lse=PTR, out=PTR, decay=1.0, off=cu):
        return L.sd_kv4_observe(ctypes.byref(c), PTR, 512, 4, lse, PTR, off.ctypes.data, off.size - 1, None, None,
                                None, 0, decay, out, None, None)
    assert obs(lse=None) == 1 and obs(out=None) == 1 and obs(out=PTR + 4) == 1
    assert obs(decay=-1.0) == 1 and obs(decay=float("nan")) == 1 and obs(off=_cu(0, 65)) == 2


def test_eviction_refusals(L):
    a, b = _cache(), _cache(pos=2 * PTR, weight=2 * PTR, ctx_len=2 * PTR)
    def call(src=a, dst=b, R=1, budget=64, recent=8, sinks=4, w=PTR, n=1 << 20):
        return L.sd_kv4_evict(ctypes.byref(src), ctypes.byref(dst), R, budget, recent, sinks, w, n, None, None)
    assert call(budget=0) == 1 and call(recent=-1) == 1 and call(sinks=-1) == 1 and call(recent=61) == 1
    assert call(budget=257) == 1            # dst holds 4 pages of 64
    assert call(dst=a) == 1                 # dst must have arrays of its own
    assert call(w=None) == 1 and call(w=PTR + 64) == 1 and call(n=64 * 2 * 4 - 1) == 9
    c = _cache(pos=2 * PTR, weight=2 * PTR, ctx_len=2 * PTR, n_kv_heads=4)
    assert call(dst=c) == 1
    c = _cache(pos=2 * PTR, weight=2 * PTR, ctx_len=2 * PTR, head_dim=64)
    assert call(dst=c) == 1
    assert L.sd_kv4_evict_workspace(3, 2, 64) == 3 * 2 * 64 * 4 and L.sd_kv4_evict_workspace(0, 2, 64) == 0


def test_binding_refusals(L):
    from speculative_decoding_tree_bit_gb300 import model as M
    for cu in ([1, 2], [0], [0, 3, 2], [[0, 1]]):
        with pytest.raises(ValueError):
            M.RequestRows(cu, device="cpu")
    rows = M.RequestRows([0, 2], device="cpu")
    with pytest.raises(ValueError):
        M.KV4Cache(np.zeros((1, 1)), 1, 2, 80, 64, device="cpu")
    with pytest.raises(ValueError):
        M.KV4Cache(np.zeros((1, 1)), 1, 2, 128, 40, device="cpu")
    c = M.KV4Cache(np.zeros((1, 1)), 1, 2, 128, 64, device="cpu")
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    for bad in (k.half(), k.float(), k[:, :1], k.transpose(1, 2), k[..., ::2]):
        with pytest.raises(ValueError):
            c.append(bad, k, rows)
    with pytest.raises(ValueError):
        c.append(k, k, M.RequestRows([0, 1, 2], device="cpu"))
    with pytest.raises(ValueError):
        c.append(k, k, rows, pos=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        c.append(k, k, rows, at=3)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        c.attend(q, rows, k=k)
    with pytest.raises(ValueError):
        c.attend(q[:, :3], rows)
    with pytest.raises(ValueError):
        c.attend(q, rows, anc=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        c.observe(q, torch.zeros(1), rows)
    with pytest.raises(ValueError):
        c.evict(c, 16)
    with pytest.raises(ValueError):
        M.KV4Score(slopes=torch.zeros(4, dtype=torch.float64))


def test_the_definition_holds_its_bound():
    """A value is at most half a step off, or what the rounding of s and m to
    bf16 takes at the row's ends: 15 s 2^-9 + |m| 2^-9 + half a step."""
    g = torch.Generator().manual_seed(3)
    x = ref.bf16(torch.randn(200, 128, generator=g).double() * 3 + torch.randn(200, 1, generator=g).double())
    c, s, m = ref.quantise(x)
    assert c.min() == 0 and c.max() == 15
    err = (ref.values(x) - x).abs()
    assert (err <= (s * (0.5 + 15 / 512) + m.abs() / 256)[:, None]).all()
    assert torch.equal(ref.values(torch.full((1, 64), 2.5).double()), torch.full((1, 64), 2.5).double())

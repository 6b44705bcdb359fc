"""Rotary tables, and what the rotary, prompt and sampling calls refuse before
anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

import request_ref as ref
import speculative_decoding_tree_bit_gb300 as sdv
from speculative_decoding_tree_bit_gb300 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return sdv.lib()


@pytest.fixture(scope="module")
def M(L):
    from speculative_decoding_tree_bit_gb300 import model
    return model


KINDS = {"plain": {}, "linear": dict(factor=3.0), "bands": dict(factor=8.0, original=8192.0, low=1.0, high=4.0),
         "ramp": dict(factor=16.0, original=4096.0, low=1.0, high=32.0)}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rot,base", [(2, 1e4), (20, 1e4), (64, 5e5), (128, 1e6)])
def test_turns_are_the_frequencies(L, kind, rot, base):
    """As fractions of 2^64, so that pos turns mod 2^64 is the angle of any position."""
    a = KINDS[kind]
    args = sdv.RopeScalingArgs(list(KINDS).index(kind), a.get("factor", 1), a.get("original", 1), a.get("low", 1), a.get("high", 2), 0)
    turns, amp = np.zeros(rot // 2, np.uint64), ctypes.c_float()
    assert L.sd_rope_turns_host(rot, base, ctypes.byref(args), turns.ctypes.data, ctypes.byref(amp)) == 0
    freq = ref.frequencies(rot, base, kind, **a)
    # cut to a whole number (one), both sides' pow and log in 64 bits (2^-43 of the value)
    want = freq / (2 * math.pi) * 2.0 ** 64
    assert (np.abs(turns.astype(np.float64) - want) <= 1 + 1e-13 * want).all()
    assert amp.value == np.float32(0.1 * math.log(a["factor"]) + 1 if kind == "ramp" else 1.0)
    for pos in (1, 4097, 2 ** 20, -5):
        frac = (int(turns[0]) * pos % 2 ** 64) / 2.0 ** 64
        assert abs(math.cos(2 * math.pi * frac) - math.cos(pos * freq[0])) < 1e-9


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rot,base", [(2, 1e4), (20, 1e4), (64, 5e5), (96, 1e7), (128, 1e6), (256, 1e4)])
def test_turns_against_60_digits(L, kind, rot, base):
    """All pairs, off by at most the documented 2^-53 of a turn a position: of f <= 1 and f / 2 pi <= 0.16 the power is
    off by its own rounding (2^-53) and its exponent's (y e^-y 2^-53, at most 0.4), the scaling by four
    roundings (2^-53 each) and the quotient by its own and pi's (2^-54): (1 + 0.4 + 4) 0.16 2^-53 + 0.16 2^-52."""
    a = KINDS[kind]
    args = sdv.RopeScalingArgs(list(KINDS).index(kind), a.get("factor", 1), a.get("original", 1), a.get("low", 1), a.get("high", 2), 0)
    turns, amp = np.zeros(rot // 2, np.uint64), ctypes.c_float()
    assert L.sd_rope_turns_host(rot, base, ctypes.byref(args), turns.ctypes.data, ctypes.byref(amp)) == 0
    want = ref.exact_turns(rot, base, kind, **a)
    off = [abs(float(int(t) - w * 2 ** 64)) for t, w in zip(turns, want)]
    assert max(off) <= 2.0 ** (64 - 53)
    for pos in (2 ** 31 - 1, -2 ** 31, 2 ** 20, -5):
        for t, w in zip(turns, want):
            d = float((int(t) * pos - w * pos * 2 ** 64) % 2 ** 64) / 2.0 ** 64
            assert min(d % 1.0, 1.0 - d % 1.0) <= abs(pos) * 2.0 ** -53


def test_turns_refusals(L):
    out, amp = np.zeros(64, np.uint64), ctypes.c_float()
    call = lambda rot=128, base=1e6, s=None: L.sd_rope_turns_host(  # noqa: E731
        rot, base, None if s is None else ctypes.byref(sdv.RopeScalingArgs(*s)), out.ctypes.data, ctypes.byref(amp))
    assert call() == 0
    nan, inf = math.nan, math.inf
    assert [call(rot=r) for r in (0, -2, 3)] == [1, 1, 1]
    assert [call(base=b) for b in (0.0, -1.0, nan, inf)] == [1] * 4
    assert call(s=(4, 1, 1, 1, 2, 0)) == 1 and call(s=(-1, 1, 1, 1, 2, 0)) == 1
    for f in (0.0, -1.0, nan, inf):
        assert call(s=(1, f, 1, 1, 2, 0)) == 1 and call(s=(2, 2, f, 1, 2, 0)) == 1 and call(s=(3, 2, 1, f, 2, 0)) == 1
    assert call(s=(2, 2, 10, 4, 4, 0)) == 1 and call(s=(3, 2, 10, 4, 1, 0)) == 1
    assert call(s=(1, 2, 1, 1, 2, nan)) == 1
    assert call(base=1.0, s=(3, 2, 10, 1, 4, 0)) == 1
    assert call(s=(1, 2, 0, 0, 0, 0)) == 0  # what a kind does not use is not looked at
    assert L.sd_rope_turns_host(4, 1e4, None, None, ctypes.byref(amp)) == 1


def rope(L, q=1 << 20, k=1 << 21, q_out=1 << 22, k_out=1 << 23, rows=4, hq=4, hk=2, d=64, rot=64, qs=256, ks=128, qos=256, kos=128,
         turns=1 << 10, pos=1 << 12):
    v = lambda x: ctypes.c_void_p(x)  # noqa: E731
    return L.sd_rope(v(turns), 1.0, d, rot, 0, v(pos), rows, v(q), qs, hq, v(q_out), qos, v(k), ks, hk, v(k_out), kos, None)


def test_rope_refusals(L):
    """No call here passes: nothing would be launched."""
    assert rope(L, rows=0) == 0
    for kw in (dict(rows=-1), dict(hq=0), dict(hk=-1), dict(d=0), dict(d=2048), dict(rot=63), dict(rot=0), dict(rot=66), dict(turns=0),
               dict(pos=0), dict(q=0), dict(q_out=0), dict(k=0), dict(k_out=0), dict(hk=0), dict(qs=255), dict(ks=127),
               dict(qos=255), dict(kos=100)):
        assert rope(L, **kw) == 1, kw
    # outputs over other tensors, or shifted over their own
    q = 1 << 20
    for kw in (dict(q_out=q + 16), dict(k_out=q), dict(k_out=q + 100), dict(k_out=1 << 22), dict(q_out=1 << 21), dict(q_out=q, qos=512),
               dict(k=q, k_out=q, hk=4, ks=256, kos=256), dict(q_out=q, k_out=q + 512, kos=256)):
        assert rope(L, **kw) == 1, kw


def test_rope_binding_refuses(M):
    for kw in (dict(head_dim=0), dict(rot_dim=3), dict(rot_dim=256), dict(rot_dim=0)):
        with pytest.raises(ValueError):
            M.Rope(device="cpu", **kw)
    with pytest.raises(sdv.SdvError):
        M.Rope(base=-1.0, device="cpu")
    with pytest.raises(sdv.SdvError):
        M.Rope(scaling=M.RopeScaling.bands(2.0, 100.0, low=4.0, high=1.0), device="cpu")
    op = M.Rope(64, device="cpu")
    q = torch.zeros(3, 4, 64).bfloat16()
    with pytest.raises(ValueError, match="CPU"):
        op(q, None, torch.zeros(3, dtype=torch.int32))


def test_prompt_refusals(L):
    v = lambda x: ctypes.c_void_p(x)  # noqa: E731
    cu, ck = np.array([0, 3, 5], np.int32), np.array([0, 3, 9], np.int32)

    def call(q=256, qs=512, hq=8, k=256, vv=256, ks=128, hk=2, d=64, cuq=256, cuqh=cu, cuk=256, cukh=ck, R=2, score=None, out=256,
             ws=256, n=1 << 40):
        p = lambda a: None if a is None else a.ctypes.data  # noqa: E731
        return L.sd_prompt_attn(v(q), qs, hq, v(k), v(vv), ks, hk, d, v(cuq), p(cuqh), v(cuk), p(cukh), R, score, v(out), None,
                                v(ws), n, None, None)

    for kw in (dict(d=96), dict(d=0), dict(hq=7), dict(hk=0), dict(hq=0), dict(hq=258)):
        assert call(**kw) == 2, kw
    for kw in (dict(R=0), dict(cuq=0), dict(cuqh=None), dict(cuk=0), dict(cukh=None), dict(cuqh=np.array([1, 2, 3], np.int32)),
               dict(cuqh=np.array([0, 3, 2], np.int32)), dict(cukh=np.array([0, -1, 2], np.int32)), dict(q=0), dict(k=0), dict(vv=0),
               dict(out=0), dict(q=264), dict(k=258), dict(vv=264), dict(out=260), dict(qs=511), dict(qs=516), dict(ks=120),
               dict(ks=130), dict(ws=0), dict(ws=128)):
        assert call(**kw) == 1, kw
    assert call(n=16) == 9
    for s in (sdv.KV4ScoreArgs(-1.0, 0, None, 0, None), sdv.KV4ScoreArgs(0, math.nan, None, 0, None), sdv.KV4ScoreArgs(0, 0, None, -1, None),
              sdv.KV4ScoreArgs(0, 0, None, 0, 256)):
        assert call(score=ctypes.byref(s)) == 1
    assert call(cuqh=np.array([0, 0, 0], np.int32)) == 0  # no rows: nothing to do
    assert L.sd_prompt_attn_workspace(96) == 0 and L.sd_prompt_attn_workspace(64) > 0


def test_prompt_output_over_an_input(L):
    """2 rows of 2 heads, 4 keys of 1: out over any part of q, k or v is refused."""
    cu, ck = np.array([0, 2], np.int32), np.array([0, 4], np.int32)
    q, k, vv = 4096, 8192, 12288  # 2 x 256 bytes; 4 rows of 128, 512 apart

    def call(out):
        v = lambda x: ctypes.c_void_p(x)  # noqa: E731
        return L.sd_prompt_attn(v(q), 128, 2, v(k), v(vv), 256, 1, 64, v(256), cu.ctypes.data, v(256), ck.ctypes.data, 1, None, v(out),
                                None, v(256), 1 << 40, None, None)

    for out in (q, q - 496, q + 496, k, k + 3 * 512 + 112, k - 496, vv, vv + 3 * 512 + 112):
        assert call(out) == 1 and b"overlaps" in L.sd_last_error(), out


def test_prompt_binding_refuses(M):
    for a in ((8, 3, 64), (8, 2, 96), (0, 1, 64), (129, 1, 64)):
        with pytest.raises(ValueError):
            M.PromptAttention(*a, device="cpu")
    op = M.PromptAttention(4, 2, 64, device="cpu")
    q, k = torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 2, 64).bfloat16()
    with pytest.raises(ValueError, match="CPU"):
        op(q, k, k, M.RequestRows([0, 3], device="cpu"))


def test_prompt_wait_refusals(L):
    assert [L.sd_debug_prompt_wait(*x) for x in ((-1, 0), (2_000_000_001, 0), (1000, -1))] == [1, 1, 1]
    assert L.sd_debug_prompt_wait(0, 0) == 0


def test_sample_refusals(L, M):
    v = lambda x: ctypes.c_void_p(x)  # noqa: E731

    def call(x=256, stride=100, rows=4, V=100, t=1.0, p=1.0, m=0.0, k=0, u=256, tokens=256, s=True):
        a = sdv.Sampling(t, p, m, k, None, None, None, None)
        return L.sd_sample(v(x), stride, rows, V, ctypes.byref(a) if s else None, v(u), v(tokens), None, None, None)

    assert call(rows=0) == 0
    for kw in (dict(x=0), dict(x=257), dict(u=0), dict(tokens=0), dict(rows=-1), dict(V=0), dict(stride=99), dict(t=-1.0), dict(t=math.nan),
               dict(t=math.inf), dict(p=0.0), dict(p=-1.0), dict(p=math.nan), dict(m=-0.1), dict(m=1.1), dict(m=math.nan), dict(k=-1),
               dict(s=False)):
        assert call(**kw) == 1, kw
    assert call(V=524161, stride=524161) == 2
    with pytest.raises(ValueError, match="CPU"):
        M.sample(torch.zeros(2, 10).bfloat16(), torch.zeros(2))


def test_counts_past_32_bits_are_the_most(M):
    """Not their low bits: a window or a top_k of 2^32 + 5 keeps everything."""
    assert [M.KV4Score(window=w).args.window for w in (2 ** 32 + 5, 2 ** 31, 7, -2 ** 32 + 3)] == [2 ** 31 - 1, 2 ** 31 - 1, 7, -2 ** 31]

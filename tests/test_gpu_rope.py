"""Rotary positions against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import request_ref as ref

pytestmark = pytest.mark.gpu
KINDS = {"plain": {}, "linear": dict(factor=4.0), "bands": dict(factor=8.0, original=8192.0, low=1.0, high=4.0),
         "ramp": dict(factor=4.0, original=4096.0, low=1.0, high=32.0)}


@pytest.fixture(scope="module")
def M():
    from speculative_decoding_tree_bit_gb300 import model
    return model


def scaling(M, kind):
    a = KINDS[kind]
    return {"plain": lambda: None, "linear": lambda: M.RopeScaling.linear(a["factor"]),
            "bands": lambda: M.RopeScaling.bands(a["factor"], a["original"], low=a["low"], high=a["high"]),
            "ramp": lambda: M.RopeScaling.ramp(a["factor"], a["original"], fast=a["high"], slow=a["low"])}[kind]()


def rows(n, heads, d, seed):
    return torch.randn(n, heads, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def same(got, x, pos, freq, amplitude, interleaved):
    want, slack = ref.rotate(x.cpu().double(), pos.cpu(), freq, amplitude, interleaved)
    rot = 2 * len(freq)
    off = (got.cpu().double() - want).abs() - slack
    assert (off[..., :rot] <= ref.BF16 * (want.abs() + slack)[..., :rot]).all()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 32), (64, 64), (64, 16), (80, 20), (96, 96), (256, 64), (10, 6), (5, 2), (2, 2)])
def test_layouts_and_scalings(M, d, rot, kind, interleaved):
    base = 1e6 if d > 64 else 1e4
    op = M.Rope(d, rot, base, interleaved, scaling(M, kind))
    freq = ref.frequencies(rot, base, kind, **KINDS[kind])
    amp = 0.1 * np.log(4.0) + 1 if kind == "ramp" else 1.0
    q, k = rows(37, 4, d, 1), rows(37, 2, d, 2)
    pos = torch.randint(0, 1 << 20, (37,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    pos[:4] = torch.tensor([0, 1, -7, 2 ** 31 - 1])
    q2, k2 = op(q, k, pos)
    same(q2, q, pos, freq, amp, interleaved)
    same(k2, k, pos, freq, amp, interleaved)


@pytest.mark.parametrize("n,hq,hk", [(0, 4, 1), (1, 1, 1), (1, 32, 8), (16, 40, 8), (4099, 5, 1), (700, 128, 3)])
def test_sizes(M, n, hq, hk):
    op = M.Rope()
    freq = ref.frequencies(128, 1e6)
    q, k = rows(n, hq, 128, n), rows(n, hk, 128, n + 1)
    pos = torch.arange(n, dtype=torch.int32).cuda() + 2048
    q2, k2 = op(q, k, pos)
    same(q2, q, pos, freq, 1.0, False)
    same(k2, k, pos, freq, 1.0, False)
    q3, none = op(q, None, pos)
    assert none is None and torch.equal(q2, q3)


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (80, 20)])
def test_in_place_on_slices_of_one_projection(M, d, rot):
    """q and k as slices of [rows][heads + 2 kv heads][dim]; v and what lies between stays."""
    op = M.Rope(d, rot, 1e4)
    qkv = rows(50, 12, d, 4)
    before = qkv.clone()
    pos = torch.arange(50, dtype=torch.int32).cuda()
    q, k = qkv[:, :8], qkv[:, 8:10]
    want = op(q, k, pos)
    op(q, k, pos, q_out=q, k_out=k)
    assert torch.equal(qkv[:, :8], want[0]) and torch.equal(qkv[:, 8:10], want[1])
    assert torch.equal(qkv[:, 10:], before[:, 10:])


@pytest.mark.parametrize("kind", KINDS)
def test_the_last_positions(M, kind):
    """Against angles to 60 digits: 2^31 positions off by 2^-53 of a turn each, the turn cut at 2^-32 and as fp32 2^-26,
    sine and cosine 2^-22 and the products 2^-23 of themselves."""
    op = M.Rope(64, 64, 5e5, False, scaling(M, kind))
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 4097, 1 << 20]
    x = rows(4, 3, 64, 11)
    got = op(x, None, torch.tensor(pos, dtype=torch.int32).cuda())[0].cpu().double()
    amp = 0.1 * np.log(4.0) + 1 if kind == "ramp" else 1.0
    turns = ref.exact_turns(64, 5e5, kind, **KINDS[kind])
    angle = torch.tensor([[float(t * p % 1) for t in turns] for p in pos], dtype=torch.float64) * (2 * np.pi)
    c, s = (amp * torch.cos(angle))[:, None], (amp * torch.sin(angle))[:, None]
    x = x.cpu().double()
    a, b = x[..., :32], x[..., 32:]
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    slack = amp * (a.abs() + b.abs()).repeat(1, 1, 2) * (2 * np.pi * (2.0 ** -22 + 2.0 ** -32 + 2.0 ** -26) + 2.0 ** -22 + 2.0 ** -22)
    assert ((got - want).abs() <= ref.BF16 * (want.abs() + slack) + slack).all()


def test_unaligned_rows(M):
    """Addresses that 16-byte pieces do not fit."""
    op = M.Rope(64, 64, 1e4)
    flat = torch.randn(20 * 70 * 3 + 1, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    q = flat[1:].view(20, 210)[:, :64 * 3].unflatten(1, (3, 64))
    pos = torch.arange(20, dtype=torch.int32).cuda() * 1000
    same(op(q, None, pos)[0], q, pos, ref.frequencies(64, 1e4), 1.0, False)


def test_a_negative_position_turns_back_and_is_the_gradient(M):
    """<R x, y> = <x, R' y>: R' is the gradient; against differences, in 64 bits."""
    op = M.Rope(64, 32, 1e4, interleaved=True)
    x, y = rows(9, 3, 64, 6), rows(9, 3, 64, 7)
    pos = torch.randint(1, 5000, (9,), generator=torch.Generator().manual_seed(8), dtype=torch.int32).cuda()
    fx, by = op(x, None, pos)[0].double(), op(y, None, -pos)[0].double()
    left, right = (fx * y.double()).sum(-1), (x.double() * by).sum(-1)
    size = (x.double().norm(dim=-1) * y.double().norm(dim=-1))
    assert ((left - right).abs() <= 2 * ref.BF16 * 1.01 * size).all()
    freq = ref.frequencies(32, 1e4)
    f = lambda z: (ref.rotate(z, pos.cpu(), freq, 1.0, True)[0] * y.cpu().double()).sum()  # noqa: E731
    z, h = x.cpu().double(), 2.0 ** -10
    for at in ((0, 0, 0), (3, 1, 17), (8, 2, 31), (4, 0, 50)):
        e = torch.zeros_like(z)
        e[at] = h
        assert abs((f(z + e) - f(z - e)).item() / (2 * h) - by[at].item()) <= ref.BF16 * abs(by[at].item()) + 2.0 ** -17


def test_rows_past_32_bit_offsets(M):
    """2^31 elements and more, in place: the last rows as a call of their own turns them."""
    op, n = M.Rope(128), 430_000
    x = torch.randn(64, 40, 128, device="cuda").bfloat16().repeat(n // 64 + 1, 1, 1)[:n].contiguous()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    last = x[-100:].clone()
    want_q, want_k = op(last[:, :32], last[:, 32:], pos[-100:].clone())
    op(x[:, :32], x[:, 32:], pos, q_out=x[:, :32], k_out=x[:, 32:])
    assert torch.equal(x[-100:, :32], want_q) and torch.equal(x[-100:, 32:], want_k)


def test_graph_and_stream(M):
    op = M.Rope()
    q, k, pos = rows(33, 8, 128, 1), rows(33, 2, 128, 2), torch.arange(33, dtype=torch.int32).cuda()
    want = op(q, k, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = op(q, k, pos, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = op(q, k, pos)
    pos.add_(1000)
    graph.replay()
    want = op(q, k, pos)
    assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])


def test_as_the_models_own_rotation(M):
    """The half layout at base 1e6 is what the q/k/v product's epilogue applies."""
    op = M.Rope(128, 128, 1e6)
    x = rows(20, 2, 128, 9)
    pos = torch.arange(20, dtype=torch.int32).cuda() * 200
    i = np.arange(64)
    th = pos.cpu().numpy()[:, None] * 1e6 ** (-2.0 * i / 128)
    c, s = (torch.from_numpy(f(th).astype(np.float32)).double()[:, None] for f in (np.cos, np.sin))
    a, b = x.cpu().double()[..., :64], x.cpu().double()[..., 64:]
    want = torch.cat([a * c - b * s, b * c + a * s], -1)
    got = op(x, None, pos)[0].cpu().double()
    assert ((got - want).abs() <= ref.BF16 * want.abs() + 2.0 ** -18 * (a.abs() + b.abs()).repeat(1, 1, 2)).all()

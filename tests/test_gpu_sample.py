"""Sampled tokens against the definition in 64 bits, token by token."""
import math

import numpy as np
import pytest
import torch

import request_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from speculative_decoding_tree_bit_gb300 import model
    return model


def check(M, logits, u, **kw):
    """logits bf16 [rows][V] on the GPU; every row against the definition."""
    got = M.sample(logits, u, **kw)
    t, k, p, m = (kw.get("temperature", 1.0), kw.get("top_k", 0), kw.get("top_p", 1.0), kw.get("min_p", 0.0))
    at = lambda x, r: x[r].item() if isinstance(x, torch.Tensor) else torch.tensor(x, dtype=torch.float32).item()  # noqa: E731
    tokens, logprob, kept = (got[n].cpu() for n in ("tokens", "logprob", "kept"))
    rows = logits.cpu().double()
    for r in range(rows.shape[0]):
        want = ref.sample_row(rows[r], u[r].item(), at(t, r), int(at(k, r)), at(p, r), at(m, r))
        assert (tokens[r].item(), kept[r].item()) == (want[0], want[2]), (r, tokens[r], kept[r], want)
        if want[0] >= 0:
            # three fp32 steps and a logarithm of 1 + x, the weight in fp32
            assert abs(logprob[r].item() - want[1]) <= 2.0 ** -20 * (abs(want[1]) + min(1.0, abs(want[1]))) + 2.0 ** -43, (r, want)
        else:
            assert logprob[r].item() == -math.inf
    return got


def normal(rows, V, spread=2.5, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, V, generator=g)).bfloat16().cuda(), torch.rand(rows, generator=g).cuda()


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_p=0.9), dict(top_k=1), dict(top_k=40, temperature=1.3),
            dict(min_p=0.05), dict(top_k=100, top_p=0.8, min_p=0.01, temperature=0.9), dict(top_p=1e-6), dict(min_p=1.0),
            dict(temperature=1e-3), dict(temperature=50.0, top_p=0.99), dict(temperature=1e-40), dict(temperature=1e30)]


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 127, 1000, 4099, 65528, 65529, 151936])
def test_sizes(M, V):
    x, u = normal(5, V, seed=V)
    for kw in SETTINGS[:7]:
        check(M, x, u, **kw)


@pytest.mark.parametrize("kw", SETTINGS)
def test_settings(M, kw):
    x, u = normal(9, 3001, seed=3)
    check(M, x, u, **kw)
    # few distinct logits: ties at every cut
    check(M, (x * 0.6).round().bfloat16(), u, **kw)


@pytest.mark.parametrize("rows", [1, 3, 40, 160, 300])
def test_rows_and_clusters(M, rows):
    """One row takes up to eight CTAs, many rows one each."""
    x, u = normal(rows, 16000, seed=rows)
    check(M, x, u, top_k=50, top_p=0.95)
    check(M, x, u)


def test_settings_by_row(M):
    x, u = normal(24, 5000, seed=5)
    g = torch.Generator().manual_seed(6)
    t = torch.tensor([0.0, 0.5, 1.0, 2.0]).repeat(6).cuda()
    k = torch.randint(0, 60, (24,), generator=g, dtype=torch.int32).cuda()
    p = (1 - 0.6 * torch.rand(24, generator=g)).cuda()
    m = (0.1 * torch.rand(24, generator=g)).cuda()
    check(M, x, u, temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("rows", [6, 200])
def test_an_infinite_temperature_of_a_row(M, rows):
    """Every token weighs 1, beside rows of other temperatures."""
    x, u = normal(rows, 3000, seed=41)
    t = torch.tensor([math.inf, 1.0, math.inf, 50.0]).repeat(rows // 4 + 1)[:rows].cuda()
    for kw in (dict(), dict(min_p=0.5), dict(min_p=1.0), dict(top_k=7, min_p=0.1), dict(top_p=0.5)):
        check(M, x, u, temperature=t, **kw)


@pytest.mark.parametrize("rows", [3, 200])
def test_min_p_of_any_size(M, rows):
    """Down to the least fp32 number, beside weights as small, and beside an infinity, where the others weigh 0."""
    x, u = normal(rows, 1000, seed=43)
    x[:, 0] = 100.0
    x[:, 1:20] = torch.linspace(0.0, 30.0, 19).bfloat16().cuda()
    x[1, 5] = math.inf
    for p in (2.0 ** -119, 1e-37, 1e-40, 1e-45):
        check(M, x, u, min_p=p)


def test_logits_further_apart_than_fp32(M):
    x, u = normal(4, 500, seed=44)
    big = torch.finfo(torch.bfloat16).max
    x[0, 3], x[0, 4] = big, -big
    x[1], x[1, 9] = -big, big
    x[2, 3], x[2, 4] = big / 2, -big
    rows = x.cpu().double()
    for t in (3e37, 1e38, 2.9e38):
        for kw in (dict(), dict(top_p=0.5), dict(min_p=0.2)):
            got = M.sample(x, u, temperature=t, **kw)
            f = lambda v: torch.tensor(v, dtype=torch.float32).item()  # noqa: E731
            for r in range(4):
                token, logprob, kept = ref.sample_row(rows[r], u[r].item(), f(t), 0, f(kw.get("top_p", 1.0)), f(kw.get("min_p", 0.0)))
                assert (got["tokens"][r].item(), got["kept"][r].item()) == (token, kept), (t, kw, r)
                # as check, and 500 weights each rounded to a multiple of 2^-44 (row 1: weights of 2^-32 beside one of 1),
                # of which the logarithm of 1 + x takes no more than x
                off = abs(got["logprob"][r].item() - logprob)
                assert off <= 2.0 ** -20 * (abs(logprob) + min(1.0, abs(logprob))) + 2.0 ** -43 + 500 * 2.0 ** -45, (t, kw, r)


def test_a_top_k_past_32_bits_keeps_everything(M):
    x, u = normal(3, 500, seed=45)
    got, want = M.sample(x, u, top_k=2 ** 32 + 5), M.sample(x, u)
    assert torch.equal(got["kept"], want["kept"]) and torch.equal(got["tokens"], want["tokens"])
    with pytest.raises(Exception, match="top_k"):
        M.sample(x, u, top_k=-2 ** 32 + 3)


@pytest.mark.parametrize("rows", [4, 160])
def test_settings_of_a_row_past_their_range(M, rows):
    """Numbers that are refused for all rows are taken as the header says where rows have their own."""
    x, u = normal(rows, 700, seed=46)
    pair = lambda a, b, dtype=torch.float32: torch.tensor([a, b], dtype=dtype).repeat(rows // 2).cuda()  # noqa: E731
    for name, a, b, as_a, as_b in (("temperature", -1.0, math.nan, 0.0, 0.0), ("top_p", 0.0, -2.0, 1e-6, 1e-6), ("top_p", math.nan, 3.0, 1.0, 1.0),
                                   ("min_p", 7.0, -1.0, 1.0, 0.0), ("min_p", math.nan, 0.5, 0.0, 0.5)):
        got, want = M.sample(x, u, **{name: pair(a, b)}), check(M, x, u, **{name: pair(as_a, as_b)})
        for k in want:
            assert torch.equal(got[k], want[k]), (name, a, b, k)
    got, want = M.sample(x, u, top_k=pair(-5, 9, torch.int32)), check(M, x, u, top_k=pair(0, 9, torch.int32))
    for k in want:
        assert torch.equal(got[k], want[k])


def test_ties_take_the_lowest_index(M):
    x = torch.zeros(4, 70000).bfloat16().cuda()
    u = torch.tensor([0.0, 0.25, 0.5, 1 - 2.0 ** -24]).cuda()
    check(M, x, u)
    check(M, x, u, top_k=3)
    check(M, x, u, temperature=0.0)
    x[1, ::2] = -0.0  # equal to 0
    check(M, x, u, top_k=5)


def test_masked_rows_and_special_values(M):
    x, u = normal(8, 2000, seed=8)
    x[0] = -math.inf                       # nothing left
    x[1] = math.nan
    x[2, 5:] = -math.inf
    x[3, ::2] = math.nan
    x[4, 77] = x[4, 1500] = math.inf       # everything else weighs 0
    x[5] = torch.finfo(torch.bfloat16).min  # a mask of the lowest value
    x[5, 900] = 0.0
    x[6] = torch.finfo(torch.bfloat16).min
    x[7, 0], x[7, 1] = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).min
    for kw in SETTINGS:
        check(M, x, u, **kw)


def test_tiny_magnitudes_keep_their_order(M):
    """Logits of all binades, subnormal ones too: ordered by value."""
    g = torch.Generator().manual_seed(11)
    bits = torch.randint(-32768, 32768, (6, 4000), generator=g, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.bfloat16).clone()
    x = torch.where(x.abs() < 4, x, torch.zeros_like(x)).cuda()
    u = torch.rand(6, generator=g).cuda()
    check(M, x, u)
    check(M, x, u, top_k=1500)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=7, temperature=0.8), dict(top_p=0.7, min_p=0.01), dict(temperature=0.0)])
def test_many_rows_with_special_values(M, kw):
    """Many rows, some with magnitudes past 2^15 or below 2^-24, infinities, masks of every kind, nothing left."""
    x, u = normal(220, 1501, seed=14)
    x[3] = -math.inf
    x[10, 5] = 1e30
    x[11, 5], x[11, 700] = -1e30, 1e-30
    x[40] = torch.finfo(torch.bfloat16).min
    x[41, 9] = math.inf
    x[42, :1500] = -math.inf
    x[43, ::3] = math.nan
    x[44] = 0.0
    x[45] = (x[45].float() * 1e-9).bfloat16()
    x[46] = torch.finfo(torch.bfloat16).min
    x[46, 1500] = 3.0
    x[219] = math.nan
    check(M, x, u, **kw)


def test_long_rows_one_cta_each(M):
    x, u = normal(160, 40000, seed=15)
    check(M, x[:, 3:], u, temperature=1.2)
    x = torch.zeros(153, 140000).bfloat16().cuda()  # one key, more than 16 bits of it
    u = torch.rand(153, generator=torch.Generator().manual_seed(3)).cuda()
    got = M.sample(x, u)
    want = torch.floor(u.double() * 140000).to(torch.int32)
    assert torch.equal(got["tokens"], want) and (got["kept"] == 140000).all()


@pytest.mark.parametrize("special", [False, True])
def test_rows_past_32_bit_offsets(M, special):
    """2^31 elements and more: the last rows as a call of their own samples them."""
    V, n = 151936, 14200
    row, u = normal(40, V, seed=31)
    if special:  # magnitudes that the kernel of many rows leaves to the other one
        row[7::13, 5] = 1e30
    x = row.repeat(n // 40, 1)
    us = u.repeat(n // 40)
    got, want = M.sample(x, us, temperature=0.9, top_p=0.95), M.sample(row, u, temperature=0.9, top_p=0.95)
    for k in want:
        assert torch.equal(got[k].reshape(-1, 40), want[k].expand(n // 40, 40)), k


def test_u_is_clamped(M):
    x, _ = normal(5, 300, seed=2)
    u = torch.tensor([-1.0, math.nan, 1.0, 7.0, math.inf]).cuda()
    got = M.sample(x, u)["tokens"]
    want = M.sample(x, torch.tensor([0.0, 0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24]).cuda())["tokens"]
    assert torch.equal(got, want)


def test_strided_rows_anywhere(M):
    """Rows that begin at any 2-byte address, and what lies beside them is not read into them."""
    g = torch.Generator().manual_seed(4)
    wide = (3 * torch.randn(6, 1237, generator=g)).bfloat16().cuda()
    u = torch.rand(6, generator=g).cuda()
    for off in range(9):
        x = wide.clone()
        x[:, :off], x[:, off + 1009:] = math.inf, math.inf
        check(M, x[:, off:off + 1009], u, top_k=30)
        bits = x.view(torch.int16)[:, off:off + 1009]
        assert torch.equal(M.sample(bits, u, top_k=30)["tokens"], M.sample(x[:, off:off + 1009], u, top_k=30)["tokens"])


def test_frequencies_match_the_weights(M):
    """Many u over one row: every token as often as its weight says (u on a grid: to one of the grid's steps)."""
    x, _ = normal(1, 50, seed=9)
    n = 20000
    u = ((torch.arange(n) + 0.5) / n).cuda()
    got = torch.bincount(M.sample(x.expand(n, 50).contiguous(), u)["tokens"].cpu().long(), minlength=50)
    want = torch.softmax(x[0].cpu().double(), 0) * n
    assert (got - want).abs().max() <= 1.0 + 1e-6


def test_replay_and_streams(M):
    x, u = normal(4, 30000, seed=1)
    want = M.sample(x, u, top_p=0.9)["tokens"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = M.sample(x, u, top_p=0.9, stream=s)["tokens"]
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = M.sample(x, u, top_p=0.9)
    for seed in (21, 22):
        y, w = normal(4, 30000, seed=seed)
        x.copy_(y), u.copy_(w)
        graph.replay()
        assert torch.equal(held["tokens"], M.sample(x, u, top_p=0.9)["tokens"])


def test_sampled_tokens_walk_a_tree(M):
    """In the argmax's place of sd_accept: the walk accepts what sampling token by token gives."""
    import ctypes  # noqa: F401

    from speculative_decoding_tree_bit_gb300 import check as ck, lib, stream_ptr
    g = torch.Generator().manual_seed(12)
    V, m = 40, 16
    parents = [-1] + [int(torch.randint(max(0, i - 4), i, (1,), generator=g)) for i in range(1, m)]
    logits, u = normal(m, V, spread=1.0, seed=13)
    drawn = M.sample(logits, u, temperature=0.5)["tokens"]
    # half of the drafts are what their parent's row gave
    tokens = torch.randint(0, V, (m,), generator=g, dtype=torch.int32)
    for i in range(1, m, 2):
        tokens[i] = drawn[parents[i]].item()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    tok, par = tokens.cuda(), torch.tensor(parents, dtype=torch.int32).cuda()
    length, path_tokens, bonus, path, status = i32(1), i32(m), i32(1), i32(m + 1), i32(1)
    ck(lib().sd_accept(tok.data_ptr(), par.data_ptr(), drawn.data_ptr(), m, length.data_ptr(), path_tokens.data_ptr(),
                       bonus.data_ptr(), path.data_ptr(), status.data_ptr(), stream_ptr()))
    ok, depth = [True] + [False] * (m - 1), [0] * m
    for i in range(1, m):
        depth[i] = depth[parents[i]] + 1
        ok[i] = ok[parents[i]] and tokens[i].item() == drawn[parents[i]].item()
    best = max((i for i in range(m) if ok[i]), key=lambda i: (depth[i], -i))
    assert status.item() == 0 and length.item() == depth[best] and bonus.item() == drawn[best].item()


def test_no_rows(M):
    out = M.sample(torch.zeros(0, 100).bfloat16().cuda(), torch.zeros(0).cuda())
    assert out["tokens"].numel() == 0

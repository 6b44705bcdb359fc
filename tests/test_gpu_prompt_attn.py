"""Attention over packed prompts against the definition in 64 bits."""
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


def inputs(m, keys, hq, hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    n, s = sum(m), sum(keys)
    q = (1.5 * torch.randn(n, hq, d, generator=g)).bfloat16().cuda()
    k = (torch.randn(s, hkv, d, generator=g) * (0.5 + torch.rand(hkv, d, generator=g)) + 0.5 * torch.randn(hkv, d, generator=g)).bfloat16().cuda()
    v = torch.randn(s, hkv, d, generator=g).bfloat16().cuda()
    return q, k, v


def run(M, m, keys, q, k, v, score=None, stream=None, **kw):
    op = M.PromptAttention(q.shape[1], k.shape[1], q.shape[2])
    rows = M.RequestRows(np.cumsum([0] + list(m)))
    held = M.RequestRows(np.cumsum([0] + list(keys)))
    out, lse = op(q, k, v, rows, held, score=score, stream=stream, **kw)
    torch.cuda.synchronize()
    assert op.status() == 0
    return out, lse


def same(out, lse, m, keys, q, k, v, **kw):
    f = lambda t: t.cpu().double()  # noqa: E731
    want, want_lse, tol, tol_lse = ref.attend(f(q), f(k), f(v), np.cumsum([0] + list(m)), np.cumsum([0] + list(keys)), **kw)
    out, lse = f(out), f(lse)
    assert torch.equal(torch.isinf(lse), torch.isinf(want_lse))
    some = ~torch.isinf(want_lse)
    assert ((lse - want_lse).abs()[some] <= tol_lse[some]).all(), (lse - want_lse).abs()[some].max()
    bad = (out - want).abs() > tol
    assert not bad.any(), (bad.nonzero()[:5], (out - want).abs()[bad].max(), int(bad.sum()))


def check(M, m, keys, hq, hkv, d, seed=0, cap=0.0, slopes=None, window=0, scale=0.0):
    q, k, v = inputs(m, keys, hq, hkv, d, seed)
    sl = None if slopes is None else slopes.cuda()
    out, lse = run(M, m, keys, q, k, v, M.KV4Score(scale=scale, softcap=cap, slopes=sl, window=window))
    same(out, lse, m, keys, q, k, v, cap=cap, slopes=slopes, window=window, scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700])
def test_one_prompt(M, n, d):
    check(M, [n], [n], 8, 2, d, seed=n)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (5, 1), (8, 1), (7, 7), (10, 2), (32, 8), (16, 1), (33, 1), (64, 1), (65, 1),
                                    (100, 1), (128, 1)])
def test_head_groups(M, hq, hkv):
    check(M, [70, 3], [70, 3], hq, hkv, 128, seed=hq)
    check(M, [70, 3], [200, 140], hq, hkv, 64, seed=hq + 1)


@pytest.mark.parametrize("d", [64, 128])
def test_packed_ragged(M, d):
    """Requests without rows, without keys, of one token; rows before the keys see nothing."""
    m = [5, 0, 1, 130, 0, 64, 300, 7, 3]
    keys = [5, 40, 1, 130, 0, 200, 300, 3, 0]
    check(M, m, keys, 8, 2, d, seed=1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("m,past", [(1, 1), (1, 127), (1, 128), (1, 5000), (17, 1000), (64, 2049), (200, 3000)])
def test_next_chunk(M, m, past, d):
    check(M, [m], [m + past], 8, 2, d, seed=m)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 500, 100000])
@pytest.mark.parametrize("d", [64, 128])
def test_window(M, window, d):
    check(M, [300, 20, 1], [300, 700, 900], 4, 2, d, seed=window, window=window)


def test_options(M):
    slopes = torch.exp2(-torch.arange(1, 9).float())
    for d in (64, 128):
        check(M, [150, 9], [150, 400], 8, 4, d, cap=20.0)
        check(M, [150, 9], [150, 400], 8, 4, d, slopes=slopes)
        check(M, [150, 9], [150, 400], 8, 4, d, cap=50.0, slopes=slopes, window=70)
        check(M, [150, 9], [150, 400], 8, 4, d, scale=0.3)


@pytest.mark.parametrize("d", [64, 128])
def test_many_requests_of_few_rows(M, d):
    rng = np.random.default_rng(3)
    m = rng.integers(0, 6, 200).tolist()
    keys = [int(x + rng.integers(0, 300)) for x in m]
    check(M, m, keys, 4, 1, d, seed=2)


@pytest.mark.parametrize("d", [64, 128])
def test_single_rows_over_one_and_few_steps_of_keys(M, d):
    """Units of one step of 128 keys and of two or three behind one another in a CTA: only one of the
    two groups of rows has a use for the first one's values, and both for the next one's."""
    keys = [(1 + 37 * i % 128, 129 + 91 * i % 256, 1 + 53 * i % 128, 257 + 29 * i % 128, 513 + i % 7)[i % 5] for i in range(900)]
    check(M, [1] * 900, keys, 2, 1, d, seed=21)
    # between prompts, whose units hold two tiles
    m = [1, 1, 300, 1, 1, 1, 129] * 40
    keys = [m[i] + (0, 200, 0, 100, 380, 17, 260)[i % 7] for i in range(280)]
    check(M, m, keys, 2, 1, d, seed=22)


def test_long_contexts(M):
    """Work split over the keys and joined; far offsets."""
    check(M, [2, 1], [20011, 9000], 4, 1, 128, seed=4)
    check(M, [40], [20000], 5, 1, 64, seed=5)


def test_keys_past_32_bit_offsets(M):
    """K and V of 2^31 elements and more: one token's greatest key near the end, the rest as one value."""
    n, hkv, d = 2_200_000, 8, 128
    k = torch.zeros(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    k[n - 5], v[n - 5] = 4.0, -3.0  # score 4 sqrt(d): weight e^45 for 1
    k[3], v[3] = 4.0, 5.0
    q = torch.ones(1, 16, d).bfloat16().cuda()
    out, lse = run(M, [1], [n], q, k, v)
    x = 4 * math.sqrt(d)
    # two equal weights of 1 - 2^-40: (5 - 3) / 2
    assert (out.double() - 1.0).abs().max() <= ref.BF16
    assert (lse.double() - (x + math.log(2.0))).abs().max() <= 2.0 ** -18 * x
    window = M.KV4Score(window=1000)
    out, lse = run(M, [1], [n], q, k, v, window)
    assert (out.double() + 3.0).abs().max() <= 3 * ref.BF16


def test_large_and_small_scores(M):
    """Softmax statistics over a wide range: a maximum that keeps growing, and one key that takes all."""
    m = keys = [400]
    q, k, v = inputs(m, keys, 4, 2, 128, 6)
    k = (k.float() * torch.linspace(0.01, 6.0, 400, device="cuda")[:, None, None]).bfloat16()
    out, lse = run(M, m, keys, q, k, v)
    same(out, lse, m, keys, q, k, v)
    k = k.flip(0).contiguous()
    out, lse = run(M, m, keys, q, k, v)
    same(out, lse, m, keys, q, k, v)
    out, lse = run(M, m, keys, (q.float() * 1e-30).bfloat16(), k, v)
    same(out, lse, m, keys, (q.float() * 1e-30).bfloat16(), k, v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [(3,), (63,), (64,), (127,), (128, 200), (10, 70, 140, 260, 330), (399,)])
def test_scores_that_leap(M, at, d):
    """A key whose score passes all before it by hundreds, in either half of a step of 128 keys."""
    m, keys = [400, 30], [400, 300]
    q, k, v = inputs(m, keys, 4, 2, d, 8)
    q = (q.abs() + 0.5).bfloat16()
    size = 40.0
    for j in at:
        for first in (0, 400):
            if j < (400 if first == 0 else 300):
                k[first + j] = size
        size *= 1.5
    out, lse = run(M, m, keys, q, k, v)
    same(out, lse, m, keys, q, k, v)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [10, 18, 26, 55])
def test_scores_whose_last_place_passes_an_exponent(M, power, d):
    """Scores of 2^25 to 2^116: the last place of one is more than an exponent holds.  All
    keys but one have one score: rows before it average what they see, the others take it,
    and every weight is 0 or 1."""
    m, keys = [300, 40], [300, 400]
    _, _, v = inputs(m, keys, 4, 2, d, 9)
    q = torch.full((340, 4, d), 3.0 * 2.0 ** power).bfloat16().cuda()
    k = torch.full((700, 2, d), -1.5 * 2.0 ** power).bfloat16().cuda()
    for j in (70, 300 + 377):
        k[j] = 2.0 ** power
    out, lse = run(M, m, keys, q, k, v)
    f = lambda t: t.cpu().double()  # noqa: E731
    want, want_lse, _, _ = ref.attend(f(q), f(k), f(v), np.cumsum([0] + m), np.cumsum([0] + keys))
    assert torch.isfinite(out).all()
    # the output in bf16, a sum of at most 400 values in fp32
    assert ((f(out) - want).abs() <= ref.BF16 * want.abs() + 400 * 2.0 ** -24 * f(v).abs().max()).all()
    assert ((f(lse) - want_lse).abs() <= 2.0 ** -20 * want_lse.abs()).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e30, 1e34, 1e36, 1e38])
@pytest.mark.parametrize("m,n", [(1, 128), (300, 300), (40, 1000), (3, 40000)])
def test_finite_values_give_finite_outputs(M, d, size, m, n):
    """Values of one sign and of both near the type's end, under equal weights and under keys of a later
    half step that weigh 2^7, 2^18.8 and 2^20 times the first ones."""
    g = torch.Generator().manual_seed(n)
    q = torch.ones(m, 2, d).bfloat16().cuda()
    values = ((0.5 + 0.5 * torch.rand(n, 1, d, generator=g)) * size).bfloat16()
    signs = torch.sign(torch.randn(n, 1, d, generator=g)).bfloat16()
    for at in (0.0, 5.0, 13.0, 14.0):
        k = torch.zeros(n, 1, d).bfloat16()
        k[100::128] = at / math.sqrt(d)
        for v in (values, values * signs):
            out, lse = run(M, [m], [n], q, k.cuda(), v.cuda())
            same(out, lse, [m], [n], q, k, v)
    slopes, score = torch.tensor([0.5, -0.01]), dict(cap=20.0, window=600)
    out, lse = run(M, [m], [n], q, k.cuda(), v.cuda(), M.KV4Score(softcap=20.0, slopes=slopes.cuda(), window=600))
    same(out, lse, [m], [n], q, k, v, slopes=slopes, **score)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1e-30, 1e-34, 1e-36])
@pytest.mark.parametrize("m,n", [(1, 128), (300, 300), (3, 40000)])
def test_small_values_keep_their_bits(M, d, size, m, n):
    """An output relative to its own size, all values positive: both roundings (2^-8) and the fp32 steps
    (request_ref), and of the sums, held in multiples of 2^-149, eight a half step's product: a row's weights
    come to 2^-15 at least."""
    q, k, _ = inputs([m], [n], 2, 1, d, 3)
    v = ((0.5 + 0.5 * torch.rand(n, 1, d, generator=torch.Generator().manual_seed(n))) * size).bfloat16().cuda()
    out, lse = run(M, [m], [n], q, k, v)
    f = lambda t: t.cpu().double()  # noqa: E731
    want, _, tol, _ = ref.attend(f(q), f(k), f(v), [0, m], [0, n])
    lost = 2.0 ** -149 * 8 * (n // 64 + 2) * 2.0 ** 15
    assert ((f(out) - want).abs() <= tol - 2.0 ** -130 + lost).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slope", [1e10, 1e25])
def test_slopes_that_leave_the_nearest_key(M, slope, d):
    m, keys = [150, 3], [150, 300]
    q, k, v = inputs(m, keys, 4, 2, d, 10)
    slopes = torch.full((4,), slope)
    out, lse = run(M, m, keys, q, k, v, M.KV4Score(slopes=slopes.cuda()))
    own = torch.cat([v[:150], v[150 + 297:]]).repeat_interleave(2, 1)
    assert torch.equal(out, own)
    assert (lse.abs().cpu() <= 300 * slope * 2.0 ** -21 + 1e3).all()  # far keys' distance is taken off again


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,slope", [(1e-14, 1e25), (1e-39, 0.25), (1e-30, 1e9), (1e-3, 0.5), (100.0, 1e36), (1e-39, 1e36), (1e-39, 0.0)])
def test_slopes_beside_any_scale(M, scale, slope, d):
    """Scale and slope a range apart that fp32 does not hold."""
    m, keys = [150, 3], [150, 300]
    q, k, v = inputs(m, keys, 4, 2, d, 10)
    slopes = torch.full((4,), slope)
    out, lse = run(M, m, keys, q, k, v, M.KV4Score(scale=scale, slopes=slopes.cuda()))
    if slope < 1e20:
        same(out, lse, m, keys, q, k, v, scale=scale, slopes=slopes)
    else:  # the nearest key alone
        assert torch.equal(out, torch.cat([v[:150], v[150 + 297:]]).repeat_interleave(2, 1)) and torch.isfinite(lse).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_only_reach_the_rows_that_see_them(M, bad, d):
    """In a key or a value: earlier rows, other requests and other kv heads stay as they were."""
    m, keys = [200, 150, 30], [200, 150, 400]
    q, k, v = inputs(m, keys, 4, 2, d, 7)
    clean, clean_lse = run(M, m, keys, q, k, v)
    for key, of in ((60, "v"), (199, "v"), (200 + 149, "v"), (130, "k"), (350 + 399, "v"), (350 + 398, "k"), (350, "v")):
        k2, v2 = k.clone(), v.clone()
        (k2 if of == "k" else v2)[key, 1, 5] = bad
        out, lse = run(M, m, keys, q, k2, v2)
        r = 0 if key < 200 else 1 if key < 350 else 2
        at, first = key - [0, 200, 350][r], [0, 200, 350][r]
        row0 = first + max(0, at - (keys[r] - m[r]))  # the first row that sees it
        end = first + m[r]
        hit = torch.zeros(sum(m), 4, dtype=torch.bool, device="cuda")
        hit[row0:end, 2:] = True
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit]), (key, of)
        if of == "v":
            assert (~torch.isfinite(out[hit][:, 5].float())).all(), (key, of)
            rest = [i for i in range(d) if i != 5]
            assert torch.equal(out[hit][:, rest], clean[hit][:, rest]) and torch.equal(lse[hit], clean_lse[hit])


def test_nothing_beyond_the_last_row_is_written(M):
    q, k, v = inputs([70], [70], 4, 2, 128)
    big, big_lse = torch.full((75, 4, 128), 7.0).bfloat16().cuda(), torch.full((75, 4), 7.0).cuda()
    out, lse = run(M, [70], [70], q, k, v, out=big[:70], lse=big_lse[:70])
    assert (big[70:] == 7).all() and (big_lse[70:] == 7).all()
    same(out, lse, [70], [70], q, k, v)


def test_strided_rows(M):
    """q, k and v as slices of one projection's output; bits in int16."""
    qkv = torch.randn(190, 8 + 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    out, lse = run(M, [100, 90], [100, 90], q, k, v)
    same(out, lse, [100, 90], [100, 90], q, k, v)
    b = qkv.view(torch.int16)
    out2, _ = run(M, [100, 90], [100, 90], b[:, :8], b[:, 8:10], b[:, 10:])
    assert out2.dtype is torch.int16 and torch.equal(out2.view(torch.bfloat16), out)


def test_same_bits_every_time_and_on_streams_and_graphs(M):
    m, keys = [3, 500, 40], [4000, 500, 40]
    q, k, v = inputs(m, keys, 8, 2, 128, 9)
    want, want_lse = run(M, m, keys, q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        out, lse = run(M, m, keys, q, k, v, stream=stream)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    op = M.PromptAttention(8, 2, 128)
    rows, held = M.RequestRows(np.cumsum([0] + m)), M.RequestRows(np.cumsum([0] + keys))
    op(q, k, v, rows, held)
    graphs = []
    for _ in range(2):  # two graphs and eager calls between their replays
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, *op(q, k, v, rows, held)))
    q.copy_(q.flip(0))
    want, want_lse = op(q, k, v, rows, held)
    with torch.cuda.stream(s):
        graphs[0][0].replay()
    graphs[1][0].replay()
    again, _ = op(q, k, v, rows, held)
    torch.cuda.synchronize()
    for _, out, lse in graphs:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.equal(again, want)


@pytest.mark.parametrize("loads", [0, 1, 2, 5])
@pytest.mark.parametrize("m,keys,d,window", [([900], [900], 128, 0), ([700, 30], [900, 2000], 64, 130), ([1, 1, 2], [3000, 700, 5000], 128, 0),
                                             ([40] * 30, [700] * 30, 128, 0)])
def test_a_wait_that_runs_out_ends_the_call(M, loads, m, keys, d, window):
    """Values that do not come (after `loads` steps of a CTA's): every wait for what they would bring gives up after
    20 ms, the call ends with its status and writes nothing past its rows, and the next one is right."""
    import time

    from speculative_decoding_tree_bit_gb300 import check as ck, lib
    q, k, v = inputs(m, keys, 4, 2, d, 12)
    n = sum(m)
    big, big_lse = torch.full((n + 9, 4, d), 7.0).bfloat16().cuda(), torch.full((n + 9, 4), 7.0).cuda()
    op = M.PromptAttention(4, 2, d)
    rows, held = M.RequestRows(np.cumsum([0] + m)), M.RequestRows(np.cumsum([0] + keys))
    score = M.KV4Score(window=window)
    torch.cuda.synchronize()
    try:
        ck(lib().sd_debug_prompt_wait(20_000_000, loads))
        t0 = time.perf_counter()
        op(q, k, v, rows, held, score=score, out=big[:n], lse=big_lse[:n])
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        ck(lib().sd_debug_prompt_wait(0, 0))
    done = op.status()
    assert done == 6 if loads == 0 else done in (0, 6)  # a CTA with no more steps than that ends as ever
    assert dt < 1.5 and (done == 0 or dt >= 0.018)
    assert (big[n:] == 7).all() and (big_lse[n:] == 7).all()
    out, lse = run(M, m, keys, q, k, v, score)
    same(out, lse, m, keys, q, k, v, window=window)


@pytest.mark.parametrize("m,keys,d,window", [([900] * 20, [900] * 20, 128, 0), ([700, 30] * 30, [900, 2000] * 30, 64, 130),
                                             ([1, 1, 2] * 50, [3000, 100, 300] * 50, 128, 0)])
def test_waits_of_a_microsecond(M, m, keys, d, window):
    """A limit that any wait may pass: a call ends early with its status or is right, and writes nothing past its rows."""
    from speculative_decoding_tree_bit_gb300 import check as ck, lib
    q, k, v = inputs(m, keys, 4, 2, d, 13)
    n = sum(m)
    op = M.PromptAttention(4, 2, d)
    rows, held = M.RequestRows(np.cumsum([0] + m)), M.RequestRows(np.cumsum([0] + keys))
    score = M.KV4Score(window=window)
    want, want_lse = op(q, k, v, rows, held, score=score)
    assert op.status() == 0
    for limit in (1, 1000, 3000, 10000) * 3:
        big, big_lse = torch.full((n + 9, 4, d), 7.0).bfloat16().cuda(), torch.full((n + 9, 4), 7.0).cuda()
        torch.cuda.synchronize()
        try:
            ck(lib().sd_debug_prompt_wait(limit, 2 ** 31))
            op(q, k, v, rows, held, score=score, out=big[:n], lse=big_lse[:n])
            torch.cuda.synchronize()
        finally:
            ck(lib().sd_debug_prompt_wait(0, 0))
        done = op.status()
        assert done in (0, 6) and (big[n:] == 7).all() and (big_lse[n:] == 7).all()
        if done == 0:
            assert torch.equal(big[:n], want) and torch.equal(big_lse[:n], want_lse)
    out, lse = op(q, k, v, rows, held, score=score)
    assert op.status() == 0 and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_no_rows(M):
    q, k, v = inputs([0, 0], [5, 0], 4, 2, 64)
    out, lse = run(M, [0, 0], [5, 0], q, k, v)
    assert out.numel() == 0 and lse.numel() == 0

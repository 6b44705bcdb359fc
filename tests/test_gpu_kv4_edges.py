"""The 4-bit cache on the GPU where it can go wrong: positions that do not lie
behind the cache, rows that are NaN, values of very different sizes, calls
without rows, streams and graphs.  Against the 64-bit definition.

Tolerances, from the number formats.  With p the softmax weights and R_k the
greatest magnitude of the held value row k, an output is off by at most
  2^-8 |out|              its rounding to bf16,
  3 2^-12 sum(p R)        the roundings of a weight, of a value and of m - 8 s to
                          fp16's 11 bits (the last two on the tensor cores alone),
  2 e sum(p R)            a score off by e, as a factor of each weight,
  n 2^-24 sum(p R)        weights below fp16's normal range, n keys.
e: the dot product's D + 16 roundings to fp32 of its terms' sizes, 2^-20 for the
exponential, (1 + cap / 8) times that with a cap, and 2^-23 of the slope's term."""
import math

import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    from speculative_decoding_tree_bit_gb300 import model
    return model


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def dev(x):
    return x.to(torch.bfloat16).cuda()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def make(M, K, V, pos, room=0, page=32, extra=2):
    """A cache whose request r holds the rows K[r], V[r] ([ctx][hkv][D]) at positions pos[r]."""
    R, hkv, D = len(K), K[0].shape[1], K[0].shape[2]
    pages = max(1, -(-(max(k.shape[0] for k in K) + room) // page))
    n = R * pages + extra
    table = np.random.default_rng(R + n).permutation(n)[:R * pages].reshape(R, pages)
    c = M.KV4Cache(table, n, hkv, D, page)
    c.blocks.fill_(0xFF)
    rows = M.RequestRows(np.cumsum([0] + [k.shape[0] for k in K]))
    if rows.n:
        c.append(dev(torch.cat(K)), dev(torch.cat(V)), rows, pos=i32(torch.cat(pos)))
    assert c.status() == 0
    return c


def expect(q, K, V, q_pos, k_pos, sees, cap=0.0, slope=0.0, window=0, start=None):
    """One query head in 64 bits: (out, lse, scores, weights, tolerance of out, e)."""
    D = q.shape[1]
    z, size = ref.scores(q, K, q_pos, k_pos, 1 / math.sqrt(D), cap, slope, window, start)
    z = z.masked_fill(~sees, -math.inf)
    p, lse = ref.softmax(z)
    far = float((q_pos[:, None] - k_pos[None]).abs().max()) * abs(slope) if K.shape[0] and q.shape[0] else 0.0
    e = (D + 16) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + cap / 8) + 2.0 ** -23 * far
    out = p @ V
    big = V.abs().amax(-1) if V.shape[0] else V.new_zeros(0)
    tol = H * out.abs() + ((3 * 2.0 ** -12 + 2 * e + V.shape[0] * 2.0 ** -24) * (p @ big))[:, None]
    return out, lse, z, p, tol, e


def compare(got, got_lse, want, lse, tol, e, what=()):
    none = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, none), what
    err = (got - want).abs()
    assert (err <= tol).all(), (*what, float((err / tol.clamp(min=1e-300)).max()))
    err = (got_lse - lse)[~none].abs()
    assert (err <= e + 2.0 ** -22 * lse[~none].abs() + 2.0 ** -18).all(), (*what, float(err.max()))


# -------------------------------- rows that do not stand behind the cache --

def attend_and_observe(M, c, K, V, pos, rows_of, q, G, q_pos, score_kw, own=None, posd=True):
    """attend and observe of every request against the definition; q_pos: per request."""
    rows = M.RequestRows(np.cumsum([0] + rows_of))
    start = score_kw.get("start")
    score = M.KV4Score(window=score_kw.get("window", 0), start=i32(start) if start is not None else None)
    pd = i32([p for r in q_pos for p in r]) if posd else None
    out, lse = c.attend(dev(q), rows, pos=pd, score=score)
    w0 = torch.rand(c.weight.shape, generator=torch.Generator().manual_seed(7))
    c.weight.copy_(w0)
    w = c.observe(dev(q), lse, rows, pos=pd, score=score, decay=0.5, out=torch.full_like(c.weight, -3.0))
    assert c.status() == 0
    out, lse, w = out.double().cpu(), lse.double().cpu(), w.double().cpu()
    for r in range(len(K)):
        a, b = int(rows.cu[r]), int(rows.cu[r + 1])
        qp = torch.tensor(q_pos[r], dtype=torch.int64)
        hkv = K[r].shape[1]
        want_w = 0.5 * w0[r, :, :K[r].shape[0]].double()
        e_max = 0.0
        for h in range(hkv * G):
            held = ref.values(K[r][:, h // G]), ref.values(V[r][:, h // G])
            kp = pos[r] if pos[r].dim() == 1 else pos[r][h // G]
            sees = torch.ones(b - a, kp.numel(), dtype=torch.bool)
            want, l, z, p, tol, e = expect(q[a:b, h], *held, qp, kp, sees, window=score_kw.get("window", 0),
                                           start=start[r] if start is not None else None)
            compare(out[a:b, h], lse[a:b, h], want, l, tol, e, (r, h))
            want_w[h // G] += torch.exp(z - torch.where(l == -math.inf, math.inf, lse[a:b, h])[:, None]).sum(0)
            e_max = max(e_max, e)
        err = (w[r, :, :K[r].shape[0]] - want_w).abs()
        assert (err <= (e_max + 2.0 ** -18) * want_w + 1e-12).all(), r


@pytest.mark.parametrize("G", [2, 40])
def test_a_token_that_is_cached_already_sees_its_whole_window(M, G):
    """Append, then attend without own keys: the row's own key is the cache's
    last, and the oldest key of the window may be alone in its group of 32."""
    g = torch.Generator().manual_seed(G)
    hkv, D = 1 if G > 16 else 2, 64
    m, G = (5, 16) if G > 16 else (1, G)  # 80 rows a kv head: the tensor-core kernel
    lens = list(range(100, 135))
    K = [ref.bf16(rnd(g, n, hkv, D)) for n in lens]
    V = [ref.bf16(rnd(g, n, hkv, D)) for n in lens]
    pos = [torch.arange(n) for n in lens]
    c = make(M, K, V, pos)
    q = ref.bf16(rnd(g, m * len(lens), hkv * G, D))
    q_pos = [[n - m + i for i in range(m)] for n in lens]
    for kw in (dict(window=40), dict(window=1), dict(window=65), dict(start=[n - 34 for n in lens]),
               dict(start=[n - 1 for n in lens], window=70), dict(start=[33] * len(lens))):
        attend_and_observe(M, c, K, V, pos, [m] * len(lens), q, G, q_pos, kw)


@pytest.mark.parametrize("m,G", [(8, 2), (64, 4)])
def test_rows_that_are_all_cached_already(M, m, G):
    g = torch.Generator().manual_seed(m)
    hkv, D, n = 2, 128, 300
    K, V = [ref.bf16(rnd(g, n, hkv, D))], [ref.bf16(rnd(g, n, hkv, D))]
    pos = [torch.arange(n) * 2]
    c = make(M, K, V, pos)
    q = ref.bf16(rnd(g, m, hkv * G, D))
    q_pos = [[2 * (n - m + i) for i in range(m)]]
    for kw in (dict(window=33), dict(window=64), dict(start=[2 * (n - 90)]), dict(start=[2 * (n - m)], window=300)):
        attend_and_observe(M, c, K, V, pos, [m], q, G, q_pos, kw)


@pytest.mark.parametrize("m,G", [(1, 2), (6, 16)])
@pytest.mark.parametrize("posd", [False, True])
def test_positions_after_an_eviction(M, m, G, posd):
    """The kept keys' positions pass ctx_len, and differ between the kv heads:
    by default the rows stand at ctx_len + i, before most of the cache."""
    g = torch.Generator().manual_seed(3 * m + G)
    hkv, D, n, budget = 2, 64, 2000, 400
    K, V = [ref.bf16(rnd(g, n, hkv, D)) for _ in range(2)], [ref.bf16(rnd(g, n, hkv, D)) for _ in range(2)]
    c = make(M, K, V, [torch.arange(n)] * 2)
    c.weight.copy_(torch.rand(c.weight.shape, generator=g))
    dst = M.KV4Cache(np.arange(2 * 13).reshape(2, 13), 26, hkv, D, 32)
    kept = c.evict(dst, budget, recent=20, sinks=4).long().cpu()
    assert c.status() == 0
    K = [torch.stack([K[r][kept[r, h], h] for h in range(hkv)], 1) for r in range(2)]
    V = [torch.stack([V[r][kept[r, h], h] for h in range(hkv)], 1) for r in range(2)]
    pos = [kept[r] for r in range(2)]
    q = ref.bf16(rnd(g, 2 * m, hkv * G, D))
    q_pos = [[(n if posd else budget) + i for i in range(m)]] * 2
    for kw in (dict(window=150), dict(window=512), dict(start=[300, 0]), dict(start=[1000, 450], window=600)):
        attend_and_observe(M, dst, K, V, pos, [m, m], q, G, q_pos, kw, posd=posd)


# ------------------------------------------------------ NaN and its reach --

@pytest.mark.parametrize("kw", [dict(), dict(window=40), dict(start=[30])])
@pytest.mark.parametrize("m,G", [(3, 4), (33, 4)])
def test_a_nan_row_gives_no_weight(M, m, G, kw):
    """A bad own value leaves lse NaN in the row that sees it; the weights that
    the other rows give stay, and the hidden keys' too."""
    g = torch.Generator().manual_seed(m)
    hkv, D, n = 2, 128, 120
    K, V = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, n, hkv, D))
    c = make(M, [K], [V], [torch.arange(n)])
    q, k, v = (ref.bf16(rnd(g, m, h, D)) for h in (hkv * G, hkv, hkv))
    v[1, 0, 5] = math.nan
    qd = dev(q)
    qd[2, 1, 7] = math.inf  # and a query that is not finite
    rows = M.RequestRows([0, m])
    anc = torch.tensor([1 << i for i in range(m)], dtype=torch.int64).cuda()
    qp = torch.full((m,), n, dtype=torch.int64)
    score = M.KV4Score(window=kw.get("window", 0), start=i32(kw["start"]) if "start" in kw else None)
    out, lse = c.attend(qd, rows, dev(k), dev(v), anc=anc, pos=i32(qp), score=score)
    lse = lse.double().cpu()
    assert torch.isnan(lse[1, :G]).all() and torch.isfinite(lse[1, G:]).all() and torch.isnan(lse[2, 1])
    w0 = torch.rand(c.weight.shape, generator=g)
    c.weight.copy_(w0)
    got = c.observe(qd, lse.float().cuda(), rows, pos=i32(qp), score=score, decay=0.5)[0, :, :n].double().cpu()
    want = 0.5 * w0[0, :, :n].double()
    e_max = 0.0
    for h in range(hkv * G):
        _, _, z, _, _, e = expect(q[:, h], ref.values(K[:, h // G]), ref.values(V[:, h // G]), qp, torch.arange(n),
                                  torch.ones(m, n, dtype=torch.bool), window=kw.get("window", 0),
                                  start=kw["start"][0] if "start" in kw else None)
        fine = torch.isfinite(lse[:, h])
        want[h // G] += torch.exp(z[fine] - lse[fine, h][:, None]).sum(0)
        e_max = max(e_max, e)
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= (e_max + 2.0 ** -18) * want).all()


# ------------------------------------------------------- keys held as NaN --

def test_a_key_held_as_nan_collects_nothing(M):
    """Seen by a row of weight 0 alone, or by a row whose lse it has made NaN."""
    g = torch.Generator().manual_seed(4)
    hkv, D, n = 1, 64, 64
    K, V = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, n, hkv, D))
    bad = K.clone()
    bad[20] = math.nan
    c = make(M, [bad], [V], [torch.arange(n)])
    q = ref.bf16(rnd(g, 3, 2, D))
    rows, qp = M.RequestRows([0, 3]), torch.tensor([n - 20, n + 10, n + 12])
    score = M.KV4Score(window=40)  # the first row sees key 20, the others do not
    _, lse = c.attend(dev(q), rows, pos=i32(qp), score=score)
    assert torch.isnan(lse[0]).all() and torch.isfinite(lse[1:]).all()
    for weight in ([0.0, 1.0, 1.0], [1.0, 1.0, 0.5]):
        got = c.observe(dev(q), lse, rows, pos=i32(qp), score=score, row_weight=torch.tensor(weight).cuda(),
                        out=torch.zeros_like(c.weight))[0, 0, :n].double().cpu()
        want = torch.zeros(n, dtype=torch.float64)
        for h in range(2):
            z, size = ref.scores(q[:, h], ref.values(K[:, 0]), qp, torch.arange(n), 1 / 8.0, window=40)
            for r in (1, 2):
                want += weight[r] * torch.exp(z[r] - float(lse[r, h]))
        assert got[20] == 0 and torch.isfinite(got).all()
        e = (D + 16) * 2.0 ** -24 * size + 2.0 ** -18
        assert ((got - want).abs() <= e * want).all()


# ----------------------------------------- values of very different sizes --

def check_values(M, K, V, q, k, v, G, anc, pos=None, start=None, page=32):
    """One request, against the definition with the tolerance above."""
    n, hkv, D = K.shape
    m = q.shape[0]
    kp = torch.arange(n) if pos is None else pos
    qp = torch.full((m,), int(kp[-1]) + 1 if n else 0, dtype=torch.int64)
    c = make(M, [K], [V], [kp], page=page)
    score = M.KV4Score(start=i32([start])) if start is not None else None
    ancd = torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64).cuda()
    out, lse = c.attend(dev(q), M.RequestRows([0, m]), dev(k), dev(v), anc=ancd, pos=i32(qp), score=score)
    assert c.status() == 0
    out, lse = out.double().cpu(), lse.double().cpu()
    own = torch.tensor([[bool(a >> j & 1) for j in range(m)] for a in anc])
    for h in range(hkv * G):
        Kh = torch.cat([ref.values(K[:, h // G]), k[:, h // G]])
        Vh = torch.cat([ref.values(V[:, h // G]), v[:, h // G]])
        sees = torch.cat([torch.ones(m, n, dtype=torch.bool), own], 1)
        want, l, _, _, tol, e = expect(q[:, h], Kh, Vh, qp, torch.cat([kp, qp]), sees, start=start)
        compare(out[:, h], lse[:, h], want, l, tol, e, (h,))


SHAPES = [(1, 4, 128), (6, 4, 128), (7, 2, 64), (20, 4, 128), (17, 4, 64), (30, 8, 128)]  # 4 to 240 rows a kv head


@pytest.mark.parametrize("m,G,D", SHAPES)
def test_values_from_2_to_the_minus_14_to_2_to_the_14(M, m, G, D):
    g = torch.Generator().manual_seed(m * G)
    n, hkv = 333, 2
    K, k = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    size = lambda r: torch.exp2((28 * torch.rand(r, hkv, 1, generator=g, dtype=torch.float64) - 14).round())  # noqa: E731
    V, v = ref.bf16(rnd(g, n, hkv, D) * size(n)), ref.bf16(rnd(g, m, hkv, D) * size(m))
    anc = [(1 << i) | 1 for i in range(m)]
    check_values(M, K, V, ref.bf16(2 * rnd(g, m, hkv * G, D)), k, v, G, anc)


@pytest.mark.parametrize("m,G,D", SHAPES)
@pytest.mark.parametrize("where", ["own", "cached", "both"])
@pytest.mark.parametrize("huge", [1e30, 2.0 ** 20])
def test_a_huge_value_that_no_row_or_one_row_sees(M, m, G, D, where, huge):
    """A draft row that is nobody's ancestor but its own (its output is its
    affair), and cached keys before the document, leave the others as they are."""
    g = torch.Generator().manual_seed(m + G)
    n, hkv = 290, 2
    K, k = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    V, v = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    if where != "cached":
        v[m - 1] *= huge
    if where != "own":
        V[3], V[70], V[99] = V[3] * huge, V[70] * huge, V[99] * -huge
    anc = [(1 << i) | 1 for i in range(m)]
    check_values(M, K, ref.bf16(V), ref.bf16(1.5 * rnd(g, m, hkv * G, D)), k, ref.bf16(v), G, anc,
                 start=100 if where != "own" else None)


@pytest.mark.parametrize("m,G,D", SHAPES)
def test_the_greatest_finite_values_where_no_row_sees_them(M, m, G, D):
    g = torch.Generator().manual_seed(m + 7 * G)
    n, hkv = 290, 2
    K, k = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    V, v = rnd(g, n, hkv, D), rnd(g, m, hkv, D)
    huge = lambda *s: 1e38 + 2e38 * torch.rand(*s, generator=g, dtype=torch.float64)  # noqa: E731
    V[3], V[64:70], V[99] = huge(hkv, D), huge(6, hkv, D), -huge(hkv, D)
    V[50] = 2.4e38 + 0.45 * huge(hkv, D) - 0.45e38  # 8 s + m passes fp32
    anc = [(1 << i) | 1 for i in range(m)]
    if m > 1:
        v[m - 1] = huge(hkv, D)
        anc[m - 1] = 1  # nobody's, not even its own
    check_values(M, K, ref.bf16(V), ref.bf16(1.5 * rnd(g, m, hkv * G, D)), k, ref.bf16(v), G, anc, start=100)


@pytest.mark.parametrize("m,G,D", SHAPES)
def test_a_large_value_of_little_weight(M, m, G, D):
    """Seen, but with a weight that makes it count as little as the others."""
    g = torch.Generator().manual_seed(m + 3 * G)
    n, hkv = 160, 1
    V, v = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    q = torch.zeros(m, G, D, dtype=torch.float64)
    q[..., 0] = 16.0
    K, k = 0.01 * rnd(g, n, hkv, D), 0.01 * rnd(g, m, hkv, D)
    K[77, 0, 0] = k[0, 0, 0] = -0.69 * 24 * math.sqrt(D) / 16  # a weight of 2^-24
    V[77] *= 2.0 ** 22
    v[0] *= 2.0 ** 22
    check_values(M, ref.bf16(K), ref.bf16(V), q, ref.bf16(k), ref.bf16(v), G, [(1 << i) | 1 for i in range(m)])


@pytest.mark.parametrize("m,G,D", [(6, 4, 128), (20, 4, 128), (30, 8, 64)])
def test_values_of_zero_and_of_one_size(M, m, G, D):
    """Rows of zeros, constant rows, and rows near the least and greatest sizes."""
    g = torch.Generator().manual_seed(m + 5 * G)
    n, hkv = 200, 1
    K, k = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, m, hkv, D))
    q = ref.bf16(rnd(g, m, G, D))
    anc = [(2 << i) - 1 for i in range(m)]
    V, v = torch.zeros(n, hkv, D, dtype=torch.float64), torch.zeros(m, hkv, D, dtype=torch.float64)
    check_values(M, K, V, q, k, v, G, anc)
    V[40:90], v[2] = 3.0, -0.5
    check_values(M, K, V, q, k, v, G, anc)
    for size in (2.0 ** -80, 2.0 ** 80):
        check_values(M, K, ref.bf16(size * rnd(g, n, hkv, D)), q, k, ref.bf16(size * rnd(g, m, hkv, D)), G, anc)


@pytest.mark.parametrize("m,G,D", [(20, 4, 64), (64, 4, 64), (24, 4, 128)])
def test_values_far_larger_and_smaller_in_a_long_context(M, m, G, D):
    """Enough keys that a CTA walks more than 64 units of 64, some of them with a
    value 2^9 larger or smaller than the others', some hidden by the document.
    Roundings of different keys add up as squares do: four times 3 2^-12."""
    ctx, hkv, start = 131149, 8, 1000
    g = torch.Generator(device="cuda").manual_seed(m + D)
    c = M.KV4Cache(np.arange(-(-ctx // 128))[None][:, ::-1], -(-ctx // 128), hkv, D, 128)
    K = torch.randn(ctx, hkv, D, generator=g, device="cuda").bfloat16()
    V = torch.randn(ctx, hkv, D, generator=g, device="cuda")
    V[::1777] *= 2.0 ** 9
    V[5::1313] *= 2.0 ** -9
    V[700] *= 1e30
    V = V.bfloat16()
    q = (1.5 * torch.randn(m, hkv * G, D, generator=g, device="cuda")).bfloat16()
    k, v = (torch.randn(m, hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    c.append(K, V, M.RequestRows([0, ctx]))
    out, lse = c.attend(q, M.RequestRows([0, m]), k, v, score=M.KV4Score(start=i32([start])))
    assert c.status() == 0
    own = torch.tril(torch.ones(m, m, dtype=torch.bool, device="cuda"))
    for h in range(0, hkv, 3):
        kd = torch.cat([ref.values(K[start:, h].double()), k[:, h].double()])
        vd = torch.cat([ref.values(V[start:, h].double()), v[:, h].double()])
        for hq in (h * G, h * G + G - 1):
            z = (q[:, hq].double() @ kd.T) / math.sqrt(D)
            z[:, ctx - start:] = z[:, ctx - start:].masked_fill(~own, -math.inf)
            l = torch.logsumexp(z, 1)
            p = torch.exp(z - l[:, None])
            o = p @ vd
            assert ((lse[:, hq].double() - l).abs() <= 2.0 ** -16).all()
            big = vd.abs().amax(1)
            tol = H * o.abs() + (4 * 3 * 2.0 ** -12 * (p ** 2 @ big ** 2).sqrt() + 2.0 ** -14 * (p @ big))[:, None]
            err = (out[:, hq].double() - o).abs()
            assert (err <= tol).all(), (hq, float((err / tol).max()))


# ----------------------------------------------------- calls without rows --

def test_calls_without_rows(M):
    g = torch.Generator().manual_seed(1)
    K, V = [ref.bf16(rnd(g, 70, 2, 64)), ref.bf16(rnd(g, 3, 2, 64))], [ref.bf16(rnd(g, 70, 2, 64)), ref.bf16(rnd(g, 3, 2, 64))]
    c = make(M, K, V, [torch.arange(70), torch.arange(3)])
    none = M.RequestRows([0, 0, 0])
    kv, q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    before = c.blocks.clone()
    c.append(kv, kv, none)
    assert c.ctx_len.tolist() == [70, 3] and torch.equal(before, c.blocks)
    k, v = c.read(none)
    assert k.shape == v.shape == (0, 2, 64)
    out, lse = c.attend(q, none, kv, kv)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = c.attend(q, none)
    for score in (None, M.KV4Score(window=5)):
        w0 = torch.rand_like(c.weight)
        c.weight.copy_(w0)
        c.observe(q, lse, none, decay=0.25, score=score)  # the weights fade all the same
        assert c.status() == 0
        for r, n in enumerate((70, 3)):
            assert torch.equal(c.weight[r, :, :n], 0.25 * w0[r, :, :n]) and torch.equal(c.weight[r, :, n:], w0[r, :, n:])


# -------------------------------------------------- append from no source --

def test_append_from_no_rows_at_all(M):
    """n_src = 0: no source row exists, so none is read."""
    import ctypes
    from speculative_decoding_tree_bit_gb300 import check, lib, stream_ptr
    c = M.KV4Cache([[0]], 1, 1, 64, 32)
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    rows, src, before = M.RequestRows([0, 2]), i32([0, -1]), c.blocks.clone()
    def call(count):
        check(lib().sd_kv4_append(ctypes.byref(c._s), x.data_ptr(), x.data_ptr(), 64, 0, rows.cu_dev.data_ptr(),
                                  rows.cu.ctypes.data, 1, src.data_ptr(), count.data_ptr(), None, None,
                                  c._status.data_ptr(), stream_ptr()))
    zero, two = i32([0]), i32([2])
    call(zero)
    assert c.status() == 0 and c.ctx_len.tolist() == [0]
    call(two)
    assert c.status() == 7 and torch.equal(before, c.blocks)


# -------------------------------------------------------------- bad pages --

def test_a_row_of_a_bad_page_is_nan_after_an_eviction_and_when_read(M):
    """Not what the destination's page held before, which may be another request's."""
    g = torch.Generator().manual_seed(13)
    K, V = [ref.bf16(rnd(g, 200, 2, 128))], [ref.bf16(rnd(g, 200, 2, 128))]
    c = make(M, K, V, [torch.arange(200)])
    dst = make(M, [ref.bf16(rnd(g, 128, 2, 128))], [ref.bf16(rnd(g, 128, 2, 128))], [torch.arange(128)])
    c.page_table[0, 4] = -4  # slots 128 .. 159
    kept = c.evict(dst, 100, recent=100)
    assert c.status() == 7
    k, v = dst.read(M.RequestRows([0, 100]))
    want = (kept[0].t() >= 128) & (kept[0].t() < 160)
    assert want.any() and not want.all()
    assert torch.equal(torch.isnan(k).all(-1), want) and torch.equal(torch.isnan(v).all(-1), want)
    assert torch.equal(torch.isnan(k).any(-1), want) and torch.equal(torch.isnan(v).any(-1), want)
    k, v = c.read(M.RequestRows([0, 200]))
    assert c.status() == 7
    want = (torch.arange(200) >= 128) & (torch.arange(200) < 160)
    for x in (k, v):
        assert torch.equal(torch.isnan(x).flatten(1).all(1).cpu(), want)
        assert torch.equal(torch.isnan(x).flatten(1).any(1).cpu(), want)


# ----------------------------------------------------- streams and graphs --

@pytest.mark.parametrize("m", [4, 40])
def test_the_first_call_on_another_stream(M, m):
    """The workspace is made ready on the stream of the call, whatever the
    current stream is busy with."""
    g = torch.Generator().manual_seed(m)
    K, V = [ref.bf16(rnd(g, 3000, 2, 64))], [ref.bf16(rnd(g, 3000, 2, 64))]
    c, d = (make(M, K, V, [torch.arange(3000)]) for _ in range(2))
    q, rows = dev(rnd(g, m, 8, 64)), M.RequestRows([0, m])
    want, want_lse = d.attend(q, rows)
    pages = np.arange(8)[None]
    dst, dst2 = M.KV4Cache(pages, 8, 2, 64, 32), M.KV4Cache(pages, 8, 2, 64, 32)
    want_kept = d.evict(dst2, 200).clone()
    # memory that the allocator may hand out again is not zero
    junk = [torch.full((1 << 24,), 3, dtype=torch.int32, device="cuda") for _ in range(4)]
    del junk
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second on the current stream
    out, lse = c.attend(q, rows, stream=other)
    kept = c.evict(dst, 200, stream=other)
    other.synchronize()
    got = [t.clone() for t in (out, lse, kept)]
    torch.cuda.synchronize()
    assert c.status() == 0
    assert torch.equal(got[0], want) and torch.equal(got[1], want_lse) and torch.equal(got[2], want_kept)


def test_a_capture_before_any_other_call(M):
    """The first attend inside a graph capture: eager calls before the first
    replay, and replays after them, see a workspace that is ready."""
    g = torch.Generator().manual_seed(2)
    K, V = [ref.bf16(rnd(g, 3000, 2, 64))], [ref.bf16(rnd(g, 3000, 2, 64))]
    c, d = (make(M, K, V, [torch.arange(3000)]) for _ in range(2))
    q, rows = dev(rnd(g, 4, 8, 64)), M.RequestRows([0, 4])
    want, want_lse = d.attend(q, rows)
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(q, rows, out=out, lse=lse)
    for _ in range(2):
        a, b = c.attend(q, rows)
        assert torch.equal(a, want) and torch.equal(b, want_lse)
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert c.status() == 0


# ----------------------------------------------- second kernels in graphs --

def test_append_and_evict_in_a_graph(M):
    """Their second kernels begin while the first end; replayed, they do what
    the eager calls do."""
    g = torch.Generator().manual_seed(6)
    n = [150, 64, 0]
    K, V = [ref.bf16(rnd(g, x, 2, 128)) for x in n], [ref.bf16(rnd(g, x, 2, 128)) for x in n]
    def fresh():
        c = make(M, K, V, [torch.arange(x) for x in n], room=90)
        c.weight.copy_(torch.rand(c.weight.shape, generator=torch.Generator().manual_seed(5)))
        return c, M.KV4Cache(np.arange(12).reshape(3, 4), 12, 2, 128, 32)
    rows, x = M.RequestRows([0, 5, 6, 10]), dev(rnd(g, 10, 2, 128))
    y, count = dev(rnd(g, 10, 2, 128)), i32([3, 1, 4])
    def step(c, dst):
        c.append(x, y, rows, count=count)
        c.evict(dst, 100, recent=10, sinks=2)
    c, dst = fresh()
    step(c, dst)  # the workspace
    eager = []
    c, dst = fresh()
    for _ in range(3):
        step(c, dst)
        eager.append([t.clone() for t in (c.ctx_len, c.pos, c.blocks, dst.ctx_len, dst.pos, dst.weight)] +
                     list(dst.read(M.RequestRows(np.cumsum([0] + dst.ctx_len.tolist())))))
    c, dst = fresh()
    first = [t.clone() for t in (c.ctx_len, c.pos, c.blocks, c.weight)]
    step(c, dst)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, dst)
    for t, v in zip((c.ctx_len, c.pos, c.blocks, c.weight), first):
        t.copy_(v)
    dst.pos.zero_(), dst.weight.zero_(), dst.ctx_len.zero_()
    for want in eager:
        graph.replay()
        torch.cuda.synchronize()
        got = [c.ctx_len, c.pos, c.blocks, dst.ctx_len, dst.pos, dst.weight]
        got += list(dst.read(M.RequestRows(np.cumsum([0] + dst.ctx_len.tolist()))))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert c.status() == 0 and c.ctx_len.tolist() == [159, 67, 12]

"""The 4-bit key/value cache on the GPU against its 64-bit definition.

Tolerances, from the number formats: an output is rounded to bf16 (half a
step: 2^-8 of its value); the softmax weights enter the products as two bf16
terms (2^-15 of the greatest value seen); a score carries the rounding of a
dot product of D terms in fp32 ((D + 16) 2^-24 of the sum of its terms' sizes)
and of its cap, slope and exponential (2^-20)."""
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


class Setup:
    """A cache of requests holding `ctxs` keys, and the same on the host."""

    def __init__(self, M, ctxs, hkv=2, D=128, page=64, seed=0, room=0, gaps=False, extra_pages=3):
        g = self.g = torch.Generator().manual_seed(seed)
        self.ctxs, self.hkv, self.D, self.R = ctxs, hkv, D, len(ctxs)
        pages = max(1, -(-(max(ctxs) + room) // page))
        n = self.R * pages + extra_pages
        self.table = torch.randperm(n, generator=g)[:self.R * pages].reshape(self.R, pages).numpy()
        self.cache = M.KV4Cache(self.table, n, hkv, D, page)
        self.cache.blocks.fill_(0xFF)  # records of slots nobody wrote: NaN scales
        self.K = [ref.bf16(rnd(g, c, hkv, D) * (0.5 + torch.rand(hkv, D, generator=g)) + 0.5 * rnd(g, hkv, D))
                  for c in ctxs]
        self.V = [ref.bf16(rnd(g, c, hkv, D)) for c in ctxs]
        self.pos = []
        for c in ctxs:
            step = torch.ones(c, dtype=torch.int64)
            if gaps:
                step += torch.randint(0, 9, (c,), generator=g)
            self.pos.append(torch.cumsum(step, 0) - 1)
        rows = M.RequestRows(np.cumsum([0] + list(ctxs)))
        if rows.n:
            self.cache.append(dev(torch.cat(self.K)), dev(torch.cat(self.V)), rows,
                              pos=torch.cat(self.pos).int().cuda())
        assert self.cache.status() == 0
        assert self.cache.ctx_len.tolist() == list(ctxs)

    def next_pos(self, r):
        return int(self.pos[r][-1]) + 1 if self.ctxs[r] else 0


def tree(g, m, chain):
    anc, depth = [], []
    for i in range(m):
        p = i - 1 if chain or i == 0 else int(torch.randint(0, i, (1,), generator=g))
        anc.append((anc[p] if i else 0) | 1 << i)
        depth.append(depth[p] + 1 if i else 0)
    return anc, depth


def signed(anc):
    return torch.tensor([a - (1 << 64) if a >> 63 else a for a in anc], dtype=torch.int64).cuda()


def check_attention(M, s, ms, G=4, chain=False, own=True, cap=0.0, slopes=False, window=0, start=None, anc_given=True,
                    pos_given=True, strided=False, q_scale=1.5, stream=None, max_ctx=0, scale=0.0):
    """Runs attend and compares; returns what observe's check needs."""
    g, D, hkv = s.g, s.D, s.hkv
    hq, n = G * hkv, sum(ms)
    rows = M.RequestRows(np.cumsum([0] + list(ms)))
    q = ref.bf16(q_scale * rnd(g, n, hq, D))
    k, v = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, n, hkv, D))
    trees = [tree(g, m, chain) for m in ms]
    anc = [a for t in trees for a in t[0]] if anc_given else [(2 << i) - 1 for m in ms for i in range(m)]
    if pos_given:
        pos = [s.next_pos(r) + d for r, t in enumerate(trees) for d in t[1]]
    else:
        pos = [s.ctxs[r] + i for r, m in enumerate(ms) for i in range(m)]
    sl = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq) if slopes else None
    st = torch.tensor(start, dtype=torch.int32) if start is not None else None
    score = M.KV4Score(scale=scale, softcap=cap, slopes=sl.float().cuda() if slopes else None, window=window,
                       start=st.cuda() if start is not None else None)
    if strided:  # rows cut out of a wider one, as a fused projection leaves them
        wide = torch.zeros(n, hq + 2 * hkv + 1, D, dtype=torch.bfloat16, device="cuda")
        wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:hq + 2 * hkv] = dev(q), dev(k), dev(v)
        qd, kd, vd = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:hq + 2 * hkv]
    else:
        qd, kd, vd = dev(q), dev(k), dev(v)
    posd = torch.tensor(pos, dtype=torch.int32).cuda() if pos_given else None
    out, lse = s.cache.attend(qd, rows, kd if own else None, vd if own else None,
                              anc=signed(anc) if anc_given else None, pos=posd, score=score, stream=stream,
                              max_ctx=max_ctx)
    torch.cuda.synchronize()
    assert s.cache.status() == 0
    assert out.shape == q.shape and out.dtype == qd.dtype
    got, got_lse = out.double().cpu(), lse.double().cpu()
    eps = []
    for r in range(s.R):
        a, b = int(rows.cu[r]), int(rows.cu[r + 1])
        K, V, kp = ref.values(s.K[r]), ref.values(s.V[r]), s.pos[r]
        sees = torch.ones(b - a, s.ctxs[r], dtype=torch.bool)
        qp = torch.tensor(pos[a:b], dtype=torch.int64)
        if own:
            K, V, kp = torch.cat([K, k[a:b]]), torch.cat([V, v[a:b]]), torch.cat([kp, qp])
            sees = torch.cat([sees, torch.tensor([[bool(anc[a + i] >> j & 1) for j in range(b - a)]
                                                  for i in range(b - a)]).reshape(b - a, b - a).bool()], 1)
        for h in range(hq):
            z, size = ref.scores(q[a:b, h], K[:, h // G], qp, kp, scale or 1 / math.sqrt(D), cap,
                                 float(sl[h]) if slopes else 0.0, window, int(st[r]) if start is not None else None)
            z = z.masked_fill(~sees, -math.inf)
            p, l = ref.softmax(z)
            far = float((qp[:, None] - kp[None]).abs().max()) * float(sl[h]) if slopes and kp.numel() and b > a else 0.0
            e = (D + 16) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + cap / 8) + 2.0 ** -23 * far
            eps.append(e)
            want = p @ V[:, h // G]
            top = V[:, h // G].abs().max().item() if V.shape[0] else 0.0
            err = (got[a:b, h] - want).abs()
            assert (err <= H * want.abs() + (2.0 ** -15 + 2 * e) * top).all(), (r, h, float(err.max()))
            inf = l == -math.inf
            assert torch.equal(got_lse[a:b, h] == -math.inf, inf)
            assert (got[a:b, h][inf] == 0).all()
            err = (got_lse[a:b, h] - l)[~inf].abs()
            assert (err <= e + 2.0 ** -22 * l[~inf].abs()).all(), (r, h, float(err.max()))
    return dict(rows=rows, q=q, qd=qd, lse=lse, pos=pos, posd=posd, score=score, sl=sl, cap=cap, window=window, st=st,
                G=G, scale=scale, eps=max(eps) if eps else 0.0)


def check_observe(M, s, o, decay=1.0, row_weight=None, in_place=False, max_ctx=0):
    g, hkv, G = s.g, s.hkv, o["G"]
    w0 = torch.rand(s.R, hkv, s.cache.cap, generator=g)
    s.cache.weight.copy_(w0)
    rw = row_weight
    out = None if in_place else torch.full_like(s.cache.weight, -7.0)
    got = s.cache.observe(o["qd"], o["lse"], o["rows"], pos=o["posd"],
                          row_weight=None if rw is None else torch.tensor(rw).float().cuda(), score=o["score"],
                          decay=decay, out=out, max_ctx=max_ctx)
    torch.cuda.synchronize()
    assert s.cache.status() == 0
    got = got.double().cpu()
    rest = w0.double() if in_place else torch.full_like(got, -7.0)
    for r in range(s.R):
        a, b = int(o["rows"].cu[r]), int(o["rows"].cu[r + 1])
        c = s.ctxs[r]
        K, qp = ref.values(s.K[r]), torch.tensor(o["pos"][a:b], dtype=torch.int64)
        want = decay * w0[r, :, :c].double()
        for h in range(G * hkv):
            z, _ = ref.scores(o["q"][a:b, h], K[:, h // G], qp, s.pos[r], o["scale"] or 1 / math.sqrt(s.D), o["cap"],
                              float(o["sl"][h]) if o["sl"] is not None else 0.0, o["window"],
                              int(o["st"][r]) if o["st"] is not None else None)
            lse = o["lse"][a:b, h].double().cpu()
            p = torch.exp(z - torch.where(lse == -math.inf, math.inf, lse)[:, None])
            if rw is not None:
                p = p * torch.tensor(rw[a:b]).double()[:, None]
            want[h // G] += p.sum(0)
        err = (got[r, :, :c] - want).abs()
        assert (err <= (o["eps"] + 2.0 ** -19) * want + 1e-12).all(), (r, float((err / want.clamp(min=1e-9)).max()))
        assert torch.equal(got[r, :, c:], rest[r, :, c:])  # slots past the context are not touched


# ----------------------------------------------------------- append, read --

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,ctxs", [(32, [1]), (64, [33, 0, 200]), (96, [95, 97, 1, 64])])
def test_append_stores_the_defined_codes(M, D, page, ctxs):
    s = Setup(M, ctxs, hkv=3, D=D, page=page, seed=D + page)
    blocks = s.cache.blocks.cpu().numpy()
    for r, c in enumerate(ctxs):
        for h in range(3):
            ck, sk, mk = ref.quantise(s.K[r][:, h])
            cv, sv, mv = ref.quantise(s.V[r][:, h])
            for t0 in range(0, c, 32):
                n = min(32, c - t0)
                rec = blocks[s.table[r, t0 // page], h, t0 % page // 32]
                kc, ksm, vc, vsm = ref.parse_record(rec, D)
                for codes, sm, wc, ws, wm in ((kc, ksm, ck, sk, mk), (vc, vsm, cv, sv, mv)):
                    assert np.array_equal(codes[:n], wc[t0:t0 + n].numpy())
                    assert np.array_equal(sm[:n, 0], ws[t0:t0 + n].float().numpy())
                    assert np.array_equal(sm[:n, 1], wm[t0:t0 + n].float().numpy())
        assert torch.equal(s.cache.pos[r, :, :c].cpu(), s.pos[r].int().expand(3, -1))
    rows = M.RequestRows(np.cumsum([0] + ctxs))
    k, v = s.cache.read(rows)
    for got, want in ((k, torch.cat(s.K)), (v, torch.cat(s.V))):
        want = ref.values(want)
        assert ((got.double().cpu() - want).abs() <= H * want.abs()).all()


def test_append_of_special_rows(M):
    D = 128
    x = torch.zeros(9, 1, D, dtype=torch.float64)
    x[1] = 2.5                                     # constant
    x[2, 0, ::2], x[2, 0, 1::2] = 1e30, -1e30      # wide
    x[3, 0, 5] = math.nan
    x[4, 0, 7] = math.inf
    x[5, 0, 9] = -math.inf
    x[6] = 2.0 ** -130                             # below the normal range
    x[6, 0, 3] = 2.0 ** -126
    x[7] = torch.arange(D) - 64.0                  # ties of the rounding
    x[8, 0, 0] = -0.0
    x = ref.bf16(x)
    c = M.KV4Cache([[0]], 1, 1, D, 32)
    rows = M.RequestRows([0, 9])
    c.append(dev(x), dev(x.flip(0)), rows)
    k, v = c.read(rows)
    want = ref.values(x)
    for got, w in ((k.double().cpu(), want), (v.double().cpu(), want.flip(0))):
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert [bool(t) for t in torch.isnan(w).flatten(1).any(1)].count(True) == 3
        f = ~torch.isnan(w)
        assert ((got - w)[f].abs() <= H * w[f].abs() + 2.0 ** -133).all()


def test_append_of_an_accepted_path(M):
    """The verified tree's accepted nodes only, at the context's end."""
    s = Setup(M, [40, 0, 63], room=8, seed=5)
    g = s.g
    n, hkv, D = 24, 2, 128
    k, v = ref.bf16(rnd(g, n, hkv, D)), ref.bf16(rnd(g, n, hkv, D))
    rows = M.RequestRows([0, 8, 16, 24])
    src = torch.arange(n, dtype=torch.int32)
    path = {0: [0, 3, 7], 1: [0], 2: [0, 1, 2, 4, 5, 6]}
    for r, p in path.items():
        src[8 * r:8 * r + len(p)] = 8 * r + torch.tensor(p)
    count = torch.tensor([3, 1, 6], dtype=torch.int32)
    s.cache.append(dev(k), dev(v), rows, src=src.cuda(), count=count.cuda())
    assert s.cache.status() == 0
    assert s.cache.ctx_len.tolist() == [43, 1, 69]
    got, _ = s.cache.read(M.RequestRows([0, 3, 4, 10]), at=torch.tensor([40, 0, 63], dtype=torch.int32).cuda())
    want = ref.values(torch.cat([k[[8 * r + i for i in p]] for r, p in path.items()]))
    assert ((got.double().cpu() - want).abs() <= H * want.abs()).all()
    assert s.cache.pos[0, 0, 40:43].tolist() == [40, 41, 42]
    # at set: the given slots, and the length follows from them
    s.cache.append(dev(k[:3]), dev(v[:3]), M.RequestRows([0, 1, 2, 3]),
                   at=torch.tensor([10, 1, 20], dtype=torch.int32).cuda())
    assert s.cache.ctx_len.tolist() == [11, 2, 21]


def test_append_past_the_capacity_or_with_a_bad_page_stores_nothing(M):
    c = M.KV4Cache([[0], [1]], 2, 1, 64, 32)
    x = torch.ones(40, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.append(x, x, M.RequestRows([0, 33, 40]))
    assert c.ctx_len.tolist() == [0, 7] and int(c.pos[0].abs().sum()) == 0
    assert c.status() == 7
    c.page_table.fill_(5)
    before = c.blocks.clone()
    c.append(x[:2], x[:2], M.RequestRows([0, 1, 2]), at=0)
    assert c.status() == 7 and torch.equal(before, c.blocks)
    src = torch.tensor([0, 40], dtype=torch.int32).cuda()
    c.page_table.copy_(torch.tensor([[0], [1]]))
    c.append(x, x, M.RequestRows([0, 1, 2]), at=0, src=src)
    assert c.status() == 7


# -------------------------------------------------------------- attention --

@pytest.mark.parametrize("ctx", [0, 1, 31, 32, 33, 64, 65, 255, 700])
@pytest.mark.parametrize("D", [64, 128])
def test_one_token(M, ctx, D):
    s = Setup(M, [ctx], D=D, seed=ctx)
    check_observe(M, s, check_attention(M, s, [1]))


@pytest.mark.parametrize("G,hkv,m", [(1, 1, 1), (1, 3, 9), (2, 2, 4), (3, 2, 5), (4, 2, 16), (5, 1, 13), (8, 1, 64),
                                     (16, 1, 17), (16, 2, 64)])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_and_rows(M, G, hkv, m, D):
    s = Setup(M, [150], hkv=hkv, D=D, seed=G * 100 + m, page=32)
    check_observe(M, s, check_attention(M, s, [m], G=G))


@pytest.mark.parametrize("page", [32, 64, 96, 256])
@pytest.mark.parametrize("own", [True, False])
def test_ragged_batches(M, page, own):
    s = Setup(M, [500, 1, 0, 33, 260, 96], page=page, seed=page + own)
    o = check_attention(M, s, [3, 1, 8, 0, 40, 2], own=own)
    check_observe(M, s, o, decay=0.5, row_weight=[float(i % 3) / 2 for i in range(54)])
    check_observe(M, s, o, in_place=True)


@pytest.mark.parametrize("opt", [dict(cap=30.0), dict(slopes=True), dict(window=1), dict(window=40),
                                 dict(window=100000), dict(start=[0, 100, 10 ** 6]),
                                 dict(cap=5.0, slopes=True, window=77, start=[3, 40, 0]), dict(scale=0.3)])
@pytest.mark.parametrize("D,gaps", [(64, True), (128, False), (128, True)])
def test_score_options(M, opt, D, gaps):
    s = Setup(M, [300, 129, 5], D=D, gaps=gaps, seed=11 + D)
    check_observe(M, s, check_attention(M, s, [5, 16, 2], **opt), decay=0.25)


@pytest.mark.parametrize("opt", [dict(window=3), dict(start=[10 ** 7, 10 ** 7])])
def test_rows_that_see_nothing(M, opt):
    """No own keys and every cached key hidden: zeros and -inf, weight 0."""
    s = Setup(M, [90, 0], seed=2)
    s.pos[0] = s.pos[0]
    o = check_attention(M, s, [4, 2], own=False, **({"start": opt["start"]} if "start" in opt else {}))
    check_observe(M, s, o)
    if "window" in opt:
        check_observe(M, s, check_attention(M, s, [4, 2], own=False, chain=True, window=3))


@pytest.mark.parametrize("kw", [dict(anc_given=False), dict(pos_given=False), dict(anc_given=False, pos_given=False,
                                window=20), dict(strided=True), dict(chain=True, q_scale=30.0), dict(q_scale=0.0),
                                dict(max_ctx=64), dict(max_ctx=1)])
def test_defaults_strides_and_sharp_scores(M, kw):
    s = Setup(M, [190, 64], seed=21)
    o = check_attention(M, s, [16, 7], **kw)
    check_observe(M, s, o, max_ctx=kw.get("max_ctx", 0))


def test_many_requests(M):
    """More requests than a warp, some empty, and a table of shared pages."""
    ctxs = [(37 * i) % 140 for i in range(70)]
    s = Setup(M, ctxs, hkv=1, D=64, page=32, seed=8)
    check_observe(M, s, check_attention(M, s, [(i * 7) % 5 for i in range(70)], G=2))


@pytest.mark.parametrize("ctx,m,G,D", [(20000, 1, 4, 128), (9000, 16, 4, 128), (12345, 1, 1, 64), (5000, 64, 5, 128)])
def test_long_contexts(M, ctx, m, G, D):
    s = Setup(M, [ctx, 77], D=D, hkv=2, seed=ctx)
    check_observe(M, s, check_attention(M, s, [m, 1], G=G))


def test_a_shared_page_serves_several_requests(M):
    s = Setup(M, [64, 64], seed=4)
    s.cache.page_table[1] = s.cache.page_table[0]
    s.K[1], s.V[1] = s.K[0], s.V[0]
    check_attention(M, s, [2, 3])


def test_masked_and_unwritten_slots_do_not_leak(M):
    """NaN and infinity in keys that no row may see, and NaN scales past the
    end of the context, leave the outputs alone; a NaN that is seen shows."""
    s = Setup(M, [100], seed=6)
    bad = torch.full((30, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    bad[10:20] = math.inf
    s.cache.append(bad, bad, M.RequestRows([0, 30]), at=torch.zeros(1, dtype=torch.int32).cuda(),
                   pos=torch.arange(30, dtype=torch.int32).cuda())
    s.cache.ctx_len.fill_(100)
    o = check_attention(M, s, [5], start=[30])
    check_observe(M, s, o)
    check_attention(M, s, [5], window=60, chain=True)
    rows = M.RequestRows([0, 1])
    q = torch.ones(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = s.cache.attend(q, rows)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_bad_pages_and_lengths_set_the_status(M):
    s = Setup(M, [100, 40], seed=7)
    q = torch.ones(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    rows = M.RequestRows([0, 1, 2])
    good, _ = s.cache.attend(q, rows)
    s.cache.page_table[0, 1] = 1 << 20
    out, lse = s.cache.attend(q, rows)
    assert s.cache.status() == 7
    assert torch.equal(out[1], good[1]) and torch.isfinite(out).all()
    s.cache.observe(q, lse, rows)
    assert s.cache.status() == 7
    s.cache.page_table[0, 1] = -1
    s.cache.attend(q, rows)
    assert s.cache.status() == 7
    s.cache.page_table.copy_(torch.from_numpy(s.table))
    s.cache.ctx_len.copy_(torch.tensor([-5, 40]))
    out, _ = s.cache.attend(q, rows)
    assert s.cache.status() == 7
    assert torch.equal(out[1], good[1]) and (out[0] == 0).all()


def test_another_stream_and_a_graph(M):
    s = Setup(M, [333], seed=9)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o = check_attention(M, s, [8])
    torch.cuda.current_stream().wait_stream(st)
    q, rows = o["qd"], o["rows"]
    out, lse = torch.empty_like(q), torch.empty_like(o["lse"])
    w = torch.zeros_like(s.cache.weight)
    s.cache.attend(q, rows, pos=o["posd"], out=out, lse=lse)
    s.cache.observe(q, lse, rows, pos=o["posd"], out=w)
    torch.cuda.synchronize()
    want = (out.clone(), lse.clone(), w.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.cache.attend(q, rows, pos=o["posd"], out=out, lse=lse)
        s.cache.observe(q, lse, rows, pos=o["posd"], out=w)
    for _ in range(3):
        out.zero_(), lse.zero_(), w.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, lse, w), want))


def test_many_rows_in_a_graph(M):
    """Over 64 rows a kv head, a context whose parts are joined by a second
    kernel, replayed with another context length and other rows."""
    s = Setup(M, [5000, 700], seed=12)
    cu = [0, 40, 70]
    o = check_attention(M, s, [40, 30], G=8)
    q, rows = o["qd"], o["rows"]
    out, lse = torch.empty_like(q), torch.empty_like(o["lse"])
    w = torch.zeros_like(s.cache.weight)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.cache.attend(q, rows, pos=o["posd"], out=out, lse=lse)
        s.cache.observe(q, lse, rows, pos=o["posd"], out=w)
    assert rows.cu.tolist() == cu
    for ctxs in ([5000, 700], [64, 0], [4999, 699]):
        s.cache.ctx_len.copy_(torch.tensor(ctxs))
        want = s.cache.attend(q, rows, pos=o["posd"])
        want_w = s.cache.observe(q, want[1], rows, pos=o["posd"], out=torch.zeros_like(w))
        out.zero_(), lse.zero_(), w.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.equal(w, want_w)
    assert s.cache.status() == 0


def test_the_same_call_gives_the_same_bits(M):
    s = Setup(M, [4000, 900], seed=10)
    q = dev(rnd(s.g, 20, 8, 128))
    rows = M.RequestRows([0, 16, 20])
    a = s.cache.attend(q, rows)
    w = s.cache.observe(q, a[1], rows, out=torch.zeros_like(s.cache.weight))
    for _ in range(5):
        b = s.cache.attend(q, rows)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.equal(w, s.cache.observe(q, a[1], rows, out=torch.zeros_like(w)))


def test_a_cache_beyond_32_bit_offsets(M):
    """Pages past 4 GB of blocks, read and written by one request."""
    D, hkv, page = 128, 8, 128
    per = hkv * (page // 32) * 4352
    n = (1 << 32) // per + 40
    table = np.array([[n - 1, 3, n - 2, n // 2 + 5]])
    c = M.KV4Cache(table, n, hkv, D, page)
    assert c.blocks.numel() > 1 << 32
    g = torch.Generator().manual_seed(1)
    s = object.__new__(Setup)
    s.g, s.ctxs, s.hkv, s.D, s.R, s.table, s.cache = g, [500], hkv, D, 1, table, c
    s.K, s.V = [ref.bf16(rnd(g, 500, hkv, D))], [ref.bf16(rnd(g, 500, hkv, D))]
    s.pos = [torch.arange(500)]
    c.append(dev(s.K[0]), dev(s.V[0]), M.RequestRows([0, 500]))
    check_observe(M, s, check_attention(M, s, [3], G=2))


# --------------------------------------------------------------- eviction --

@pytest.mark.parametrize("budget,recent,sinks", [(64, 16, 4), (1, 0, 0), (100, 100, 0), (33, 0, 33), (32, 5, 1),
                                                 (350, 20, 2), (1000, 10, 3)])
@pytest.mark.parametrize("D,kind", [(64, "mixed"), (128, "mixed"), (128, "ties"), (128, "odd")])
def test_eviction_keeps_the_heaviest(M, budget, recent, sinks, D, kind):
    ctxs = [400, 64, 0, 33, 1100]
    s = Setup(M, ctxs, hkv=2, D=D, page=32, gaps=True, seed=budget)
    w = torch.rand(5, 2, s.cache.cap, generator=s.g) ** 6
    if kind == "ties":
        w = (w * 4).round()
    if kind == "odd":
        w[0, 0, ::7], w[0, 1, ::5], w[4, 0, ::3], w[4, 1, 1::2] = math.nan, math.inf, -1.0, -0.0
        w[4, 1, 2::4] = 0.0
    s.cache.weight.copy_(w)
    pages = -(-budget // 64)
    dst = M.KV4Cache(np.arange(5 * pages)[::-1].reshape(5, pages), 5 * pages, 2, D, 64)
    src_before = s.cache.blocks.clone()
    kept = s.cache.evict(dst, budget, recent=recent, sinks=sinks)
    torch.cuda.synchronize()
    assert s.cache.status() == 0 and torch.equal(src_before, s.cache.blocks)
    n = [min(c, budget) for c in ctxs]
    assert dst.ctx_len.tolist() == n and s.cache.ctx_len.tolist() == ctxs
    k, v = dst.read(M.RequestRows(np.cumsum([0] + n)))
    k, v, off = k.double().cpu(), v.double().cpu(), 0
    for r, c in enumerate(ctxs):
        for h in range(2):
            want = ref.keep(w[r, h, :c].tolist(), budget, recent, sinks)
            assert kept[r, h, :n[r]].tolist() == want, (r, h)
            i = torch.tensor(want, dtype=torch.int64)
            assert torch.equal(dst.pos[r, h, :n[r]].cpu(), s.pos[r].int()[i])
            got = dst.weight[r, h, :n[r]].cpu()
            assert torch.equal(torch.nan_to_num(got, -5.0), torch.nan_to_num(w[r, h][i], -5.0))
            for x, y in ((k, s.K), (v, s.V)):
                ex = ref.values(y[r][:, h])[i]
                assert ((x[off:off + n[r], h] - ex).abs() <= H * ex.abs()).all()
        off += n[r]


def test_attention_after_an_eviction(M):
    s = Setup(M, [300, 90], seed=12)
    w = torch.rand(2, 2, s.cache.cap, generator=s.g)
    s.cache.weight.copy_(w)
    dst = M.KV4Cache([[0, 1], [2, 3]], 4, 2, 128, 64)
    kept = s.cache.evict(dst, 100, recent=20, sinks=2).cpu()
    q = ref.bf16(rnd(s.g, 2, 4, 128))
    out, lse = dst.attend(dev(q), M.RequestRows([0, 1, 2]))
    for r, n in ((0, 100), (1, 90)):
        for h in range(4):
            i = kept[r, h // 2, :n].long()
            z = q[r, h][None] @ ref.values(s.K[r][:, h // 2])[i].T / math.sqrt(128)
            p, l = ref.softmax(z)
            want = (p @ ref.values(s.V[r][:, h // 2])[i])[0]
            assert ((out[r, h].double().cpu() - want).abs() <= H * want.abs() + 2.0 ** -13).all()
            assert abs(float(lse[r, h]) - float(l)) < 2.0 ** -16


def test_a_bad_page_in_an_eviction_sets_the_status(M):
    s = Setup(M, [200], seed=13)
    dst = M.KV4Cache([[0, 9]], 2, 2, 128, 64)
    s.cache.evict(dst, 100, recent=100)
    assert s.cache.status() == 7
    s.cache.page_table[0, 3] = -4
    dst = M.KV4Cache([[0, 1]], 2, 2, 128, 64)
    s.cache.evict(dst, 100, recent=100)
    assert s.cache.status() == 7


# ------------------------------------- many rows a kv head (tensor cores) --

@pytest.mark.parametrize("ms,G", [([25, 3, 12, 0, 1], 4), ([64, 1], 2), ([20, 13], 5), ([64, 2, 9], 16), ([33, 64], 3)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("opt", [dict(), dict(cap=20.0, slopes=True, gaps=True), dict(own=False, window=150)])
def test_many_rows_and_mixed_requests(M, ms, G, D, opt):
    """Requests of many and of few rows in one call: whole tiles, copies of
    rows, rows over several segments."""
    opt = dict(opt)
    ctxs = [700, 40, 257, 64, 0][:len(ms)]
    s = Setup(M, ctxs, D=D, page=32, gaps=opt.pop("gaps", False), seed=sum(ms) + G + D)
    o = check_attention(M, s, ms, G=G, **opt)
    check_observe(M, s, o, row_weight=[float(i % 2) for i in range(sum(ms))])


@pytest.mark.parametrize("m,G", [(1, 1), (12, 1), (25, 4), (64, 5)])
def test_a_long_context_against_64_bits_on_the_gpu(M, m, G):
    """Enough keys that a warp walks many records: 131149 keys, 8 kv heads."""
    D, hkv, ctx = 64, 8 if m * G > 64 else 32, 131149
    g = torch.Generator(device="cuda").manual_seed(m)
    c = M.KV4Cache(np.arange(-(-ctx // 128))[None][:, ::-1], -(-ctx // 128), hkv, D, 128)
    K = torch.randn(ctx, hkv, D, generator=g, device="cuda").bfloat16()
    V = torch.randn(ctx, hkv, D, generator=g, device="cuda").bfloat16()
    q = (1.5 * torch.randn(m, hkv * G, D, generator=g, device="cuda")).bfloat16()
    keys, rows = M.RequestRows([0, ctx]), M.RequestRows([0, m])
    c.append(K, V, keys)
    out, lse = c.attend(q, rows)
    w = c.observe(q, lse, rows, out=torch.zeros_like(c.weight))
    assert c.status() == 0
    for h in range(0, hkv, 5):
        kd, vd = ref.values(K[:, h].double()), ref.values(V[:, h].double())
        want_w = torch.zeros(ctx, dtype=torch.float64, device="cuda")
        for hq in range(h * G, h * G + G):
            z = q[:, hq].double() @ kd.T / math.sqrt(D)
            l = torch.logsumexp(z, 1)
            p = torch.exp(z - l[:, None])
            o = p @ vd
            want_w += torch.exp(z - lse[:, hq].double()[:, None]).sum(0)
            assert ((lse[:, hq].double() - l).abs() <= 2.0 ** -16).all()
            # the softmax weights' 11 bits, over many keys: 2^-12 of the norm of p v
            tol = H * o.abs() + 4 * 2.0 ** -12 * (p ** 2 @ vd ** 2).sqrt() + 2.0 ** -16
            assert ((out[:, hq].double() - o).abs() <= tol).all()
        assert ((w[0, h, :ctx].double() - want_w).abs() <= 2.0 ** -15 * want_w).all()


@pytest.mark.parametrize("m,G", [(4, 2), (16, 4), (20, 4), (64, 4)])
def test_a_bad_own_value_shows_only_where_it_is_seen(M, m, G):
    s = Setup(M, [200], seed=m)
    q, k, v = dev(rnd(s.g, m, 2 * G, 128)), dev(rnd(s.g, m, 2, 128)), dev(rnd(s.g, m, 2, 128))
    rows = M.RequestRows([0, m])
    anc = [1 << i | 1 for i in range(m)]  # a star: everyone sees the root and itself
    good, _ = s.cache.attend(q, rows, k, v, anc=signed(anc))
    v[2, 1, 7] = math.nan
    v[3, 0, 100] = math.inf
    out, lse = s.cache.attend(q, rows, k, v, anc=signed(anc))
    torch.cuda.synchronize()
    bad = torch.zeros(m, 2 * G, dtype=torch.bool, device="cuda")
    bad[2, G:], bad[3, :G] = True, True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(out[~bad], good[~bad]) and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("ms,G", [([1, 1, 1], 4), ([8, 3, 16], 4), ([40, 2, 64], 4), ([64, 64, 5], 2)])
def test_the_same_bits_from_cold_and_warm_caches(M, ms, G):
    s = Setup(M, [1500, 260, 77], page=32, seed=33)
    n = sum(ms)
    q, k, v = dev(1.5 * rnd(s.g, n, 2 * G, 128)), dev(rnd(s.g, n, 2, 128)), dev(rnd(s.g, n, 2, 128))
    rows = M.RequestRows(np.cumsum([0] + ms))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    want = s.cache.attend(q, rows, k, v)
    w = s.cache.observe(q, want[1], rows, out=torch.zeros_like(s.cache.weight))
    for i in range(60):
        if i % 2:
            flush.zero_()
        out, lse = s.cache.attend(q, rows, k, v)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        if i % 4 == 0:
            assert torch.equal(w, s.cache.observe(q, lse, rows, out=torch.zeros_like(w)))
    assert s.cache.status() == 0


@pytest.mark.parametrize("ms", [[1, 1], [40, 64]])
def test_a_bad_page_leaves_the_other_requests_alone(M, ms):
    s = Setup(M, [300, 90], page=32, seed=17)
    q = dev(rnd(s.g, sum(ms), 8, 128))
    rows = M.RequestRows(np.cumsum([0] + ms))
    good, lse = s.cache.attend(q, rows)
    s.cache.page_table[0, 4] = -1
    out, _ = s.cache.attend(q, rows)
    assert s.cache.status() == 7
    assert torch.equal(out[ms[0]:], good[ms[0]:]) and torch.isfinite(out).all()
    s.cache.observe(q, lse, rows)
    assert s.cache.status() == 7


def test_the_serving_loop_example_runs(M):
    import os
    import runpy
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = runpy.run_path(os.path.join(root, "examples", "kv4_serving.py"))["main"](steps=12, seed=1, quiet=True)
    assert r["status"] == 0 and r["evictions"] > 0 and max(r["ctx"]) <= r["limit"]
    # against attention over the same keys in bf16: what 4 bits cost
    assert r["error"] < 0.2

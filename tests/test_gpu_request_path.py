"""A request from its prompt to its accepted tokens, by the operators in a row:
rotary positions, attention over the packed prompts, the prompts' keys into the
4-bit cache, a draft tree's rows turned and attended over it, tokens sampled, the
accepted path, its rows stored.  Each stage is compared with its definition in 64 bits on
what the stage before it gave, and the whole is captured and replayed.

Tolerances: of rotary positions, prompts and samples as in request_ref; of the cache's
attention an output is rounded to bf16 (2^-8 of its value), weights enter as two bf16
terms (2^-15 of the greatest value), scores carry a dot product of D terms in fp32."""
import math

import numpy as np
import pytest
import torch

import kv4_ref
import request_ref as ref

pytestmark = pytest.mark.gpu

HQ, HKV, VOCAB, NODES = 8, 2, 97, 7
PARENTS = [-1, 0, 0, 1, 1, 2, 5]
DEPTH = [0, 1, 1, 2, 2, 2, 3]


@pytest.fixture(scope="module")
def M():
    from speculative_decoding_tree_bit_gb300 import model
    return model


class Layer:
    """One attention layer and a head of random weights, and what a call of the path needs."""

    def __init__(self, M, lengths, d, seed):
        self.M, self.lengths, self.d, self.R = M, lengths, d, len(lengths)
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
        n, t = sum(lengths), self.R * NODES
        self.prompt, self.draft = rnd(n, HQ + 2 * HKV, d), rnd(t, HQ + 2 * HKV, d)
        self.head = rnd(HQ * d, VOCAB)
        self.u = torch.rand(t, generator=g).cuda()
        self.rope = M.Rope(d, base=1e4, scaling=M.RopeScaling.ramp(2.0, 64))
        self.attention = M.PromptAttention(HQ, HKV, d)
        self.score = M.KV4Score(softcap=30.0)
        self.rows = M.RequestRows(np.cumsum([0] + lengths))
        self.tree = M.RequestRows(np.arange(self.R + 1) * NODES)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.pos = i32([i for m in lengths for i in range(m)])
        self.draft_pos = i32([m + x for m in lengths for x in DEPTH])
        anc = []
        for i, p in enumerate(PARENTS):
            anc.append((anc[p] if i else 0) | 1 << i)
        self.bits = anc
        self.anc = torch.tensor(anc * self.R).cuda()
        self.tokens, self.parents = i32([[0] + [int(x) for x in torch.randint(0, 4, (NODES - 1,), generator=g)] for _ in range(self.R)]), i32(PARENTS)
        pages = -(-(max(lengths) + NODES) // 32)
        self.cache = M.KV4Cache(np.arange(self.R * pages).reshape(self.R, pages), self.R * pages, HKV, d, 32)
        self.status = i32([0])

    def accept(self, drawn):
        """The walk of each request's tree; src and count as KV4Cache.append takes them."""
        from speculative_decoding_tree_bit_gb300 import check, lib, stream_ptr
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        length, bonus, path, toks, src = z(self.R), z(self.R), z(self.R, 65), z(self.R, NODES), z(self.R * NODES)
        for r in range(self.R):
            check(lib().sd_accept(self.tokens[r].data_ptr(), self.parents.data_ptr(), drawn[r * NODES:].data_ptr(), NODES,
                                  length[r:].data_ptr(), toks[r].data_ptr(), bonus[r:].data_ptr(), path[r].data_ptr(),
                                  self.status.data_ptr(), stream_ptr()))
            src[r * NODES:(r + 1) * NODES] = path[r, :NODES].clamp(0, NODES - 1) + r * NODES
        return length + 1, src, bonus

    def __call__(self):
        """From the projections to the accepted rows' place in the cache."""
        r = {}
        x = r["prompt"] = self.prompt.clone()  # turned in place, as a projection leaves it
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        self.rope(q, k, self.pos, q_out=q, k_out=k)
        r["out"], r["lse"] = self.attention(q, k, v, self.rows, score=self.score)
        self.cache.append(k, v, self.rows, pos=self.pos, at=0)
        y = r["draft"] = self.draft.clone()
        q, k, v = y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]
        self.rope(q, k, self.draft_pos, q_out=q, k_out=k)
        r["tree"], _ = self.cache.attend(q, self.tree, k, v, anc=self.anc, pos=self.draft_pos, score=self.score)
        r["logits"] = 0.05 * (r["tree"].flatten(1) @ self.head)
        r["logits"][:, 4:] -= 3.0  # the drafts' tokens are likely ones
        r.update(self.M.sample(r["logits"], self.u, temperature=0.8, top_p=0.95))
        r["count"], r["src"], r["bonus"] = self.accept(r["tokens"])
        self.cache.append(k, v, self.tree, pos=self.draft_pos[r["src"].long()].contiguous(), src=r["src"], count=r["count"])
        return r


def host(t):
    return t.cpu().double()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[70, 1, 33], [1], [200, 129]])
def test_from_prompt_to_accepted_rows(M, lengths, d):
    s = Layer(M, lengths, d, seed=sum(lengths) + d)
    r = s()
    torch.cuda.synchronize()
    assert s.attention.status() == 0 and s.cache.status() == 0 and s.status.item() == 0

    # rotary positions, in place beside values that stay
    freq, amplitude = ref.frequencies(d, 1e4, "ramp", 2.0, 64.0, 1.0, 32.0), 0.1 * math.log(2.0) + 1.0
    for x, y, pos in ((s.prompt, r["prompt"], s.pos), (s.draft, r["draft"], s.draft_pos)):
        want, slack = ref.rotate(host(x)[:, :HQ + HKV], pos.cpu(), freq, amplitude)
        err = (host(y)[:, :HQ + HKV] - want).abs()
        assert (err <= ref.BF16 * want.abs() + 2 * slack).all()  # the slack is rounded with the value
        assert torch.equal(x[:, HQ + HKV:], y[:, HQ + HKV:])

    # attention over the prompts
    q, k, v = (host(r["prompt"])[:, a:b] for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    want, lse, tol, tol_lse = ref.attend(q, k, v, s.rows.cu, s.rows.cu, cap=30.0)
    assert ((host(r["out"]) - want).abs() <= tol).all() and ((host(r["lse"]) - lse).abs() <= tol_lse).all()

    # the tree's rows over the cached prompt and their ancestors
    held_k, held_v = kv4_ref.values(k), kv4_ref.values(v)
    tq, tk, tv = (host(r["draft"])[:, a:b] for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    for i in range(s.R * NODES):
        b, node = divmod(i, NODES)
        own = [b * NODES + j for j in range(NODES) if s.bits[node] >> j & 1]
        a, e = int(s.rows.cu[b]), int(s.rows.cu[b + 1])
        K, V = torch.cat([held_k[a:e], tk[own]]), torch.cat([held_v[a:e], tv[own]])
        for h in range(HQ):
            z = K[:, h // (HQ // HKV)] @ tq[i, h] / math.sqrt(d)
            size = float((K[:, h // (HQ // HKV)].abs() @ tq[i, h].abs()).max()) / math.sqrt(d)
            want = torch.softmax(30.0 * torch.tanh(z / 30.0), 0) @ V[:, h // (HQ // HKV)]
            eps = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20 * (1 + 30.0 / 8)
            off = (host(r["tree"][i, h]) - want).abs()
            assert (off <= 2.0 ** -8 * want.abs() + (2.0 ** -15 + 2 * eps) * float(V.abs().max())).all()

    # the tokens, and the path that they accept
    drawn = []
    t, p = (torch.tensor(x, dtype=torch.float32).item() for x in (0.8, 0.95))
    for i, row in enumerate(host(r["logits"])):
        token, logprob, kept = ref.sample_row(row, s.u[i].item(), t, 0, p)
        assert (r["tokens"][i].item(), r["kept"][i].item()) == (token, kept)
        drawn.append(token)
    for b in range(s.R):
        ok = [True] * NODES
        for j in range(1, NODES):
            ok[j] = ok[PARENTS[j]] and s.tokens[b, j].item() == drawn[b * NODES + PARENTS[j]]
        best = max((j for j in range(NODES) if ok[j]), key=lambda j: (DEPTH[j], -j))
        path = [j for j in range(NODES) if s.bits[best] >> j & 1]
        count = r["count"][b].item()
        assert count == len(path) and r["bonus"][b].item() == drawn[b * NODES + best]
        assert r["src"][b * NODES:b * NODES + count].tolist() == [b * NODES + j for j in path]
        assert s.cache.ctx_len[b].item() == lengths[b] + count

    # what the cache holds of the accepted rows
    kept = M.RequestRows(np.cumsum([0] + [lengths[b] + r["count"][b].item() for b in range(s.R)]))
    got_k, _ = s.cache.read(kept)
    for b in range(s.R):
        path = r["src"][b * NODES:b * NODES + r["count"][b].item()].cpu().long()
        a, e = int(kept.cu[b]) + lengths[b], int(kept.cu[b + 1])
        want = kv4_ref.values(tk[path])
        assert ((host(got_k)[a:e] - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -130).all()


def test_a_prompt_in_chunks_is_the_whole(M):
    """Three chunks, each over all keys so far, against one call; then one token at a time."""
    s = Layer(M, [150, 40], 128, seed=5)
    q, k, v = (s.prompt[:, a:b].contiguous() for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
    q, k = s.rope(q, k, s.pos)
    f = lambda t: t.cpu().double()  # noqa: E731
    want, lse, tol, tol_lse = ref.attend(f(q), f(k), f(v), s.rows.cu, s.rows.cu)
    ends = [(0, 0), (64, 7), (149, 39), (150, 40)]
    for (a0, a1), (b0, b1) in zip(ends[:-1], ends[1:]):
        at = torch.cat([torch.arange(a0, b0), 150 + torch.arange(a1, b1)])
        keys = torch.cat([torch.arange(0, b0), 150 + torch.arange(0, b1)])
        out, l = s.attention(q[at.cuda()], k[keys.cuda()], v[keys.cuda()], M.RequestRows(np.array([0, b0 - a0, b0 - a0 + b1 - a1])),
                             M.RequestRows(np.array([0, b0, b0 + b1])))
        assert ((f(out) - want[at]).abs() <= tol[at]).all() and ((f(l) - lse[at]).abs() <= tol_lse[at]).all()
    assert s.attention.status() == 0


def test_the_path_in_a_graph(M):
    """Captured once, replayed on other inputs: the same bits as the calls by themselves."""
    s = Layer(M, [90, 31], 64, seed=8)
    s()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = s()
    for seed in (1, 2):
        other = Layer(M, [90, 31], 64, seed=seed)
        for a in ("prompt", "draft", "head", "u", "tokens"):
            getattr(s, a).copy_(getattr(other, a))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: x.clone() for n, x in held.items()}
        ctx = s.cache.ctx_len.clone()
        want = s()
        for n in want:
            assert torch.equal(got[n], want[n]), n
        assert torch.equal(ctx, s.cache.ctx_len)
    assert s.attention.status() == 0 and s.cache.status() == 0 and s.status.item() == 0


def test_the_readme_s_prompt(M):
    """Slices of one projection, turned in place, attended and stored; k turned into a tensor of its own is refused
    beside a slice of v, and taken with a v of its own."""
    m, d = [70, 9], 128
    qkv = torch.randn(79, HQ + 2 * HKV, d, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    kept = qkv.clone()
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    pos = torch.tensor([i for n in m for i in range(n)], dtype=torch.int32).cuda()
    rope, prompts, attention = M.Rope(d), M.RequestRows(np.cumsum([0] + m)), M.PromptAttention(HQ, HKV, d)
    cache = M.KV4Cache(np.arange(6).reshape(2, 3), 6, HKV, d, 32)
    rope(q, k, pos, q_out=q, k_out=k)
    out, lse = attention(q, k, v, prompts)
    cache.append(k, v, prompts)
    q2, k2 = rope(kept[:, :HQ], kept[:, HQ:HQ + HKV], pos)
    assert torch.equal(q2, q) and torch.equal(k2, k)
    with pytest.raises(ValueError, match="one row stride"):
        attention(q2, k2, v, prompts)
    again, lse2 = attention(q2, k2, v.contiguous(), prompts)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    assert cache.ctx_len.tolist() == m and attention.status() == 0 and cache.status() == 0

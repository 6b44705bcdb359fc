"""The 4-bit key/value cache in a serving loop: one attention layer, a batch
of requests, draft trees verified step by step.

Each step attends the trees' nodes over the cache and their own keys, walks the
accepted path (the library's sd_accept, on random target tokens here), stores
the accepted rows' keys and values in 4 bits, adds the weight that those rows
gave to the cached keys, and brings requests that grew past a limit back to a
budget, into the pages of a second cache.

    python examples/kv4_serving.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_tree_bit_gb300 import check, lib, stream_ptr  # noqa: E402
from speculative_decoding_tree_bit_gb300 import model as sdv  # noqa: E402

HQ, HKV, D = 32, 8, 128


def tree_masks(parents, cu):
    """Ancestor bits and depths of every request's tree (sd_tree_info)."""
    n = parents.numel()
    anc = torch.empty(n, dtype=torch.int64, device="cuda")
    depth, pos = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for a, b in zip(cu[:-1], cu[1:]):
        check(lib().sd_tree_info(parents[a:].data_ptr(), int(b - a), 0, anc[a:].data_ptr(), depth[a:].data_ptr(),
                                 pos[a:].data_ptr(), status.data_ptr(), stream_ptr()))
    return anc, depth


def accept(tokens, parents, argmax, cu):
    """Per request: accepted rows (root included) and their node ids, laid
    out as `src` of KV4Cache.append (sd_accept)."""
    R, n, dev = len(cu) - 1, tokens.numel(), "cuda"
    length = torch.zeros(R, dtype=torch.int32, device=dev)
    toks, bonus = torch.zeros(n, dtype=torch.int32, device=dev), torch.zeros(R, dtype=torch.int32, device=dev)
    path = torch.zeros(R, 65, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    src = torch.zeros(n, dtype=torch.int32, device=dev)
    for r in range(R):
        a, m = int(cu[r]), int(cu[r + 1] - cu[r])
        check(lib().sd_accept(tokens[a:].data_ptr(), parents[a:].data_ptr(), argmax[a:].data_ptr(), m,
                              length[r:].data_ptr(), toks[a:].data_ptr(), bonus[r:].data_ptr(), path[r].data_ptr(),
                              status.data_ptr(), stream_ptr()))
        src[a:a + m] = path[r, :m].clamp(0, m - 1) + a
    return length + 1, src


def main(steps=40, R=4, nodes=16, prompt=300, limit=340, budget=256, seed=0, quiet=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    new = lambda n: torch.randn(n, HKV, D, generator=g, device="cuda").bfloat16()  # noqa: E731
    pages = -(-(limit + nodes) // 64)
    caches = [sdv.KV4Cache(np.arange(R * pages).reshape(R, pages), R * pages, HKV, D, 64) for _ in range(2)]
    cache, spare = caches
    score = sdv.KV4Score(softcap=50.0)

    lengths = [prompt - 17 * r for r in range(R)]
    rows = sdv.RequestRows(np.cumsum([0] + lengths))
    K, V = new(rows.n), new(rows.n)
    cache.append(K, V, rows)
    # the same keys in bf16, for the comparison at the end
    bf16 = [[(K[a:b], V[a:b])] for a, b in zip(rows.cu[:-1], rows.cu[1:])]

    cu = np.arange(R + 1) * nodes
    tree = sdv.RequestRows(cu)
    parents = np.concatenate([[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, nodes)] for _ in range(R)])
    parents = torch.from_numpy(parents.astype(np.int32)).cuda()
    anc, depth = tree_masks(parents, cu)
    next_pos = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ctx, evictions, error = list(lengths), 0, 0.0
    for step in range(steps):
        q = (1.5 * torch.randn(R * nodes, HQ, D, generator=g, device="cuda")).bfloat16()
        k, v = new(R * nodes), new(R * nodes)
        pos = (next_pos.repeat_interleave(nodes) + depth).to(torch.int32)
        out, lse = cache.attend(q, tree, k, v, anc=anc, pos=pos, score=score)
        if step == 0:
            error = _against_bf16(q, k, v, out, anc, bf16, nodes, score)
        # a random target: half of the drafts come true
        tokens = torch.randint(0, 2, (R * nodes,), generator=g, device="cuda", dtype=torch.int32)
        argmax = torch.randint(0, 2, (R * nodes,), generator=g, device="cuda", dtype=torch.int32)
        count, src = accept(tokens, parents, argmax, cu)
        # accepted rows: their weight counts, their keys and values stay
        first = torch.arange(nodes, device="cuda").repeat(R) < count.repeat_interleave(nodes)
        weight = torch.zeros(R * nodes, device="cuda").index_fill_(0, src[first].long(), 1.0)
        cache.observe(q, lse, tree, pos=pos, row_weight=weight, score=score, decay=0.95)
        cache.append(k, v, tree, pos=pos[src.long()].contiguous(), src=src, count=count)
        next_pos += count
        ctx = cache.ctx_len.tolist()
        if max(ctx) + nodes > limit:
            cache.evict(spare, budget, recent=64, sinks=4)
            cache, spare = spare, cache
            ctx, evictions = cache.ctx_len.tolist(), evictions + 1
        if not quiet:
            print(f"step {step}: accepted {count.tolist()}, cached {ctx}")
    torch.cuda.synchronize()
    status = caches[0].status() or caches[1].status()
    if not quiet:
        print(f"{evictions} evictions, status {status}, first step off bf16 attention by {error:.3f} of its norm")
    return {"status": status, "evictions": evictions, "ctx": ctx, "limit": limit, "error": error}


def _against_bf16(q, k, v, out, anc, held, nodes, score):
    off = norm = 0.0
    for r, parts in enumerate(held):
        a = r * nodes
        K = torch.cat([p[0] for p in parts] + [k[a:a + nodes]]).float()
        V = torch.cat([p[1] for p in parts] + [v[a:a + nodes]]).float()
        own = (anc[a:a + nodes, None] >> torch.arange(nodes, device="cuda")) & 1
        sees = torch.cat([torch.ones(nodes, K.shape[0] - nodes, device="cuda"), own], 1) > 0
        for h in range(HQ):
            z = q[a:a + nodes, h].float() @ K[:, h // (HQ // HKV)].T / D ** 0.5
            z = score.args.softcap * torch.tanh(z / score.args.softcap)
            want = torch.softmax(z.masked_fill(~sees, -torch.inf), 1) @ V[:, h // (HQ // HKV)]
            off += float((out[a:a + nodes, h].float() - want).square().sum())
            norm += float(want.square().sum())
    return (off / norm) ** 0.5


if __name__ == "__main__":
    main()

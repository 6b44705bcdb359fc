"""Cases of the 4-bit key/value cache: storing rows, attention over them, the
attention weight that each key collects, and eviction by that weight.

The cache holds every key and value row (one token, one kv head) as 4-bit codes
with a scale s and a middle m, both bf16: value = s * (code - 8) + m.  With lo
and hi the row's least and greatest value, s = bf16((hi - lo) / 15), m =
bf16(lo + 8 s) and code = round_half_even((x - m) / s) + 8 clamped to 0..15;
where s is 0 the code is 8 and m = bf16(lo).

A request holds ctx keys; its rows (draft-tree nodes, chain tokens, or a single
token) see the cached keys and, among their own bf16 keys, their ancestors.
score = cap * tanh(q.k * scale / cap) + slope * (position of k - position of q),
cap and slope optional; a key is visible when it lies in the request's document
(position >= start) and less than `window` positions back.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases --

def _case(name, op, **kw):
    c = dict(name=name, op=op, R=1, m=1, chain=False, hq=32, hkv=8, d=128, lo=1, hi=1, page=64, cap=0.0, alibi=False,
             window=0, docs=False, own_keys=True, gaps=False, decay=1.0, budget=0, recent=0, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # what a batched verify step commits: 32 requests, up to 8 accepted rows each
        _case("append_batch_32x8", "append", R=32, m=8, chain=True, lo=1024, hi=4096),
        # a prompt's keys and values stored at once
        _case("append_prompt_16384", "append", R=1, m=16384, chain=True, lo=0, hi=0),
        # one request, one token, a short context: latency
        _case("token_1x331", "attend", R=1, m=1, lo=331, hi=331),
        # the decode step of a batch: one token for each request, ragged contexts
        _case("tokens_32x8k", "attend", R=32, m=1, lo=1500, hi=8192),
        # the 8B-class decoder's draft tree of 16 nodes over 2048 keys
        _case("tree16_2k", "attend", R=1, m=16, lo=2048, hi=2048),
        # the batched step: 32 requests, chains of 8 rows, capped scores
        _case("chains_32x8_4k_cap", "attend", R=32, m=8, chain=True, lo=1024, hi=4096, cap=50.0),
        # the 27B-class decoder's tree of 64 nodes over a long context
        _case("tree64_128k", "attend", R=1, m=64, hq=40, hkv=8, lo=131072, hi=131072, page=128),
        # heads of their own with distance slopes, a sliding window and packed documents, after evictions
        _case("window_4x5_mha64", "attend", R=4, m=5, hq=16, hkv=16, d=64, lo=700, hi=5001, page=32, alibi=True,
              window=1024, docs=True, gaps=True),
        # the weights that a verified tree's rows give to the keys of one request
        _case("weights_tree16_2k", "observe", R=1, m=16, lo=2048, hi=2048),
        # the same for a batch's accepted rows, older weight fading
        _case("weights_32x5_8k", "observe", R=32, m=5, lo=1500, hi=8192, decay=0.9, gaps=True),
        # one request brought back to 1024 keys
        _case("evict_1x2304_1024", "evict", R=1, lo=2304, hi=2304, budget=1024, recent=256, sinks=4, gaps=True),
        # a batch of long requests brought back to 2048 keys
        _case("evict_16x16k_2048", "evict", R=16, lo=5000, hi=16384, budget=2048, recent=512, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "observe", "evict"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    page = rng.choice([32, 64, 96, 128])
    R = _log(rng, 1, 32)
    if op == "append":
        m = _log(rng, 1, max(1, 16384 // R))
        lo = _log(rng, 1, 4096)
        return _case("", op, R=R, m=m, chain=True, hq=hkv, hkv=min(hkv, 8), d=d, lo=lo, hi=lo + _log(rng, 1, 1000),
                     page=page, gaps=rng.random() < 0.3)
    hi = _log(rng, 1, 131072 // R if op == "attend" else 16384)
    if op == "attend" and R == 1 and rng.random() < 0.15:
        hi = 131072 - rng.randrange(1000)
    lo = int(hi * rng.uniform(0.0, 1.0))
    # no dearer than the largest listed case: rows x heads x keys
    m = max(1, min(64, 40 * 64 * 131072 // (R * hq * max(hi, 1024)), _log(rng, 1, 64)))
    bias = dict(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                window=rng.choice([0, 0, 0, _log(rng, 2, 8192)]), docs=rng.random() < 0.25, gaps=rng.random() < 0.3)
    shape = dict(R=R, m=m, chain=rng.random() < 0.4, hq=hq, hkv=hkv, d=d, lo=lo, hi=hi, page=page)
    if op == "attend":
        return _case("", op, own_keys=rng.random() < 0.85, **shape, **bias)
    if op == "observe":
        shape["m"] = min(m, 16)
        return _case("", op, decay=rng.choice([1.0, 0.9, 0.5]), **shape, **bias)
    budget = _log(rng, 16, 4096)
    recent = rng.randrange(0, budget // 2)
    shape.update(R=min(R, 16), m=1, hkv=min(hkv, 8), hq=min(hkv, 8))
    return _case("", op, budget=budget, recent=recent, sinks=rng.randrange(0, min(8, budget - recent)),
                 gaps=bias["gaps"], **shape)


def _spread(lo, hi, n):
    """n whole numbers over lo..hi, the first one hi: the same for every seed."""
    return [hi - int((hi - lo) * ((i * 0.6180339887) % 1.0)) for i in range(n)]


def _sizes(c):
    """(keys held, rows) of each request."""
    return _spread(c["lo"], c["hi"], c["R"]), _spread(max(1, c["m"] // 2), c["m"], c["R"])


# ------------------------------------------------------------------ inputs --

def _inputs(c, seed):
    """The tensors of a case from its seed: bf16 keys, values and queries, trees, positions, weights."""
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    ctx, rows = _sizes(c)
    R, C, n = c["R"], max(max(ctx), 1), sum(rows)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    mean, spread = 0.5 * normal(hkv, d), 0.5 + torch.rand(hkv, d, device="cuda", generator=g)  # keys' channels differ
    x = {"ctx": ctx, "rows": rows, "C": C, "n": n}
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    x["cu"] = cu
    step = torch.ones(R, C, dtype=torch.int64, device="cuda")
    if c["gaps"]:  # positions that eviction left
        step += (torch.rand(R, C, device="cuda", generator=g) < 0.4) * torch.randint(1, 9, (R, C), device="cuda", generator=g)
    pos = torch.cumsum(step, 1) - step[:, :1]
    x["pos"] = pos.to(torch.int32)                                   # [R][C] position of the cached keys
    ctx_t = torch.tensor(ctx, device="cuda")
    after = torch.where(ctx_t > 0, pos.gather(1, (ctx_t - 1).clamp(min=0)[:, None])[:, 0] + 1, 0)
    if c["op"] != "append":
        x["K"] = (normal(R, C, hkv, d) * spread + mean).bfloat16()   # [R][C][hkv][d]
        x["V"] = normal(R, C, hkv, d).bfloat16()
    if c["op"] != "evict":
        x["k"] = (normal(n, hkv, d) * spread + mean).bfloat16()      # the rows' own keys and values
        x["v"] = normal(n, hkv, d).bfloat16()
    # trees: parents of random earlier nodes, or chains
    local = torch.cat([torch.arange(r) for r in rows])
    if c["op"] in ("attend", "observe"):
        x["q"] = (1.5 * normal(n, hq, d)).bfloat16()
        anc, depth = [], []
        for r, m in enumerate(rows):
            pick = torch.rand(m, generator=torch.Generator().manual_seed(seed * 131 + r)).tolist()
            bits, deep = [], []
            for i in range(m):
                p = i - 1 if c["chain"] or i == 0 else int(pick[i] * i)
                bits.append((bits[p] if i else 0) | (1 << i))
                deep.append(deep[p] + 1 if i else 0)
            anc += [b - (1 << 64) if b >> 63 else b for b in bits]
            depth += deep
        x["anc"] = torch.tensor(anc, dtype=torch.int64, device="cuda")
        local = torch.tensor(depth)
    req = torch.repeat_interleave(torch.arange(R), torch.tensor(rows))
    x["req"] = req.cuda()
    x["at"] = torch.cat([torch.arange(r) for r in rows]).cuda()
    x["row_pos"] = (after[x["req"]] + local.cuda()).to(torch.int32)  # [n] position of the rows
    if c["alibi"]:
        x["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq).float()
    if c["docs"]:
        x["start"] = (pos.gather(1, ctx_t[:, None] // 3)[:, 0]).to(torch.int32)
    if c["op"] in ("observe", "evict"):
        x["weight"] = torch.rand(R, hkv, C, device="cuda", generator=g) ** 8 * 4   # few keys hold most of it
        x["weight"] *= torch.arange(C, device="cuda")[None, None] < ctx_t[:, None, None]
    if c["op"] == "observe":
        x["row_weight"] = (torch.rand(n, device="cuda", generator=g) < 0.7).float()  # accepted rows count
        x["row_weight"][torch.tensor(cu[:-1], device="cuda")] = 1.0
    return x


def _slots(c, keys):
    return -(-keys // c["page"]) * c["page"]


def _held(rows):
    """The 4-bit form of bf16 rows: codes (two a byte), (scale, middle)."""
    x = rows.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).bfloat16().float()
    m = (lo + 8 * s).bfloat16().float()
    code = torch.where(s > 0, torch.round((x - m) / s) + 8, 8).clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.cat([s, m], -1).bfloat16()


def _value(code, sm):
    c = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    s, m = sm[..., :1].float(), sm[..., 1:].float()
    return s * (c.float() - 8) + m


# ------------------------------------------------------------------ passes --

def prepare(case, seed):
    c, x = case, _inputs(case, seed)
    st = _given(c, x)
    ctx = st["ctx"]
    most = x["C"] + (max(x["rows"]) if c["op"] == "append" else 0)
    st["keep"] = [min(k, c["budget"]) for k in x["ctx"]]
    st["kept"] = (torch.repeat_interleave(torch.arange(c["R"]), torch.tensor(st["keep"])).cuda(),
                  torch.cat([torch.arange(k) for k in st["keep"]]).cuda())
    if c["op"] == "observe":
        st["lse"] = _lse(c, x)
    if own:
        from speculative_decoding_tree_bit_gb300 import model as sdv
        pages = -(-most // c["page"])
        table = torch.randperm(c["R"] * pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        cache = sdv.KV4Cache(table.reshape(c["R"], pages).numpy(), c["R"] * pages, c["hkv"], c["d"], c["page"])
        if c["op"] != "append":
            keys = sdv.RequestRows(torch.tensor([0] + x["ctx"]).cumsum(0).numpy())
            held = torch.arange(x["C"], device="cuda")[None] < ctx[:, None]
            cache.append(x["K"][held], x["V"][held], keys, pos=x["pos"][held])
            if x.get("weight") is not None:
                cache.weight[:, :, :x["C"]] = x["weight"]
        st["cache"], st["rows"] = cache, sdv.RequestRows(x["cu"])
        if c["op"] in ("attend", "observe"):
            st["score"] = sdv.KV4Score(softcap=c["cap"], slopes=st["slopes"], window=c["window"], start=st["start"])
        if c["op"] == "observe":
            st["out"] = torch.zeros_like(cache.weight)
        if c["op"] == "evict":
            pages = -(-c["budget"] // c["page"])
            table = torch.arange(c["R"] * pages, dtype=torch.int32).flip(0).reshape(c["R"], pages)
            st["dst"] = sdv.KV4Cache(table.numpy(), c["R"] * pages, c["hkv"], c["d"], c["page"])
            st["rows"] = sdv.RequestRows(torch.tensor([0] + st["keep"]).cumsum(0).numpy())
    elif c["op"] != "append":
        _plain_cache(st, x)
    return st


def _given(c, x):
    st = {"c": c, "req": x["req"], "at": x["at"], "row_pos": x["row_pos"], "m": max(x["rows"])}
    for name in ("q", "k", "v", "anc", "slopes", "start", "weight", "row_weight"):
        st[name] = x.get(name)
    st["ctx"] = torch.tensor(x["ctx"], dtype=torch.int32, device="cuda")
    st["cap"] = _slots(c, x["C"] + (max(x["rows"]) if c["op"] == "append" else 0))
    st["pos"] = x["pos"][:, None].expand(-1, c["hkv"], -1).contiguous()
    st["scale"] = 1.0 / math.sqrt(c["d"])
    return st


def _lse(c, x):
    """The rows' log-sum-exp that the weights' case takes as an input."""
    return _plain_attend(_plain_cache(_given(c, x), x), lse_only=True)


def _plain_cache(st, x):
    st["kc"], st["ks"] = _held(x["K"])
    st["vc"], st["vs"] = _held(x["V"])
    return st


def run(state):
    return {"append": _append, "attend": _attend, "observe": _observe, "evict": _evict}[state["c"]["op"]](state)


def _append(st):
    if own:
        cache = st["cache"]
        cache.append(st["k"], st["v"], st["rows"], pos=st["row_pos"], at=st["ctx"])
        k, v = cache.read(st["rows"], at=st["ctx"])
        return {"k": k, "v": v, "ctx": cache.ctx_len, "pos": cache.pos}
    c = st["c"]
    k, v = _value(*_held(st["k"])).bfloat16(), _value(*_held(st["v"])).bfloat16()
    count = torch.zeros(c["R"], dtype=torch.int32, device="cuda").index_add_(
        0, st["req"], torch.ones_like(st["req"], dtype=torch.int32))
    pos = torch.zeros(c["R"], c["hkv"], st["cap"], dtype=torch.int32, device="cuda")
    pos[st["req"], :, st["ctx"].long()[st["req"]] + st["at"]] = st["row_pos"][:, None]
    return {"k": k, "v": v, "ctx": st["ctx"] + count, "pos": pos}


def _grouped(st, t):
    """Rows [n][heads][d] laid out by request and kv head, in 32 bits: [R][hkv][group][m][d]."""
    c = st["c"]
    out = torch.zeros(c["R"], st["m"], *t.shape[1:], device="cuda")
    out[st["req"], st["at"]] = t.float()
    return out.reshape(c["R"], st["m"], c["hkv"], -1, *t.shape[2:]).permute(0, 2, 3, 1, *range(4, t.dim() + 2))


def _scores(st, q, k, k_pos):
    """Capped and biased scores [R][hkv][group][m][keys], -inf where the window or the document hides a key."""
    c = st["c"]
    s = (q @ k[:, :, None].transpose(-1, -2)) * st["scale"]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    q_pos = torch.zeros(c["R"], st["m"], dtype=torch.int32, device="cuda")
    q_pos[st["req"], st["at"]] = st["row_pos"]
    back = (q_pos[:, None, None, :, None] - k_pos[:, :, None, None, :])
    if st["slopes"] is not None:
        s = s - st["slopes"].reshape(1, c["hkv"], -1, 1, 1) * back.float()
    if c["window"]:
        s = s.masked_fill(back >= c["window"], -math.inf)
    if st["start"] is not None:
        s = s.masked_fill(k_pos[:, :, None, None, :] < st["start"][:, None, None, None, None], -math.inf)
    return s


def _plain_attend(st, lse_only=False):
    c = st["c"]
    q = _grouped(st, st["q"])
    k = _value(st["kc"], st["ks"]).transpose(1, 2)
    s = _scores(st, q, k, st["pos"])
    held = torch.arange(k.shape[2], device="cuda")[None] < st["ctx"][:, None]
    s = s.masked_fill(~held[:, None, None, None], -math.inf)
    if c["own_keys"]:
        k2 = _grouped(st, st["k"])[:, :, 0]
        p2 = torch.zeros(c["R"], st["m"], dtype=torch.int32, device="cuda")
        p2[st["req"], st["at"]] = st["row_pos"]
        s2 = _scores(st, q, k2, p2[:, None].expand(-1, c["hkv"], -1))
        anc = torch.zeros(c["R"], st["m"], dtype=torch.int64, device="cuda")
        anc[st["req"], st["at"]] = st["anc"]
        sees = (anc[:, :, None] >> torch.arange(st["m"], device="cuda")) & 1
        s = torch.cat([s, s2.masked_fill((sees == 0)[:, None, None], -math.inf)], -1)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]          # [R][hkv][group][m]
    lse = lse.permute(0, 3, 1, 2)[st["req"], st["at"]].reshape(-1, c["hq"])
    if lse_only:
        return lse
    v = _value(st["vc"], st["vs"]).transpose(1, 2)
    if c["own_keys"]:
        v = torch.cat([v, _grouped(st, st["v"])[:, :, 0]], 2)
    o = p @ v[:, :, None] / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4)[st["req"], st["at"]].reshape(-1, c["hq"], c["d"])
    return o.bfloat16(), lse


def _attend(st):
    c = st["c"]
    if own:
        k, v = (st["k"], st["v"]) if c["own_keys"] else (None, None)
        out, lse = st["cache"].attend(st["q"], st["rows"], k, v, anc=st["anc"], pos=st["row_pos"], score=st["score"])
    else:
        out, lse = _plain_attend(st)
    return {"out": out, "lse": lse}


def _observe(st):
    c = st["c"]
    if own:
        return st["cache"].observe(st["q"], st["lse"], st["rows"], pos=st["row_pos"], row_weight=st["row_weight"],
                                   score=st["score"], decay=c["decay"], out=st["out"])
    q = _grouped(st, st["q"])
    s = _scores(st, q, _value(st["kc"], st["ks"]).transpose(1, 2), st["pos"])
    lse = torch.zeros(c["R"], st["m"], c["hq"], device="cuda")
    lse[st["req"], st["at"]] = st["lse"]
    lse = lse.reshape(c["R"], st["m"], c["hkv"], -1).permute(0, 2, 3, 1)[..., None]
    w = torch.zeros(c["R"], st["m"], device="cuda")
    w[st["req"], st["at"]] = st["row_weight"]
    p = torch.where(lse > -math.inf, torch.exp(s - lse), 0.0) * w[:, None, None, :, None]
    held = torch.arange(s.shape[-1], device="cuda")[None, None] < st["ctx"][:, None, None]
    out = torch.zeros(c["R"], c["hkv"], st["cap"], device="cuda")
    out[:, :, :s.shape[-1]] = torch.where(held, c["decay"] * st["weight"] + p.sum((2, 3)), 0.0)
    return out


def _evict(st):
    c = st["c"]
    if own:
        dst = st["dst"]
        st["cache"].evict(dst, c["budget"], recent=c["recent"], sinks=c["sinks"])
        k, v = dst.read(st["rows"], at=0)
        return {"k": k, "v": v, "ctx": dst.ctx_len, "pos": dst.pos, "weight": dst.weight}
    C, B = st["weight"].shape[-1], c["budget"]
    slot = torch.arange(C, device="cuda")
    ctx = st["ctx"][:, None, None]
    safe = (slot < c["sinks"]) | (slot >= ctx - c["recent"])
    w = torch.where(safe, math.inf, st["weight"])
    w = torch.where(slot < ctx, w, -math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :B]   # ties: the lower slot
    if best.shape[-1] < B:
        best = torch.cat([best, best.new_full((*best.shape[:-1], B - best.shape[-1]), C)], -1)
    best = torch.sort(torch.where(torch.arange(B, device="cuda") < ctx, best, C), -1).values
    there = best < C
    best = torch.where(there, best, 0)
    cap = _slots(c, B)
    pos = torch.zeros(c["R"], c["hkv"], cap, dtype=torch.int32, device="cuda")
    weight = torch.zeros(c["R"], c["hkv"], cap, device="cuda")
    pos[..., :B] = torch.where(there, st["pos"].gather(2, best), 0)
    weight[..., :B] = torch.where(there, st["weight"].gather(2, best), 0)
    r, h = torch.arange(c["R"], device="cuda")[:, None, None], torch.arange(c["hkv"], device="cuda")[None, :, None]
    k = _value(st["kc"][r, best, h], st["ks"][r, best, h]).bfloat16().transpose(1, 2)[st["kept"]]
    v = _value(st["vc"][r, best, h], st["vs"][r, best, h]).bfloat16().transpose(1, 2)[st["kept"]]
    return {"k": k, "v": v, "ctx": st["ctx"].clamp(max=B), "pos": pos, "weight": weight}


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    ctx, rows = _sizes(c)
    n, hq, hkv, d = sum(rows), c["hq"], c["hkv"], c["d"]
    row = d + 8                                     # a key's and a value's codes, scales and middles
    if c["op"] == "append":                         # bf16 rows in; codes, positions and the values held out
        return {"bytes": n * hkv * (4 * d + row + 4 + 4 * d) + 4 * n, "flops": 10.0 * n * hkv * d}
    if c["op"] == "evict":                          # every weight; the kept rows in and out; their values out
        kept = sum(min(k, c["budget"]) for k in ctx)
        return {"bytes": hkv * (4 * sum(ctx) + kept * (2 * row + 12 + 4 * d)), "flops": float(hkv * sum(ctx))}
    if c["docs"]:
        ctx = [k - k // 3 for k in ctx]
    seen = [min(k, c["window"]) if c["window"] else k for k in ctx]
    key_pos = 4 if c["window"] or c["alibi"] or c["docs"] else 0
    if c["op"] == "observe":                        # the keys' half of the rows; weights in and out
        byt = hkv * (sum(seen) * (row // 2 + key_pos) + 8 * sum(_sizes(c)[0])) + n * hq * (2 * d + 4) + 8 * n
        return {"bytes": byt, "flops": 2.0 * d * hq * sum(m * k for m, k in zip(rows, seen))}
    pairs = sum(m * (k + ((m + 1) / 2 if c["own_keys"] else 0)) for m, k in zip(rows, seen))
    byt = hkv * sum(seen) * (row + key_pos) + n * hq * (4 * d + 4) + (n * hkv * 4 * d if c["own_keys"] else 0) + 12 * n
    return {"bytes": byt, "flops": 4.0 * d * hq * pairs}


# ------------------------------------------------------- 64-bit definition --

def _held64(x):
    """The values a bf16 row [..., d] is held as, in 64 bits."""
    x = x.double()
    least, most = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
    s = ((most - least) / 15).bfloat16().double()
    m = (least + s * 8).bfloat16().double()
    steps = ((x - m) / torch.where(s == 0, 1.0, s)).round().clamp(-8, 7)
    return torch.where(s == 0, m, m + s * steps)


def exact(case, seed):
    c, x = case, _inputs(case, seed)
    R, hq, hkv, d, G = c["R"], c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["op"] == "append":
        return {"k": _held64(x["k"]), "v": _held64(x["v"]), "ctx": None, "pos": None}
    if c["op"] == "evict":
        ks, vs = [], []
        for r, keys in enumerate(x["ctx"]):
            per_head = []
            for h in range(hkv):
                w = x["weight"][r, h, :keys].tolist()
                always = set(range(min(c["sinks"], keys))) | set(range(max(0, keys - c["recent"]), keys))
                rest = sorted((j for j in range(keys) if j not in always), key=lambda j: (-w[j], j))
                kept = sorted(always | set(rest[:max(0, c["budget"] - len(always))]))
                kept = torch.tensor(kept, device="cuda")
                per_head.append((_held64(x["K"][r, kept, h]), _held64(x["V"][r, kept, h])))
            ks.append(torch.stack([a for a, _ in per_head], 1))
            vs.append(torch.stack([b for _, b in per_head], 1))
        return {"k": torch.cat(ks), "v": torch.cat(vs), "ctx": None, "pos": None, "weight": None}
    lse_in = _lse(c, x).double() if c["op"] == "observe" else None
    outs, lses = [], []
    sums = torch.zeros(R, hkv, _slots(c, x["C"]), **f64)
    for r in range(R):
        a, b, keys = x["cu"][r], x["cu"][r + 1], x["ctx"][r]
        K, V = _held64(x["K"][r, :keys]), _held64(x["V"][r, :keys])
        kp = x["pos"][r, :keys].double()
        sees = torch.ones(b - a, keys, dtype=torch.bool, device="cuda")
        if c["op"] == "attend" and c["own_keys"]:
            K, V = torch.cat([K, x["k"][a:b].double()]), torch.cat([V, x["v"][a:b].double()])
            kp = torch.cat([kp, x["row_pos"][a:b].double()])
            own_sees = torch.tensor([[bool(w >> j & 1) for j in range(b - a)] for w in x["anc"][a:b].tolist()],
                                    device="cuda")
            sees = torch.cat([sees, own_sees], 1)
        qp = x["row_pos"][a:b].double()
        far = qp[:, None] - kp[None]
        if c["window"]:
            sees = sees & (far < c["window"])
        if c["docs"]:
            sees = sees & (kp >= x["start"][r])[None]
        o_heads, l_heads = [], []
        for h in range(hq):
            z = x["q"][a:b, h].double() @ K[:, h // G].T / math.sqrt(d)
            if c["cap"]:
                z = torch.tanh(z / c["cap"]) * c["cap"]
            if c["alibi"]:
                z = z - x["slopes"][h].double() * far
            if c["op"] == "observe":
                p = torch.exp(z - lse_in[a:b, h][:, None]) * sees * (lse_in[a:b, h] > -math.inf)[:, None]
                sums[r, h // G, :keys] += (p.nan_to_num(0.0) * x["row_weight"][a:b].double()[:, None]).sum(0)
                continue
            z = z.masked_fill(~sees, -math.inf)
            lse = torch.logsumexp(z, 1)
            o_heads.append(torch.nan_to_num(torch.softmax(z, 1), 0.0) @ V[:, h // G])
            l_heads.append(lse)
        if c["op"] == "observe":
            sums[r, :, :keys] += c["decay"] * x["weight"][r, :, :keys].double()
        else:
            outs.append(torch.stack(o_heads, 1))
            lses.append(torch.stack(l_heads, 1))
    return sums if c["op"] == "observe" else {"out": torch.cat(outs), "lse": torch.cat(lses)}

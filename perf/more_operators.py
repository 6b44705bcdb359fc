"""Cases of a request's way around the verify step: rotary positions of its
queries and keys, causal attention over packed prompts, and tokens sampled from
logits.

Rotary: pair i of a head's first `rot` dims turns by pos * f_i, f_i = base^(-2i /
rot), scaled for contexts longer than the trained one:
  linear  f / factor
  bands   t = original f / 2 pi turns in the trained context: f where t > high, f /
          factor where t < low, between them in proportion to (t - low) / (high - low)
  ramp    f where i <= lo, f / factor where i >= hi, in proportion between them, lo
          and hi being the pairs that make `fast` and `slow` turns in the trained
          context (rounded outwards); sines and cosines times 0.1 ln(factor) + 1.
Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved.

Attention: query i of a request of m rows and n keys stands at position n - m + i and
sees the keys up to itself, less than `window` back.  score = cap tanh(q.k scale /
cap) + slope (j - position), cap and slope optional.

Sampling, of a row's tokens by falling logit, equal ones by index: weight exp((logit -
most) / temperature); the first top_k are kept, of those the ones of at least min_p,
of those the shortest run that holds top_p of their sum; the token is the first whose
running sum passes u times the sum of what is kept.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases --

def _rope(name, **kw):
    c = dict(name=name, op="rope", n=1, hq=32, hkv=8, d=128, rot=128, base=1e6, interleaved=False, scaling="none",
             factor=1.0, low=1.0, high=4.0, fast=32.0, slow=1.0, original=4096, far=2048, tree=False)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", R=1, m_lo=1, m_hi=1, past_lo=0, past_hi=0, hq=32, hkv=8, d=128, cap=0.0, alibi=False,
             window=0)
    c.update(kw)
    return c


def _sample(name, **kw):
    c = dict(name=name, op="sample", n=1, V=151936, spread=2.5, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
             mixed=False)
    c.update(kw)
    return c


def listed():
    return [
        # the rows of one draft tree of the 8B-class decoder: latency
        _rope("rope_tree_16", n=16, tree=True),
        # a long prompt of the 27B-class decoder, past the trained context
        _rope("rope_prompt_16384_ramp", n=16384, hq=40, scaling="ramp", factor=4.0, original=8192, far=0),
        # rows of many requests at far positions, part of smaller heads, neighbours paired
        _rope("rope_far_part_4099", n=4099, hq=16, hkv=16, d=64, rot=32, base=5e5, interleaved=True, scaling="bands",
              factor=8.0, original=8192, far=1 << 20),
        # one short prompt: latency
        _attend("prompt_1x331", m_lo=331, m_hi=331),
        # a batch of prompts, packed
        _attend("prompts_8x2k", R=8, m_lo=500, m_hi=2048),
        # one long prompt
        _attend("prompt_16384", m_lo=16384, m_hi=16384),
        # the next chunk of a prompt whose first 32768 tokens are done
        _attend("chunk_512_past_32k", m_lo=512, m_hi=512, past_lo=32768, past_hi=32768, hq=40),
        # heads of their own, capped scores, distance slopes, a sliding window, ragged prompts
        _attend("window_5x3k_mha64_cap", R=5, m_lo=1, m_hi=3001, past_lo=0, past_hi=900, hq=16, hkv=16, d=64, cap=50.0,
                alibi=True, window=1024),
        # one token of each of a batch over keys in bf16
        _attend("tokens_16x8k", R=16, m_lo=1, m_hi=1, past_lo=1500, past_hi=8191),
        # the next token of one request: latency
        _sample("sample_1", temperature=0.8, top_p=0.95),
        # the rows of a batched step of 32 requests, each with its own settings
        _sample("sample_256_mixed", n=256, mixed=True),
        # an odd vocabulary, so that rows start anywhere
        _sample("sample_33_odd", n=33, V=50021, temperature=1.3, top_k=50, min_p=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "sample"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 128])
        hkv = rng.choice([1, 2, 4, 8])
        return _rope("", n=_log(rng, 1, 16384), hq=hkv * rng.choice([1, 2, 4, 5]), hkv=hkv, d=d,
                     rot=rng.choice([d, d, d // 2, d // 4]), base=rng.choice([1e4, 5e5, 1e6]),
                     interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "bands", "ramp"]),
                     factor=rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([2048, 4096, 8192]),
                     far=rng.choice([0, _log(rng, 1, 1 << 20)]), tree=rng.random() < 0.2)
    if op == "sample":
        n = _log(rng, 1, 256)
        return _sample("", n=n, V=_log(rng, 1000, 151936), spread=rng.uniform(1.0, 4.0),
                       temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.5]), top_k=rng.choice([0, 0, 1, _log(rng, 2, 1000)]),
                       top_p=rng.choice([1.0, rng.uniform(0.1, 0.999)]), min_p=rng.choice([0.0, 0.0, rng.uniform(0.0, 0.3)]),
                       mixed=rng.random() < 0.3)
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 4, 5, 8])
    R = _log(rng, 1, 16)
    m = _log(rng, 1, 8192)
    past = rng.choice([0, 0, _log(rng, 1, 32768)])
    # no dearer than the longest listed prompt: heads x rows x keys
    most = 32 * 128 * 16384 * 8192
    while R * hq * d * m * (past + (m + 1) / 2) > most:
        R, m, past = max(1, R // 2), max(1, m // 2), past // 2
    lo = rng.uniform(0.0, 1.0)
    return _attend("", R=R, m_lo=int(m * lo), m_hi=m, past_lo=int(past * rng.uniform(0.0, 1.0)), past_hi=past, hq=hq, hkv=hkv,
                   d=d, cap=rng.choice([0.0, 0.0, 0.0, 50.0]), alibi=rng.random() < 0.2,
                   window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]))


def _spread(lo, hi, n, start=0):
    """n whole numbers over lo..hi, the first one hi: the same for every seed."""
    return [hi - int((hi - lo) * (((i + start * (i > 0)) * 0.6180339887) % 1.0)) for i in range(n)]


def _sizes(c):
    """(rows, keys) of each request."""
    rows, past = _spread(c["m_lo"], c["m_hi"], c["R"]), _spread(c["past_lo"], c["past_hi"], c["R"], 3)
    return rows, [m + p for m, p in zip(rows, past)]


def _sums(lengths):
    cu = [0]
    for x in lengths:
        cu.append(cu[-1] + x)
    return cu


# ------------------------------------------------------------------ inputs --

def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    if c["op"] == "rope":
        n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
        at = torch.arange(n, device="cuda")
        if c["tree"]:                                                  # nodes of a tree stand at a few depths
            at = (uniform(n) * 8).long()
        far = torch.zeros(n, dtype=torch.int64, device="cuda")
        if c["far"]:
            far = far + c["far"] if c["tree"] else (uniform(n) * c["far"]).long()
        qkv = normal(n, hq + 2 * hkv, d).bfloat16()                    # as one projection leaves them
        return {"q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "pos": (at + far).to(torch.int32)}
    if c["op"] == "sample":
        n, V = c["n"], c["V"]
        logits = c["spread"] * normal(n, V)
        each = V // 64
        likely = torch.arange(64, device="cuda") * each + (uniform(n, 64) * each).long()   # a few tokens stand out
        logits.scatter_(1, likely, 4.0 * c["spread"] + 2.0 * normal(n, 64))
        x = {"logits": logits.bfloat16(), "u": uniform(n)}
        if c["mixed"]:
            pick = torch.randint(0, 4, (n,), device="cuda", generator=g)
            x["temperature"] = torch.tensor([0.0, 0.6, 1.0, 1.4], device="cuda")[pick]
            x["top_k"] = torch.tensor([0, 40, 0, 500], dtype=torch.int32, device="cuda")[(pick + 1) % 4]
            x["top_p"] = 1.0 - 0.5 * uniform(n) ** 3
            x["min_p"] = torch.tensor([0.0, 0.0, 0.05, 0.01], device="cuda")[(pick + 2) % 4]
        return x
    rows, keys = _sizes(c)
    n, s = sum(rows), sum(keys)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    mean, spread = 0.5 * normal(hkv, d), 0.5 + uniform(hkv, d)         # keys' channels differ
    x = {"q": (1.5 * normal(n, hq, d)).bfloat16(), "k": (normal(s, hkv, d) * spread + mean).bfloat16(),
         "v": normal(s, hkv, d).bfloat16(), "rows": _sums(rows), "keys": _sums(keys)}
    if c["alibi"]:
        x["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq).float()
    return x


def prepare(case, seed):
    c = case
    st = {"c": c, **_inputs(c, seed)}
    if c["op"] == "rope":
        st["freq"], st["amplitude"] = _frequencies(c)
    if c["op"] == "sample":
        st["set"] = {k: st.get(k, c[k]) for k in ("temperature", "top_k", "top_p", "min_p")}
    if own:
        from speculative_decoding_tree_bit_gb300 import model as sdv
        if c["op"] == "rope":
            scaling = {"none": lambda: None, "linear": lambda: sdv.RopeScaling.linear(c["factor"]),
                       "bands": lambda: sdv.RopeScaling.bands(c["factor"], c["original"], low=c["low"], high=c["high"]),
                       "ramp": lambda: sdv.RopeScaling.ramp(c["factor"], c["original"], fast=c["fast"],
                                                            slow=c["slow"])}[c["scaling"]]()
            st["op"] = sdv.Rope(c["d"], c["rot"], c["base"], interleaved=c["interleaved"], scaling=scaling)
        elif c["op"] == "sample":
            st["op"] = sdv.sample
        else:
            st["op"] = sdv.PromptAttention(c["hq"], c["hkv"], c["d"])
            st["rows"], st["keys"] = sdv.RequestRows(st["rows"]), sdv.RequestRows(st["keys"])
            st["score"] = sdv.KV4Score(softcap=c["cap"], slopes=st.get("slopes"), window=c["window"])
    return st


def _frequencies(c):
    """(64-bit frequencies of the pairs, what sines and cosines are multiplied by), on the GPU."""
    rot, base, factor, original = c["rot"], c["base"], c["factor"], c["original"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f, amplitude = base ** (-2.0 * i / rot), 1.0
    if c["scaling"] == "linear":
        f = f / factor
    elif c["scaling"] == "bands":
        turns = original * f / (2 * math.pi)
        part = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0.0, 1.0)
        f = part * f + (1 - part) * f / factor
    elif c["scaling"] == "ramp":
        lo, hi = (rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (c["fast"], c["slow"]))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        part = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f, amplitude = (1 - part) * f + part * f / factor, 0.1 * math.log(factor) + 1.0
    return f, amplitude


# ------------------------------------------------------------------ passes --

def run(state):
    return {"rope": _run_rope, "attend": _run_attend, "sample": _run_sample}[state["c"]["op"]](state)


def _run_rope(st):
    if own:
        q, k = st["op"](st["q"], st["k"], st["pos"])
        return {"q": q, "k": k}
    c = st["c"]
    angle = st["pos"].double()[:, None] * st["freq"]                   # far positions: the angle in 64 bits
    cos, sin = (st["amplitude"] * torch.cos(angle)).float()[:, None], (st["amplitude"] * torch.sin(angle)).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        y, rot = x.clone(), c["rot"]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        out[name] = y.bfloat16()
    return out


def _run_attend(st):
    if own:
        out, lse = st["op"](st["q"], st["k"], st["v"], st["rows"], st["keys"], score=st["score"])
        return {"out": out, "lse": lse}
    c = st["c"]
    G, scale = c["hq"] // c["hkv"], 1.0 / math.sqrt(c["d"])
    out = torch.zeros_like(st["q"])
    lse = torch.full(st["q"].shape[:2], -math.inf, device="cuda")
    for r in range(c["R"]):
        a, b, ka, kb = st["rows"][r], st["rows"][r + 1], st["keys"][r], st["keys"][r + 1]
        if a == b:
            continue
        back = torch.arange(kb - ka - (b - a), kb - ka, device="cuda")[:, None] - torch.arange(kb - ka, device="cuda")
        hidden = back < 0
        if c["window"]:
            hidden = hidden | (back >= c["window"])
        for h in range(c["hq"]):
            s = (st["q"][a:b, h].float() * scale) @ st["k"][ka:kb, h // G].float().T
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["alibi"]:
                s = s - st["slopes"][h] * back.float()
            s.masked_fill_(hidden, -math.inf)
            top = s.amax(-1, keepdim=True)
            s = torch.exp_(s - top)                                    # a row always sees itself
            total = s.sum(-1, keepdim=True)
            lse[a:b, h] = (top + torch.log(total))[:, 0]
            out[a:b, h] = (s @ st["v"][ka:kb, h // G].float() / total).bfloat16()
    return {"out": out, "lse": lse}


def _run_sample(st):
    c, p = st["c"], st["set"]
    if own:
        return st["op"](st["logits"], st["u"], **p)
    n, V = c["n"], c["V"]

    def rowwise(x):
        return x.double()[:, None] if isinstance(x, torch.Tensor) else torch.full((n, 1), x, dtype=torch.float64, device="cuda")

    # the settings are 32-bit numbers, the running sums 64-bit ones: tokens lie next to a border often
    t, top_k, top_p, min_p = (rowwise(p[k] if isinstance(p[k], torch.Tensor) else torch.tensor(p[k]).float().item())
                              for k in ("temperature", "top_k", "top_p", "min_p"))
    x, order = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(t > 0, t, 1.0))
    rank = torch.arange(V, device="cuda")
    keep = ((rank < top_k) | (top_k <= 0)) & (w >= min_p) & ((t > 0) | (rank < 1))
    w = w * keep
    run_sum = torch.cumsum(w, 1)
    before = run_sum - w
    keep = keep & ((before < top_p * run_sum[:, -1:]) | (top_p >= 1) | (rank < 1))
    kept = keep.sum(1)
    w = w * keep
    total = run_sum.gather(1, kept[:, None] - 1)
    at = (run_sum <= st["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    at = torch.minimum(at, kept[:, None] - 1)
    logprob = torch.log(w.gather(1, at) / total)[:, 0].float()
    return {"tokens": order.gather(1, at)[:, 0].to(torch.int32), "logprob": logprob, "kept": kept.to(torch.int32)}


# -------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "rope":                            # rows in and out, positions; a pair is four products, two sums
        heads = c["n"] * (c["hq"] + c["hkv"])
        return {"bytes": 4 * c["d"] * heads + 4 * c["n"], "flops": 3.0 * c["rot"] * heads}
    if c["op"] == "sample":                          # the logits; settings, a token, its logarithm and a count
        return {"bytes": c["n"] * (2 * c["V"] + 16 + 16 * c["mixed"]), "flops": 2.0 * c["n"] * c["V"]}
    rows, keys = _sizes(c)
    pairs = seen = 0
    for m, s in zip(rows, keys):
        w = c["window"] or s
        first = max(s - m + 1, 1)                    # keys up to the first row
        short = max(0, min(s, w) - first + 1)        # rows whose keys the window does not cut
        pairs += short * (first + min(s, w)) // 2 + (m - min(short, m)) * w if m else 0
        seen += min(s, w + m - 1) if m else 0
    n, hq, hkv, d = sum(rows), c["hq"], c["hkv"], c["d"]
    return {"bytes": n * hq * (4 * d + 4) + seen * hkv * 4 * d, "flops": 4.0 * d * hq * pairs}


# ------------------------------------------------------- 64-bit definition --

def exact(case, seed):
    x = _inputs(case, seed)
    return {"rope": _exact_rope, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](case, x)


def _exact_rope(c, x):
    rot, factor = c["rot"], c["factor"]
    freq = []
    amplitude = 1 + math.log(factor) / 10 if c["scaling"] == "ramp" else 1.0
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(c["base"]))
        if c["scaling"] == "linear":
            f /= factor
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > c["original"] / c["low"]:
                f /= factor
            elif wave >= c["original"] / c["high"]:
                share = (c["original"] / wave - c["low"]) / (c["high"] - c["low"])
                f = f / factor + share * (f - f / factor)
        elif c["scaling"] == "ramp":
            def pair_of(turns):
                return rot / 2 * math.log(c["original"] / (turns * 2 * math.pi)) / math.log(c["base"])
            lo, hi = max(0, math.floor(pair_of(c["fast"]))), min(rot - 1, math.ceil(pair_of(c["slow"])))
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - share + share / factor)
        freq.append(f)
    turn = torch.polar(torch.full((c["n"], rot // 2), amplitude, dtype=torch.float64, device="cuda"),
                       x["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))[:, None]
    out = {}
    for name in ("q", "k"):
        head = x[name].double()
        part = head[..., :rot]
        pairs = part.unflatten(-1, (-1, 2)) if c["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        turned = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
        out[name] = torch.cat([turned, head[..., rot:]], -1)
    return out


def _exact_attend(c, x):
    G = c["hq"] // c["hkv"]
    out = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(x["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for r in range(c["R"]):
        a, b, ka, kb = x["rows"][r], x["rows"][r + 1], x["keys"][r], x["keys"][r + 1]
        past = (kb - ka) - (b - a)
        for i in range(0, b - a, 2048):              # rows i .. j see keys first .. past + j
            j = min(b - a, i + 2048)
            first = max(0, past + i - c["window"] + 1) if c["window"] else 0
            K = x["k"][ka + first:ka + past + j].double()
            V = x["v"][ka + first:ka + past + j].double()
            at = torch.arange(past + i, past + j, device="cuda")[:, None]
            key = torch.arange(first, past + j, device="cuda")[None]
            sees = key <= at
            if c["window"]:
                sees = sees & (at - key < c["window"])
            for h in range(c["hq"]):
                z = x["q"][a + i:a + j, h].double() @ K[:, h // G].T / math.sqrt(c["d"])
                if c["cap"]:
                    z = torch.tanh(z / c["cap"]) * c["cap"]
                if c["alibi"]:
                    z = z + x["slopes"][h].double() * (key - at)
                z = torch.where(sees, z, -math.inf)
                lse[a + i:a + j, h] = torch.logsumexp(z, 1)
                out[a + i:a + j, h] = torch.softmax(z, 1) @ V[:, h // G]
    return {"out": out, "lse": lse}


def _exact_sample(c, x):
    """The logarithm of each token's share, row by row over the distinct logits."""
    def of(name, r):
        v = x[name][r].item() if name in x else c[name]
        return v if name == "top_k" else torch.tensor(v, dtype=torch.float32).item()

    logprob = []
    for r in range(c["n"]):
        t, k, top_p, min_p, u = of("temperature", r), of("top_k", r), of("top_p", r), of("min_p", r), x["u"][r].item()
        if t <= 0:
            logprob.append(0.0)
            continue
        value, count = torch.unique(x["logits"][r].double(), return_counts=True)
        value, count = value.flip(0), count.flip(0)
        w = torch.exp((value - value[0]) / t)
        if k > 0:
            count = torch.minimum(count, (k - (torch.cumsum(count, 0) - count)).clamp(min=0))
        count = torch.where(w >= min_p, count, 0)
        mass = count * w
        if top_p < 1:
            lack = top_p * mass.sum() - (torch.cumsum(mass, 0) - mass)
            count = torch.minimum(count, torch.ceil(lack / w).clamp(min=0).long())
            count[0] = max(int(count[0]), 1)
            mass = count * w
        run_sum = torch.cumsum(mass, 0)
        at = int((run_sum <= u * run_sum[-1]).sum())
        logprob.append(math.log(w[at].item() / run_sum[-1].item()))
    return {"tokens": None, "logprob": torch.tensor(logprob, dtype=torch.float64, device="cuda"), "kept": None}

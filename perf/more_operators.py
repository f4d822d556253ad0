"""Measured cases of the operators that bound a long context: attention over a
window with sinks, attention of a batch that shares a prefix, the weight that
attention gives each cached token, and eviction by that weight.

A chunk is the newest n tokens of some requests (one each in a decode step, a
few draft tokens, a piece of a prompt).  Token i of a request's chunk sits at
position ctx_len - n + i.  Rows of a call are laid out request after request
(layer by layer where a call has several layers).

  window   a query at position p attends over the tokens t <= p with t < sinks
           or t > p - window
  shared   a query attends over the first tokens of one request, which the batch
           has in common, and over its own request's tokens up to its own
  weights  per cached token the sum of the probabilities that the chunk's queries
           give it, all heads together, from the attention's log-sum-exp
  evict    of every layer's tokens the first, the last, and of the rest those
           with the largest weights stay; the context closes up

`own` chooses between elementary torch operations on the cache's tensors and
the library's calls.
"""
import math

import torch

own = False

KV_HEADS, HEAD_DIM, Q_HEADS, GROUP = 4, 128, 16, 4
INDEX_DIM = 64
ROW = {"bf16": 2048, "fp8": 1040}
K_BYTES = {"bf16": 1024, "fp8": 520}
SCALE = HEAD_DIM ** -0.5
FULL = 1 << 30                       # a window that no context reaches past


def listed():
    return [
        # one request decodes one token over a short window: latency
        {"name": "window token", "op": "window", "requests": 1, "tokens": 1, "context": 8192, "sinks": 4,
         "window": 1024, "rows": "bf16"},
        # a serving batch decodes over FP8 rows
        {"name": "window batch", "op": "window", "requests": 32, "tokens": 1, "context": 16384, "sinks": 4,
         "window": 4096, "rows": "fp8"},
        # a piece of a long prompt
        {"name": "window prompt", "op": "window", "requests": 1, "tokens": 4096, "context": 16384, "sinks": 16,
         "window": 4096, "rows": "bf16"},
        # a prompt's end with every earlier token in sight, FP8 rows
        {"name": "causal prompt", "op": "window", "requests": 2, "tokens": 1023, "context": 8191, "sinks": 0,
         "window": FULL, "rows": "fp8"},
        # two answers to one short prompt
        {"name": "shared pair", "op": "shared", "requests": 2, "tokens": 1, "prefix": 2047, "context": 61,
         "copies": True, "rows": "bf16"},
        # a batch behind one long system prompt, which only one request holds
        {"name": "shared batch", "op": "shared", "requests": 64, "tokens": 1, "prefix": 16384, "context": 512,
         "copies": False, "rows": "bf16"},
        # draft tokens of requests that branched from one long document
        {"name": "shared draft", "op": "shared", "requests": 8, "tokens": 4, "prefix": 65536, "context": 1000,
         "copies": False, "rows": "fp8"},
        # a decode step notes what its tokens attend to
        {"name": "weights token", "op": "weights", "requests": 8, "tokens": 1, "context": 8192, "sinks": 0,
         "window": FULL, "rows": "bf16"},
        # a prompt's last tokens judge a long context
        {"name": "weights prompt", "op": "weights", "requests": 1, "tokens": 64, "context": 131072, "sinks": 0,
         "window": FULL, "rows": "fp8"},
        # every token of a piece of a prompt judges what it sees
        {"name": "weights chunk", "op": "weights", "requests": 1, "tokens": 1024, "context": 32768, "sinks": 4,
         "window": 16384, "rows": "bf16"},
        # a short request goes back to half of its tokens
        {"name": "evict short", "op": "evict", "context": 2047, "keep": 1021, "first": 4, "last": 128, "layers": 12,
         "rows": "fp8"},
        # a long one
        {"name": "evict long", "op": "evict", "context": 32768, "keep": 16384, "first": 4, "last": 1024, "layers": 12,
         "rows": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["window", "window", "shared", "weights", "evict"])
    rows = rng.choice(["bf16", "fp8"])
    if op == "evict":
        context = _spread(rng, 256, 32768)
        keep = rng.randint(context // 4, context - 1)
        return {"op": op, "context": context, "keep": keep, "first": rng.randint(0, 16), "last": rng.randint(0, keep // 4),
                "layers": rng.choice([1, 4, 12]), "rows": rows}
    requests = rng.choice([1, 1, 2, 3, 8, 32, 64])
    tokens = rng.choice([1, rng.randint(2, 8), _spread(rng, 1, max(1, 2048 // requests))])
    if op == "shared":
        tokens = min(tokens, 512 // requests)
        return {"op": op, "requests": requests, "tokens": tokens, "prefix": _spread(rng, 64, 32768),
                "context": tokens + _spread(rng, 1, 2048), "copies": requests <= 8 and rng.random() < 0.5, "rows": rows}
    context = tokens + _spread(rng, 8, min(32768, 131072 // requests))
    return {"op": op, "requests": requests, "tokens": tokens if op == "window" else min(tokens, 1024 // requests),
            "context": context, "sinks": rng.choice([0, 1, 4, 37, 128]),
            "window": rng.choice([FULL if tokens * requests <= 256 else 4096, _spread(rng, 64, 4096)]), "rows": rows}


# -------------------------------------------------------------------- sizes

def _lengths(case):
    """(context, tokens) of each request of a chunk: ragged over the batch.  For
    a shared prefix the context counts the request's own tokens alone."""
    out = []
    for r in range(case["requests"]):
        n = max(1, case["tokens"] - r % 4)
        out.append((max(n, case["context"] - 13 * (r % 16)), n))
    return out


def _seen(case, p):
    """Tokens that a query at position p sees."""
    low = max(0, p - case["window"] + 1)
    return p + 1 - low + min(case["sinks"], low)


def work(case):
    op, row = case["op"], ROW[case["rows"]]
    if op == "evict":
        n, k, L = case["context"], case["keep"], case["layers"]
        moved = k * (n - k) // n
        return {"bytes": L * (4 * n + k * (2 * (INDEX_DIM + 2) + 8 + 8) + 2 * moved * row), "flops": 0}
    lens = _lengths(case)
    rows = sum(n for _, n in lens)
    io = rows * Q_HEADS * (4 * HEAD_DIM + 4)
    if op == "shared":
        pairs = sum(n * case["prefix"] + n * c - n * (n - 1) // 2 for c, n in lens)
        return {"bytes": (case["prefix"] + sum(c for c, _ in lens)) * row + io, "flops": 4 * HEAD_DIM * Q_HEADS * pairs}
    pairs = sum(_seen(case, p) for c, n in lens for p in range(c - n, c))
    tokens = sum(c - max(0, c - n - case["window"] + 1) + min(case["sinks"], max(0, c - n - case["window"] + 1))
                 for c, n in lens)
    if op == "window":
        return {"bytes": tokens * row + io, "flops": 4 * HEAD_DIM * Q_HEADS * pairs}
    return {"bytes": tokens * K_BYTES[case["rows"]] + rows * Q_HEADS * (2 * HEAD_DIM + 4) + 4 * sum(c for c, _ in lens),
            "flops": 2 * HEAD_DIM * Q_HEADS * pairs}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _queries(g, rows, common):
    """Queries with a part that they have in common, as trained heads have."""
    return (1.5 * _randn(g, rows, Q_HEADS, HEAD_DIM) + common).bfloat16()


def _kv_rows(g, n, kind, common, sinks=0):
    """KV rows; the keys of the first `sinks` tokens lie along the queries' common
    part and draw much of the attention."""
    x = _randn(g, n, 8, HEAD_DIM)
    x[:sinks, :KV_HEADS] += 3.0 * common
    x = x.bfloat16()
    if kind == "bf16":
        return x.view(n, 1024).view(torch.uint8)
    x = x.float()
    sc = (x.abs().amax(2) / 448).half()
    codes = (x / sc.float()[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.cat([codes.view(n, 1024).view(torch.uint8), sc.view(torch.uint8).view(n, 16)], 1)


def _cache(case, requests, capacity, layers, pool_rows):
    """The cache's tensors, and (for the library) the cache itself."""
    kind = case["rows"]
    if own:
        import sparse_attention_decode_qsa_gb300 as Q
        c = Q.Cache(n_layers=layers, max_requests=requests, ctx_capacity=capacity, hbm_pool_rows=pool_rows,
                    ring_tokens=64, staging_rows=0, kv_format=Q.KV_FP8 if kind == "fp8" else Q.KV_BF16)
        return {"cache": c, "pool": c.pool, "keys": c.index_keys, "scales": c.index_scales, "slots": c.slot_table}
    empty = lambda dtype, *shape: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    return {"pool": empty(torch.uint8, pool_rows, ROW[kind]),
            "keys": torch.zeros(requests, layers, capacity, INDEX_DIM, dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros(requests, layers, capacity, dtype=torch.float16, device="cuda"),
            "slots": torch.full((requests, layers, capacity), -1, dtype=torch.int32, device="cuda")}


def _begin(s, r, ctx, layers, base):
    """Lease request r, all of its rows in the pool from row `base` on."""
    if own:
        return s["cache"].request_begin(ctx)
    s["slots"][r, :, :ctx] = base + torch.arange(layers * ctx, dtype=torch.int32, device="cuda").view(layers, ctx)
    return r


def prepare(case, seed):
    g = _gen(seed)
    s = _prepare_evict(case, g) if case["op"] == "evict" else _prepare_chunk(case, g)
    return dict(s, case=case)


def _prepare_evict(case, g):
    n, L, k = case["context"], case["layers"], case["keep"]
    s = _cache(case, 1, n, L, L * n)
    s["request"] = _begin(s, 0, n, L, 0)
    s["pool"].copy_(torch.randint(0, 256, s["pool"].shape, generator=g, device="cuda", dtype=torch.uint8))
    s["keys"][0] = torch.randint(0, 127, (L, n, INDEX_DIM), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"][0] = _randn(g, L, n).abs().half()
    # a few tokens have most of the weight, as attention leaves it
    s["weights"] = (2.0 * _randn(g, L, n)).exp()
    s["weights_out"] = torch.zeros(L, k, device="cuda")
    s["kept"] = torch.zeros(L, k, dtype=torch.int32, device="cuda")
    if own:
        need = s["cache"].evict_workspace_bytes(s["request"], k)
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


def _prepare_chunk(case, g):
    lens = _lengths(case)
    shared = case["op"] == "shared"
    R, rows = len(lens), sum(n for _, n in lens)
    common = 0.5 * _randn(g, HEAD_DIM)
    sinks = 4
    # a request's own tokens lie behind its copy of the prefix, or alone
    P = case["prefix"] if shared else 0
    lead = P if shared and case["copies"] else 0
    ctx = [lead + c for c, _ in lens] + ([P] if shared else [])
    bases = [sum(ctx[:r]) for r in range(len(ctx))]
    total = sum(ctx)
    s = _cache(case, len(ctx), max(ctx), 1, total)
    s["requests"] = [_begin(s, r, c, 1, bases[r]) for r, c in enumerate(ctx)]
    s.update(ctx=ctx, tokens=[n for _, n in lens], own_first=lead)
    first = [sum(n for _, n in lens[:r]) for r in range(R)]
    s["first"] = first
    for r, c in enumerate(ctx):
        s["pool"][bases[r]:bases[r] + c] = _kv_rows(g, c, case["rows"], common, min(sinks, c) if not shared or r == R else 0)
    if lead:
        for r in range(R):
            s["pool"][bases[r]:bases[r] + P] = s["pool"][bases[R]:bases[R] + P]
    s["q"] = _queries(g, rows, common)
    if shared:
        s["prefix"] = s["requests"].pop()
    if case["op"] == "weights":
        s["weights"] = torch.zeros(R, max(ctx), device="cuda")
        s["lse"] = torch.empty(rows, Q_HEADS, device="cuda")
        for r in range(R):
            for h in range(Q_HEADS):
                a, n = first[r], s["tokens"][r]
                t, mask = _visible(s, case, r)
                k = _values(s, case, r, t)[0][:, h // GROUP]
                x = (s["q"][a:a + n, h].float() @ k.T) * SCALE
                s["lse"][a:a + n, h] = x.masked_fill(~mask, -math.inf).logsumexp(1)
        return s
    s["out"] = torch.zeros(rows, Q_HEADS, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(rows, Q_HEADS, device="cuda")
    if own:
        c = s["cache"]
        need = (c.shared_attn_workspace_bytes(s["requests"], s["tokens"], 0, 1, s["prefix"], P, lead) if shared else
                c.window_attn_workspace_bytes(s["requests"], s["tokens"], 0, 1, case["sinks"], case["window"]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- runs

def _visible(s, case, r):
    """Tokens that any query of request r's chunk sees, and which query sees which."""
    c, n = s["ctx"][r], s["tokens"][r]
    at = torch.arange(c - n, c, device="cuda")[:, None]
    low = max(min(case["sinks"], c), c - n - case["window"] + 1)
    t = torch.cat([torch.arange(min(case["sinks"], c), device="cuda"), torch.arange(low, c, device="cuda")])
    return t, (t <= at) & ((t < case["sinks"]) | (t > at - case["window"]))


def _values(s, case, r, tokens):
    """K and V of some tokens of request r in fp32: [tokens][4][128] each."""
    rows = s["pool"][s["slots"][r, 0][tokens].long()]
    if case["rows"] == "bf16":
        kv = rows.view(torch.bfloat16).float().view(-1, 2, KV_HEADS, HEAD_DIM)
    else:
        kv = (rows[:, :1024].view(torch.float8_e4m3fn).float().view(-1, 2, KV_HEADS, HEAD_DIM) *
              rows[:, 1024:].view(torch.float16).float().view(-1, 2, KV_HEADS, 1))
    return kv[:, 0], kv[:, 1]


def _logits(q, k):
    """[KV heads][rows * group][tokens] from q [rows][16][128] and k [tokens][4][128]."""
    q = q.float().view(-1, KV_HEADS, GROUP, HEAD_DIM).transpose(0, 1).reshape(KV_HEADS, -1, HEAD_DIM)
    return torch.bmm(q * SCALE, k.permute(1, 2, 0))


def _by_row(x):
    """[KV heads][rows * group][...] -> [rows][16][...]"""
    return x.unflatten(1, (-1, GROUP)).transpose(0, 1).flatten(1, 2)


def _store(s, a, n, out, lse):
    s["out"][a:a + n] = _by_row(out).bfloat16()
    s["lse"][a:a + n] = _by_row(lse)[..., 0]


def _window(s):
    case = s["case"]
    if own:
        s["cache"].window_attn(s["requests"], s["tokens"], 0, 1, s["q"], case["sinks"], case["window"], SCALE,
                               s["out"], s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    for r in range(len(s["tokens"])):
        a, n = s["first"][r], s["tokens"][r]
        t, mask = _visible(s, case, r)
        k, v = _values(s, case, r, t)
        x = _logits(s["q"][a:a + n], k).masked_fill_(~mask.repeat_interleave(GROUP, 0), -math.inf)
        m = x.amax(-1, keepdim=True)
        p = x.sub_(m).exp_()
        z = p.sum(-1, keepdim=True)
        _store(s, a, n, torch.bmm(p, v.transpose(0, 1)) / z, m + z.log())
    return s["out"], s["lse"]


def _shared(s):
    case = s["case"]
    P = case["prefix"]
    if own:
        s["cache"].shared_attn(s["requests"], s["tokens"], 0, 1, s["prefix"], P, s["own_first"], s["q"], SCALE,
                               s["out"], s["lse"], workspace=s["workspace"])
        return s["out"], s["lse"]
    R = len(s["tokens"])
    k, v = _values(s, case, R, torch.arange(P, device="cuda"))
    x = _logits(s["q"], k)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    z, o = p.sum(-1, keepdim=True), torch.bmm(p, v.transpose(0, 1))
    for r in range(R):
        a, n = s["first"][r], s["tokens"][r]
        c = s["ctx"][r]
        t = torch.arange(s["own_first"], c, device="cuda")
        mask = t <= torch.arange(c - n, c, device="cuda")[:, None]
        k, v = _values(s, case, r, t)
        x = _logits(s["q"][a:a + n], k).masked_fill_(~mask.repeat_interleave(GROUP, 0), -math.inf)
        rows = slice(a * GROUP, (a + n) * GROUP)
        mr = torch.maximum(m[:, rows], x.amax(-1, keepdim=True))
        p = (x - mr).exp()
        f = (m[:, rows] - mr).exp()
        zr = z[:, rows] * f + p.sum(-1, keepdim=True)
        _store(s, a, n, (o[:, rows] * f + torch.bmm(p, v.transpose(0, 1))) / zr, mr + zr.log())
    return s["out"], s["lse"]


def _weights(s):
    case = s["case"]
    if own:
        s["cache"].window_weights(s["requests"], s["tokens"], 0, 1, s["q"], s["lse"], case["sinks"], case["window"],
                                  SCALE, s["weights"])
        return s["weights"]
    for r in range(len(s["tokens"])):
        a, n = s["first"][r], s["tokens"][r]
        t, mask = _visible(s, case, r)
        x = _logits(s["q"][a:a + n], _values(s, case, r, t)[0])
        lse = s["lse"][a:a + n].view(n, KV_HEADS, GROUP).transpose(0, 1).reshape(KV_HEADS, -1, 1)
        p = x.sub_(lse).exp_().masked_fill_(~mask.repeat_interleave(GROUP, 0), 0.0)
        s["weights"][r, :s["ctx"][r]] = 0
        s["weights"][r, t] = p.sum((0, 1))
    return s["weights"]


def _evict(s):
    case = s["case"]
    n, L, keep, lo, hi = case["context"], case["layers"], case["keep"], case["first"], case["context"] - case["last"]
    # the request has its whole context again
    if own:
        s["cache"].request_end(s["request"])
    s["request"] = _begin(s, 0, n, L, 0)
    if own:
        s["cache"].evict(s["request"], s["weights"], keep, lo, case["last"], s["kept"], s["weights_out"],
                         workspace=s["workspace"])
    else:
        at = torch.arange(n, device="cuda")
        w = s["weights"].masked_fill((at < lo) | (at >= hi), math.inf)
        kept = w.sort(dim=1, descending=True, stable=True).indices[:, :keep].sort(1).values
        s["kept"].copy_(kept)
        s["weights_out"].copy_(s["weights"].gather(1, kept))
        s["keys"][0, :, :keep] = s["keys"][0].gather(1, kept[:, :, None].expand(L, keep, INDEX_DIM))
        s["scales"][0, :, :keep] = s["scales"][0].gather(1, kept)
        # rows past the kept ones' number go to the free rows before it, in order
        base = n * torch.arange(L, device="cuda")[:, None]
        row = s["slots"][0].long().gather(1, kept) - base
        used = torch.zeros(L, n, dtype=torch.bool, device="cuda").scatter_(1, row, True)[:, :keep]
        free = (~used).nonzero()
        moves = (row >= keep).nonzero()
        to, source = free[:, 1] + n * free[:, 0], row[row >= keep] + n * moves[:, 0]
        s["pool"][to] = s["pool"][source]
        row[row >= keep] = free[:, 1]
        s["slots"][0, :, :keep] = (row + base).int()
    return (s["kept"], s["weights_out"].view(torch.int32), s["keys"][0, :, :keep], s["scales"][0, :, :keep].view(torch.int16),
            s["slots"][0, :, :keep], s["pool"].view(torch.int32))


def run(s):
    return {"window": _window, "shared": _shared, "weights": _weights, "evict": _evict}[s["case"]["op"]](s)


# ------------------------------------------------------------ exact results

def _exact_rows(s, case, r):
    """All of request r's K and V in 64 bits, one row of the pool after the other."""
    c = s["ctx"][r]
    base = sum(s["ctx"][:r])
    rows = s["pool"][base:base + c]
    if case["rows"] == "bf16":
        kv = rows.view(torch.bfloat16).double().view(c, 8, HEAD_DIM)
    else:
        codes = rows[:, :1024].contiguous().view(torch.float8_e4m3fn).float().double().view(c, 8, HEAD_DIM)
        kv = codes * rows[:, 1024:].contiguous().view(torch.float16).double().view(c, 8, 1)
    return kv[:, :4], kv[:, 4:]


def exact(case, seed):
    """From the definitions, in 64 bits, head by head."""
    if case["op"] == "evict":
        return None       # copies and whole numbers: equal or not
    global own
    before, own = own, False
    s = prepare(case, seed)
    own = before
    rows = s["q"].shape[0]
    out = torch.zeros(rows, Q_HEADS, HEAD_DIM, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, Q_HEADS, dtype=torch.float64, device="cuda")
    weights = torch.zeros(len(s["tokens"]), max(s["ctx"]), dtype=torch.float64, device="cuda")
    if case["op"] == "shared":
        kp, vp = _exact_rows(s, case, len(s["tokens"]))
    for r, n in enumerate(s["tokens"]):
        a, c = s["first"][r], s["ctx"][r]
        k, v = _exact_rows(s, case, r)
        t = torch.arange(c, device="cuda")
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            p = torch.arange(c - n + i0, c - n + i1, device="cuda")[:, None]
            if case["op"] == "shared":
                see = (t >= s["own_first"]) & (t <= p)
            else:
                see = (t <= p) & ((t < case["sinks"]) | (p - t < case["window"]))
            for h in range(Q_HEADS):
                q = s["q"][a + i0:a + i1, h].double()
                x = (q @ k[:, h // 4].T / math.sqrt(HEAD_DIM)).masked_fill(~see, -math.inf)
                if case["op"] == "weights":
                    weights[r, :c] += (x - s["lse"][a + i0:a + i1, h, None].double()).exp().sum(0)
                    continue
                values = v[:, h // 4]
                if case["op"] == "shared":
                    x = torch.cat([q @ kp[:, h // 4].T / math.sqrt(HEAD_DIM), x], 1)
                    values = torch.cat([vp[:, h // 4], values])
                lse[a + i0:a + i1, h] = x.logsumexp(1)
                out[a + i0:a + i1, h] = torch.softmax(x, 1) @ values
    return weights if case["op"] == "weights" else (out, lse)

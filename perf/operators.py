"""Measured cases of the chunk operators (several queries of a request at once)
and of the operators on a cache's pages.

A chunk is the newest n tokens of some requests: a piece of a prompt, or draft
tokens to verify.  Token i of a request's chunk sits at position
ctx_len - n + i, and its query sees the tokens up to that position.  Rows of a
call are laid out request after request (layer by layer where a call has
several layers).

  append   quantise and store the index keys and KV rows of a chunk
  score    index scores of every query of a chunk, reduced to blocks of four tokens
  select   the best blocks of every query, in ascending order
  attend   attention of every query over its own selected blocks
  fork     a new request that starts with the first tokens of another one
  compact  live requests slide to the front of the pool once one has ended

`own` chooses between elementary torch operations on the cache's tensors and
the library's calls.
"""
import math

import torch

own = False

KV_HEADS, HEAD_DIM, Q_HEADS, GROUP = 4, 128, 16, 4
INDEX_HEADS, INDEX_DIM = 8, 64
ROW = {"bf16": 2048, "fp8": 1040}
BUDGET = 2048


def listed():
    return [
        # four draft tokens of eight requests are stored at one layer: latency
        {"name": "append draft", "op": "append", "requests": 8, "tokens": 4, "context": 8192, "layers": 1, "rows": "bf16"},
        # a piece of a long prompt, kept as FP8 rows
        {"name": "append prompt", "op": "append", "requests": 1, "tokens": 8191, "context": 32768, "layers": 4, "rows": "fp8"},
        # draft tokens scored against long contexts, queries as the decode step has them
        {"name": "score draft", "op": "score", "requests": 4, "tokens": 4, "context": 65536, "query": "f32"},
        # a piece of a long prompt late in it
        {"name": "score prompt", "op": "score", "requests": 1, "tokens": 2048, "context": 131072, "query": "bf16"},
        # selections of draft tokens
        {"name": "select draft", "op": "select", "requests": 8, "tokens": 4, "context": 131072},
        # selections of a piece of a prompt
        {"name": "select prompt", "op": "select", "requests": 1, "tokens": 2048, "context": 131072},
        # draft tokens attend over FP8 rows
        {"name": "attend draft", "op": "attend", "requests": 8, "tokens": 4, "context": 65536, "rows": "fp8", "spread": 0.4},
        # a piece of a prompt attends over BF16 rows
        {"name": "attend prompt", "op": "attend", "requests": 1, "tokens": 2048, "context": 32768, "rows": "bf16", "spread": 0.4},
        # a second answer from a short prompt
        {"name": "fork short", "op": "fork", "context": 2047, "prefix": 1021, "layers": 12, "rows": "fp8"},
        # a conversation branches late
        {"name": "fork long", "op": "fork", "context": 32768, "prefix": 32001, "layers": 12, "rows": "bf16"},
        # short requests come and go
        {"name": "compact short", "op": "compact", "requests": 3, "context": 509, "layers": 12, "rows": "fp8"},
        # the pool is closed up behind a long request
        {"name": "compact long", "op": "compact", "requests": 4, "context": 16384, "layers": 12, "rows": "bf16"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "score", "select", "attend", "attend", "fork", "compact"])
    rows = rng.choice(["bf16", "fp8"])
    requests = rng.choice([1, 1, 2, 3, 5, 8])
    if op == "append":
        tokens = _spread(rng, 1, 8192 // requests)
        return {"op": op, "requests": requests, "tokens": tokens, "context": tokens + _spread(rng, 8, 16384),
                "layers": rng.choice([1, 1, 2, 3]), "rows": rows}
    if op == "score":
        tokens = _spread(rng, 1, 2048 // requests)
        return {"op": op, "requests": requests, "tokens": tokens, "context": tokens + _spread(rng, 8, 120000),
                "query": rng.choice(["f32", "bf16"])}
    if op == "select":
        tokens = _spread(rng, 1, 2048 // requests)
        return {"op": op, "requests": requests, "tokens": tokens, "context": tokens + _spread(rng, 2500, 120000)}
    if op == "attend":
        tokens = _spread(rng, 1, 2048 // requests)
        return {"op": op, "requests": requests, "tokens": tokens, "context": tokens + _spread(rng, 8, 60000),
                "rows": rows, "spread": rng.choice([0.2, 0.4, 0.8])}
    if op == "fork":
        context = _spread(rng, 64, 32768)
        return {"op": op, "context": context, "prefix": rng.randint(context // 2, context),
                "layers": rng.choice([1, 4, 12]), "rows": rows}
    return {"op": op, "requests": rng.choice([2, 3, 4]), "context": _spread(rng, 64, 16384),
            "layers": rng.choice([1, 4, 12]), "rows": rows}


# -------------------------------------------------------------------- sizes

def _lengths(case):
    """(context, tokens) of each request of a chunk: ragged over the batch."""
    out = []
    for r in range(case.get("requests", 1)):
        n = max(1, case["tokens"] - r)
        out.append((max(n, case["context"] - 37 * r), n))
    return out


def _visible(ctx, n):
    """Blocks that each query of a request's chunk sees."""
    return [(ctx - n + i) // 4 + 1 for i in range(n)]


def work(case):
    op = case["op"]
    row = ROW[case.get("rows", "bf16")]
    if op == "fork":
        return {"bytes": case["layers"] * case["prefix"] * (2 * (row + INDEX_DIM + 2) + 4), "flops": 0}
    if op == "compact":
        n = case["layers"] * case["context"]
        return {"bytes": (case["requests"] - 1) * n * (2 * row + 8) + 4 * n, "flops": 0}
    lens = _lengths(case)
    rows = sum(n for _, n in lens)
    if op == "append":
        return {"bytes": case["layers"] * rows * (4 * INDEX_DIM + 2048 + INDEX_DIM + 2 + row + 4), "flops": 0}
    blocks = sum(sum(_visible(c, n)) for c, n in lens)
    if op == "score":
        q = 4 if case["query"] == "f32" else 2
        pairs = sum(n * (2 * c - n + 1) // 2 for c, n in lens)
        return {"bytes": sum(c for c, _ in lens) * 66 + rows * INDEX_HEADS * (INDEX_DIM * q + 4) + 4 * blocks,
                "flops": pairs * INDEX_HEADS * (2 * INDEX_DIM + 2)}
    k = BUDGET // 4
    kept = sum(min(k, v) for c, n in lens for v in _visible(c, n))
    if op == "select":
        return {"bytes": 4 * blocks + 4 * kept + 4 * rows, "flops": 0}
    used = sum(min(c, 4 * sum(min(k, v) for v in _visible(c, n))) for c, n in lens)
    return {"bytes": used * row + 4 * kept + rows * Q_HEADS * (HEAD_DIM * 4 + 4),
            "flops": 4 * kept * Q_HEADS * HEAD_DIM * 4}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _keys(g, n):
    """Index keys as they are stored: e4m3 codes and one fp16 scale a token."""
    k = _randn(g, n, INDEX_DIM)
    sc = (k.abs().amax(1) / 448).half()
    return (k / sc.float()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), sc


def _kv_rows(g, n, kind):
    x = _randn(g, n, 8, HEAD_DIM).bfloat16()
    if kind == "bf16":
        return x.view(n, 1024).view(torch.uint8)
    x = x.float()
    sc = (x.abs().amax(2) / 448).half()
    codes = (x / sc.float()[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.cat([codes.view(n, 1024).view(torch.uint8), sc.view(torch.uint8).view(n, 16)], 1)


def _cache(case, requests, context, layers, pool_rows):
    """The cache's tensors, and (for the library) the cache itself."""
    kind = case.get("rows", "bf16")
    if own:
        import sparse_attention_decode_qsa_gb300 as Q
        c = Q.Cache(n_layers=layers, max_requests=requests, ctx_capacity=context, hbm_pool_rows=pool_rows,
                    budget_tokens=BUDGET, ring_tokens=64, staging_rows=0,
                    kv_format=Q.KV_FP8 if kind == "fp8" else Q.KV_BF16)
        return {"cache": c, "pool": c.pool, "keys": c.index_keys, "scales": c.index_scales, "slots": c.slot_table}
    empty = lambda dtype, *shape: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    return {"pool": empty(torch.uint8, pool_rows, ROW[kind]),
            "keys": torch.zeros(requests, layers, context, INDEX_DIM, dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros(requests, layers, context, dtype=torch.float16, device="cuda"),
            "slots": torch.full((requests, layers, context), -1, dtype=torch.int32, device="cuda")}


def _begin(s, r, ctx, layers, base):
    """Lease request r, all of its rows in the pool from row `base` on."""
    if own:
        return s["cache"].request_begin(ctx)
    s["slots"][r, :, :ctx] = base + torch.arange(layers * ctx, dtype=torch.int32, device="cuda").view(layers, ctx)
    return r


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "fork":
        n, L = case["context"], case["layers"]
        s = _cache(case, 2, n, L, 2 * L * n)
        s["parent"] = _begin(s, 0, n, L, 0)
        s["pool"][:L * n] = torch.randint(0, 256, (L * n, s["pool"].shape[1]), generator=g, device="cuda", dtype=torch.uint8)
        s["pool"][L * n:] = 0
        s["keys"][0] = torch.randint(0, 127, (L, n, INDEX_DIM), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"][0] = _randn(g, L, n).abs().half()
    elif op == "compact":
        n, L, R = case["context"], case["layers"], case["requests"]
        s = _cache(case, R, n, L, R * L * n)
        s["live"] = [_begin(s, r, n, L, r * L * n) for r in range(R)]
        s["pool"].copy_(torch.randint(0, 256, s["pool"].shape, generator=g, device="cuda", dtype=torch.uint8))
    else:
        s = _prepare_chunk(case, g)
    return dict(s, case=case)


def _prepare_chunk(case, g):
    op = case["op"]
    L = case.get("layers", 1)
    lens = _lengths(case)
    R, cap = len(lens), max(c for c, _ in lens)
    kept = op in ("append", "attend")           # the paths that touch KV rows
    bases = [L * sum(c for c, _ in lens[:r]) for r in range(R)]
    total = L * sum(c for c, _ in lens)
    s = _cache(case, R, cap, L, total)
    s["requests"] = [_begin(s, r, c, L, bases[r]) for r, (c, _) in enumerate(lens)]
    s.update(tokens=[n for _, n in lens], ctx=[c for c, _ in lens], bases=bases)
    rows = sum(n for _, n in lens)
    first = [sum(n for _, n in lens[:r]) for r in range(R)]
    s.update(n_rows=rows, first=first)
    positions = torch.cat([torch.arange(c - n, c, device="cuda") for c, n in lens])
    s["positions"] = positions
    if kept:
        for a in range(0, total, 1 << 18):
            e = min(total, a + (1 << 18))
            s["pool"][a:e] = _kv_rows(g, e - a, case["rows"])
    if op == "append":
        s["k_new"] = _randn(g, L * rows, INDEX_DIM)
        s["kv_new"] = _kv_rows(g, L * rows, "bf16")
    stride = (cap + 3) // 4
    K = BUDGET // 4
    if op == "score":
        for r, (c, _) in enumerate(lens):
            s["keys"][r, 0, :c], s["scales"][r, 0, :c] = _keys(g, c)
        q = _randn(g, rows, INDEX_HEADS, INDEX_DIM)
        s["q_idx"] = q if case["query"] == "f32" else q.bfloat16()
        s["w"] = torch.rand(rows, INDEX_HEADS, generator=g, device="cuda")
        s["blk"] = torch.full((rows, stride), -math.inf, device="cuda")
    if op in ("select", "attend"):
        # block scores of neighbouring queries go together: a part that all
        # share, one that 16 share, one of their own; the first block and the
        # newest ones always count
        seen = positions // 4
        noise = case.get("spread", 0.4)
        blk = torch.empty(rows, stride, device="cuda")
        for r in range(R):
            a, e = first[r], first[r] + s["tokens"][r]
            part = _randn(g, (e - a + 15) // 16, stride).repeat_interleave(16, 0)[:e - a]
            blk[a:e] = _randn(g, stride) + 0.7 * part + noise * _randn(g, e - a, stride)
        at = torch.arange(stride, device="cuda")
        blk += 6.0 * ((at == 0) | (at > seen[:, None] - 16))
        s["blk"] = blk
        s["sel"] = torch.full((rows, K), -1, dtype=torch.int32, device="cuda")
        s["n_sel"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    if op == "attend":
        blk = blk.masked_fill(at > seen[:, None], -math.inf)
        k = min(K, stride)
        top = blk.topk(k, dim=1).indices
        s["n_sel"] = (seen + 1).clamp(max=K).int()
        top = top.masked_fill(torch.arange(k, device="cuda") >= s["n_sel"][:, None], 1 << 30).sort(1).values
        s["sel"][:, :k] = torch.where(top == 1 << 30, -1, top).int()
        del s["blk"]
        s["q"] = _randn(g, rows, Q_HEADS, HEAD_DIM).bfloat16()
        s["out"] = torch.zeros(rows, Q_HEADS, HEAD_DIM, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(rows, Q_HEADS, device="cuda")
        if own:
            need = s["cache"].chunk_attn_workspace_bytes(s["requests"], s["tokens"], 0, 1, BUDGET)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------- runs

def run(s):
    return {"append": _append, "score": _score, "select": _select, "attend": _attend,
            "fork": _fork, "compact": _compact}[s["case"]["op"]](s)


def _quantise(x):
    """(e4m3 codes, fp16 scale) of vectors in the last dimension."""
    sc = (x.abs().amax(-1, keepdim=True) / 448).clamp(max=65504).half()
    f = sc.float()
    codes = torch.where(f > 0, x / torch.where(f > 0, f, 1.0), 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes, sc[..., 0]


def _region(s, r):
    """KV rows of request r: [layers][context][row bytes]."""
    L, c, b = s["case"].get("layers", 1), s["ctx"][r], s["bases"][r]
    return s["pool"][b:b + L * c].view(L, c, -1)


def _of_chunk(s, x, r):
    """Rows of request r in a tensor of the chunk's rows, with the layers in front."""
    L = s["case"].get("layers", 1)
    return x.view(L, s["n_rows"], *x.shape[1:])[:, s["first"][r]:s["first"][r] + s["tokens"][r]]


def _stored(s, r):
    """What an append leaves of request r's chunk: codes, scales, rows, slots."""
    c, n = s["ctx"][r], s["tokens"][r]
    rows = _region(s, r)[:, c - n:]
    kv = ([rows.view(torch.bfloat16)] if s["case"]["rows"] == "bf16" else
          [rows[..., :1024].view(torch.float8_e4m3fn), rows[..., 1024:].view(torch.float16)])
    return [s["keys"][r, :, c - n:c].view(torch.float8_e4m3fn), s["scales"][r, :, c - n:c],
            s["slots"][r, :, c - n:c], *kv]


def _append_one(s, r):
    L, c, n = s["case"]["layers"], s["ctx"][r], s["tokens"][r]
    codes, sc = _quantise(_of_chunk(s, s["k_new"], r))
    s["keys"][r, :, c - n:c] = codes.view(torch.uint8)
    s["scales"][r, :, c - n:c] = sc
    kv = _of_chunk(s, s["kv_new"], r)
    if s["case"]["rows"] == "fp8":
        x, xs = _quantise(kv.contiguous().view(torch.bfloat16).float().view(L, n, 8, HEAD_DIM))
        kv = torch.cat([x.view(torch.uint8).view(L, n, 1024), xs.contiguous().view(torch.uint8).view(L, n, 16)], -1)
    _region(s, r)[:, c - n:] = kv
    at = torch.arange(c - n, c, dtype=torch.int32, device="cuda")
    s["slots"][r, :, c - n:c] = s["bases"][r] + c * torch.arange(L, dtype=torch.int32, device="cuda")[:, None] + at


def _append(s):
    if own:
        s["cache"].append_chunk(s["requests"], s["tokens"], 0, s["case"]["layers"], s["k_new"], s["kv_new"])
    else:
        [_append_one(s, r) for r in range(len(s["ctx"]))]
    return [_stored(s, r) for r in range(len(s["ctx"]))]


def _score_one(s, r):
    a, n, c = s["first"][r], s["tokens"][r], s["ctx"][r]
    key = s["keys"][r, 0, :c].view(torch.float8_e4m3fn).float() * s["scales"][r, 0, :c].float()[:, None]
    y = (s["q_idx"][a:a + n].float().view(n * INDEX_HEADS, INDEX_DIM) @ key.T).relu_().view(n, INDEX_HEADS, c)
    y = torch.bmm(s["w"][a:a + n].float()[:, None], y)[:, 0]
    y = y.masked_fill(torch.arange(c, device="cuda") > s["positions"][a:a + n, None], -math.inf)
    nb = (c + 3) // 4
    s["blk"][a:a + n, :nb] = torch.nn.functional.pad(y, (0, 4 * nb - c), value=-math.inf).view(n, nb, 4).amax(2)


def _score(s):
    if own:
        s["cache"].chunk_index_score(s["requests"], s["tokens"], 0, 1, s["q_idx"], s["w"], s["blk"])
    else:
        [_score_one(s, r) for r in range(len(s["ctx"]))]
    return s["blk"]


def _select(s):
    if own:
        s["cache"].chunk_select_topk(s["requests"], s["tokens"], 0, 1, s["blk"], BUDGET, s["sel"], s["n_sel"])
    else:
        blocks = s["positions"] // 4 + 1
        K = min(BUDGET // 4, s["blk"].shape[1])
        x = (s["blk"] + 0.0).masked_fill(torch.arange(s["blk"].shape[1], device="cuda") >= blocks[:, None], -math.inf)
        order = x.sort(dim=1, descending=True, stable=True).indices[:, :K]
        s["n_sel"].copy_(blocks.clamp(max=BUDGET // 4))
        there = torch.arange(K, device="cuda") < s["n_sel"][:, None]
        ids = order.masked_fill(~there, 1 << 30).sort(1).values
        s["sel"][:, :K] = torch.where(there, ids.int(), s["sel"][:, :K])
    return s["sel"], s["n_sel"]


def _attend_one(s, r):
    a, n = s["first"][r], s["tokens"][r]
    at = s["positions"][a:a + n]
    sel = s["sel"][a:a + n].long()
    there = torch.arange(sel.shape[1], device="cuda") < s["n_sel"][a:a + n, None]
    tok = (sel[:, :, None] * 4 + torch.arange(4, device="cuda")).view(n, -1)
    there = there.repeat_interleave(4, 1) & (tok <= at[:, None])
    rows = s["pool"][s["slots"][r, 0][torch.where(there, tok, 0)].long()]
    if s["case"]["rows"] == "bf16":
        kv = rows.view(torch.bfloat16).float().view(n, -1, 2, KV_HEADS, HEAD_DIM)
    else:
        kv = (rows[..., :1024].view(torch.float8_e4m3fn).float().view(n, -1, 2, KV_HEADS, HEAD_DIM) *
              rows[..., 1024:].view(torch.float16).float().view(n, -1, 2, KV_HEADS, 1))
    q = s["q"][a:a + n].float().view(n, KV_HEADS, GROUP, HEAD_DIM) * HEAD_DIM ** -0.5
    x = torch.matmul(q, kv[:, :, 0].permute(0, 2, 3, 1)).masked_fill(~there[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    z = p.sum(-1, keepdim=True)
    s["out"][a:a + n] = (torch.matmul(p, kv[:, :, 1].transpose(1, 2)) / z).view(n, Q_HEADS, HEAD_DIM).bfloat16()
    s["lse"][a:a + n] = (m + z.log()).view(n, Q_HEADS)


def _attend(s):
    if own:
        s["cache"].chunk_sparse_attn(s["requests"], s["tokens"], 0, 1, s["q"], s["sel"], s["n_sel"], BUDGET,
                                     HEAD_DIM ** -0.5, s["out"], s["lse"], workspace=s["workspace"])
    else:
        [_attend_one(s, r) for r in range(len(s["ctx"]))]
    return s["out"], s["lse"]


def _fork(s):
    n, L, k = s["case"]["context"], s["case"]["layers"], s["case"]["prefix"]
    base = L * n
    if own:
        child = s["cache"].request_fork(s["parent"], k)
        s["cache"].request_end(child)
    else:
        s["keys"][1, :, :k] = s["keys"][0, :, :k]
        s["scales"][1, :, :k] = s["scales"][0, :, :k]
        s["pool"][base:base + L * k] = s["pool"][:L * n].view(L, n, -1)[:, :k].reshape(L * k, -1)
        s["slots"][1, :, :k] = base + torch.arange(L * k, dtype=torch.int32, device="cuda").view(L, k)
    return (s["keys"][1, :, :k], s["scales"][1, :, :k].view(torch.int16),
            s["pool"][base:base + L * k].view(torch.int32), s["slots"][1, :, :k])


def _compact(s):
    n, L = s["case"]["context"], s["case"]["layers"]
    size = L * n
    gone = s["live"].pop(0)
    if own:
        s["cache"].request_end(gone)
        s["cache"].compact()
    else:
        s["pool"][:-size] = s["pool"][size:].clone()
        s["slots"] -= size
    s["live"].append(_begin(s, gone, n, L, size * len(s["live"])))
    return s["pool"].view(torch.int32), s["slots"]


# ------------------------------------------------------------ exact results

def exact(case, seed):
    """From the definitions, in 64 bits."""
    if case["op"] in ("select", "fork", "compact"):
        return None       # copies and whole numbers: equal or not
    global own
    before, own = own, False
    s = prepare(case, seed)
    own = before
    return {"append": _exact_append, "score": _exact_score, "attend": _exact_attend}[case["op"]](s)


def _exact_append(s):
    """Scales and quotients before their roundings."""
    out = []
    for r in range(len(s["ctx"])):
        k = _of_chunk(s, s["k_new"], r).double()
        top = k.abs().amax(-1)
        kv = _of_chunk(s, s["kv_new"], r).contiguous().view(torch.bfloat16).double()
        rows = [kv]
        if s["case"]["rows"] == "fp8":
            x = kv.unflatten(-1, (8, HEAD_DIM))
            most = x.abs().amax(-1)
            rows = [(x * (448 / most)[..., None]).flatten(-2), most / 448]
        out.append([k * (448 / top)[..., None], top / 448, None, *rows])
    return out


def _exact_score(s):
    out = torch.full(s["blk"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r in range(len(s["ctx"])):
        c = s["ctx"][r]
        key = (s["keys"][r, 0, :c].view(torch.float8_e4m3fn).float().double() *
               s["scales"][r, 0, :c].double()[:, None]).T.contiguous()
        for a in range(0, s["tokens"][r], 64):
            rows = slice(s["first"][r] + a, s["first"][r] + min(a + 64, s["tokens"][r]))
            total = 0
            for h in range(INDEX_HEADS):
                total = total + s["w"][rows, h].double()[:, None] * (s["q_idx"][rows, h].double() @ key).clamp(min=0)
            for i in range(4):      # the i-th token of every block
                part = total[:, i::4]
                at = torch.arange(i, c, 4, device="cuda")
                part = part.masked_fill(at > s["positions"][rows, None], -math.inf)
                out[rows, :part.shape[1]] = torch.maximum(out[rows, :part.shape[1]], part)
    return out


def _exact_attend(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    n_sel, positions = s["n_sel"].tolist(), s["positions"].tolist()
    for r in range(len(s["ctx"])):
        region = _region(s, r)[0]
        if s["case"]["rows"] == "bf16":
            kv = region.view(torch.bfloat16).double().view(-1, 8, HEAD_DIM)
        else:
            kv = (region[:, :1024].view(torch.float8_e4m3fn).float().double().view(-1, 8, HEAD_DIM) *
                  region[:, 1024:].view(torch.float16).double().view(-1, 8, 1))
        k, v = kv[:, :4].repeat_interleave(GROUP, 1), kv[:, 4:].repeat_interleave(GROUP, 1)
        for i in range(s["first"][r], s["first"][r] + s["tokens"][r]):
            t = (4 * s["sel"][i, :n_sel[i], None].long() + torch.arange(4, device="cuda")).flatten()
            t = t[t <= positions[i]]
            x = torch.einsum("hd,thd->ht", s["q"][i].double(), k[t]) / math.sqrt(HEAD_DIM)
            lse[i] = torch.logsumexp(x, 1)
            out[i] = torch.einsum("ht,thd->hd", torch.softmax(x, 1), v[t])
    return out, lse

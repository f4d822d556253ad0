"""Attention over a window with sinks, attention over a shared prefix and the
attention weight of each cached token on the GPU, against plain implementations
in float64, at the lengths, windows and placements where they can go wrong; and
the refusals.

Tolerances.  Attention: the probabilities go into the product as bf16 beside BF16
rows and as f16 beside FP8 rows (at most 2^-8 of each term of sum p|v|), the
output is rounded once to bf16 (2^-8 of it), fp32 sums add less than 1e-4 of
sum p|v|.  lse: 128 products in fp32 (2^-17 of scale * sum |q_d k_d|) and a sum of
up to 2^13 terms (1e-5).  Weights: a term's logit is off by 2^-17 of scale *
sum |q_d k_d| and by 2^-22 of its distance to the lse (under 64 here: 2^-16), the
sum of up to 2^12 terms by 2^-12 of itself at most."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from oracle import qsa_oracle as O
from tests import qsa_check as QC
from tests.test_gpu_chunk import NEG, SCALE, Filled, _clean, _queries
from tests.test_gpu_planned_misses import _planned

pytestmark = pytest.mark.gpu

FULL = (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _seen(p, sinks, window):
    return [t for t in range(p + 1) if t < sinks or t > p - window]


def _attend(q_bits, K, V, scale=SCALE):
    """out, lse, sum p|v| and the bound of the logits' sizes, all heads at once."""
    q = O.decode_bf16(q_bits).reshape(16, 128)
    if len(K) == 0:
        return np.zeros((16, 128)), np.full(16, -np.inf), np.zeros((16, 128)), np.zeros(16)
    Kh, Vh = K[:, np.arange(16) // 4], V[:, np.arange(16) // 4]
    x = scale * np.einsum("thd,hd->ht", Kh, q)
    m = x.max(1, keepdims=True)
    p = np.exp(x - m)
    z = p.sum(1, keepdims=True)
    size = abs(scale) * np.einsum("thd,hd->ht", np.abs(Kh), np.abs(q)).max(1)
    return np.einsum("ht,thd->hd", p, Vh) / z, (m + np.log(z))[:, 0], np.einsum("ht,thd->hd", p, np.abs(Vh)) / z, size


def _check(rows, q, out, lse, values, scale=SCALE, sample=20):
    """rows: one key per row; values(key) -> K, V of its tokens."""
    assert len(rows) == len(out)
    idx = range(len(rows)) if len(rows) <= sample else \
        sorted(set(np.random.RandomState(3).choice(len(rows), sample, replace=False)) | {0, len(rows) - 1})
    for x in idx:
        o, ls, mag, size = _attend(QC.bits16(q[x]), *values(rows[x]), scale)
        got = out[x].double().cpu().numpy()
        big = 2.0 ** -16 * size.max() if abs(scale) > SCALE else 0.0
        assert np.all(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4 + big) * mag + 1e-30), \
            (x, rows[x], np.abs(got - o).max())
        if lse is not None:
            gl = lse[x].double().cpu().numpy()
            if np.all(ls == -np.inf):
                assert np.all(gl == -np.inf) and np.all(got == 0), (x, rows[x])
            else:
                assert np.all(np.abs(gl - ls) <= 2.0 ** -17 * size + 1e-5), (x, rows[x], np.abs(gl - ls).max())


def _rows(f, n_tokens, layers=1):
    return [(l, r, p) for l in range(layers) for r, p in f.positions(n_tokens)]


def _window(f, n_tokens, q, sinks, window, layers=1, layer0=0, scale=SCALE, **kw):
    out = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:2], float("nan"), device=q.device)
    f.c.window_attn(f.hs, n_tokens, layer0, layers, q, sinks, window, scale, out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


CASES = [
    ([1], [1], 0, 1, 1), ([1], [1], 4, 0, 1), ([6], [6], 2, 0, 1), ([6], [6], 0, 0, 1),
    ([5, 130, 64], [1, 1, 1], 4, 16, 1), ([700, 3, 257], [129, 3, 64], 5, 100, 1), ([300], [300], 0, FULL, 1),
    ([2500], [70], 17, 513, 1), ([900, 40], [0, 7], 3, 33, 2), ([64, 65, 66, 127, 128, 129], [2, 3, 4, 5, 6, 1], 1, 64, 1),
    ([400], [33], 1000, 7, 1), ([1500, 1400], [5, 4], 128, FULL, 1), ([3000], [1], 4, FULL, 2),
    ([200] * 40, [1, 2, 3, 4] * 10, 0, 128, 1), ([385], [385], 130, 1, 1), ([1100], [40], 600, 200, 1),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,sinks,window,layers", CASES)
def test_window_attention_matches_float64(fp8, ctxs, n_tokens, sinks, window, layers):
    f = Filled(ctxs, layers=layers + 1, fp8=fp8, seed=3)
    try:
        q = _queries(layers * sum(n_tokens), 5, f.dev, 1.5)
        out, lse = _window(f, n_tokens, q, sinks, window, layers, layer0=1)
        _clean(f.c)
        _check(_rows(f, n_tokens, layers), q, out, lse, lambda k: f.values(k[1], k[0] + 1, _seen(k[2], sinks, window)))
        out2 = torch.full_like(q, float("nan"))
        f.c.window_attn(f.hs, n_tokens, 1, layers, q, sinks, window, SCALE, out2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_tokens", [[1, 1, 1], [40, 3, 70]])
def test_window_attention_reads_rings_hosts_and_pool_alike(fp8, n_tokens):
    f = Filled([500, 500, 260], [Q.KV_HOST_RING, Q.KV_HOST, Q.KV_HBM], fp8=fp8, seed=5, ring=64, layers=2)
    try:
        q = _queries(2 * sum(n_tokens), 5, f.dev)
        out, lse = _window(f, n_tokens, q, 4, 200, layers=2)
        _clean(f.c)
        _check(_rows(f, n_tokens, 2), q, out, lse, lambda k: f.values(k[1], k[0], _seen(k[2], 4, 200)))
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [2, 70])
def test_window_and_shared_attention_and_weights_complete_a_pending_plan(fp8, tokens):
    f = Filled([800], [Q.KV_HOST_RING], layers=2, ring=16, hot_rows=128, budget=128, fp8=fp8, seed=9)
    try:
        q = _queries(tokens, 7, f.dev)
        values = lambda k: f.values(k[1], 1, _seen(k[2], 4, 700))  # noqa: E731
        _planned(f, 1)
        out, lse = _window(f, [tokens], q, 4, 700, layer0=1)
        _check(_rows(f, [tokens]), q, out, lse, values)
        _planned(f, 1)
        out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
        f.c.shared_attn(f.hs, [tokens], 1, 1, f.hs[0], 300, 300, q, SCALE, out2, lse2)
        _check(_rows(f, [tokens]), q, out2, lse2, lambda k: f.values(k[1], 1, list(range(k[2] + 1))))
        _planned(f, 1)
        w = torch.zeros(1, 800, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 1, 1, q, lse, 4, 700, SCALE, w)
        assert abs(w.double().sum().item() - 16 * tokens) < 1e-3 * 16 * tokens
        # the plan is done: nothing is pending, and the next reads see the same rows
        out3, lse3 = _window(f, [tokens], q, 4, 700, layer0=1)
        assert torch.equal(out, out3) and torch.equal(lse, lse3)
        _clean(f.c)
    finally:
        f.close()


# ------------------------------------------------------------ shared prefix

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("own,n_tokens,prefix_len,own_first,layers", [
    ([1], [1], 1, 0, 1), ([30, 70], [1, 1], 333, 0, 1), ([90, 41, 200], [5, 41, 64], 700, 0, 2),
    ([50, 60], [2, 3], 0, 10, 1), ([20], [20], 129, 1000, 1), ([140] * 20, [1, 3, 2, 4] * 5, 515, 0, 1),
    ([300, 20], [130, 3], 64, 100, 1), ([33] * 70, [1] * 70, 1000, 32, 1), ([40, 50], [0, 9], 100, 7, 2),
    ([25], [1], 5000, 0, 1), ([25, 30], [25, 30], 0, 0, 1), ([10], [4], 0, 1000, 1)])
def test_shared_attention_matches_float64(fp8, own, n_tokens, prefix_len, own_first, layers):
    """The last request holds the prefix; the others' tokens follow it."""
    f = Filled(own + [max(prefix_len, 1) + 3], layers=layers + 1, fp8=fp8, seed=3)
    try:
        R = len(own)
        q = _queries(layers * sum(n_tokens), 5, f.dev, 1.5)
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=f.dev)
        f.c.shared_attn(f.hs[:R], n_tokens, 1, layers, f.hs[R], prefix_len, own_first, q, SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(f.c)

        def values(k):
            a, b = f.values(R, k[0] + 1, list(range(prefix_len))), f.values(k[1], k[0] + 1, list(range(own_first, k[2] + 1)))
            return [np.concatenate(x) for x in zip(a, b)]
        _check(_rows(f, n_tokens, layers), q, out, lse, values)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_batch_of_forks_attends_as_each_of_its_requests_alone(fp8):
    """Requests that hold copies of the prefix: shared attention equals window
    attention over each one's whole context; the parent is one of the batch."""
    f = Filled([600], fp8=fp8, seed=4, grow=40, spare=2 * 640)
    try:
        hs = [f.hs[0]] + [f.c.request_fork(f.hs[0], 600, max_ctx=640) for _ in range(2)]
        g = torch.Generator().manual_seed(3)
        n_tokens = [3, 5, 1]
        for h, n in zip(hs, n_tokens):
            f.c.advance(h, n)
        total = sum(n_tokens)
        kv = torch.randn(total, 1024, generator=g).bfloat16().view(torch.uint8).to(f.dev)
        f.c.append_chunk(hs, n_tokens, 0, 1, torch.randn(total, 64, generator=g).to(f.dev), kv)
        q = _queries(total, 8, f.dev)
        a = [torch.zeros_like(q), torch.zeros(total, 16, device=f.dev)]
        b = [torch.zeros_like(q), torch.zeros(total, 16, device=f.dev)]
        f.c.window_attn(hs, n_tokens, 0, 1, q, 0, FULL, SCALE, *a)
        f.c.shared_attn(hs, n_tokens, 0, 1, hs[0], 600, 600, q, SCALE, *b)
        torch.cuda.synchronize()
        _clean(f.c)
        # both are within their roundings of the same values: 2^-8 of the output
        # each, and 2^-8 of sum p|v| each (|v| < 6, as N(0, 1) over these sizes)
        assert (a[1] - b[1]).abs().max() <= 4e-5
        assert (a[0].float() - b[0].float()).abs().max() <= 2 ** -7 * a[0].float().abs().max() + 2 ** -7
    finally:
        f.close()


@pytest.mark.parametrize("place", [Q.KV_HOST_RING, Q.KV_HOST])
def test_a_shared_prefix_in_host_memory(place):
    f = Filled([50, 60, 300], [Q.KV_HBM, Q.KV_HOST, place], layers=2, ring=64, seed=7)
    try:
        q = _queries(2 * 9, 5, f.dev)
        out, lse = torch.zeros_like(q), torch.zeros(18, 16, device=f.dev)
        f.c.shared_attn(f.hs[:2], [5, 4], 0, 2, f.hs[2], 299, 0, q, SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(f.c)

        def values(k):
            a, b = f.values(2, k[0], list(range(299))), f.values(k[1], k[0], list(range(k[2] + 1)))
            return [np.concatenate(x) for x in zip(a, b)]
        _check(_rows(f, [5, 4], 2), q, out, lse, values)
    finally:
        f.close()


# ---------------------------------------------------------- values and slots

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("tokens", [3, 70])
def test_values_that_are_not_finite_reach_only_the_queries_that_see_them(fp8, value, tokens):
    f = Filled([400], seed=6, fp8=fp8)
    try:
        sinks, window = 4, 90
        p0 = 400 - tokens
        bad = [10, p0 - window + 1, 399]      # never seen; seen by the first query alone; by the last alone
        c = f.c
        for i, r_ in enumerate(c.slot_table[f.hs[0].index, 0, bad].tolist()):
            if fp8:
                c.pool[r_, 1024:].view(torch.float16)[4 if i % 2 else 0:8] = value
            else:
                c.pool[r_].view(torch.bfloat16)[512 if i % 2 else 0:] = value
        q = _queries(tokens, 7, f.dev)
        out, lse = _window(f, [tokens], q, sinks, window)
        rows = _rows(f, [tokens])
        hit = [any(b in _seen(k[2], sinks, window) for b in bad) for k in rows]
        assert 0 < sum(hit) < tokens
        for x, k in enumerate(rows):
            if hit[x]:
                assert not bool(out[x].isfinite().all()), x
            else:
                _check([k], q[x:x + 1], out[x:x + 1], lse[x:x + 1], lambda k: f.values(0, 0, _seen(k[2], sinks, window)))
        # weights: tokens that no query sees and queries that do not see them
        w = torch.full((1, 400), NEG, device=f.dev)
        good = torch.tensor([not h for h in hit], device=f.dev)
        ls = torch.where(good[:, None], lse, -math.inf)
        c.window_weights(f.hs, [tokens], 0, 1, q, ls, sinks, window, SCALE, w)
        assert w[0, 10].item() == 0.0 and bool(w.isfinite().all())
        assert abs(w.double().sum().item() - 16 * (tokens - sum(hit))) <= 1e-3 * 16 * tokens
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -SCALE, 8 * SCALE])
@pytest.mark.parametrize("n_tokens", [[2, 1], [40, 33]])
def test_softmax_scales_of_any_sign_and_size(fp8, scale, n_tokens):
    f = Filled([700, 650], fp8=fp8, seed=4)
    try:
        q = _queries(sum(n_tokens), 3, f.dev)
        out, lse = _window(f, n_tokens, q, 4, 600, scale=scale)
        _clean(f.c)
        _check(_rows(f, n_tokens), q, out, lse, lambda k: f.values(k[1], 0, _seen(k[2], 4, 600)), scale=scale)
    finally:
        f.close()


@pytest.mark.parametrize("n_tokens", [[2], [70]])
def test_bad_slots_are_reported_and_their_tokens_left_out(n_tokens):
    f = Filled([300], seed=10)
    try:
        c = f.c
        c.slot_table[f.hs[0].index, 0, 250] = c.pool.shape[0]
        c.slot_table[f.hs[0].index, 0, 200] = -1                 # cold, but there is no host history
        q = _queries(n_tokens[0], 7, f.dev)
        out, lse = _window(f, n_tokens, q, 2, 150)
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        seen = lambda p: [t for t in _seen(p, 2, 150) if t not in (200, 250)]  # noqa: E731
        _check(_rows(f, n_tokens), q, out, lse, lambda k: f.values(0, 0, seen(k[2])))
        w = torch.zeros(1, 300, device=f.dev)
        c.window_weights(f.hs, n_tokens, 0, 1, q, lse, 2, 150, SCALE, w)
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        assert w[0, 200].item() == 0.0 and w[0, 250].item() == 0.0
        assert abs(w.double().sum().item() - 16 * n_tokens[0]) <= 1e-3 * 16 * n_tokens[0]
        # every slot of the context bad: rows without tokens
        c.slot_table[f.hs[0].index, 0, :] = -5
        out, lse = _window(f, n_tokens, q, 2, 150)
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    finally:
        f.close()


# ------------------------------------------------------------------- weights

def _weights(f, n_tokens, q, lse, sinks, window, layers, layer0):
    """In float64, and the tolerance of every entry."""
    out = np.zeros((layers * len(n_tokens), max(f.ctxs)))
    tol = np.zeros_like(out)
    x = 0
    for l in range(layers):
        for r, n in enumerate(n_tokens):
            K, _ = f.values(r, l + layer0, list(range(f.ctxs[r])))
            Kh = K[:, np.arange(16) // 4]
            for i in range(n):
                p = f.ctxs[r] - n + i
                seen = np.array(_seen(p, sinks, window), dtype=int)
                qd = O.decode_bf16(QC.bits16(q[x])).reshape(16, 128)
                ls = lse[x].double().cpu().numpy()
                x += 1
                if len(seen) == 0 or np.all(ls == -np.inf):
                    continue
                e = np.exp(SCALE * np.einsum("thd,hd->th", Kh[seen], qd) - ls)
                size = SCALE * np.einsum("thd,hd->th", np.abs(Kh[seen]), np.abs(qd))
                out[l * len(n_tokens) + r, seen] += e.sum(1)
                tol[l * len(n_tokens) + r, seen] += (e * (2.0 ** -17 * size + 2.0 ** -16)).sum(1)
    return out, tol + 2.0 ** -12 * out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,sinks,window,layers", CASES)
def test_weights_match_float64(fp8, ctxs, n_tokens, sinks, window, layers):
    f = Filled(ctxs, layers=layers + 1, fp8=fp8, seed=3)
    try:
        q = _queries(layers * sum(n_tokens), 5, f.dev, 1.5)
        _, lse = _window(f, n_tokens, q, sinks, window, layers, layer0=1)
        units, stride = layers * len(ctxs), max(ctxs) + 5
        w = torch.full((units, stride), NEG, device=f.dev)
        f.c.window_weights(f.hs, n_tokens, 1, layers, q, lse, sinks, window, SCALE, w)
        torch.cuda.synchronize()
        _clean(f.c)
        want, tol = _weights(f, n_tokens, q, lse, sinks, window, layers, 1)
        got = w.double().cpu().numpy()
        for u in range(units):
            n = ctxs[u % len(ctxs)]
            assert np.all(np.abs(got[u, :n] - want[u, :n]) <= tol[u, :n]), (u, np.abs(got[u, :n] - want[u, :n]).max())
            assert np.all(got[u, n:] == np.float32(NEG))
        # again, to the bit; and added to what is there (one rounding)
        w2 = torch.full_like(w, NEG)
        f.c.window_weights(f.hs, n_tokens, 1, layers, q, lse, sinks, window, SCALE, w2)
        assert torch.equal(w, w2)
        base = torch.rand_like(w)
        w3 = base.clone()
        f.c.window_weights(f.hs, n_tokens, 1, layers, q, lse, sinks, window, SCALE, w3, accumulate=True)
        for u in range(units):
            n = ctxs[u % len(ctxs)]
            assert torch.equal(w3[u, :n], base[u, :n] + w[u, :n]) and torch.equal(w3[u, n:], base[u, n:])
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_of_every_row_add_up_to_one(fp8):
    f = Filled([1000, 777], fp8=fp8, seed=3)
    try:
        for n_tokens in ([1, 1], [130, 300], [1000, 5]):
            q = _queries(sum(n_tokens), 5, f.dev)
            _, lse = _window(f, n_tokens, q, 0, FULL)
            w = torch.zeros(2, 1000, device=f.dev)
            f.c.window_weights(f.hs, n_tokens, 0, 1, q, lse, 0, FULL, SCALE, w)
            s = w.double().sum(1)
            for u in range(2):
                assert abs(s[u].item() - 16 * n_tokens[u]) <= 2e-4 * 16 * n_tokens[u]
    finally:
        f.close()


# -------------------------------------------------- streams, graphs, workspaces

def test_captured_calls_replay_and_streams_keep_apart():
    f = Filled([3000, 2000, 900], seed=8)
    try:
        c, dev = f.c, f.dev
        bufs = []
        for i, nt in enumerate(([70, 0], [1, 45], [2, 1])):
            rows = sum(nt)
            ws = c.window_attn_workspace_bytes(f.hs[:2], nt, 0, 1, 4, 2500)
            ws2 = c.shared_attn_workspace_bytes(f.hs[:2], nt, 0, 1, f.hs[2], 800, 1500)
            # the call stays inside its workspace
            guard = [torch.full((n + 4096,), 77, dtype=torch.uint8, device=dev) for n in (ws, ws2)]
            bufs.append(dict(nt=nt, q=_queries(rows, i, dev), guard=guard, ws=guard[0][:ws], ws2=guard[1][:ws2],
                             out=torch.zeros(rows, 16, 128, dtype=torch.bfloat16, device=dev),
                             out2=torch.zeros(rows, 16, 128, dtype=torch.bfloat16, device=dev),
                             lse=torch.zeros(rows, 16, device=dev), lse2=torch.zeros(rows, 16, device=dev),
                             w=torch.zeros(2, 3000, device=dev)))

        def step(b):
            c.window_attn(f.hs[:2], b["nt"], 0, 1, b["q"], 4, 2500, SCALE, b["out"], b["lse"], workspace=b["ws"])
            c.window_weights(f.hs[:2], b["nt"], 0, 1, b["q"], b["lse"], 4, 2500, SCALE, b["w"])
            c.shared_attn(f.hs[:2], b["nt"], 0, 1, f.hs[2], 800, 1500, b["q"], SCALE, b["out2"], b["lse2"],
                          workspace=b["ws2"])

        names, want = ("out", "lse", "out2", "lse2", "w"), []
        for b in bufs:
            step(b)
            torch.cuda.synchronize()
            want.append([b[k].clone() for k in names])
            for g in b["guard"]:
                assert bool((g[-4096:] == 77).all())
        streams = [torch.cuda.Stream() for _ in bufs]
        graphs = []
        for b, s in zip(bufs, streams):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(b)
            graphs.append(g)
        for _ in range(5):
            for b in bufs:
                for k in names:
                    b[k].zero_()
                b["ws"].fill_(255)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for b, w in zip(bufs, want):
                for k, x in zip(names, w):
                    assert torch.equal(b[k], x), k
        b = bufs[0]
        b["q"].neg_()
        graphs[0].replay()
        torch.cuda.synchronize()
        o = b["out"].clone()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(o, b["out"]) and not torch.equal(o, want[0][0])
        _clean(c)
    finally:
        f.close()


def test_rows_past_32_bits_of_bytes_and_many_rows():
    """A request behind four gigabytes of other rows, and as many queries as a
    prompt's piece has."""
    n, behind = 1500, 2_200_000
    c = Q.Cache(n_layers=1, max_requests=2, ctx_capacity=behind, hbm_pool_rows=behind + n, staging_rows=0)
    try:
        c.request_begin(behind)
        h = c.request_begin(n)
        base = c.request_info(h).hbm_row_base
        assert base * 2048 > 1 << 32
        dev = c.pool.device
        g = torch.Generator(device=dev).manual_seed(2)
        kv = torch.randn(n, 2, 4, 128, generator=g, device=dev).bfloat16()
        c.pool[base:base + n] = kv.view(n, 1024).view(torch.uint8)
        for tokens in (1, n):
            q = _queries(tokens, 5, dev)
            out, lse, w = torch.zeros_like(q), torch.zeros(tokens, 16, device=dev), torch.zeros(1, n, device=dev)
            c.window_attn([h], [tokens], 0, 1, q, 3, 1000, SCALE, out, lse)
            c.window_weights([h], [tokens], 0, 1, q, lse, 3, 1000, SCALE, w)
            at = torch.arange(n - tokens, n, device=dev)[:, None]
            t = torch.arange(n, device=dev)
            see = (t <= at) & ((t < 3) | (t > at - 1000))
            total = torch.zeros(n, dtype=torch.float64, device=dev)
            for hd in range(16):
                x = (q[:, hd].double() @ kv[:, 0, hd // 4].double().T * SCALE).masked_fill(~see, -math.inf)
                p = torch.softmax(x, 1)
                v = kv[:, 1, hd // 4].double()
                tol = 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 1e-4) * (p @ v.abs())
                assert bool(((out[:, hd].double() - p @ v).abs() <= tol).all())
                assert (lse[:, hd].double() - x.logsumexp(1)).abs().max().item() <= 2e-4
                total += (x - lse[:, hd, None].double()).exp().sum(0)
            assert bool(((w[0].double() - total).abs() <= 1e-3 * total + 1e-6).all())
        _clean(c)
    finally:
        c.close()


# ----------------------------------------------------------------- refusals

def test_refusals_leave_everything_alone():
    f = Filled([200, 100], [Q.KV_HBM, Q.KV_HBM], seed=2)
    try:
        c, dev = f.c, f.dev
        q = _queries(5, 1, dev)
        out = torch.full_like(q, 3.0)
        lse = torch.full((5, 16), 3.0, device=dev)
        w = torch.full((2, 200), 3.0, device=dev)

        def refused(status, fn, *a, **kw):
            with pytest.raises(Q.QsaError) as e:
                fn(*a, **kw)
            assert e.value.status == status, e.value
        ok = (f.hs, [3, 2], 0, 1, q)
        stale = Q._native.Handle(f.hs[0].index, f.hs[0].generation + 1)
        INV = Q.ERR_INVALID_ARG
        refused(INV, c.window_attn, *ok, -1, 5, SCALE, out, lse)
        refused(INV, c.window_attn, *ok, 0, -1, SCALE, out, lse)
        refused(INV, c.window_attn, *ok, 0, 5, float("nan"), out, lse)
        refused(INV, c.window_attn, f.hs, [201, 2], 0, 1, _queries(203, 1, dev), 0, 5, SCALE, torch.zeros(203, 16, 128, dtype=torch.bfloat16, device=dev))
        refused(INV, c.window_attn, [f.hs[0], f.hs[0]], [3, 2], 0, 1, q, 0, 5, SCALE, out, lse)
        refused(INV, c.window_attn, f.hs, [3, 2], 1, 1, q, 0, 5, SCALE, out, lse)
        some = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
        refused(Q.ERR_STALE_HANDLE, c.window_attn, [stale], [5], 0, 1, q, 0, 5, SCALE, out, lse, workspace=some)
        small = torch.zeros(128, dtype=torch.uint8, device=dev)
        refused(INV, c.window_attn, *ok, 0, 5, SCALE, out, lse, workspace=small)
        args = (f.hs[1], 50, 0, q, SCALE, out, lse)
        refused(INV, c.shared_attn, f.hs, [3, 2], 0, 1, f.hs[1], 101, 0, q, SCALE, out, lse)
        refused(INV, c.shared_attn, f.hs, [3, 2], 0, 1, f.hs[1], -1, 0, q, SCALE, out, lse)
        refused(INV, c.shared_attn, f.hs, [3, 2], 0, 1, f.hs[1], 50, -1, q, SCALE, out, lse)
        refused(Q.ERR_STALE_HANDLE, c.shared_attn, f.hs, [3, 2], 0, 1, stale, 50, 0, q, SCALE, out, lse, workspace=some)
        refused(INV, c.shared_attn, f.hs, [3, 2], 0, 1, *args, workspace=small)
        refused(INV, c.window_weights, *ok, lse, 0, -2, SCALE, w)
        refused(INV, c.window_weights, *ok, lse, -1, 2, SCALE, w)
        refused(INV, c.window_weights, *ok, lse, 0, 5, SCALE, torch.zeros(2, 199, device=dev))
        refused(INV, c.window_weights, *ok, lse, 0, 5, float("nan"), w)
        for bad in (dict(q=q.float()), dict(q=q[:4]), dict(out=out.float()), dict(lse=lse[:, :8]), dict(q=q.cpu()),
                    dict(out=out.transpose(0, 1).contiguous().transpose(0, 1))):
            kw = dict(q=q, out=out, lse=lse, **{})
            kw.update(bad)
            with pytest.raises(ValueError):
                c.window_attn(f.hs, [3, 2], 0, 1, kw["q"], 0, 5, SCALE, kw["out"], kw["lse"])
            with pytest.raises(ValueError):
                c.shared_attn(f.hs, [3, 2], 0, 1, f.hs[1], 50, 0, kw["q"], SCALE, kw["out"], kw["lse"])
        with pytest.raises(ValueError):
            c.window_weights(f.hs, [3, 2], 0, 1, q, lse, 0, 5, SCALE, w[:1])
        # no rows: nothing to do
        none = torch.zeros(0, 16, 128, dtype=torch.bfloat16, device=dev)
        c.window_attn(f.hs, [0, 0], 0, 1, none, 0, 5, SCALE, none)
        c.shared_attn(f.hs, [0, 0], 0, 1, f.hs[0], 5, 0, none, SCALE, none)
        torch.cuda.synchronize()
        assert bool((out == 3).all()) and bool((lse == 3).all()) and bool((w == 3).all())
        # weights without rows: zero, or as they were
        c.window_weights(f.hs, [0, 0], 0, 1, none, lse[:0], 0, 5, SCALE, w, accumulate=True)
        assert bool((w == 3).all())
        c.window_weights(f.hs, [0, 0], 0, 1, none, lse[:0], 0, 5, SCALE, w)
        assert bool((w[0] == 0).all()) and bool((w[1, :100] == 0).all()) and bool((w[1, 100:] == 3).all())
        _clean(c)
    finally:
        f.close()

"""Window and shared-prefix attention and attention weights where values lie far
apart, and in size: logits of tokens that a query does not see, V scales from
2^-24 to 2^15 in one row, query elements far below the largest, contexts of tens
of thousands of tokens, many tiles to a CTA.  Against float64.

Tolerances of the attention as in test_gpu_chunk_range.py (the same roundings): per
element 2^-8 of the output, and of sum p|v| 2^-8 beside BF16 rows or 2^-11 beside FP8
rows, 2^-16 of the logits' sizes and 1e-4; FP8 rows also 2^-19 of a row's largest
product times the codes.  Weights as in test_gpu_window.py."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries
from tests.test_gpu_chunk_range import SIGNS, _check, _set_logits, _set_v_scales, _store
from tests.test_gpu_window import FULL, _window

pytestmark = pytest.mark.gpu

LAYOUTS = [([600], [1]), ([600], [3]), ([600], [40]), ([300] * 39, [3] * 39), ([260] * 39, [7] * 39)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _all(f, n_tokens):
    """Every block up to a query's own: causal attention as a selection."""
    sel = [np.arange(p // 4 + 1) for _, p in f.positions(n_tokens)]
    return sel, [len(s) for s in sel]


def _run(f, n_tokens, q, rows=None):
    out, lse = _window(f, n_tokens, q, 0, FULL)
    _clean(f.c)
    sel, nsel = _all(f, n_tokens)
    step = max(1, len(sel) // 40)
    _check(f, n_tokens, q, sel, nsel, out, lse, range(0, len(sel), step) if rows is None else rows)
    return out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("logit", [-20.0, -60.0])
@pytest.mark.parametrize("ctx", [1, 2, 15, 17, 33, 129])
def test_places_past_the_list_leave_low_logits_alone(fp8, logit, ctx):
    for tokens in {1, min(ctx, 6)}:
        f = Filled([ctx], fp8=fp8, seed=3)
        try:
            _set_logits(f, 0, [logit] * ctx)
            _run(f, [tokens], SIGNS.bfloat16().expand(tokens, 16, 128).contiguous().to(f.dev))
        finally:
            f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("step", [4.0, 12.0, 40.0])
@pytest.mark.parametrize("ctxs,n_tokens", [([400], [4]), ([400], [70]), ([9000], [70]), ([300] * 39, [5] * 39)])
def test_later_tokens_do_not_reach_a_query(fp8, step, ctxs, n_tokens):
    """In the chunk, every token's logit is `step` nats above that of the token
    before it, for four tokens at a time."""
    f = Filled(ctxs, fp8=fp8, seed=3)
    try:
        rng = np.random.RandomState(8)
        for r, (n, k) in enumerate(zip(ctxs, n_tokens)):
            logits = rng.randn(n)
            at = np.arange(n - k, n)
            logits[at] = step * (at % 4)
            _set_logits(f, r, logits)
        _run(f, n_tokens, SIGNS.bfloat16().expand(sum(n_tokens), 16, 128).contiguous().to(f.dev))
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("signed", [False, True])
def test_v_scales_of_every_size(ctxs, n_tokens, signed):
    f = Filled(ctxs, fp8=True, seed=3)
    try:
        rng = np.random.RandomState(5)
        for r, n in enumerate(ctxs):
            v = np.exp2(rng.uniform(-24, 15.9, n)) * (rng.choice([-1, 1], n) if signed else 1)
            v[rng.rand(n) < 0.1] = 0
            _set_v_scales(f, r, np.arange(n), v)
            _store(f, r)
        _run(f, n_tokens, _queries(sum(n_tokens), 5, f.dev, scale=3.0))
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("logit", [0.0, 30.0, 55.0, 90.0])
def test_small_values_behind_tokens_without_any(ctxs, n_tokens, logit):
    """The first 160 tokens' V rows are zero, with scale 0, their logits `logit`
    nats above the others'; the rest have scales of 2^-20."""
    f = Filled(ctxs, fp8=True, seed=3)
    try:
        rng = np.random.RandomState(5)
        for r, n in enumerate(ctxs):
            _set_logits(f, r, np.where(np.arange(n) < 160, logit, 0.0) + rng.randn(n))
            _set_v_scales(f, r, np.arange(n), np.where(np.arange(n) < 160, 0.0, 2.0 ** -20 * (1 + rng.rand(n))))
            f.kv[r][0][:160, 512:1024] = 0
            _store(f, r)
        _run(f, n_tokens, SIGNS.bfloat16().expand(sum(n_tokens), 16, 128).contiguous().to(f.dev))
    finally:
        f.close()


@pytest.mark.parametrize("tokens", [3, 40])
@pytest.mark.parametrize("value,scale", [(float("inf"), 2.0 ** -19), (float("nan"), 2.0 ** -19), (1e4, 1.0), (3e4, 2.0 ** -10)])
def test_an_outlier_that_is_not_seen_costs_no_bits(tokens, value, scale):
    """The newest token's V scale is infinite, NaN or large; only the last query
    sees it."""
    f = Filled([500], fp8=True, seed=3)
    try:
        rng = np.random.RandomState(5)
        v = scale * (1 + rng.rand(500))
        v[499] = value
        _set_v_scales(f, 0, np.arange(500), v)
        _store(f, 0)
        q = _queries(tokens, 5, f.dev)
        out, _ = _run(f, [tokens], q, range(tokens - 1 if not np.isfinite(value) else tokens))
        if not np.isfinite(value):
            assert not bool(out[-1].isfinite().all())
    finally:
        f.close()


@pytest.mark.parametrize("tokens", [1, 4, 40])
def test_query_elements_far_apart_beside_fp8_rows(tokens):
    """Elements log-uniform over [2^-36, 1] of the largest, and rows of 2^60 and 2^-60
    (with a softmax scale that makes up for it)."""
    f = Filled([300], fp8=True, seed=3)
    try:
        g = torch.Generator().manual_seed(5)
        e = torch.exp2(-36 * torch.rand(tokens, 16, 128, generator=g))
        q = (e * torch.sign(torch.randn(tokens, 16, 128, generator=g))).bfloat16().to(f.dev)
        out, lse = _run(f, [tokens], q)
        for power in (60, -60):
            o = torch.empty_like(out)
            l = torch.empty_like(lse)
            f.c.window_attn(f.hs, [tokens], 0, 1, (q.float() * 2.0 ** power).bfloat16(), 0, FULL, SCALE * 2.0 ** -power, o, l)
            assert torch.equal(o, out) and torch.equal(l, lse)
    finally:
        f.close()


def _on_device(c, hs, fp8):
    """K and V of every request in float64, from the pool."""
    out = []
    for h in hs:
        n = c.request_info(h).ctx_len
        rows = c.pool[c.slot_table[h.index, 0, :n].long()]
        if fp8:
            kv = rows[:, :1024].contiguous().view(torch.float8_e4m3fn).float().double().view(n, 2, 4, 128)
            kv = kv * rows[:, 1024:].contiguous().view(torch.float16).double().view(n, 2, 4, 1)
        else:
            kv = rows.view(torch.bfloat16).double().view(n, 2, 4, 128)
        out.append((kv[:, 0], kv[:, 1]))
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,sinks,window", [
    ([70001], [1], 4, FULL), ([70001], [2], 4, 50000), ([50000, 30], [4, 30], 130, 41000), ([60001], [6], 3, FULL),
    ([41000], [100], 5, FULL), ([45000, 40000], [33, 70], 300, 39300), ([3000] * 12, [6] * 12, 9, 2500),
    ([9000] * 6, [130] * 6, 0, FULL), ([5000] * 100, [1] * 100, 4, 900)])
def test_long_contexts_and_many_tiles(fp8, ctxs, n_tokens, sinks, window):
    """Shares and pieces at their most, tiles of 256 tokens, several tiles to a CTA;
    attention, its weights, and the same tokens as a shared prefix."""
    total = sum(ctxs)
    c = Q.Cache(n_layers=1, max_requests=len(ctxs) + 1, ctx_capacity=max(ctxs), hbm_pool_rows=total + 8, staging_rows=0,
                kv_format=Q.KV_FP8 if fp8 else Q.KV_BF16)
    try:
        dev = c.pool.device
        hs = [c.request_begin(n) for n in ctxs]
        g = torch.Generator(device=dev).manual_seed(2)
        for a in range(0, total, 1 << 16):
            x = torch.randn(min(total, a + (1 << 16)) - a, 8, 128, generator=g, device=dev).bfloat16()
            if fp8:
                sc = (x.float().abs().amax(2) / 448).half()
                codes = (x.float() / sc.float()[:, :, None]).to(torch.float8_e4m3fn)
                c.pool[a:a + len(x), :1024] = codes.view(len(x), 1024).view(torch.uint8)
                c.pool[a:a + len(x), 1024:] = sc.view(torch.uint8)
            else:
                c.pool[a:a + len(x)] = x.view(len(x), 1024).view(torch.uint8)
        rows = sum(n_tokens)
        q = _queries(rows, 5, dev, 1.5)
        out, lse = torch.full_like(q, float("nan")), torch.full((rows, 16), float("nan"), device=dev)
        w = torch.full((len(ctxs), max(ctxs)), -3.0, device=dev)
        c.window_attn(hs, n_tokens, 0, 1, q, sinks, window, SCALE, out, lse)
        c.window_weights(hs, n_tokens, 0, 1, q, lse, sinks, window, SCALE, w)
        whole = window >= max(ctxs)
        if whole:                # all but the chunk's tokens come from the first request itself
            o2, l2 = torch.empty_like(out), torch.empty_like(lse)
            P = ctxs[0] - n_tokens[0]
            c.shared_attn(hs[:1], n_tokens[:1], 0, 1, hs[0], P, P, q[:n_tokens[0]], SCALE, o2[:n_tokens[0]], l2[:n_tokens[0]])
        torch.cuda.synchronize()
        _clean(c)
        x = 0
        for r, (K, V) in enumerate(_on_device(c, hs, fp8)):
            n, k = ctxs[r], n_tokens[r]
            at, t = torch.arange(n - k, n, device=dev)[:, None], torch.arange(n, device=dev)
            see = (t <= at) & ((t < sinks) | (t > at - window))
            total_w, tol_w = torch.zeros(n, dtype=torch.float64, device=dev), torch.zeros(n, dtype=torch.float64, device=dev)
            for h in range(16):
                qd = q[x:x + k, h].double()
                z = (qd @ K[:, h // 4].T * SCALE).masked_fill(~see, -math.inf)
                size = (qd.abs() @ K[:, h // 4].abs().T * SCALE)
                p = torch.softmax(z, 1)
                want, mag = p @ V[:, h // 4], p @ V[:, h // 4].abs()
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 1e-4) * mag
                for o, l in [(out, lse)] + ([(o2, l2)] if whole and r == 0 else []):
                    assert bool(((o[x:x + k, h].double() - want).abs() <= tol).all()), (r, h)
                    err = (l[x:x + k, h].double() - z.logsumexp(1)).abs()
                    assert bool((err <= 2.0 ** -17 * size.amax(1) + 1e-5).all()), (r, h, err.max())
                e = (z - lse[x:x + k, h, None].double()).exp()
                total_w += e.sum(0)
                tol_w += (e * (2.0 ** -17 * size + 2.0 ** -16)).sum(0)
            got = w[r, :n].double()
            assert bool(((got - total_w).abs() <= tol_w + 2.0 ** -12 * total_w).all()), (r, (got - total_w).abs().max())
            assert bool((w[r, n:] == -3.0).all())
            assert bool((got[~see.any(0)] == 0).all())
            x += k
    finally:
        c.close()


@pytest.mark.parametrize("tokens", [1, 4, 40])
def test_every_code_as_a_key(tokens):
    """Token t's K codes are all the code t: its weight is that of the code's value,
    subnormal codes among them; a NaN code makes its own token's weight NaN alone."""
    f = Filled([300], fp8=True, seed=3)
    try:
        raw = f.kv[0][0]
        raw[:256, :512] = torch.arange(256, dtype=torch.uint8)[:, None]
        raw[:256, 1024:1032] = torch.tensor([2.0 ** -6] * 4, dtype=torch.float16).view(torch.uint8)
        _store(f, 0)
        q = _queries(tokens, 5, f.dev, 0.25)
        lse = torch.full((tokens, 16), 2.5, device=f.dev)
        w = torch.zeros(1, 300, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 0, 1, q, lse, 0, FULL, SCALE, w)
        _clean(f.c)
        codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        x = SCALE * 2.0 ** -6 * codes[None, None] * q.double().cpu().sum(2)[:, :, None]
        want = (x - 2.5).exp().sum((0, 1))
        bad = codes.isnan()
        assert bad.nonzero().flatten().tolist() == [127, 255]
        got = w[0, :256].double().cpu()
        assert torch.equal(got.isnan(), bad)
        # logits up to 10: 2^-17 of scale sum |q k|, 2^-16 and 2^-12 as for the weights elsewhere
        size = SCALE * 2.0 ** -6 * codes.abs()[None, None] * q.double().cpu().abs().sum(2)[:, :, None]
        tol = ((x - 2.5).exp() * (2.0 ** -17 * size + 2.0 ** -16)).sum((0, 1)) + 2.0 ** -12 * want
        assert bool(((got - want).abs() <= tol)[~bad].all())
        assert bool(w[0, 256:].isfinite().all())
    finally:
        f.close()

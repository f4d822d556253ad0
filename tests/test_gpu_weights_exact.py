"""Attention weights where float64 leaves little room: logits whose products and sums
are exact in fp32, one term to a weight, so that what remains is the exponential and
its argument; infinite queries; softmax scales of any sign; host rows entry by entry.

Tolerance of a weight exp(z - lse) whose dot product is exact (one dim of the key is
not zero; 8 bits of the query times 8 of the key, or 4 and 11 of code and scale).  The
argument y = z log2 e - lse log2 e is two multiply-adds, each rounded at the size of y
(2^-24 |y|, times ln 2 in the weight); scale and lse are in two parts, exact to 2^-46
of sizes under 2^10; 2^y by ex2.approx (2^-22), the factor that the lse's second part
makes by exp2f (2 ulp: 2^-22), their product and the term's sum (2^-24 each)."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries
from tests.test_gpu_chunk_range import _store
from tests.test_gpu_window import FULL

pytestmark = pytest.mark.gpu

F32 = float(np.float32(SCALE))    # what the library is given


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _one_dim(f, value, dim):
    """Every token's key is zero but for one dim, about value[t] there; what it holds
    after the format's rounding."""
    raw, n = f.kv[0][0], len(value)
    v = torch.as_tensor(value, dtype=torch.float32)
    if f.fp8:
        scale = (v.abs() / 400).half()
        codes = torch.zeros(n, 4, 128, dtype=torch.float8_e4m3fn)
        codes[:, :, dim] = (v / scale.float()).to(torch.float8_e4m3fn)[:, None]
        raw[:, :512] = codes.view(torch.uint8).view(n, 512)
        raw[:, 1024:1032] = scale[:, None].repeat(1, 4).view(torch.uint8)
        held = codes[:, 0, dim].double() * scale.double()
    else:
        k = torch.zeros(n, 4, 128, dtype=torch.bfloat16)
        k[:, :, dim] = v.bfloat16()[:, None]
        raw[:, :1024] = k.view(n, 512).view(torch.uint8)
        held = k[:, 0, dim].double()
    _store(f, 0)
    return held


@pytest.mark.parametrize("tokens", [1, 3, 40, 300])
@pytest.mark.parametrize("lse", [10.0, 40.3, 300.7])
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_of_exact_logits(fp8, lse, tokens):
    n = 2000
    f = Filled([n], fp8=fp8, seed=3)
    try:
        g = torch.Generator().manual_seed(2)
        q = torch.randn(tokens, 16, 128, generator=g).bfloat16()
        q[tokens // 2, 9, 77] = 1.3671875
        # logits within 4 nats of the lse (and what the row format makes of them)
        z = lse + 8 * torch.rand(n, generator=g) - 4
        held = _one_dim(f, z / (F32 * 1.3671875), 77)
        ls = torch.full((tokens, 16), -math.inf)
        ls[tokens // 2, 9] = lse
        w = torch.zeros(1, n, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 0, 1, q.to(f.dev), ls.to(f.dev), 0, FULL, SCALE, w)
        torch.cuda.synchronize()
        _clean(f.c)
        y = F32 * 1.3671875 * held - float(np.float32(lse))
        want = y.exp()
        want[n - tokens + tokens // 2 + 1:] = 0
        tol = want * (2 * 2.0 ** -22 + 2 * 2.0 ** -24 + 2 * y.abs() * 2.0 ** -24)
        if tokens > 4 and not fp8:
            # these logits take a factor of 1 + 1.1 * 2^-23 for what the tensor core cuts
            # off of other sums: 1.1 * 2^-23 |z| in the exponent
            tol += want * torch.expm1(1.1 * 2.0 ** -23 * (y + lse).abs())
        err = (w[0].double().cpu() - want).abs()
        assert bool((err <= tol).all()), (err / want).nan_to_num(0).max()
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 40])
def test_infinite_queries(fp8, tokens):
    """An infinite element of a query against keys that are zero elsewhere: weights
    infinite or zero by the sign."""
    n = 300
    f = Filled([n], fp8=fp8, seed=3)
    try:
        g = torch.Generator().manual_seed(2)
        held = _one_dim(f, torch.randn(n, generator=g).sign() * (1 + torch.rand(n, generator=g)), 5)
        q = torch.randn(tokens, 16, 128, generator=g).bfloat16()
        q[0, :, 5] = math.inf
        ls = torch.full((tokens, 16), -math.inf)
        ls[0] = 3.0
        w = torch.zeros(1, n, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 0, 1, q.to(f.dev), ls.to(f.dev), 0, FULL, SCALE, w)
        seen = n - tokens + 1
        want = torch.where(held > 0, math.inf, 0.0).float()
        want[seen:] = 0
        assert torch.equal(w[0].cpu(), want)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 4, 40, 70])
def test_a_lse_of_infinity(fp8, tokens):
    """exp(z - inf): nothing for finite logits, no value for an infinite one, whatever
    other rows of the chunk have no weight at all."""
    n = 300
    f = Filled([n], fp8=fp8, seed=3)
    try:
        g = torch.Generator().manual_seed(2)
        held = _one_dim(f, torch.randn(n, generator=g).sign() * (1 + torch.rand(n, generator=g)), 5)
        q = torch.randn(tokens, 16, 128, generator=g).bfloat16()
        ls = torch.full((tokens, 16), math.inf)
        ls[0, 3] = -math.inf
        w = torch.full((1, n), 7.0, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 0, 1, q.to(f.dev), ls.to(f.dev), 0, FULL, SCALE, w)
        assert bool((w == 0).all())
        q[0, :, 5] = math.inf
        f.c.window_weights(f.hs, [tokens], 0, 1, q.to(f.dev), ls.to(f.dev), 0, FULL, SCALE, w)
        _clean(f.c)
        seen = torch.arange(n) <= n - tokens
        got = w[0].cpu()
        assert torch.equal(got.isnan(), (held > 0) & seen) and bool((got[(held < 0) | ~seen] == 0).all())
    finally:
        f.close()


def _weights(f, n_tokens, q, lse, sinks, window, scale):
    """In float64, and the tolerance of every entry: a term's logit is off by 2^-17 of
    |scale| sum |q_d k_d| and by 2^-22 of its distance to the lse, the exponential by
    2^-21; the sum of up to 2^12 terms by 2^-12 of itself; weights below 2^-126 are 0."""
    out, tol, x = [], [], 0
    for r, n in enumerate(n_tokens):
        K, _ = f.values(r, 0, list(range(f.ctxs[r])))
        Kh, t = K[:, np.arange(16) // 4], np.arange(f.ctxs[r])
        w, e_w = np.zeros(f.ctxs[r]), np.zeros(f.ctxs[r])
        for i in range(n):
            p = f.ctxs[r] - n + i
            see = (t <= p) & ((t < sinks) | (t > p - window))
            qd, ls = q[x].double().cpu().numpy(), lse[x].double().cpu().numpy()
            x += 1
            if not see.any():
                continue
            d = scale * np.einsum("thd,hd->th", Kh[see], qd) - ls
            size = abs(scale) * np.einsum("thd,hd->th", np.abs(Kh[see]), np.abs(qd))
            e = np.exp(d)
            w[see] += e.sum(1)
            e_w[see] += (e * np.expm1(2.0 ** -17 * size + 2.0 ** -22 * np.abs(d) + 2.0 ** -21)).sum(1)
        out.append(w)
        tol.append(e_w + 2.0 ** -12 * w + 16 * n * 2.0 ** -126)
    return out, tol


def _entry_by_entry(f, n_tokens, sinks, window, scale):
    q = _queries(sum(n_tokens), 5, f.dev, 1.5)
    out, lse = torch.zeros_like(q), torch.zeros(sum(n_tokens), 16, device=f.dev)
    f.c.window_attn(f.hs, n_tokens, 0, 1, q, sinks, window, scale, out, lse)
    w = torch.full((len(n_tokens), max(f.ctxs)), -3.0, device=f.dev)
    f.c.window_weights(f.hs, n_tokens, 0, 1, q, lse, sinks, window, scale, w)
    torch.cuda.synchronize()
    _clean(f.c)
    want, tol = _weights(f, n_tokens, q, lse, sinks, window, float(np.float32(scale)))
    for r, n in enumerate(f.ctxs):
        got = w[r, :n].double().cpu().numpy()
        assert np.all(np.abs(got - want[r]) <= tol[r]), (r, np.abs(got - want[r]).max())
        assert np.all(got[want[r] == 0] == 0) and bool((w[r, n:] == -3).all())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -SCALE, 6 * SCALE, SCALE / 50])
@pytest.mark.parametrize("n_tokens", [[2, 1], [4, 40], [300, 33]])
def test_softmax_scales_of_any_sign_and_size(fp8, scale, n_tokens):
    f = Filled([700, 650], fp8=fp8, seed=4)
    try:
        _entry_by_entry(f, n_tokens, 4, 600, scale)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_tokens", [[1, 2, 3], [40, 3, 70]])
def test_weights_over_rings_hosts_and_pool(fp8, n_tokens):
    f = Filled([500, 500, 260], [Q.KV_HOST_RING, Q.KV_HOST, Q.KV_HBM], fp8=fp8, seed=5, ring=64)
    try:
        _entry_by_entry(f, n_tokens, 4, 200, SCALE)
    finally:
        f.close()

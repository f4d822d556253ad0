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
from tests.test_gpu_chunk import SCALE, Filled, _clean
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

"""Window and shared-prefix attention over keys and values that are not finite, where
the tokens are cut into shares: an answer may not depend on which share such a token
falls into, nor on whether a row sees anything else there.  Against float64: an
element is finite exactly where the definition's is.

Tolerances of the finite elements as in test_gpu_window.py."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from oracle import qsa_oracle as O
from tests import qsa_check as QC
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries
from tests.test_gpu_chunk_range import SIGNS, _set_logits, _store
from tests.test_gpu_window import FULL, _window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _check(rows, q, out, lse, values):
    """rows: one key per row; values(key) -> K, V of its tokens.  Returns how many
    elements are not finite."""
    bad = 0
    for x, key in enumerate(rows):
        K, V = values(key)
        qd = O.decode_bf16(QC.bits16(q[x])).reshape(16, 128)
        Kh, Vh = K[:, np.arange(16) // 4], V[:, np.arange(16) // 4]
        with np.errstate(all="ignore"):
            z = SCALE * np.einsum("thd,hd->ht", Kh, qd)
            m = z.max(1, keepdims=True)
            p = np.exp(z - m)
            total = p.sum(1, keepdims=True)
            want, mag = [np.einsum("ht,thd->hd", p, v) / total for v in (Vh, np.abs(Vh))]
            ls = (m + np.log(total))[:, 0]
            size = SCALE * np.einsum("thd,hd->th", np.abs(Kh), np.abs(qd))
            size = np.where(np.isfinite(size), size, 0).max(0)
        got, gl = out[x].double().cpu().numpy(), lse[x].double().cpu().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), fin), (x, key, np.argwhere(np.isfinite(got) != fin)[:4])
        assert np.all(np.abs(got - want)[fin] <= (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 1e-4) * mag)[fin]), (x, key)
        fin_l = np.isfinite(ls)
        assert np.array_equal(np.isfinite(gl), fin_l), (x, key)
        assert np.all(np.abs(gl - ls)[fin_l] <= (2.0 ** -17 * size + 1e-5)[fin_l]), (x, key)
        bad += int((~fin).sum())
    return bad


def _poison_keys(f, r, toks, value):
    """One dim of every head's key, or every head's K scale."""
    raw = f.kv[r][0]
    for t in toks:
        if f.fp8:
            raw[t, 1024:1032] = torch.full((4,), value, dtype=torch.float16).view(torch.uint8)
        else:
            raw[t, :1024].view(torch.bfloat16)[5::128] = value
    _store(f, r)


# contexts that are cut into shares; the poisoned tokens fill a share, or all that a row sees of it
SHARES = [(1025, 1, range(1024, 1025)), (1025, 1, range(992, 1024)), (1025, 4, range(992, 1024)), (160, 1, range(128, 160)),
          (2944, 40, range(2600, 2944)), (600, 40, range(384, 600)), (600, 40, range(0, 300))]


@pytest.mark.parametrize("fp8,value", [(False, float("nan")), (False, float("inf")), (False, -float("inf")),
                                       (True, float("nan"))])
@pytest.mark.parametrize("ctx,tokens,bad", SHARES)
def test_keys_that_are_not_finite_and_fill_a_share(fp8, value, ctx, tokens, bad):
    f = Filled([ctx], fp8=fp8, seed=6)
    try:
        _poison_keys(f, 0, bad, value)
        q = _queries(tokens, 7, f.dev)
        out, lse = _window(f, [tokens], q, 0, FULL)
        _clean(f.c)
        pos = [p for _, p in f.positions([tokens])]
        assert _check(pos, q, out, lse, lambda p: f.values(0, 0, list(range(p + 1)))) > 0
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests", [3, 10])
def test_keys_that_are_not_finite_at_the_end_of_a_shared_prefix(fp8, requests):
    f = Filled([40] * requests + [1000], fp8=fp8, seed=6)
    try:
        _poison_keys(f, requests, range(768, 1000), float("nan"))
        q = _queries(requests, 7, f.dev)
        for prefix_len in (768, 1000):
            out, lse = torch.zeros_like(q), torch.zeros(requests, 16, device=f.dev)
            f.c.shared_attn(f.hs[:requests], [1] * requests, 0, 1, f.hs[requests], prefix_len, 0, q, SCALE, out, lse)
            torch.cuda.synchronize()
            _clean(f.c)

            def values(r):
                a, b = f.values(requests, 0, list(range(prefix_len))), f.values(r, 0, list(range(40)))
                return [np.concatenate(x) for x in zip(a, b)]
            n = _check(range(requests), q, out, lse, values)
            assert n == (0 if prefix_len == 768 else requests * 16 * 128)
    finally:
        f.close()


@pytest.mark.parametrize("ctx,tokens", [(1025, 1), (1025, 3), (160, 1), (600, 40)])
def test_values_that_are_not_finite_behind_logits_far_below(ctx, tokens):
    """The first tokens' logits are 200 below the others' (their share counts 2^-288 in
    the join), their values infinite in one dim."""
    f = Filled([ctx], seed=6)
    try:
        first = 256 if tokens > 4 else 32
        _set_logits(f, 0, np.where(np.arange(ctx) < first, -200.0, 0.0))
        f.kv[0][0][:first, 1024:].view(torch.bfloat16)[:, 3::128] = float("inf")
        _store(f, 0)
        q = SIGNS.bfloat16().expand(tokens, 16, 128).contiguous().to(f.dev)
        out, lse = _window(f, [tokens], q, 0, FULL)
        _clean(f.c)
        pos = [p for _, p in f.positions([tokens])]
        assert _check(pos, q, out, lse, lambda p: f.values(0, 0, list(range(p + 1)))) == tokens * 16
    finally:
        f.close()


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,tokens,bad", SHARES + [(20, 1, range(7, 8)), (20, 9, range(2, 3)), (300, 70, range(150, 151))])
def test_infinite_k_scales(value, ctx, tokens, bad):
    """Codes of both signs times an infinite scale: logits without a value (for the
    sum of the codes' products they would have one, and -inf leave the token out)."""
    f = Filled([ctx], fp8=True, seed=6)
    try:
        _poison_keys(f, 0, bad, value)
        q = _queries(tokens, 7, f.dev)
        out, lse = _window(f, [tokens], q, 0, FULL)
        pos = [p for _, p in f.positions([tokens])]
        assert _check(pos, q, out, lse, lambda p: f.values(0, 0, list(range(p + 1)))) > 0
        # the weights: NaN for those tokens, the others' as if these were not there
        lse = torch.full((tokens, 16), 3.0, device=f.dev)
        w, w0 = torch.zeros(1, ctx, device=f.dev), torch.zeros(1, ctx, device=f.dev)
        f.c.window_weights(f.hs, [tokens], 0, 1, q, lse, 0, FULL, SCALE, w)
        _poison_keys(f, 0, bad, 1.0)
        f.c.window_weights(f.hs, [tokens], 0, 1, q, lse, 0, FULL, SCALE, w0)
        _clean(f.c)
        at = torch.zeros(ctx, dtype=torch.bool, device=f.dev)
        at[list(bad)] = True
        assert torch.equal(w[0].isnan(), at) and torch.equal(w[0, ~at], w0[0, ~at])
    finally:
        f.close()

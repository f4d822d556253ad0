"""Window and shared-prefix attention as a server calls them: right behind the kernels
that write what they read, and batches that mix single tokens with pieces of prompts."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries
from tests.test_gpu_window import FULL, _check, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("own_first", [0, 10000])
def test_calls_read_what_the_kernels_before_them_wrote(own_first, fp8):
    """64 requests of one token behind a prefix: the prefix's tiles and the requests'
    own tokens (all of them, or none) are two kernels, both behind the append and the
    queries' copy."""
    R = 64
    f = Filled([70] * R + [3000], fp8=fp8, seed=5, grow=12)
    try:
        c, dev, hs = f.c, f.dev, f.hs[:R]
        g = torch.Generator(device=dev).manual_seed(3)
        q = _queries(R, 1, dev)
        ws = torch.empty(c.shared_attn_workspace_bytes(hs, [1] * R, 0, 1, f.hs[R], 3000, own_first) + (1 << 22), dtype=torch.uint8,
                         device=dev)
        steps = [(torch.randn(R, 64, generator=g, device=dev),
                  torch.randn(R, 1024, generator=g, device=dev).bfloat16().view(torch.uint8),
                  _queries(R, 10 + i, dev)) for i in range(10)]
        outs = [[torch.zeros_like(q), torch.zeros(R, 16, device=dev)] for _ in range(20)]

        def attend(i, o):
            q.copy_(steps[i][2])
            c.shared_attn(hs, [1] * R, 0, 1, f.hs[R], 3000, own_first, q, SCALE, *o, workspace=ws)

        torch.cuda.synchronize()
        for i in range(10):          # one behind the other
            for h in hs:
                c.advance(h, 1)
            c.append_token(hs, 0, 1, *steps[i][:2])
            attend(i, outs[i])
        torch.cuda.synchronize()
        for i in range(9, -1, -1):   # each alone
            for h in hs:
                c.truncate(h, 71 + i)
            torch.cuda.synchronize()
            q.copy_(steps[i][2])
            torch.cuda.synchronize()
            attend(i, outs[10 + i])
            torch.cuda.synchronize()
        for i in range(10):
            assert torch.equal(outs[i][0], outs[10 + i][0]) and torch.equal(outs[i][1], outs[10 + i][1]), i
        _clean(c)
    finally:
        f.close()


def _attend_guarded(f, n_tokens, layers, q, prefix=None):
    """Window attention over everything, or behind the prefix (request, length, own
    first), in a workspace of exactly the bytes asked for; those bytes."""
    c, hs = f.c, f.hs[:len(n_tokens)]
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=f.dev)
    if prefix is None:
        need = c.window_attn_workspace_bytes(hs, n_tokens, 0, layers, 0, FULL)
    else:
        need = c.shared_attn_workspace_bytes(hs, n_tokens, 0, layers, *prefix)
    guard = torch.full((need + 8192,), 255, dtype=torch.uint8, device=f.dev)
    if prefix is None:
        c.window_attn(hs, n_tokens, 0, layers, q, 0, FULL, SCALE, out, lse, workspace=guard[:need])
    else:
        c.shared_attn(hs, n_tokens, 0, layers, *prefix, q, SCALE, out, lse, workspace=guard[:need])
    torch.cuda.synchronize()
    _clean(c)
    assert bool((guard[need:] == 255).all())
    return out, lse, need


PIECE = 16 * (128 + 4) * 4        # bytes of a row's partial: 16 heads, O, maximum and sum


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,layers,cut", [
    # (requests, tokens each, layers, rows that may need up to 64 pieces each)
    ([4200, 9000], [4096, 1], 1, 1), ([9000, 300, 3000], [2, 0, 2700], 1, 2), ([2600, 700, 2600, 5000], [2500, 700, 3, 4], 2, 14),
    ([6000, 500, 500], [2, 70, 3], 2, 150), ([3000], [1], 1, 1), ([2000], [2000], 2, 0)])
def test_batches_of_tokens_and_pieces_of_prompts(fp8, ctxs, n_tokens, layers, cut):
    """Rows that are written at once need no workspace, whatever is beside them."""
    f = Filled(ctxs, layers=layers, fp8=fp8, seed=5)
    try:
        q = _queries(layers * sum(n_tokens), 5, f.dev, 1.5)
        out, lse, need = _attend_guarded(f, n_tokens, layers, q)
        assert need <= 256 + 64 * cut * PIECE
        _check(_rows(f, n_tokens, layers), q, out, lse, lambda k: f.values(k[1], k[0], list(range(k[2] + 1))))
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("own,n_tokens,prefix_len,own_first,layers", [
    ([900] + [40] * 30, [200] + [1] * 30, 2500, 0, 1), ([900, 40, 70], [300, 1, 2], 4000, 0, 2),
    ([3000, 30, 1200], [5, 2, 60], 700, 20, 1), ([40] * 10, [1, 9] * 5, 1500, 39, 2)])
def test_a_shared_prefix_behind_tokens_and_pieces_of_prompts(fp8, own, n_tokens, prefix_len, own_first, layers):
    f = Filled(own + [prefix_len + 3], layers=layers, fp8=fp8, seed=5)
    try:
        R = len(own)
        q = _queries(layers * sum(n_tokens), 5, f.dev, 1.5)
        out, lse, _ = _attend_guarded(f, n_tokens, layers, q, (f.hs[R], prefix_len, own_first))

        def values(k):
            a, b = f.values(R, k[0], list(range(prefix_len))), f.values(k[1], k[0], list(range(own_first, k[2] + 1)))
            return [np.concatenate(x) for x in zip(a, b)]
        _check(_rows(f, n_tokens, layers), q, out, lse, values)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layers", [90, 128])
def test_a_shared_prefix_at_as_many_layers_as_a_call_takes(layers, fp8):
    f = Filled([6, 9, 300], layers=layers, fp8=fp8, seed=5)
    try:
        q = _queries(2 * layers, 5, f.dev, 1.5)
        out, lse, _ = _attend_guarded(f, [1, 1], layers, q, (f.hs[2], 300, 0))

        def values(k):
            a, b = f.values(2, k[0], list(range(300))), f.values(k[1], k[0], list(range(k[2] + 1)))
            return [np.concatenate(x) for x in zip(a, b)]
        _check(_rows(f, [1, 1], layers), q, out, lse, values)
    finally:
        f.close()

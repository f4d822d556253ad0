"""Window and shared-prefix attention as a server calls them: right behind the kernels
that write what they read, and batches that mix single tokens with pieces of prompts."""
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries

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

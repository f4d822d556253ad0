"""Chunk attention and fork between a hot-cache plan and the attention that
fills its rows: the slots of the planned misses already name rows that hold
other tokens' bytes."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from sparse_attention_decode_qsa_gb300 import workloads
from tests import qsa_check as QC
from tests.test_gpu_chunk import SCALE, Filled, _attend, _check_attention, _clean, _queries, _run_attention
from tests.test_gpu_pages import _read

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _planned(f, layer):
    """Fill the hot rows of a layer with one selection, plan another one."""
    c, dev, h = f.c, f.dev, f.hs[0]
    n = torch.tensor([32], dtype=torch.int32, device=dev)
    old = torch.arange(0, 128, 4, dtype=torch.int32, device=dev)[None].contiguous()
    new = old + 1
    new[0, :4] = old[0, :4]                                   # some of them are there already
    new = new.sort(1).values.int().contiguous()
    c.hot_cache_fetch([h], layer, 1, old, n, 128)
    c.hot_cache_plan([h], layer, 1, new, n, 128)
    return new, n


def _decode(f, layer, sel, n):
    out = torch.zeros(1, 16, 128, device=f.dev)
    f.c.sparse_decode_attn([f.hs[0]], layer, 1, _queries(1, 5, f.dev), sel, n, 128, None, SCALE, out, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("place", [Q.KV_HOST_RING, Q.KV_HOST])
def test_chunk_attention_reads_planned_misses_from_the_host(fp8, place):
    f = Filled([800], [place], layers=2, ring=16, hot_rows=128, budget=128, fp8=fp8, seed=9)
    try:
        c = f.c
        sel, n = _planned(f, 1)
        for tokens in (3, 70):
            ids = sel[0].cpu().numpy()
            t, ns = sel.cpu().expand(tokens, -1).contiguous(), torch.full((tokens,), 32, dtype=torch.int32)
            q = _queries(tokens, 7, f.dev)
            for filled in (False, True) if tokens == 70 else (False,):
                if filled:
                    _decode(f, 1, sel, n)
                out, lse = _run_attention(f, [tokens], q, t, ns, 128, layers=1, layer0=1)
                _clean(c)
                _check_attention(f, [tokens], q, [ids] * tokens, [32] * tokens, out, lse, layer0=1)
        # a value that is not finite sends its rows through their own loop
        _planned(f, 1)
        host = f.host[0]
        if fp8:
            host[1, 4 * 5].view(torch.uint8)[1032:1040] = torch.tensor([0x00, 0x7C] * 4, dtype=torch.uint8)      # inf
        else:
            host[1, 4 * 5].view(torch.uint8)[1024:] = torch.tensor([0x80, 0x7F] * 512, dtype=torch.uint8)
        odd = [np.sort(np.append(ids[ids != 5][:20], 5)) if x % 2 else ids[ids != 5][:20] for x in range(70)]
        t = torch.full((70, 32), -1, dtype=torch.int32)
        for x, s in enumerate(odd):
            t[x, :len(s)] = torch.as_tensor(s, dtype=torch.int32)
        ns = torch.tensor([len(s) for s in odd], dtype=torch.int32)
        out, lse = _run_attention(f, [70], q, t, ns, 128, layers=1, layer0=1)
        _clean(c)
        even = list(range(0, 70, 2))
        assert bool(out[even].isfinite().all()) and not bool(out[1::2].isfinite().all(-1).any())
        for x in even:
            o, ls, mag, lmag = _attend(QC.bits16(q[x]), *f.values(0, 1, [k for b in odd[x] for k in range(4 * b, 4 * b + 4)]))
            got = out[x].double().cpu().numpy()
            assert np.all(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4) * mag), x
    finally:
        torch.cuda.synchronize()
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("child", [Q.KV_HBM, Q.KV_HOST])
def test_fork_copies_planned_misses_from_the_host(fp8, child):
    L, n = 2, 700
    f = Filled([n], [Q.KV_HOST_RING], layers=L, ring=16, hot_rows=128, budget=128, fp8=fp8, seed=9, spare=3 * L * (n + 128))
    host = workloads.alloc_host((L, n, f.c.row_bytes), f.dev, "vmm") if child != Q.KV_HBM else None
    try:
        c = f.c
        sel, k = _planned(f, 1)
        for filled in (False, True):
            if filled:
                _decode(f, 1, sel, k)
            h = c.request_fork(f.hs[0], n - 30, child, host_rows=host, max_ctx=n)
            torch.cuda.synchronize()
            _clean(c)
            for l in range(L):
                assert torch.equal(_read(c, h, l, n - 30, host), f.kv[0][l][:n - 30]), (filled, l)
            c.request_end(h)
        assert torch.equal(_read(c, f.hs[0], 1, n, f.host[0]), f.kv[0][1])
    finally:
        torch.cuda.synchronize()
        f.close()
        if host is not None:
            workloads.free_host(host)

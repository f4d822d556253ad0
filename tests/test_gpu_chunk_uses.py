"""Uses of the chunk and page operators that stand beside each other: softmax
scales of 0 and below, plans with a compaction or taken-back tokens before the
chunk, tokens appended a second time, captured calls with their own workspace,
graphs that share a cache."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from oracle import qsa_oracle as O
from sparse_attention_decode_qsa_gb300 import synth
from tests import qsa_check as QC
from tests.test_gpu_chunk import SCALE, Filled, _check_attention, _clean, _queries, _random_selection, _run_attention
from tests.test_gpu_pages import _read
from tests.test_gpu_planned_misses import _planned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -SCALE, 4 * SCALE])
@pytest.mark.parametrize("ctxs,n_tokens", [([600], [40]), ([90] * 39, [3] * 39)])
def test_softmax_scales_of_any_sign(fp8, scale, ctxs, n_tokens):
    """Rounding as in the chunk attention's other tests: 2^-8 of the output and
    2^-8 + 1e-4 of sum p|v|; logits and lse off by 2^-17 of the logits' sizes."""
    f = Filled(ctxs, fp8=fp8, seed=4, budget=256)
    try:
        sel, nsel, t, n = _random_selection(f, n_tokens, 256, 12)
        q = _queries(len(sel), 3, f.dev)
        out, lse = torch.full_like(q, float("nan")), torch.zeros(len(sel), 16, device=f.dev)
        f.c.chunk_sparse_attn(f.hs, n_tokens, 0, 1, q, t.to(f.dev), n.to(f.dev), 256, scale, out, lse)
        torch.cuda.synchronize()
        _clean(f.c)
        for x, (r, p) in enumerate(f.positions(n_tokens)):
            if x % 5:
                continue
            toks = [k for b in sel[x] for k in range(4 * b, min(4 * b + 4, p + 1))]
            K, V = f.values(r, 0, toks)
            qd = O.decode_bf16(QC.bits16(q[x])).reshape(16, 128)
            for h in range(16):
                z = scale * (K[:, h // 4] @ qd[h])
                e = np.exp(z - z.max())
                o, mag = e @ V[:, h // 4] / e.sum(), e @ np.abs(V[:, h // 4]) / e.sum()
                size = abs(scale) * (np.abs(K[:, h // 4]) @ np.abs(qd[h])).max()
                got = out[x, h].double().cpu().numpy()
                assert np.all(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -16 * size + 1e-4) * mag), (x, h)
                assert abs(lse[x, h].item() - (z.max() + np.log(e.sum()))) <= 2.0 ** -17 * size + 1e-5, (x, h)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_plan_a_compaction_and_a_chunk(fp8):
    """The planned rows have moved when the chunk completes the plan."""
    f = Filled([200, 800], [Q.KV_HBM, Q.KV_HOST_RING], layers=2, ring=16, hot_rows=128, budget=128, fp8=fp8, seed=9)
    try:
        c = f.c
        f.hs.reverse()                                        # (_planned takes the first)
        sel, n = _planned(f, 1)
        f.hs.reverse()
        c.request_end(f.hs[0])
        assert c.compact() > 0
        q = _queries(5, 7, f.dev)
        out, lse = torch.zeros_like(q), torch.zeros(5, 16, device=f.dev)
        c.chunk_sparse_attn([f.hs[1]], [5], 1, 1, q, sel.expand(5, -1).contiguous(), n.expand(5).contiguous(), 128,
                            SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(c)
        assert torch.equal(_read(c, f.hs[1], 1, 800, f.host[1]), f.kv[1][1])
        info = c.request_info(f.hs[1])
        slots = c.slot_table[f.hs[1].index, 1, (4 * sel[0].long())].cpu()
        assert bool(((slots >= info.hot_row_base + 128) & (slots < info.hot_row_base + 256)).all())
        f.ctxs, f.kv, f.host = [800], f.kv[1:], f.host[1:]
        _check_attention(f, [5], q, [sel[0].cpu().numpy()] * 5, [32] * 5, out, lse, layer0=1)
    finally:
        torch.cuda.synchronize()
        f.close()


def test_a_plan_and_tokens_taken_back():
    """Planned tokens that are taken back and appended again: the chunk reads
    the new ones, and the hot rows of the old ones come back into use."""
    f = Filled([400], [Q.KV_HOST], ring=16, hot_rows=64, budget=64, seed=9, grow=8)
    try:
        c, h, dev = f.c, f.hs[0], f.dev
        sel = torch.arange(84, 100, dtype=torch.int32, device=dev)[None].contiguous()
        n = torch.tensor([16], dtype=torch.int32, device=dev)
        c.hot_cache_plan([h], 0, 1, sel, n, 64)
        c.truncate(h, 390)
        c.advance(h, 12)
        kv = synth.kv_rows(12, 3)
        c.append_chunk([h], [12], 0, 1, torch.randn(12, 64, device=dev), kv.to(dev))
        f.kv[0] = torch.cat([f.kv[0][:, :390], kv[None]], 1)
        f.ctxs = [402]
        ids = np.append(np.arange(86, 97), [97, 98, 99, 100])
        t = torch.full((12, 16), -1, dtype=torch.int32)
        s, k = [], []
        for x in range(12):
            mine = ids[ids <= (390 + x) // 4]
            s.append(mine)
            k.append(len(mine))
            t[x, :len(mine)] = torch.from_numpy(mine).int()
        q = _queries(12, 5, dev)
        out, lse = _run_attention(f, [12], q, t, torch.tensor(k, dtype=torch.int32), 64)
        _clean(c)
        _check_attention(f, [12], q, s, k, out, lse)
        assert torch.equal(_read(c, h, 0, 402, f.host[0]), f.kv[0][0])
        for first in (0, 16, 85, 40):
            c.hot_cache_fetch([h], 0, 1, torch.arange(first, first + 16, dtype=torch.int32, device=dev)[None].contiguous(), n, 64)
            torch.cuda.synchronize()
            _clean(c)
            assert torch.equal(_read(c, h, 0, 402, f.host[0]), f.kv[0][0]), first
    finally:
        torch.cuda.synchronize()
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("place", [Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST])
def test_tokens_appended_a_second_time(fp8, place):
    """A chunk may reach back over tokens that are stored already."""
    n, k = 200, 60
    f = Filled([n], [place], layers=2, ring=16, fp8=fp8, budget=64, seed=9)
    try:
        c, h = f.c, f.hs[0]
        before = c.slot_table[h.index, :, :n].clone()
        kv = synth.kv_rows(2 * k, 3)
        c.append_chunk([h], [k], 0, 2, torch.randn(2 * k, 64, device=f.dev), kv.to(f.dev))
        torch.cuda.synchronize()
        _clean(c)
        want = (synth.fp8_kv_rows(kv) if fp8 else kv).view(2, k, -1)
        assert torch.equal(c.slot_table[h.index, :, :n], before)
        for l in range(2):
            assert torch.equal(_read(c, h, l, n, f.host[0]), torch.cat([f.kv[0][l][:n - k], want[l]]))
    finally:
        f.close()


def test_captured_calls_with_their_own_workspace():
    """Append, score, select and attend captured twice, with a workspace of the
    capture's own each; replayed in turn and at once, equal to eager calls."""
    f = Filled([900, 700], seed=4, budget=128, grow=4)
    try:
        c, dev = f.c, f.dev
        for h in f.hs:
            c.advance(h, 4)
        g0 = torch.Generator().manual_seed(1)
        sets = []
        for i, h in enumerate(f.hs):
            sets.append(dict(h=h, k=torch.randn(4, 64, generator=g0).to(dev), kv=synth.kv_rows(4, 3 + i).to(dev),
                             qi=torch.randn(4, 8, 64, generator=g0).to(dev), w=torch.rand(4, 8, generator=g0).to(dev),
                             q=_queries(4, i, dev), blk=torch.zeros(4, 232, device=dev),
                             sel=torch.zeros(4, 32, dtype=torch.int32, device=dev),
                             ns=torch.zeros(4, dtype=torch.int32, device=dev),
                             out=torch.zeros(4, 16, 128, dtype=torch.bfloat16, device=dev)))

        def step(s):
            c.append_chunk([s["h"]], [4], 0, 1, s["k"], s["kv"])
            c.chunk_index_score([s["h"]], [4], 0, 1, s["qi"], s["w"], s["blk"])
            c.chunk_select_topk([s["h"]], [4], 0, 1, s["blk"], 128, s["sel"], s["ns"])
            c.chunk_sparse_attn([s["h"]], [4], 0, 1, s["q"], s["sel"], s["ns"], 128, SCALE, s["out"])

        want = []
        for s in sets:
            step(s)
            torch.cuda.synchronize()
            want.append((s["sel"].clone(), s["out"].clone()))
        graphs, streams = [], [torch.cuda.Stream() for _ in sets]
        for s, st in zip(sets, streams):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                step(s)
            graphs.append(g)
        for together in (False, True, True):
            for s in sets:
                s["out"].zero_()
                s["sel"].zero_()
            torch.cuda.synchronize()
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
                if not together:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            for s, (a, o) in zip(sets, want):
                assert torch.equal(s["sel"], a) and torch.equal(s["out"], o)
        _clean(c)
    finally:
        f.close()


def test_repeated_calls_give_the_same_bits():
    f = Filled([9000, 700, 5000], fp8=True, seed=4, budget=2048)
    try:
        n_tokens = [70, 3, 129]
        sel, nsel, t, n = _random_selection(f, n_tokens, 2048, 12)
        q = _queries(len(sel), 3, f.dev)
        first = _run_attention(f, n_tokens, q, t, n, 2048)
        for _ in range(5):
            out, lse = _run_attention(f, n_tokens, q, t, n, 2048)
            assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    finally:
        f.close()

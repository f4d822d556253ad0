"""Fork and compaction on the GPU: after either, every live token's key and
row (found through the slot table or the host history) is what its request
holds, byte for byte."""
import random

import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from sparse_attention_decode_qsa_gb300 import workloads
from tests.test_gpu_chunk import Filled, SCALE, _check_attention, _clean, _queries, _random_selection, _run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _read(c, h, l, n, host):
    """Rows of the first n tokens as a decode step would find them."""
    slots = c.slot_table[h.index, l, :n].cpu().long()
    out = torch.empty(n, c.row_bytes, dtype=torch.uint8)
    cold = slots < 0
    out[~cold] = c.pool[slots[~cold].to(c.pool.device)].cpu()
    if bool(cold.any()):
        out[cold] = host[l][:n][cold]
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("child", [Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST])
@pytest.mark.parametrize("parent", [Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST])
def test_fork_copies_a_prefix_between_placements(parent, child, fp8):
    L, n = 2, 301
    f = Filled([40, n], [Q.KV_HBM, parent], layers=L, fp8=fp8, ring=32, grow=20, spare=3 * L * 400, budget=64)
    hist = []
    try:
        c, p = f.c, f.hs[1]
        for prefix, room in ((n, 0), (1, 5), (37, 60), (128, 0)):
            host = workloads.alloc_host((L, max(prefix, room), c.row_bytes), f.dev, "vmm") if child != Q.KV_HBM else None
            hist.append(host)
            if host is not None:
                host.fill_(0xEE)
            h = c.request_fork(p, prefix, child, host_rows=host, max_ctx=room)
            torch.cuda.synchronize()
            _clean(c)
            for l in range(L):
                assert torch.equal(c.index_keys[h.index, l, :prefix], c.index_keys[p.index, l, :prefix])
                assert torch.equal(c.index_scales[h.index, l, :prefix].view(torch.int16),
                                   c.index_scales[p.index, l, :prefix].view(torch.int16))
                assert torch.equal(_read(c, h, l, prefix, host), f.kv[1][l][:prefix]), (prefix, l)
                assert torch.equal(_read(c, p, l, n, f.host[1]), f.kv[1][l][:n])
                if host is not None:
                    assert torch.equal(host[l, :prefix], f.kv[1][l][:prefix])
                    assert bool((host[l, prefix:] == 0xEE).all())
            c.request_end(h)
    finally:
        torch.cuda.synchronize()
        f.close()
        for h in hist:
            if h is not None:
                workloads.free_host(h)


def test_fork_reads_remapped_slots_and_reports_bad_ones():
    f = Filled([100], layers=1, spare=300, budget=64)
    try:
        c, p, dev = f.c, f.hs[0], f.dev
        spare = c.request_begin(10)
        row = c.request_info(spare).hbm_row_base
        c.pool[row] = f.kv[0][0][7].to(dev)
        c.pool[c.slot_table[p.index, 0, 7].item()] = 0           # the old place no longer counts
        c.slot_table_set(p, 0, torch.tensor([7], device=dev), torch.tensor([row], dtype=torch.int32, device=dev))
        h = c.request_fork(p, 60)
        torch.cuda.synchronize()
        _clean(c)
        assert torch.equal(_read(c, h, 0, 60, None), f.kv[0][0][:60])
        c.request_end(h)
        c.slot_table[p.index, 0, 20] = c.pool.shape[0] + 5
        c.slot_table[p.index, 0, 21] = -1
        h = c.request_fork(p, 60)
        torch.cuda.synchronize()
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        ok = [t for t in range(60) if t not in (20, 21)]
        assert torch.equal(_read(c, h, 0, 60, None)[ok], f.kv[0][0][:60][ok])
    finally:
        f.close()


def test_a_fork_answers_like_its_parent_and_grows_apart():
    f = Filled([900], layers=1, grow=8, spare=1200, budget=256, seed=3)
    try:
        c, p = f.c, f.hs[0]
        h = c.request_fork(p, 900, max_ctx=905)
        f.hs.append(h)
        f.ctxs.append(900)
        f.kv.append(f.kv[0])
        n_tokens = [20, 20]
        sel, nsel, t, n = _random_selection(f, n_tokens, 256, 5)
        t[20:], n[20:] = t[:20], n[:20]
        q = _queries(40, 3, f.dev)
        q[20:] = q[:20]
        out, lse = _run_attention(f, n_tokens, q, t, n, 256)
        assert torch.equal(out[:20], out[20:]) and torch.equal(lse[:20], lse[20:])
        before = c.pool[c.request_info(p).hbm_row_base:][:900].clone()
        c.advance(h, 5)
        c.append_chunk([h], [5], 0, 1, torch.randn(5, 64, device=f.dev), torch.zeros(5, 2048, dtype=torch.uint8, device=f.dev))
        torch.cuda.synchronize()
        assert torch.equal(before, c.pool[c.request_info(p).hbm_row_base:][:900])
        _clean(c)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("holes", [[1], [3, 700], [700, 3], [64, 1, 200]])
def test_compaction_keeps_every_row(fp8, holes):
    """Gaps smaller and larger than the regions behind them (overlapping and
    plain moves), with ring and host requests between."""
    L = 2
    ctxs, places = [], []
    for i, n in enumerate(holes):
        ctxs += [n, 500 + 31 * i, 90]
        places += [Q.KV_HBM, Q.KV_HBM, Q.KV_HOST_RING if i % 2 == 0 else Q.KV_HOST]
    f = Filled(ctxs, places, layers=L, fp8=fp8, ring=16, seed=7, budget=64)
    try:
        c = f.c
        live = [r for r in range(len(ctxs)) if r % 3]
        for r in range(0, len(ctxs), 3):
            c.request_end(f.hs[r])
        moved = c.compact()
        torch.cuda.synchronize()
        _clean(c)
        assert moved > 0 and c.stats()["free_ranges"] == 1
        for r in live:
            for l in range(L):
                assert torch.equal(_read(c, f.hs[r], l, ctxs[r], f.host[r]), f.kv[r][l]), (r, l)
        assert c.compact() == 0
        h = c.request_begin(5)          # the free rows are one range: 8 spare ones and the gaps
        assert c.request_info(h).hbm_row_base + 2 * 5 <= c.pool.shape[0]
        torch.cuda.synchronize()
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gap,rows", [(45000, 70001), (45000, 30000)])
def test_compaction_of_long_regions(fp8, gap, rows):
    """Gaps wide enough for the form that moves chains side by side, with a
    region longer than the gap (overlapping move) and one shorter.  Every row
    carries its number."""
    c = Q.Cache(n_layers=1, max_requests=2, ctx_capacity=max(gap, rows), hbm_pool_rows=gap + rows, budget_tokens=64,
                staging_rows=0, kv_format=Q.KV_FP8 if fp8 else Q.KV_BF16)
    a, b = c.request_begin(gap), c.request_begin(rows)
    base = c.request_info(b).hbm_row_base
    words = c.pool.view(torch.int32)
    want = (torch.arange(rows, device=c.pool.device, dtype=torch.int32)[:, None] * 1024 +
            torch.arange(words.shape[1], device=c.pool.device, dtype=torch.int32))
    words[base:base + rows] = want
    c.request_end(a)
    assert c.compact() == rows
    torch.cuda.synchronize()
    _clean(c)
    assert c.request_info(b).hbm_row_base == base - gap
    assert torch.equal(words[base - gap:base - gap + rows], want)
    assert torch.equal(c.slot_table[b.index, 0, :rows].long(), base - gap + torch.arange(rows, device=c.pool.device))
    c.close()


def test_compaction_follows_slots_that_name_other_requests_rows():
    f = Filled([30, 40, 50], seed=7, budget=64)
    try:
        c, dev = f.c, f.dev
        a, b, d = f.hs
        tok = torch.tensor([3, 9], device=dev)
        rows = c.slot_table[d.index, 0, [11, 12]].clone()
        c.slot_table_set(b, 0, tok, rows)                        # b's tokens 3, 9 read rows of d
        torch.cuda.synchronize()
        c.request_end(a)
        assert c.compact() == 90
        torch.cuda.synchronize()
        assert torch.equal(c.slot_table[b.index, 0, [3, 9]], c.slot_table[d.index, 0, [11, 12]])
        got = _read(c, b, 0, 40, None)
        want = f.kv[1][0].clone()
        want[[3, 9]] = f.kv[2][0][[11, 12]]
        assert torch.equal(got, want)
    finally:
        f.close()


def test_compaction_between_a_plan_and_its_attention():
    """Hot rows move with their request: planned misses are filled at the new
    place, and the next step finds them there."""
    ctxs = [200, 800]
    f = Filled(ctxs, [Q.KV_HBM, Q.KV_HOST_RING], ring=16, hot_rows=128, budget=128, seed=9)
    try:
        c, dev = f.c, f.dev
        h = f.hs[1]
        sel = torch.arange(0, 128, 4, dtype=torch.int32, device=dev)[None]
        nsel = torch.tensor([32], dtype=torch.int32, device=dev)
        q = _queries(1, 5, dev)
        out, lse = torch.zeros(1, 16, 128, device=dev), torch.zeros(1, 16, device=dev)
        want = out.clone()
        c.sparse_decode_attn([h], 0, 1, q, sel, nsel, 128, None, SCALE, want, lse)   # straight from the host
        c.hot_cache_plan([h], 0, 1, sel, nsel, 128)
        c.request_end(f.hs[0])
        assert c.compact() == 16 + 128
        c.sparse_decode_attn([h], 0, 1, q, sel, nsel, 128, None, SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(c)
        assert torch.allclose(out, want, atol=1e-5)
        info = c.request_info(h)
        slots = c.slot_table[h.index, 0, :800].cpu()
        for b in sel[0].tolist():
            for t in range(4 * b, 4 * b + 4):
                assert info.hot_row_base <= slots[t] < info.hot_row_base + 128
        assert torch.equal(_read(c, h, 0, 800, f.host[1]), f.kv[1][0])
        c.hot_cache_fetch([h], 0, 1, sel + 1, nsel, 128)
        torch.cuda.synchronize()
        _clean(c)
        assert torch.equal(_read(c, h, 0, 800, f.host[1]), f.kv[1][0])
    finally:
        f.close()


def test_compaction_is_refused_on_a_capturing_stream():
    f = Filled([30, 40], seed=7, budget=64)
    try:
        c = f.c
        c.request_end(f.hs[0])
        s0 = c.stats()
        g = torch.cuda.CUDAGraph()
        x = torch.zeros(4, device=f.dev)
        with torch.cuda.graph(g):
            x += 1
            with pytest.raises(Q.QsaError) as e:
                c.compact()
        assert e.value.status == Q.ERR_INVALID_ARG
        assert c.stats() == s0
        c.compact()
    finally:
        f.close()


def test_many_requests_come_and_go():
    """Random begins, forks, ends and compactions on all placements; every
    live request keeps its rows throughout."""
    rng = random.Random(3)
    L, ring, cap = 2, 16, 400
    c = Q.Cache(n_layers=L, max_requests=8, ctx_capacity=cap, hbm_pool_rows=3000, budget_tokens=64,
                ring_tokens=ring, staging_rows=4)
    dev = c.pool.device
    live, hosts = {}, []
    try:
        for step in range(120):
            x = rng.random()
            if x < 0.4 or not live:
                place = rng.choice([Q.KV_HBM, Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST])
                parent = rng.choice(sorted(live)) if live and rng.random() < 0.5 else None
                n = rng.randint(1, cap if parent is None else live[parent][2])
                host = None
                if place != Q.KV_HBM:
                    host = workloads.alloc_host((L, n, 2048), dev, "vmm")
                    hosts.append(host)
                try:
                    h = (c.request_begin(n, place, host_rows=host) if parent is None else
                         c.request_fork(live[parent][0], n, place, host_rows=host))
                except Q.QsaError as e:
                    assert e.status in (Q.ERR_CAPACITY, Q.ERR_OUT_OF_SLOTS)
                    continue
                if parent is None:
                    kv = torch.randint(0, 256, (L, n, 2048), dtype=torch.uint8)
                    c.append_chunk([h], [n], 0, L, torch.randn(L * n, 64, device=dev), kv.view(L * n, 2048).to(dev))
                else:
                    kv = live[parent][1][:, :n]
                live[h.index] = (h, kv, n, host)
            elif x < 0.7:
                c.request_end(live.pop(rng.choice(sorted(live)))[0])
            else:
                c.compact()
            if step % 10 == 9:
                torch.cuda.synchronize()
                _clean(c)
                for h, kv, n, host in live.values():
                    for l in range(L):
                        assert torch.equal(_read(c, h, l, n, host), kv[l]), (step, h)
    finally:
        torch.cuda.synchronize()
        c.close()
        for h in hosts:
            workloads.free_host(h)

"""The chunk operators (several queries of a request at once) on the GPU,
against plain implementations in float64: what a chunk append stores, the
block scores, the selections and the attention of every query, at the sizes
and masks where they can go wrong; and the refusals.

Tolerances.  Scores: 64 products of at most fp32 precision and 8 heads, summed
in fp32: under (64 + 8 + 4) * 2^-24 < 1e-5 of sum_h |w_h sc| sum_d |q_d k_d|.
Attention: the probabilities are rounded to bf16 for the tensor cores (at most
2^-8 of each term of sum p|v|), the output once to bf16 (2^-8 of it), and fp32
sums add less than 1e-4 of sum p|v|; lse: 128 products in fp32 (2^-17 of
scale * sum |q_d k_d|) and a log-sum of up to 8192 terms (under 1e-5)."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from oracle import qsa_oracle as O
from sparse_attention_decode_qsa_gb300 import synth, workloads
from tests import qsa_check as QC

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128)
NEG = -1.5e30          # marks entries that a call must leave alone


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _clean(c):
    st, det = c.poll_error()
    assert st == 0, f"device error word {st} detail {det}"


class Filled:
    """A cache with requests of given contexts and placements, filled with
    seeded keys and rows that the test keeps for itself."""

    def __init__(self, ctxs, placements=None, layers=1, fp8=False, ring=64, budget=2048, seed=1, grow=0,
                 spare=0, hot_rows=0, cap=None):
        R = len(ctxs)
        placements = placements or [Q.KV_HBM] * R
        self.fp8, self.layers, self.ctxs, self.placements, self.ring = fp8, layers, list(ctxs), placements, ring
        rows = sum(layers * {Q.KV_HBM: n + grow, Q.KV_HOST_RING: ring + hot_rows, Q.KV_HOST: hot_rows}[p]
                   for n, p in zip(ctxs, placements))
        cap = cap or max(ctxs) + grow
        self.c = c = Q.Cache(n_layers=layers, max_requests=R + 2, ctx_capacity=cap, hbm_pool_rows=rows + spare + 8,
                             budget_tokens=budget, ring_tokens=ring, staging_rows=0, hot_rows=hot_rows,
                             kv_format=Q.KV_FP8 if fp8 else Q.KV_BF16)
        self.dev = c.pool.device
        self.host, self.hs, self.kv, self.codes, self.scales = [], [], [], [], []
        for r, (n, p) in enumerate(zip(ctxs, placements)):
            hist = None
            if p != Q.KV_HBM:
                hist = workloads.alloc_host((layers, n + grow, c.row_bytes), self.dev, "vmm")
            self.host.append(hist)
            h = c.request_begin(n, p, host_rows=hist, max_ctx=n + grow)
            self.hs.append(h)
            kv = synth.kv_rows(layers * n, synth.mix_seed(seed, 5, r))
            kv = (synth.fp8_kv_rows(kv) if fp8 else kv).view(layers, n, c.row_bytes)
            codes, sc = synth.index_keys(layers * n, synth.mix_seed(seed, 6, r))
            codes, sc = codes.view(layers, n, 64), sc.view(layers, n)
            self.kv.append(kv)
            self.codes.append(codes.numpy())
            self.scales.append(QC.bits16(sc))
            c.index_keys[h.index, :, :n] = codes.to(self.dev)
            c.index_scales[h.index, :, :n] = sc.to(self.dev)
            if hist is not None:
                hist[:, :n] = kv
            for l in range(layers):
                slots = c.slot_table[h.index, l, :n].long()
                at = (slots >= 0).nonzero().flatten()
                c.pool[slots[at]] = kv[l].to(self.dev)[at]
        torch.cuda.synchronize()

    def positions(self, n_tokens):
        """(request, position) of every row of one layer."""
        return [(r, n - k + i) for r, (n, k) in enumerate(zip(self.ctxs, n_tokens)) for i in range(k)]

    def values(self, r, l, toks):
        """K and V of tokens, float64 [m][4][128] each."""
        rows = self.kv[r][l][torch.as_tensor(toks, dtype=torch.long)].numpy()
        return O.split_kv_fp8(rows) if self.fp8 else O.split_kv(rows)

    def close(self):
        self.c.close()
        for h in self.host:
            if h is not None:
                workloads.free_host(h)


def _attend(q_bits, K, V):
    """out, lse, sum p|v|, scale * sum |q k| of the largest logit's bound."""
    q = O.decode_bf16(q_bits).reshape(16, 128)
    out, lse, mag, lmag = np.zeros((16, 128)), np.full(16, -np.inf), np.zeros((16, 128)), np.zeros(16)
    if len(K):
        for h in range(16):
            x = SCALE * (K[:, h // 4] @ q[h])
            m = x.max()
            p = np.exp(x - m)
            out[h], mag[h] = p @ V[:, h // 4] / p.sum(), p @ np.abs(V[:, h // 4]) / p.sum()
            lse[h] = m + np.log(p.sum())
            lmag[h] = SCALE * (np.abs(K[:, h // 4]) @ np.abs(q[h])).max()
    return out, lse, mag, lmag


def _check_attention(f, n_tokens, q, sel, nsel, out, lse, layers=1, sample=None, layer0=0):
    rows = [(l, r, p) for l in range(layers) for r, p in f.positions(n_tokens)]
    assert len(rows) == out.shape[0]
    idx = range(len(rows)) if sample is None or len(rows) <= sample else \
        sorted(set(np.random.RandomState(3).choice(len(rows), sample, replace=False)) | {0, len(rows) - 1})
    for x in idx:
        l, r, pos = rows[x]
        toks = [t for b in sel[x][:nsel[x]] for t in range(4 * b, min(4 * b + 4, pos + 1))]
        K, V = f.values(r, l + layer0, toks)
        o, ls, mag, lmag = _attend(QC.bits16(q[x]), K, V)
        got = out[x].double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4) * mag
        assert np.all(np.abs(got - o) <= tol + 1e-30), (x, r, pos, np.abs(got - o).max())
        if lse is not None:
            gl = lse[x].double().cpu().numpy()
            if len(toks) == 0:
                assert np.all(gl == -np.inf) and np.all(got == 0)
            else:
                assert np.all(np.abs(gl - ls) <= 2.0 ** -17 * lmag + 1e-5), (x, np.abs(gl - ls).max())


def _random_selection(f, n_tokens, budget, seed, layers=1, keep=1.0):
    """Distinct blocks of every query's context in ascending order, on the host."""
    rng = np.random.RandomState(seed)
    sel, nsel = [], []
    for _ in range(layers):
        for r, p in f.positions(n_tokens):
            nb = p // 4 + 1
            k = min(budget // 4, nb)
            if keep < 1.0:
                k = rng.randint(0, int(keep * k) + 1)
            sel.append(np.sort(rng.choice(nb, k, replace=False)))
            nsel.append(k)
    t = torch.full((len(sel), budget // 4), -7, dtype=torch.int32)
    for x, s in enumerate(sel):
        t[x, :len(s)] = torch.as_tensor(s, dtype=torch.int32)
    return sel, nsel, t, torch.tensor(nsel, dtype=torch.int32)


def _run_attention(f, n_tokens, q, t, n, budget, layers=1, layer0=0, lse=True, workspace=None):
    out = torch.full_like(q, float("nan"))
    ls = torch.full(q.shape[:2], float("nan"), device=q.device) if lse else None
    f.c.chunk_sparse_attn(f.hs, n_tokens, layer0, layers, q, t.to(f.dev), n.to(f.dev), budget, SCALE, out, ls,
                          workspace=workspace)
    torch.cuda.synchronize()
    return out, ls


def _queries(rows, seed, dev, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(rows, 16, 128, generator=g)).bfloat16().to(dev)


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("chunks", [[[1, 1, 1, 1]], [[5, 3, 40, 0], [2, 60, 1, 7]]])
def test_append_chunk_stores_what_single_appends_would(fp8, chunks):
    L, ring, grow = 2, 16, 80
    ctxs, places = [33, 5, 40, 9], [Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST_RING, Q.KV_HOST]
    f = Filled(ctxs, places, layers=L, fp8=fp8, ring=ring, grow=grow, budget=64)
    try:
        c, R = f.c, len(ctxs)
        want = [[c.slot_table[h.index, l, :n].cpu().numpy().tolist() + [None] * grow for l in range(L)]
                for h, n in zip(f.hs, ctxs)]
        new = {}
        g = torch.Generator().manual_seed(9)
        for step, counts in enumerate(chunks):
            for h, k in zip(f.hs, counts):
                if k:
                    c.advance(h, k)
            N_ = sum(counts)
            k_new = torch.randn(L * N_, 64, generator=g) * torch.exp2(torch.randint(-40, 40, (L * N_, 1), generator=g).float())
            k_new[0] = 0
            k_new[-1, 3] = 3e7
            kv_new = synth.kv_rows(L * N_, 77 + step)
            kv_new[1 % (L * N_), :256] = 0                     # an all-zero head vector
            c.append_chunk(f.hs, counts, 0, L, k_new.to(f.dev), kv_new.to(f.dev))
            x = 0
            for l in range(L):
                for r, k in enumerate(counts):
                    info = c.request_info(f.hs[r])
                    place = {Q.KV_HBM: "hbm", Q.KV_HOST_RING: "ring", Q.KV_HOST: "host"}[places[r]]
                    for i in range(k):
                        t = f.ctxs[r] + i
                        new[r, l, t] = (k_new[x].numpy(), kv_new[x].numpy())
                        for tok, slot in O.append_slot_writes(t, place, info.hbm_row_base, l, info.layer_rows, ring):
                            want[r][l][tok] = slot
                        x += 1
            for r, k in enumerate(counts):
                f.ctxs[r] += k
        torch.cuda.synchronize()
        _clean(c)
        for r, h in enumerate(f.hs):
            for l in range(L):
                n = f.ctxs[r]
                assert c.slot_table[h.index, l, :n].cpu().tolist() == want[r][l][:n], (r, l)
                for t in range(n):
                    if (r, l, t) in new:
                        key, row = new[r, l, t]
                        codes, bits = O.quantize_index_key(key)
                        row = O.quantize_kv_row_fp8(row) if fp8 else row
                        assert np.array_equal(c.index_keys[h.index, l, t].cpu().numpy(), codes), (r, l, t)
                        assert int(QC.bits16(c.index_scales[h.index, l, t:t + 1])[0]) == bits
                    else:
                        row = f.kv[r][l][t].numpy()
                        assert np.array_equal(c.index_keys[h.index, l, t].cpu().numpy(), f.codes[r][l, t])
                    if want[r][l][t] >= 0:
                        assert np.array_equal(c.pool[want[r][l][t]].cpu().numpy(), row), (r, l, t)
                    if f.host[r] is not None:
                        assert np.array_equal(f.host[r][l, t].numpy(), row), (r, l, t)
    finally:
        f.close()


# ------------------------------------------------------------------- scores

def _check_scores(f, n_tokens, q, w, blk, layers=1, sample=24):
    rows = [(l, r, p) for l in range(layers) for r, p in f.positions(n_tokens)]
    idx = range(len(rows)) if len(rows) <= sample else \
        sorted(set(np.random.RandomState(4).choice(len(rows), sample, replace=False)) | {0, len(rows) - 1})
    host = blk.double().cpu().numpy()
    for x in idx:
        l, r, pos = rows[x]
        codes, sc = f.codes[r][l, :pos + 1], f.scales[r][l, :pos + 1]
        qd, wd = q[x].double().cpu().numpy(), w[x].double().cpu().numpy()
        ref = O.c4_block_scores(O.token_scores(codes, sc, qd, wd))
        key = np.abs(O.decode_e4m3(codes)) * np.abs(O.decode_fp16(sc))[:, None]
        mag = O.c4_block_scores((key @ np.abs(qd).T) @ np.abs(wd))
        err = np.abs(host[x, :len(ref)] - ref)
        assert np.all(err <= QC.SCORE_REL_TOL * mag + 1e-30), (x, (err / (mag + 1e-30)).max())
        assert np.all(host[x, len(ref):] == np.float32(NEG)), x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,layers", [
    ([1], [1], 1), ([2, 5, 130], [2, 5, 1], 1), ([513, 700], [33, 0], 2), ([640, 641, 1023], [7, 64, 65], 1),
    ([4099], [300], 1), ([20000, 9001], [3, 130], 1), ([66000], [1], 1)])
def test_chunk_scores_match_float64(bf16, ctxs, n_tokens, layers):
    f = Filled(ctxs, layers=layers, seed=11, budget=64)
    try:
        rows = layers * sum(n_tokens)
        g = torch.Generator().manual_seed(2)
        q = torch.randn(rows, 8, 64, generator=g)
        q[0, :4] *= 1e-3
        q[rows // 2, :, ::3] *= 2.0 ** -20
        w = torch.rand(rows, 8, generator=g)
        w[rows // 3, 2] = -0.7
        w[rows // 3, 5] = 0
        q = q.bfloat16() if bf16 else q
        # some keys with no scale, some with a sign in it
        for r in range(len(ctxs)):
            f.scales[r][:, ::17] = 0
            f.scales[r][:, 3::29] |= 0x8000
            n = ctxs[r]
            f.c.index_scales[f.hs[r].index, :, :n] = torch.from_numpy(f.scales[r].view(np.int16).copy()).view(torch.float16).to(f.dev)
        stride = (max(ctxs) + 3) // 4 + 3
        blk = torch.full((rows, stride), NEG, device=f.dev)
        f.c.chunk_index_score(f.hs, n_tokens, 0, layers, q.to(f.dev), w.to(f.dev), blk)
        torch.cuda.synchronize()
        _clean(f.c)
        _check_scores(f, n_tokens, q, w, blk, layers)
    finally:
        f.close()


def test_chunk_scores_of_one_token_equal_the_decode_step_in_value():
    f = Filled([5000, 131], seed=3, budget=64)
    try:
        q, w = torch.randn(2, 8, 64, device=f.dev), torch.rand(2, 8, device=f.dev)
        a = torch.full((2, 1250), NEG, device=f.dev)
        b = a.clone()
        f.c.index_score(f.hs, 0, 1, q, w, a)
        f.c.chunk_index_score(f.hs, [1, 1], 0, 1, q, w, b)
        torch.cuda.synchronize()
        assert torch.equal(a == NEG, b == NEG)
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-4)
    finally:
        f.close()


# --------------------------------------------------------------- selections

def _check_selection(blk, positions, budget, sel, nsel, fill=-9):
    host, sel, nsel = blk.cpu().numpy(), sel.cpu().numpy(), nsel.cpu().numpy()
    for x, pos in enumerate(positions):
        nb = pos // 4 + 1
        ref = O.select_blocks(host[x, :nb], budget)
        assert nsel[x] == len(ref), x
        assert np.array_equal(sel[x, :len(ref)], ref), x
        assert np.all(sel[x, len(ref):] == fill), x


def _score_rows(rows, stride, kind, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    s = torch.randn(rows, stride, generator=g, device=dev)
    if kind == "ties":
        s = torch.round(s * 2) / 2
    elif kind == "zeros":                       # relu leaves most blocks at 0, some at -0
        s = torch.where(s > 2, s, torch.zeros_like(s))
        s[:, ::3] *= -1.0
    elif kind == "same":
        s.fill_(3.25)
    elif kind == "infinite":
        s[:, ::5] = -math.inf
        s[:, 7::11] = math.inf
    elif kind == "huge":
        s *= 1e30
    elif kind == "rising":
        s = torch.arange(stride, device=dev, dtype=torch.float32).expand(rows, stride) * 0.25 + 0 * s
    elif kind == "falling":
        s = -torch.arange(stride, device=dev, dtype=torch.float32).expand(rows, stride) + 0 * s
    elif kind == "steps":                       # long runs of equal scores
        s = (torch.arange(stride, device=dev) // 1000 % 7).float().expand(rows, stride) + 0 * s
    return s.contiguous()


@pytest.mark.parametrize("kind", ["normal", "ties", "zeros", "same", "infinite", "huge", "rising", "falling", "steps"])
@pytest.mark.parametrize("ctxs,n_tokens,budget", [
    ([1, 4, 5], [1, 2, 5], 8), ([2049, 2055], [9, 3], 2048), ([4096, 131], [2, 2], 64), ([60001], [5], 2048),
    ([131072, 9000], [3, 1], 2048), ([40000], [2], 8192), ([40000], [2], 4)])
def test_chunk_selection_matches_the_rule(kind, ctxs, n_tokens, budget):
    f = Filled([1] * len(ctxs), grow=max(ctxs) - 1, budget=8192, spare=0)
    try:
        for h, n in zip(f.hs, ctxs):
            if n > 1:
                f.c.advance(h, n - 1)
        f.ctxs = ctxs
        rows = sum(n_tokens)
        stride = (max(ctxs) + 3) // 4 + 1
        blk = _score_rows(rows, stride, kind, 5, f.dev)
        for x, (_, pos) in enumerate(f.positions(n_tokens)):
            blk[x, pos // 4 + 1:] = float("nan")        # past the query's context: never read as scores
        sel = torch.full((rows, budget // 4), -9, dtype=torch.int32, device=f.dev)
        nsel = torch.full((rows,), -9, dtype=torch.int32, device=f.dev)
        f.c.chunk_select_topk(f.hs, n_tokens, 0, 1, blk, budget, sel, nsel)
        torch.cuda.synchronize()
        _clean(f.c)
        _check_selection(blk, [p for _, p in f.positions(n_tokens)], budget, sel, nsel)
    finally:
        f.close()


@pytest.mark.parametrize("kind", ["normal", "zeros", "steps"])
def test_chunk_selection_past_a_million_tokens(kind):
    n = 1100003
    c = Q.Cache(n_layers=1, max_requests=1, ctx_capacity=n, hbm_pool_rows=n, budget_tokens=2048, staging_rows=0)
    h = c.request_begin(n)
    blk = _score_rows(3, (n + 3) // 4, kind, 6, c.pool.device)
    sel = torch.full((3, 512), -9, dtype=torch.int32, device=c.pool.device)
    nsel = torch.zeros(3, dtype=torch.int32, device=c.pool.device)
    c.chunk_select_topk([h], [3], 0, 1, blk, 2048, sel, nsel)
    torch.cuda.synchronize()
    _check_selection(blk, [n - 3, n - 2, n - 1], 2048, sel, nsel)
    c.close()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens,layers,budget", [
    ([1], [1], 1, 64), ([3, 6, 130], [3, 1, 2], 1, 64), ([257, 300, 64], [65, 0, 64], 2, 128),
    ([2100], [129], 1, 2048), ([9000, 4001, 700, 33], [4, 31, 32, 33], 1, 2048), ([30000], [3], 1, 8192),
    ([5000], [257], 1, 512)])
def test_chunk_attention_matches_float64(fp8, ctxs, n_tokens, layers, budget):
    f = Filled(ctxs, layers=layers, fp8=fp8, seed=21, budget=8192)
    try:
        sel, nsel, t, n = _random_selection(f, n_tokens, budget, 31, layers)
        q = _queries(len(sel), 41, f.dev, scale=2.0)
        out, lse = _run_attention(f, n_tokens, q, t, n, budget, layers)
        _clean(f.c)
        _check_attention(f, n_tokens, q, sel, nsel, out, lse, layers, sample=40)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_chunk_attention_reads_rings_hosts_and_pool_alike(fp8):
    ctxs, n_tokens = [3000, 2501, 700, 90], [37, 70, 1, 5]
    f = Filled(ctxs, [Q.KV_HOST_RING, Q.KV_HOST, Q.KV_HBM, Q.KV_HOST_RING], layers=2, fp8=fp8, ring=333, seed=5)
    try:
        sel, nsel, t, n = _random_selection(f, n_tokens, 512, 8, 1)
        q = _queries(len(sel), 43, f.dev)
        out, lse = _run_attention(f, n_tokens, q, t, n, 512, layers=1, layer0=1)
        _clean(f.c)
        _check_attention(f, n_tokens, q, sel, nsel, out, lse, sample=30, layer0=1)
    finally:
        f.close()


@pytest.mark.parametrize("n_tokens", [[40, 3], [1, 1], [130, 64]])
def test_rows_with_few_or_no_blocks(n_tokens):
    """Ragged counts, rows without any block, rows whose only block is their
    own, and no lse."""
    f = Filled([500, 200], seed=4, budget=256)
    try:
        sel, nsel, t, n = _random_selection(f, n_tokens, 256, 12, keep=0.4)
        pos = f.positions(n_tokens)
        for x in range(0, len(sel), 3):
            sel[x], nsel[x], n[x] = sel[x][:0], 0, 0
        for x in range(1, len(sel), 5):
            sel[x], nsel[x], n[x] = np.array([pos[x][1] // 4]), 1, 1
            t[x, 0] = pos[x][1] // 4
        q = _queries(len(sel), 3, f.dev)
        out, lse = _run_attention(f, n_tokens, q, t, n, 256)
        _clean(f.c)
        _check_attention(f, n_tokens, q, sel, nsel, out, lse)
        out2, _ = _run_attention(f, n_tokens, q, t, n, 256, lse=False)
        assert torch.equal(out, out2)
    finally:
        f.close()


def test_order_of_the_selected_blocks_does_not_matter():
    f = Filled([3000], seed=4, budget=512)
    try:
        sel, nsel, t, n = _random_selection(f, [50], 512, 12)
        q = _queries(50, 3, f.dev)
        a = _run_attention(f, [50], q, t, n, 512)
        t2 = t.clone()
        for x, s in enumerate(sel):
            t2[x, :nsel[x]] = torch.as_tensor(s[np.random.RandomState(x).permutation(len(s))].copy(), dtype=torch.int32)
        b = _run_attention(f, [50], q, t2, n, 512)
        _check_attention(f, [50], q, sel, nsel, *b)
        assert torch.equal(a[1].isfinite(), b[1].isfinite())
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_values_that_are_not_finite_reach_only_the_queries_that_select_them(fp8, value):
    """Tokens with infinite or NaN keys and values: queries that do not select
    them, and queries before them in their own block, are as without them."""
    f = Filled([400], seed=6, budget=128, fp8=fp8)
    try:
        n_tokens = [70]
        bad = [40, 41, 350, 399]              # 350: inside the chunk, its block's earlier queries must not see it
        c = f.c
        rows = c.slot_table[f.hs[0].index, 0, bad].long()
        for i, r_ in enumerate(rows.tolist()):
            if fp8:
                sc = c.pool[r_, 1024:].view(torch.float16)
                sc[4 if i % 2 else 0:8] = value
            else:
                c.pool[r_].view(torch.bfloat16)[512 if i % 2 else 0:] = value
        sel, nsel, t, n = _random_selection(f, n_tokens, 128, 5)
        pos = [p for _, p in f.positions(n_tokens)]
        q = _queries(70, 7, f.dev)
        out, lse = _run_attention(f, n_tokens, q, t, n, 128)
        hit = [any(b // 4 in sel[x] and b <= pos[x] for b in bad) for x in range(70)]
        assert 5 < sum(hit) < 65
        clean = [x for x in range(70) if not hit[x]]
        rows_ = [(0, r, p) for r, p in f.positions(n_tokens)]
        for x in clean:
            _, r, p = rows_[x]
            toks = [k for b in sel[x] for k in range(4 * b, min(4 * b + 4, p + 1))]
            o, ls, mag, lmag = _attend(QC.bits16(q[x]), *f.values(r, 0, toks))
            assert np.all(np.abs(out[x].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4) * mag), x
            assert np.all(np.abs(lse[x].double().cpu().numpy() - ls) <= 2.0 ** -17 * lmag + 1e-5), x
        for x in range(70):
            if hit[x]:
                assert not bool(out[x].isfinite().all()), x
    finally:
        f.close()


def test_large_logits_and_far_apart_rows():
    """Logits of several hundreds (one token takes all), and rows whose
    running maximum rises from tile to tile."""
    f = Filled([2048], seed=9, budget=2048)
    try:
        sel, nsel, t, n = _random_selection(f, [40], 2048, 5)
        q = _queries(40, 7, f.dev, scale=60.0)
        out, lse = _run_attention(f, [40], q, t, n, 2048)
        _check_attention(f, [40], q, sel, nsel, out, lse, sample=12)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_far_below_other_queries_tokens_keep_their_own(fp8):
    """Keys of half the blocks point along one direction with logits in the
    hundreds for every query; queries of odd rows select only the others."""
    f = Filled([1024], seed=9, budget=512, fp8=fp8)
    try:
        c = f.c
        rows = c.slot_table[f.hs[0].index, 0, :1024].long()
        kv = f.kv[0][0].numpy()
        K, V = f.values(0, 0, list(range(1024)))
        hot = [t for t in range(1024) if (t // 4) % 2 == 0]
        d = torch.randn(128, generator=torch.Generator().manual_seed(4)).bfloat16()
        raw = torch.from_numpy(kv).clone()
        if fp8:
            k = d.float().repeat(4, 1)
            v = torch.zeros(1, 8, 128)
            v[0, :4] = k
            new = synth.fp8_kv_rows(v.bfloat16().view(1, 1024).view(torch.uint8).view(1, 2048))[0]
            raw[hot, :512] = new[:512]
            raw[hot, 1024:1032] = new[1024:1032]
        else:
            raw[hot, :1024] = d.repeat(4).view(torch.uint8)
        f.kv[0] = raw[None]
        c.pool[rows] = raw.to(f.dev)
        q = (25.0 * d.float() + torch.randn(70, 16, 128, generator=torch.Generator().manual_seed(5))).bfloat16().to(f.dev)
        pos = [p for _, p in f.positions([70])]
        rng = np.random.RandomState(2)
        sel, t = [], torch.full((70, 128), -1, dtype=torch.int32)
        for x in range(70):
            ids = np.arange(pos[x] // 4 + 1)
            ids = ids[ids % 2 == 1] if x % 2 else ids
            sel.append(np.sort(rng.choice(ids, 100, replace=False)))
            t[x, :100] = torch.as_tensor(sel[x], dtype=torch.int32)
        n = torch.full((70,), 100, dtype=torch.int32)
        out, lse = _run_attention(f, [70], q, t, n, 512)
        _clean(c)
        _check_attention(f, [70], q, sel, [100] * 70, out, lse)
    finally:
        f.close()


def test_bad_blocks_counts_and_slots_are_reported_and_skipped():
    f = Filled([300], seed=10, budget=64)
    try:
        c = f.c
        sel, nsel, t, n = _random_selection(f, [20], 64, 5)
        q = _queries(20, 7, f.dev)
        pos = [p for _, p in f.positions([20])]
        # a block past the query's position, one far outside, a negative one
        for x, b in ((0, pos[0] // 4 + 1), (5, 1 << 29), (9, -3)):
            t[x, 4] = b
            sel[x] = np.delete(sel[x], 4)
        out, lse = _run_attention(f, [20], q, t, n, 64)
        assert c.poll_error()[0] == Q.ERR_BAD_BLOCK
        _check_attention(f, [20], q, sel, [len(s) for s in sel], out, lse)
        _clean(c)
        # counts outside [0, budget / 4]: the row counts as empty
        sel, nsel, t, n = _random_selection(f, [20], 64, 5)
        n[3], n[11] = 17, -1
        sel[3], sel[11] = sel[3][:0], sel[11][:0]
        out, lse = _run_attention(f, [20], q, t, n, 64)
        assert c.poll_error()[0] == Q.ERR_BAD_BLOCK
        _check_attention(f, [20], q, sel, [len(s) for s in sel], out, lse)
        # a slot outside the pool: its token is left out, for every query
        sel, nsel, t, n = _random_selection(f, [20], 64, 5)
        tok = 4 * int(sel[0][0]) + 1
        c.slot_table[f.hs[0].index, 0, tok] = c.pool.shape[0]
        c.slot_table[f.hs[0].index, 0, 4 * int(sel[0][1])] = -1          # cold, but there is no host history
        gone = {tok, 4 * int(sel[0][1])}
        out, lse = _run_attention(f, [20], q, t, n, 64)
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        for x in range(20):
            toks = [k for b in sel[x] for k in range(4 * b, min(4 * b + 4, pos[x] + 1)) if k not in gone]
            o, ls, mag, lmag = _attend(QC.bits16(q[x]), *f.values(0, 0, toks))
            assert np.all(np.abs(out[x].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4) * mag)
    finally:
        f.close()


# ----------------------------------------------------------------- refusals

def test_refusals_leave_everything_alone():
    f = Filled([300, 200], seed=10, budget=64, layers=2)
    try:
        c, dev = f.c, f.dev
        hs = f.hs
        q = torch.zeros(4, 8, 64, device=dev)
        w, blk = torch.zeros(4, 8, device=dev), torch.full((4, 75), NEG, device=dev)
        st = []

        def refused(status, call, *a, **kw):
            with pytest.raises(Q.QsaError) as e:
                call(*a, **kw)
            assert e.value.status == status, e.value
            st.append(1)

        bad = Q.ERR_INVALID_ARG
        refused(bad, c.chunk_index_score, [], [], 0, 1, q[:0], w[:0], blk[:0])
        refused(bad, c.chunk_index_score, [hs[0], hs[0]], [2, 2], 0, 1, q, w, blk)
        refused(bad, c.chunk_index_score, hs, [2, 2], 2, 1, q, w, blk)
        refused(bad, c.chunk_index_score, hs, [2, 2], -1, 1, q, w, blk)
        refused(bad, c.chunk_index_score, hs, [5, -1], 0, 1, q, w, blk)
        refused(bad, c.chunk_index_score, hs, [2, 2], 0, 1, q, w, blk[:, :74].contiguous())
        refused(bad, c.chunk_index_score, [hs[1]], [201], 0, 1, q.new_zeros(201, 8, 64), w.new_zeros(201, 8),
                blk.new_zeros(201, 75))
        refused(bad, c.chunk_index_score, hs, [2, 2], 0, 1, torch.zeros(4 * 512 + 1, device=dev)[1:].view(4, 8, 64), w, blk)
        refused(Q.ERR_STALE_HANDLE, c.chunk_index_score, [hs[0], Q.Handle(1, 9)], [2, 2], 0, 1, q, w, blk)
        sel, nsel = torch.zeros(4, 16, dtype=torch.int32, device=dev), torch.zeros(4, dtype=torch.int32, device=dev)
        refused(bad, c.chunk_select_topk, hs, [2, 2], 0, 1, blk, 68, sel.new_zeros(4, 17), nsel)
        refused(bad, c.chunk_select_topk, hs, [2, 2], 0, 1, blk, 6, sel.new_zeros(4, 1), nsel)
        qa = torch.zeros(4, 16, 128, dtype=torch.bfloat16, device=dev)
        ws = torch.zeros(c.chunk_attn_workspace_bytes(hs, [2, 2], 0, 1, 64), dtype=torch.uint8, device=dev)
        refused(bad, c.chunk_sparse_attn, hs, [2, 2], 0, 1, qa, sel, nsel, 64, SCALE, qa, workspace=ws[:-16])
        refused(bad, c.chunk_sparse_attn, hs, [2, 2], 0, 1, qa, sel, nsel, 64, float("nan"), qa, workspace=ws)
        refused(bad, c.chunk_sparse_attn, hs, [2, 2], 0, 1, qa, sel, nsel, 64, SCALE, qa,
                workspace=torch.zeros(ws.numel() + 16, dtype=torch.uint8, device=dev)[8:-8])
        with pytest.raises(ValueError):
            c.chunk_sparse_attn(hs, [2, 2], 0, 1, qa.half(), sel, nsel, 64, SCALE, qa, workspace=ws)
        with pytest.raises(ValueError):
            c.chunk_index_score(hs, [2, 2], 0, 1, q.cpu(), w, blk)
        # no rows: nothing to do
        c.chunk_index_score(hs, [0, 0], 0, 2, q[:0], w[:0], blk[:0])
        c.chunk_select_topk(hs, [0, 0], 0, 2, blk[:0], 64, sel[:0], nsel[:0])
        c.chunk_sparse_attn(hs, [0, 0], 0, 2, qa[:0], sel[:0], nsel[:0], 64, SCALE, qa[:0], workspace=ws)
        c.append_chunk(hs, [0, 0], 0, 2, q[:0, 0], torch.zeros(0, 2048, dtype=torch.uint8, device=dev))
        torch.cuda.synchronize()
        assert torch.all(blk == NEG)
        _clean(c)
    finally:
        f.close()


# ------------------------------------------------------- the steps together

def _exact_keys(n, g):
    """Index keys that quantise without rounding (scale 1, powers of two)."""
    k = torch.exp2(torch.randint(0, 6, (n, 64), generator=g).float()) * 7 * torch.randint(-1, 2, (n, 64), generator=g)
    k[:, 0] = 448.0
    return k


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("place", [Q.KV_HBM, Q.KV_HOST_RING])
def test_a_prompt_in_pieces_equals_its_tokens_one_by_one(fp8, place):
    """Two requests take the same 700 tokens at two layers, one in pieces of
    many tokens, one token by token through the decode step.  Index scores are
    whole numbers far below 2^24, so both paths' selections must be equal, ties
    included; attention agrees within the bf16 rounding of the pieces' output."""
    n, L, budget, ring = 700, 2, 256, 128
    g = torch.Generator().manual_seed(5)
    keys = [_exact_keys(n, g) for _ in range(L)]
    rows = [synth.kv_rows(n, 60 + l) for l in range(L)]
    qi = torch.randint(-2, 3, (L, n, 8, 64), generator=g).float()
    w = torch.randint(1, 4, (L, n, 8), generator=g).float()
    q = torch.randn(L, n, 16, 128, generator=g).bfloat16()
    f = Filled([1, 1], [place] * 2, layers=L, fp8=fp8, ring=ring, grow=n, budget=budget)
    try:
        c, dev = f.c, f.dev
        a, b = f.hs
        # token 0 of the second request is made that of the first
        c.index_keys[b.index, :, 0] = c.index_keys[a.index, :, 0]
        c.index_scales[b.index, :, 0] = c.index_scales[a.index, :, 0]
        for l in range(L):
            c.pool[c.slot_table[b.index, l, 0].long()] = c.pool[c.slot_table[a.index, l, 0].long()]
            if f.host[1] is not None:
                f.host[1][l, 0] = f.host[0][l, 0]
        torch.cuda.synchronize()
        got = {}
        at = 0
        for piece in (1, 2, 64, 333, 5, 200, 95):
            c.advance(a, piece)
            s = slice(at, at + piece)
            cat = lambda x: torch.cat([x[l][s] for l in range(L)]).to(dev)  # noqa: E731
            c.append_chunk([a], [piece], 0, L, cat(keys), cat(rows))
            nb = (1 + at + piece + 3) // 4
            blk = torch.full((L * piece, nb), NEG, device=dev)
            sel = torch.full((L * piece, budget // 4), -9, dtype=torch.int32, device=dev)
            nsel = torch.zeros(L * piece, dtype=torch.int32, device=dev)
            out = torch.zeros(L * piece, 16, 128, dtype=torch.bfloat16, device=dev)
            lse = torch.zeros(L * piece, 16, device=dev)
            c.chunk_index_score([a], [piece], 0, L, cat(qi), cat(w), blk)
            c.chunk_select_topk([a], [piece], 0, L, blk, budget, sel, nsel)
            c.chunk_sparse_attn([a], [piece], 0, L, cat(q), sel, nsel, budget, SCALE, out, lse)
            for l in range(L):
                for i in range(piece):
                    got[l, at + i] = (sel[l * piece + i], nsel[l * piece + i], out[l * piece + i], lse[l * piece + i])
            at += piece
        assert at == n
        torch.cuda.synchronize()
        _clean(c)
        blk = torch.empty(1, (n + 4) // 4, device=dev)
        for i in range(n):
            c.advance(b)
            for l in range(L):
                c.append_token([b], l, 1, keys[l][i:i + 1].to(dev), rows[l][i:i + 1].to(dev))
            if i % 23 and i < n - 3:
                continue
            for l in range(L):
                sel = torch.full((1, budget // 4), -9, dtype=torch.int32, device=dev)
                nsel = torch.zeros(1, dtype=torch.int32, device=dev)
                out, lse = torch.zeros(1, 16, 128, device=dev), torch.zeros(1, 16, device=dev)
                c.index_score([b], l, 1, qi[l, i:i + 1].to(dev), w[l, i:i + 1].to(dev), blk)
                c.select_c4_topk([b], l, 1, blk, budget, sel, nsel)
                c.sparse_decode_attn([b], l, 1, q[l, i:i + 1].to(dev), sel, nsel, budget, None, SCALE, out, lse)
                s2, n2, o2, l2 = got[l, i]
                assert int(n2) == int(nsel) and torch.equal(s2, sel[0]), (l, i)
                # values are below 6 in size: 2^-8 (output) + 2^-8 (probabilities) of at most that
                assert (o2.float() - out[0]).abs().max().item() <= 2 * 2.0 ** -8 * 6, (l, i)
                assert (l2 - lse[0]).abs().max().item() <= 1e-4, (l, i)
        torch.cuda.synchronize()
        _clean(c)
        for l in range(L):
            assert torch.equal(c.index_keys[a.index, l, :n + 1], c.index_keys[b.index, l, :n + 1])
    finally:
        f.close()


def test_rejected_drafts_are_taken_back():
    """Append five draft tokens, keep two, go on: the cache equals one that
    only ever saw the kept tokens."""
    f = Filled([50, 50], [Q.KV_HOST_RING] * 2, grow=30, ring=8, budget=64, seed=2)
    try:
        c, dev = f.c, f.dev
        a, b = f.hs
        g = torch.Generator().manual_seed(1)
        k, kv = torch.randn(12, 64, generator=g).to(dev), synth.kv_rows(12, 3).to(dev)
        c.advance(a, 5)
        c.append_chunk([a], [5], 0, 1, k[:5], kv[:5])
        c.truncate(a, 52)
        c.advance(a, 4)
        c.append_chunk([a], [4], 0, 1, k[6:10], kv[6:10])
        c.advance(b, 6)
        keep = [0, 1, 6, 7, 8, 9]
        c.append_chunk([b], [6], 0, 1, k[keep], kv[keep])
        torch.cuda.synchronize()
        _clean(c)
        assert torch.equal(c.index_keys[a.index, 0, 50:56], c.index_keys[b.index, 0, 50:56])
        sa, sb = c.slot_table[a.index, 0, :56].cpu(), c.slot_table[b.index, 0, :56].cpu()
        base_a, base_b = c.request_info(a).hbm_row_base, c.request_info(b).hbm_row_base
        for t in range(56):
            # a ring row that a rejected draft had taken does not come back
            if sa[t] >= 0:
                assert sa[t] - base_a == sb[t] - base_b
                assert torch.equal(c.pool[sa[t]].cpu(), f.host[0][0, t])
            else:
                assert sb[t] < 0 or t < 52
        assert torch.equal(f.host[0][0, 50:56], f.host[1][0, 50:56])
    finally:
        f.close()


def test_captured_steps_replay_and_streams_keep_apart():
    """Score, select and attend captured in a graph and replayed on new
    inputs equal eager calls; two streams with a workspace each run at once."""
    f = Filled([3000, 2000], seed=8, budget=512)
    try:
        c, dev = f.c, f.dev
        n_tokens = [[70, 0], [0, 45]]
        bufs = []
        for i, nt in enumerate(n_tokens):
            rows = sum(nt)
            bufs.append(dict(nt=nt, qi=torch.randn(rows, 8, 64, device=dev), w=torch.rand(rows, 8, device=dev),
                             blk=torch.full((rows, 750), NEG, device=dev), q=_queries(rows, i, dev),
                             sel=torch.full((rows, 128), -9, dtype=torch.int32, device=dev),
                             nsel=torch.zeros(rows, dtype=torch.int32, device=dev),
                             out=torch.zeros(rows, 16, 128, dtype=torch.bfloat16, device=dev),
                             lse=torch.zeros(rows, 16, device=dev),
                             ws=torch.empty(c.chunk_attn_workspace_bytes(f.hs, nt, 0, 1, 512), dtype=torch.uint8,
                                            device=dev)))

        def step(b):
            c.chunk_index_score(f.hs, b["nt"], 0, 1, b["qi"], b["w"], b["blk"])
            c.chunk_select_topk(f.hs, b["nt"], 0, 1, b["blk"], 512, b["sel"], b["nsel"])
            c.chunk_sparse_attn(f.hs, b["nt"], 0, 1, b["q"], b["sel"], b["nsel"], 512, SCALE, b["out"], b["lse"],
                                workspace=b["ws"])

        want = []
        for b in bufs:
            step(b)
            torch.cuda.synchronize()
            want.append((b["sel"].clone(), b["out"].clone(), b["lse"].clone()))
        streams = [torch.cuda.Stream() for _ in bufs]
        graphs = []
        for b, s in zip(bufs, streams):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(b)
            graphs.append(g)
        for _ in range(5):
            for b in bufs:
                for x in (b["sel"], b["out"], b["lse"], b["blk"]):
                    x.zero_()
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for b, (s_, o, l) in zip(bufs, want):
                assert torch.equal(b["nsel"] > 0, torch.ones_like(b["nsel"], dtype=torch.bool))
                k = b["nsel"].amin()
                assert torch.equal(b["sel"][:, :k], s_[:, :k])
                assert torch.equal(b["out"], o) and torch.equal(b["lse"], l)
        # other inputs through the same graph
        b = bufs[0]
        b["qi"].neg_()
        b["blk"].zero_()
        graphs[0].replay()
        torch.cuda.synchronize()
        o = b["out"].clone()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(o, b["out"]) and not torch.equal(o, want[0][1])
        _clean(c)
    finally:
        f.close()


@pytest.mark.parametrize("raw", [False, True])
def test_a_workspace_allocated_for_another_stream_is_that_streams_own(raw):
    """Memory freed on the current stream, which still writes to it, is not
    taken as the workspace of a call on another stream."""
    f = Filled([2500], seed=12, budget=512)
    try:
        nt = [40]
        q = _queries(40, 9, f.dev)
        _, _, t, n = _random_selection(f, nt, 512, seed=4)
        t, n = t.to(f.dev), n.to(f.dev)
        want, ls = _run_attention(f, nt, q, t, n, 512)
        out, lse = torch.zeros_like(want), torch.zeros_like(ls)
        need = f.c.chunk_attn_workspace_bytes(f.hs, nt, 0, 1, 512)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            busy = torch.empty(need, dtype=torch.uint8, device=f.dev)
            for _ in range(400):
                busy.zero_()
            del busy
            f.c.chunk_sparse_attn(f.hs, nt, 0, 1, q, t, n, 512, SCALE, out, lse,
                                  stream=side.cuda_stream if raw else side)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, ls)
        _clean(f.c)
    finally:
        f.close()


def test_fp8_codes_of_a_chunk_are_the_quotients_of_single_appends():
    """Every bf16 value, infinities and NaN among them, in head vectors of
    neighbouring values, of values far apart, and beside a largest element."""
    g = torch.Generator().manual_seed(3)
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    near, far = x, x[torch.randperm(65536, generator=g)]
    top = x.view(-1, 128).clone()
    top[:, 0] = (0x4000 + torch.arange(512) % 128).to(torch.int16)        # 2 .. 3.98
    small = torch.where(x.view(torch.bfloat16).float().view(-1, 128).abs() < 4, top, torch.zeros_like(top))
    kv = torch.cat([near, far, small.flatten()]).view(-1, 1024).contiguous().view(torch.uint8)
    n = kv.shape[0]
    Q.lib()
    c = Q.Cache(n_layers=1, max_requests=2, ctx_capacity=n + 1, hbm_pool_rows=2 * n + 2, budget_tokens=64,
                ring_tokens=64, staging_rows=0, kv_format=Q.KV_FP8)
    try:
        dev = c.pool.device
        kv, k = kv.to(dev), torch.randn(n, 64, generator=g).to(dev)
        a = c.request_begin(1, max_ctx=n + 1)
        c.advance(a, n)
        c.append_chunk([a], [n], 0, 1, k, kv)
        b = c.request_begin(1, max_ctx=n + 1)
        for i in range(n):
            c.advance(b)
            c.append_token([b], 0, 1, k[i:i + 1], kv[i:i + 1])
        torch.cuda.synchronize()
        rows = [c.pool[c.slot_table[h.index, 0, 1:n + 1].long()] for h in (a, b)]
        assert torch.equal(rows[0], rows[1])
        _clean(c)
    finally:
        c.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests", [1, 13, 37, 38, 39])
def test_lists_of_very_different_lengths_share_the_device(requests, fp8):
    """Few tiles, each with as many CTAs as its list asks for: one long list,
    short ones, empty ones; and as many tiles as there are shares, or one more."""
    ctxs = [6000 if i == requests // 2 else 5 + (37 * i) % 400 for i in range(requests)]
    n_tokens = [min(n, 33 if i == requests // 2 else 1 + i % 3) for i, n in enumerate(ctxs)]
    if requests > 13:
        n_tokens[3] = 0
    f = Filled(ctxs, fp8=fp8, seed=21, budget=1024)
    try:
        rows = sum(n_tokens)
        q = _queries(rows, 5, f.dev)
        sel, nsel, t, n = _random_selection(f, n_tokens, 1024, seed=8)
        for x in range(0, rows, 4):                  # rows without a block: whole tiles among them
            if f.positions(n_tokens)[x][0] != requests // 2:
                nsel[x] = 0
        n = torch.tensor(nsel, dtype=torch.int32)
        out, lse = _run_attention(f, n_tokens, q, t, n, 1024)
        _check_attention(f, n_tokens, q, sel, nsel, out, lse, sample=70)
        again, lse2 = _run_attention(f, n_tokens, q, t, n, 1024)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
        _clean(f.c)
    finally:
        f.close()


def _check_device_rows(c, h, pos, q, sel, out, lse):
    """Attention of one query against float64, its rows read from the pool."""
    toks = [t for b in sel for t in range(4 * b, min(4 * b + 4, pos + 1))]
    rows = c.pool[c.slot_table[h.index, 0, torch.tensor(toks, device=c.pool.device)].long()].cpu().numpy()
    K, V = O.split_kv(rows)
    o, ls, mag, lmag = _attend(QC.bits16(q), K, V)
    assert np.all(np.abs(out.double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 1e-4) * mag + 1e-30)
    assert np.all(np.abs(lse.double().cpu().numpy() - ls) <= 2.0 ** -17 * lmag + 1e-5)


def _check_device_scores(c, h, pos, q, w, got):
    """Scores of one query against float64 on the device."""
    n = pos + 1
    code = torch.from_numpy(O.decode_e4m3(np.arange(256, dtype=np.uint8))).to(c.pool.device)
    key = code[c.index_keys[h.index, 0, :n].long()] * c.index_scales[h.index, 0, :n].double()[:, None]
    wd = w.double()
    s = (key @ q.double().T).relu() @ wd
    mag = (key.abs() @ q.double().abs().T) @ wd.abs()
    pad = -n % 4
    s = torch.nn.functional.pad(s, (0, pad), value=-np.inf).view(-1, 4).amax(1)
    mag = torch.nn.functional.pad(mag, (0, pad)).view(-1, 4).amax(1)
    assert bool(((got[:len(s)].double() - s).abs() <= QC.SCORE_REL_TOL * mag + 1e-30).all())


def test_a_context_past_a_million_tokens_behind_other_requests():
    """A chunk appended to, scored, selected and attended in a request whose
    keys and rows lie past 2^31 and 2^32 bytes of their buffers."""
    n, k, R = 1100003, 70, 40
    Q.lib()
    c = Q.Cache(n_layers=1, max_requests=R, ctx_capacity=n, hbm_pool_rows=2 * n + R, budget_tokens=2048,
                ring_tokens=64, staging_rows=0)
    try:
        dev = c.pool.device
        c.request_begin(n)
        for _ in range(R - 2):
            c.request_begin(1)
        h = c.request_begin(n - k, max_ctx=n)
        assert h.index == R - 1 and c.slot_table[h.index, 0, n - k - 1].item() * 2048 > 2 ** 32
        assert h.index * n * 64 > 2 ** 31
        g = torch.Generator(device=dev).manual_seed(1)
        c.index_keys[h.index, 0] = torch.randint(0, 127, (n, 64), generator=g, device=dev, dtype=torch.uint8)
        c.index_keys[h.index, 0] |= torch.randint(0, 2, (n, 64), generator=g, device=dev, dtype=torch.uint8) << 7
        c.index_scales[h.index, 0] = torch.rand(n, generator=g, device=dev).half()
        base = c.slot_table[h.index, 0, 0].item()
        for a in range(0, n - k, 1 << 18):
            e = min(n - k, a + (1 << 18))
            c.pool[base + a:base + e] = torch.randn(e - a, 1024, generator=g, device=dev).bfloat16().view(torch.uint8)
        c.advance(h, k)
        kv = torch.randn(k, 1024, generator=g, device=dev).bfloat16().view(torch.uint8)
        c.append_chunk([h], [k], 0, 1, torch.randn(k, 64, generator=g, device=dev), kv)
        qi, w = torch.randn(k, 8, 64, generator=g, device=dev), torch.rand(k, 8, generator=g, device=dev)
        blk = torch.full((k, (n + 3) // 4), NEG, device=dev)
        sel = torch.full((k, 512), -9, dtype=torch.int32, device=dev)
        nsel = torch.zeros(k, dtype=torch.int32, device=dev)
        c.chunk_index_score([h], [k], 0, 1, qi, w, blk)
        c.chunk_select_topk([h], [k], 0, 1, blk, 2048, sel, nsel)
        sel[:, 0] = 0                                   # the first blocks and the last ones too
        sel[:, -1] = (n - k) // 4
        sel[:, -1] = torch.maximum(sel[:, -1], sel[:, -2] + 1)
        pos = torch.arange(n - k, n, device=dev)
        late = sel[:, -1] > pos // 4
        nsel -= late.int()
        q = _queries(k, 7, dev)
        out, lse = torch.zeros_like(q), torch.zeros(k, 16, device=dev)
        c.chunk_sparse_attn([h], [k], 0, 1, q, sel, nsel, 2048, SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(c)
        assert torch.equal(c.pool[base + n - k:base + n], kv)
        for x in (0, 33, k - 1):
            _check_device_scores(c, h, n - k + x, qi[x], w[x], blk[x])
            assert bool((blk[x, (n - k + x) // 4 + 1:] == NEG).all())
            _check_device_rows(c, h, n - k + x, q[x], sel[x, :nsel[x]].tolist(), out[x], lse[x])
    finally:
        c.close()


def test_as_many_rows_as_one_call_takes():
    R, m, budget = 64, 1024, 256
    f = Filled([m] * R, seed=4, budget=budget)
    try:
        c, dev, nt, rows = f.c, f.dev, [m] * R, R * m
        assert rows == 65536
        g = torch.Generator(device=dev).manual_seed(2)
        qi, w = torch.randn(rows, 8, 64, generator=g, device=dev).bfloat16(), torch.rand(rows, 8, generator=g, device=dev)
        blk = torch.full((rows, m // 4), NEG, device=dev)
        sel = torch.full((rows, budget // 4), -9, dtype=torch.int32, device=dev)
        nsel = torch.zeros(rows, dtype=torch.int32, device=dev)
        q = torch.randn(rows, 16, 128, generator=g, device=dev).bfloat16()
        out, lse = torch.zeros_like(q), torch.zeros(rows, 16, device=dev)
        c.chunk_index_score(f.hs, nt, 0, 1, qi, w, blk)
        c.chunk_select_topk(f.hs, nt, 0, 1, blk, budget, sel, nsel)
        c.chunk_sparse_attn(f.hs, nt, 0, 1, q, sel, nsel, budget, SCALE, out, lse)
        torch.cuda.synchronize()
        _clean(c)
        _check_scores(f, nt, qi, w, blk)
        at = torch.tensor([0, 1, 257, 1023, 1024, 40001, 65534, 65535])
        _check_selection(blk[at.to(dev)], [int(i) % m for i in at], budget, sel[at.to(dev)], nsel[at.to(dev)])
        _check_attention(f, nt, q, sel.cpu().numpy(), nsel.cpu().numpy(), out, lse, sample=30)
    finally:
        f.close()

"""Chunk operators where values lie far apart: logits of tokens that a query
does not see, V scales from 2^-24 to 2^15 in one selection, query elements far
below the largest.  Against float64.

Tolerances of the attention, per element and in units of mag = sum p|v|.  The
output is rounded to bf16 (2^-8 of it).  Probabilities go to the tensor cores
as bf16 beside BF16 rows (2^-8 of each term); beside FP8 rows p times the V
scale goes in as f16, off by 2^-11 of itself or by 2^-25 in units in which the
row's largest product is 2^-6 at least, so by 2^-19 of that one; where tokens
with a V scale of 0 outweigh all others, the unit is 2^100 below their weight, to
2^8, so that it is off by 2^-117 of the row's whole weight.  128 products
in fp32 leave a logit off by 2^-17 of scale * sum |q_d k_d|, a probability by
twice that (its own and the sum's), and fp32 sums add less than 1e-4."""
import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from oracle import qsa_oracle as O
from tests import qsa_check as QC
from tests.test_gpu_chunk import SCALE, Filled, _attend, _clean, _queries, _random_selection, _run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _v_scales(f, r, toks):
    rows = f.kv[r][0][torch.as_tensor(toks, dtype=torch.long)].numpy()
    return O.decode_fp16(np.ascontiguousarray(rows[:, 1032:1040]).view(np.uint16))


def _floor(q_bits, K, V, vs):
    """2^-19 of the largest p |scale| of a row, or 2^-117, times the sum of its
    codes."""
    q = O.decode_bf16(q_bits).reshape(16, 128)
    out = np.zeros((16, 128))
    for h in range(16):
        x = SCALE * (K[:, h // 4] @ q[h])
        p = np.exp(x - x.max())
        s = np.abs(vs[:, h // 4])
        codes = np.abs(V[:, h // 4]) / np.where(s > 0, s, 1)[:, None]
        out[h] = max(2.0 ** -19 * (p * s).max() / p.sum(), 2.0 ** -117) * codes.sum(0)
    return out


def _check(f, n_tokens, q, sel, nsel, out, lse, rows=None):
    pos = f.positions(n_tokens)
    for x in range(len(pos)) if rows is None else rows:
        r, p = pos[x]
        toks = [t for b in sel[x][:nsel[x]] for t in range(4 * int(b), min(4 * int(b) + 4, p + 1))]
        K, V = f.values(r, 0, toks)
        bits = QC.bits16(q[x])
        o, ls, mag, lmag = _attend(bits, K, V)
        part = (2.0 ** -11 if f.fp8 else 2.0 ** -8) + 2 * 2.0 ** -17 * lmag[:, None] + 1e-4
        tol = 2.0 ** -8 * np.abs(o) + part * mag
        if f.fp8:
            tol += _floor(bits, K, V, _v_scales(f, r, toks))
        got, gl = out[x].double().cpu().numpy(), lse[x].double().cpu().numpy()
        assert np.all(np.abs(got - o) <= tol), (x, r, p, (np.abs(got - o) / tol).max(), np.abs(got).max(), np.abs(o).max())
        assert np.all(np.abs(gl - ls) <= 2.0 ** -17 * lmag + 1e-5), (x, np.abs(gl - ls).max())


def _store(f, r):
    """The rows that the test has changed go to the pool."""
    rows = f.c.slot_table[f.hs[r].index, 0, :f.ctxs[r]].long()
    f.c.pool[rows] = f.kv[r][0].to(f.dev)


SIGNS = torch.where(torch.randn(128, generator=torch.Generator().manual_seed(4)) < 0, -1.0, 1.0)


def _set_logits(f, r, logits):
    """Keys along one direction: with the query SIGNS token t's logit is
    logits[t], up to the row format's rounding of it."""
    c = torch.as_tensor(logits, dtype=torch.float32) / (128 * SCALE)
    raw = f.kv[r][0]
    if f.fp8:
        codes = torch.where((c[:, None] < 0) != (SIGNS[None] < 0), 0xFE, 0x7E).to(torch.uint8)      # -448, 448
        raw[:, :512] = codes.repeat(1, 4)
        raw[:, 1024:1032] = (c.abs() / 448).half()[:, None].repeat(1, 4).view(torch.uint8)
    else:
        raw[:, :1024] = (c[:, None] * SIGNS).bfloat16().repeat(1, 4).view(torch.uint8)
    _store(f, r)


def _table(sel, budget):
    t = torch.full((len(sel), budget // 4), -7, dtype=torch.int32)
    for x, s in enumerate(sel):
        t[x, :len(s)] = torch.as_tensor(np.asarray(s), dtype=torch.int32)
    return t, torch.tensor([len(s) for s in sel], dtype=torch.int32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("logit", [-20.0, -60.0])
@pytest.mark.parametrize("ctx", [1, 2, 3, 5])
def test_places_past_the_context_leave_low_logits_alone(fp8, logit, ctx):
    """The last block's places without a token count as logit 0 nowhere."""
    f = Filled([ctx], fp8=fp8, budget=64, seed=3)
    try:
        _set_logits(f, 0, [logit] * ctx)
        q = SIGNS.bfloat16().expand(1, 16, 128).contiguous().to(f.dev)
        sel = [np.arange((ctx + 3) // 4)]
        out, lse = _run_attention(f, [1], q, *_table(sel, 64), 64)
        _clean(f.c)
        _check(f, [1], q, sel, [len(sel[0])], out, lse)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("step", [4.0, 12.0, 40.0])
@pytest.mark.parametrize("ctxs,n_tokens,others", [
    ([400], [70], 0), ([400], [70], 31), ([9000], [70], 400), ([300] * 39, [5] * 39, 20)])
def test_later_tokens_of_a_querys_block_do_not_reach_it(fp8, step, ctxs, n_tokens, others):
    """In the chunk, every token's logit is `step` nats above that of the token
    before it in its block; a query sees some of its own block's only.  Lists
    cut into shares and whole ones."""
    f = Filled(ctxs, fp8=fp8, budget=2048, seed=3)
    try:
        rng = np.random.RandomState(8)
        for r, (n, k) in enumerate(zip(ctxs, n_tokens)):
            logits = rng.randn(n)
            at = np.arange(n - k, n)
            logits[at] = step * (at % 4)
            _set_logits(f, r, logits)
        sel = []
        for r, p in f.positions(n_tokens):
            old = rng.choice((ctxs[r] - n_tokens[r]) // 4, others, replace=False)
            sel.append(np.sort(np.append(old, p // 4)))
        q = SIGNS.bfloat16().expand(len(sel), 16, 128).contiguous().to(f.dev)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 2048), 2048)
        _clean(f.c)
        rows = range(len(sel)) if len(sel) <= 70 else range(0, len(sel), 3)
        _check(f, n_tokens, q, sel, [len(s) for s in sel], out, lse, rows)
    finally:
        f.close()


# ------------------------------------------------------------ V scales apart

LAYOUTS = [([600], [40]), ([300] * 39, [3] * 39)]      # lists cut into shares, and whole


def _set_v_scales(f, r, toks, value):
    """V scales (fp16, a head each) of tokens: value [len(toks)] or a number."""
    raw = f.kv[r][0]
    v = torch.as_tensor(value, dtype=torch.float64).expand(len(toks))
    raw[torch.as_tensor(toks), 1032:] = v.half()[:, None].repeat(1, 4).view(torch.uint8)


def _selection_with(f, n_tokens, special, some, rng):
    """Half of the rows select the block `special`, the others do not."""
    sel = []
    for x, (r, p) in enumerate(f.positions(n_tokens)):
        ids = np.delete(np.arange(p // 4 + 1), special)
        ids = rng.choice(ids, some, replace=False)
        sel.append(np.sort(np.append(ids, special) if x % 2 else ids))
    return sel


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("block", [0, 70])
@pytest.mark.parametrize("power", [-24, -16, -9, -4, 4, 9, 16, 20, 24])
def test_v_scales_far_apart(ctxs, n_tokens, block, power):
    """One token's V scale is 2^power of the others', in the first step of the
    lists or in a later one, selected by half of the queries."""
    f = Filled(ctxs, fp8=True, budget=512, seed=3)
    try:
        rng = np.random.RandomState(power + 100)
        for r, n in enumerate(ctxs):
            base = 2.0 ** -(power // 2 + 2)
            v = base * (1 + rng.rand(n))
            v[4 * block + 1] *= 2.0 ** power
            _set_v_scales(f, r, np.arange(n), v)
            _store(f, r)
        sel = _selection_with(f, n_tokens, block, 40, rng)
        q = _queries(len(sel), 5, f.dev)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 512), 512)
        _clean(f.c)
        _check(f, n_tokens, q, sel, [len(s) for s in sel], out, lse)
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("signed", [False, True])
def test_v_scales_of_every_size(ctxs, n_tokens, signed):
    """Scales spread evenly over the whole of fp16's range, in logarithm, zeros
    among them."""
    f = Filled(ctxs, fp8=True, budget=512, seed=3)
    try:
        rng = np.random.RandomState(5)
        for r, n in enumerate(ctxs):
            v = np.exp2(rng.uniform(-24, 15.9, n)) * (rng.choice([-1, 1], n) if signed else 1)
            v[rng.rand(n) < 0.1] = 0
            _set_v_scales(f, r, np.arange(n), v)
            _store(f, r)
        sel = _selection_with(f, n_tokens, 3, 40, rng)
        q = _queries(len(sel), 5, f.dev, scale=3.0)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 512), 512)
        _clean(f.c)
        _check(f, n_tokens, q, sel, [len(s) for s in sel], out, lse)
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("logit", [0.0, 30.0, 55.0, 90.0])
def test_small_values_behind_tokens_without_any(ctxs, n_tokens, logit):
    """The first 40 blocks' V rows are zero, with scale 0, their logits
    `logit` nats above the others'; the rest have scales of 2^-20."""
    f = Filled(ctxs, fp8=True, budget=512, seed=3)
    try:
        rng = np.random.RandomState(5)
        for r, n in enumerate(ctxs):
            _set_logits(f, r, np.where(np.arange(n) < 160, logit, 0.0) + rng.randn(n))
            _set_v_scales(f, r, np.arange(n), np.where(np.arange(n) < 160, 0.0, 2.0 ** -20 * (1 + rng.rand(n))))
            f.kv[r][0][:160, 512:1024] = 0
            _store(f, r)
        sel = _selection_with(f, n_tokens, 0, 40, rng)
        q = SIGNS.bfloat16().expand(len(sel), 16, 128).contiguous().to(f.dev)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 512), 512)
        _clean(f.c)
        _check(f, n_tokens, q, sel, [len(s) for s in sel], out, lse)
        # rows over such tokens alone: zeros
        sel = [np.arange(20)] * len(sel)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 512), 512)
        _check(f, n_tokens, q, sel, [20] * len(sel), out, lse)
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens", LAYOUTS)
@pytest.mark.parametrize("value,scale", [(float("inf"), 2.0 ** -19), (float("nan"), 2.0 ** -19), (1e4, 1.0), (3e4, 2.0 ** -10)])
def test_an_outlier_that_is_not_selected_costs_no_bits(ctxs, n_tokens, value, scale):
    """Scales of `scale` to twice that beside a token of the first step whose V
    scale is infinite, NaN or large: the queries that do not select it keep
    theirs."""
    f = Filled(ctxs, fp8=True, budget=512, seed=3)
    try:
        rng = np.random.RandomState(5)
        for r, n in enumerate(ctxs):
            v = scale * (1 + rng.rand(n))
            v[5] = value
            _set_v_scales(f, r, np.arange(n), v)
            _store(f, r)
        sel = _selection_with(f, n_tokens, 1, 40, rng)
        q = _queries(len(sel), 5, f.dev)
        out, lse = _run_attention(f, n_tokens, q, *_table(sel, 512), 512)
        _clean(f.c)
        finite = bool(np.isfinite(value))
        _check(f, n_tokens, q, sel, [len(s) for s in sel], out, lse, range(0, len(sel), 1 if finite else 2))
        if not finite:
            assert not bool(out[1::2].isfinite().all(-1).any())
    finally:
        f.close()


@pytest.mark.parametrize("ctxs,n_tokens,budget", [([2100], [129], 2048), ([9000, 700, 33], [4, 33, 32], 2048), ([5000], [257], 512)])
def test_fp8_rows_lose_f16_roundings_only(ctxs, n_tokens, budget):
    f = Filled(ctxs, fp8=True, seed=21, budget=8192)
    try:
        sel, nsel, t, n = _random_selection(f, n_tokens, budget, 31)
        q = _queries(len(sel), 41, f.dev, scale=2.0)
        out, lse = _run_attention(f, n_tokens, q, t, n, budget)
        _clean(f.c)
        _check(f, n_tokens, q, sel, nsel, out, lse, range(0, len(sel), 5))
    finally:
        f.close()


# ----------------------------------------- query elements below the largest

def _keys_without_the_first_dimension(f, r, rng):
    n = f.ctxs[r]
    codes = rng.randint(0, 127, (n, 64)).astype(np.uint8) | (rng.randint(0, 2, (n, 64)) << 7).astype(np.uint8)
    codes[:, 0] = 0
    f.codes[r] = codes[None]
    f.c.index_keys[f.hs[r].index, 0, :n] = torch.from_numpy(codes).to(f.dev)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("ctxs,n_tokens", [([700], [3]), ([1300, 70], [70, 5])])
@pytest.mark.parametrize("top", [1.0, 0.5, 1.99, 1e30, 1e-30])
def test_index_query_elements_far_below_the_largest(bf16, ctxs, n_tokens, top):
    """Every head's largest element meets zero codes, so the scores are the
    others', 2^-1 to 2^-30 of it.  An fp32 element goes in within 2^-23 of
    itself, or 2^-39 of the largest, a bf16 element exactly down to 2^-31 of the
    largest (and within 2^-39 of it); 64 products and 8 heads in fp32 add (64 +
    8 + 4) 2^-24 of the sum of magnitudes."""
    f = Filled(ctxs, budget=64, seed=2)
    try:
        rng = np.random.RandomState(4)
        for r in range(len(ctxs)):
            _keys_without_the_first_dimension(f, r, rng)
        rows = sum(n_tokens)
        q = rng.randn(rows, 8, 64) * np.exp2(-rng.randint(1, 31, (rows, 8, 1)).astype(np.float64))
        q[0, :, 1:] = np.exp2(-18) * (1 + 2.0 ** -7)
        q[1, :, 1:] = 2.0 ** -13 + 2.0 ** -24
        q[..., 0] = 1
        q = torch.from_numpy(q * top).float()
        q = q.bfloat16() if bf16 else q
        w = torch.rand(rows, 8, generator=torch.Generator().manual_seed(1))
        stride = (max(ctxs) + 3) // 4
        blk = torch.zeros(rows, stride, device=f.dev)
        f.c.chunk_index_score(f.hs, n_tokens, 0, 1, q.to(f.dev), w.to(f.dev), blk)
        torch.cuda.synchronize()
        _clean(f.c)
        got = blk.double().cpu().numpy()
        for x, (r, pos) in enumerate(f.positions(n_tokens)):
            if x % 7 > 2:
                continue
            codes, sc = f.codes[r][0, :pos + 1], f.scales[r][0, :pos + 1]
            qd, wd = q[x].double().numpy(), w[x].double().numpy()
            ref = O.c4_block_scores(O.token_scores(codes, sc, qd, wd))
            key = np.abs(O.decode_e4m3(codes)) * np.abs(O.decode_fp16(sc))[:, None]
            off = 76 * 2.0 ** -24 * np.abs(qd) + 2.0 ** -39 * np.abs(qd).max(1)[:, None]
            if not bf16:
                off += 2.0 ** -23 * np.abs(qd)
            tol = O.c4_block_scores((key @ off.T) @ wd)
            assert np.all(np.abs(got[x, :len(ref)] - ref) <= tol), (x, (np.abs(got[x, :len(ref)] - ref) / tol).max())
    finally:
        f.close()


def test_query_elements_far_below_the_largest_beside_fp8_rows():
    """The largest element of every query meets K codes of 0; the others, 2^-20
    of it, meet keys 2^20 times as large."""
    f = Filled([900], fp8=True, budget=512, seed=3)
    try:
        rng = np.random.RandomState(4)
        raw = f.kv[0][0]
        raw[:, 0:512:128] = 0
        ks = raw[:, 1024:1032].clone().view(torch.float16).float() * 2.0 ** 20
        raw[:, 1024:1032] = ks.half().view(torch.uint8)
        assert bool(ks.isfinite().all()) and ks.max() < 65504
        _store(f, 0)
        q = _queries(40, 5, "cpu").float() * 2.0 ** -20
        q[..., 0] = 1
        q = q.bfloat16().to(f.dev)
        sel = [np.sort(rng.choice(860 // 4, 100, replace=False)) for _ in range(40)]
        out, lse = _run_attention(f, [40], q, *_table(sel, 512), 512)
        _clean(f.c)
        _check(f, [40], q, sel, [100] * 40, out, lse)
    finally:
        f.close()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("tokens", [3, 70])
@pytest.mark.parametrize("size", [1e34, 1e35, 1e-34])
def test_index_queries_near_the_ends_of_fp32(bf16, tokens, size):
    """Scores that fp32 holds: up to about 1e37, or down to 1e-34."""
    f = Filled([700], budget=64, seed=2)
    try:
        q = size * torch.randn(tokens, 8, 64, generator=torch.Generator().manual_seed(3))
        q = q.bfloat16() if bf16 else q
        w = torch.rand(tokens, 8, generator=torch.Generator().manual_seed(1)) + 0.5
        blk = torch.zeros(tokens, 175, device=f.dev)
        f.c.chunk_index_score(f.hs, [tokens], 0, 1, q.to(f.dev), w.to(f.dev), blk)
        torch.cuda.synchronize()
        _clean(f.c)
        got = blk.double().cpu().numpy()
        for x, (r, pos) in enumerate(f.positions([tokens])):
            codes, sc = f.codes[0][0, :pos + 1], f.scales[0][0, :pos + 1]
            qd, wd = q[x].double().numpy(), w[x].double().numpy()
            ref = O.c4_block_scores(O.token_scores(codes, sc, qd, wd))
            assert np.abs(ref).max() < 1e38
            key = np.abs(O.decode_e4m3(codes)) * np.abs(O.decode_fp16(sc))[:, None]
            mag = O.c4_block_scores((key @ np.abs(qd).T) @ wd)
            assert np.all(np.abs(got[x, :len(ref)] - ref) <= QC.SCORE_REL_TOL * mag), x
    finally:
        f.close()

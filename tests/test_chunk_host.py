"""Host-side behaviour of the operators on a cache's pages (truncate, fork,
compact) and of the chunk entry points, on host-only caches: bookkeeping
against a small model, and refusals.  No GPU needed."""
import ctypes as C
import random

import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from sparse_attention_decode_qsa_gb300 import _native as N


def _cache(**kw):
    args = dict(n_layers=3, max_requests=6, ctx_capacity=4096, hbm_pool_rows=60000, budget_tokens=64,
                ring_tokens=16, staging_rows=10, device=None)
    args.update(kw)
    return Q.Cache(**args)


def _refused(status, f, *a, **kw):
    with pytest.raises(Q.QsaError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value


def test_truncate_takes_back_tokens_and_lets_them_be_advanced_over_again():
    c = _cache()
    h = c.request_begin(100, max_ctx=120)
    c.advance(h, 20)
    c.truncate(h, 103)
    assert c.request_info(h).ctx_len == 103 and c.request_info(h).max_ctx == 120
    c.advance(h, 17)
    assert c.request_info(h).ctx_len == 120
    c.truncate(h, 120)
    for bad in (0, -1, 121):
        _refused(Q.ERR_INVALID_ARG, c.truncate, h, bad)
    c.truncate(h, 1)
    assert c.request_info(h).ctx_len == 1
    c.request_end(h)
    _refused(Q.ERR_STALE_HANDLE, c.truncate, h, 1)
    assert N.lib().qsa_request_truncate(None, h, 1) == Q.ERR_INVALID_ARG


def test_fork_leases_like_begin_and_refuses_what_the_parent_does_not_hold():
    c = _cache()
    s0 = c.stats()
    a = c.request_begin(100, max_ctx=150)
    s1 = c.stats()
    b = c.request_fork(a, 40, max_ctx=60)
    info = c.request_info(b)
    assert (info.ctx_len, info.max_ctx, info.placement, info.layer_rows) == (40, 60, Q.KV_HBM, 60)
    assert info.hbm_row_base == 30 + 3 * 150
    r = c.request_fork(a, 100, Q.KV_HOST_RING, host_rows=1 << 30)
    assert c.request_info(r).layer_rows == 16 and c.request_info(r).host_rows == 1 << 30
    n0 = c.stats()
    for kw, status in [(dict(ctx_len=101), Q.ERR_INVALID_ARG), (dict(ctx_len=0), Q.ERR_INVALID_ARG),
                       (dict(ctx_len=40, max_ctx=39), Q.ERR_INVALID_ARG),
                       (dict(ctx_len=40, placement=Q.KV_HOST), Q.ERR_INVALID_ARG),
                       (dict(ctx_len=40, max_ctx=4097), Q.ERR_CAPACITY)]:
        _refused(status, c.request_fork, a, **kw)
        assert c.stats() == n0
    # a child's host history may not overlap its parent's
    size = 3 * 100 * 2048
    for at in ((1 << 30), (1 << 30) + size - 16, (1 << 30) - size + 16):
        _refused(Q.ERR_INVALID_ARG, c.request_fork, r, 100, Q.KV_HOST, host_rows=at)
        assert c.stats() == n0
    c.request_end(c.request_fork(r, 100, Q.KV_HOST, host_rows=(1 << 30) + size))
    for h in (b, r):
        c.request_end(h)
    assert c.stats() == s1
    c.request_end(a)
    assert c.stats() == s0
    _refused(Q.ERR_STALE_HANDLE, c.request_fork, a, 1)


def test_compaction_bookkeeping_matches_a_model():
    rng = random.Random(7)
    for hot in (0, 64):
        c = _cache(hot_rows=hot)
        live = {}
        for step in range(300):
            x = rng.random()
            if x < 0.55 and len(live) < 6:
                place = rng.choice([Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST])
                n = rng.randint(1, 3000)
                try:
                    h = c.request_begin(n, place, host_rows=None if place == Q.KV_HBM else 1 << 20)
                except Q.QsaError as e:
                    assert e.status == Q.ERR_CAPACITY
                    continue
                rows = {Q.KV_HBM: 3 * n, Q.KV_HOST_RING: 3 * 16, Q.KV_HOST: 0}[place]
                rows += 3 * hot if place != Q.KV_HBM else 0
                live[h.index] = (h, rows)
            elif x < 0.9 and live:
                c.request_end(live.pop(rng.choice(sorted(live)))[0])
            else:
                held = sorted(((c.request_info(h).hbm_row_base, h, rows) for h, rows in live.values() if rows),
                              key=lambda v: v[0])
                want, at, moved = [], 30, 0
                for base, h, rows in held:
                    want.append((h, base, at, rows))
                    moved += rows if base != at else 0
                    at += rows
                hot0 = {h.index: c.request_info(h).hot_row_base for h, *_ in want}
                assert c.compact() == moved
                for h, base, to, rows in want:
                    info = c.request_info(h)
                    assert info.hbm_row_base == to
                    if hot0[h.index] >= 0:
                        assert info.hot_row_base == hot0[h.index] - (base - to)
                s = c.stats()
                assert s["free_hbm_rows"] == s["largest_free_rows"] == 60000 - at
                assert s["free_ranges"] == (1 if at < 60000 else 0)
                assert c.compact() == 0
        for h, _ in live.values():
            c.request_end(h)
        s = c.stats()
        assert s["free_hbm_rows"] == s["largest_free_rows"] == 60000 - 30
    assert N.lib().qsa_cache_compact(None, None, None) == Q.ERR_INVALID_ARG


def test_chunk_calls_on_a_cache_without_device_storage():
    c = _cache()
    h = c.request_begin(100)
    f32 = lambda *s: torch.zeros(*s)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    bf = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    _refused(Q.ERR_NO_DEVICE, c.append_chunk, [h], [2], 0, 1, f32(2, 64), torch.zeros(2, 2048, dtype=torch.uint8))
    _refused(Q.ERR_NO_DEVICE, c.chunk_index_score, [h], [2], 0, 1, f32(2, 8, 64), f32(2, 8), f32(2, 25))
    _refused(Q.ERR_NO_DEVICE, c.chunk_select_topk, [h], [2], 0, 1, f32(2, 25), 64, i32(2, 16), i32(2))
    _refused(Q.ERR_NO_DEVICE, c.chunk_sparse_attn, [h], [2], 0, 1, bf, i32(2, 16), i32(2), 64, 1.0, bf,
             workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(Q.QsaError):
        c.chunk_attn_workspace_bytes([h], [2], 0, 1, 64)
    ch = N.Chunk()
    for name, args in [("qsa_append_chunk", (None, None, None)),
                       ("qsa_chunk_index_score", (None, 0, None, None, 0, None)),
                       ("qsa_chunk_select_topk", (None, 0, 64, None, None, None)),
                       ("qsa_chunk_sparse_attn", (None, None, None, 64, 1.0, None, None, None, 0, None))]:
        assert getattr(N.lib(), name)(None, C.byref(ch), *args) == Q.ERR_INVALID_ARG, name


def test_binding_refuses_tensors_of_another_type_or_shape():
    c = _cache()
    h = c.request_begin(100)
    k, kv = torch.zeros(3, 64), torch.zeros(3, 2048, dtype=torch.uint8)
    for bad in [(k.double(), kv), (k[:2], kv), (k, kv[:, :1024]), (torch.zeros(64, 3).T, kv)]:
        with pytest.raises(ValueError):
            c.append_chunk([h], [3], 0, 1, *bad)
    with pytest.raises(ValueError):
        c.append_chunk([h], [3, 1], 0, 1, k, kv)
    with pytest.raises(ValueError):
        c.chunk_index_score([h], [3], 0, 1, torch.zeros(3, 8, 64, dtype=torch.float16), torch.zeros(3, 8),
                            torch.zeros(3, 25))

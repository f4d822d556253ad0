"""The stream that a lease, a fork and a compaction of the Python binding run
on: the one given, else the current one of the cache's device, however that
device was named.  No GPU needed: the library is replaced by a recorder."""
from types import SimpleNamespace

import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from sparse_attention_decode_qsa_gb300 import _native as N
from sparse_attention_decode_qsa_gb300 import api


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.mark.parametrize("device", [0, 1, "cuda", "cuda:0", torch.device("cuda", 0)])
def test_pages_calls_run_on_the_current_stream_of_the_caches_device(device, monkeypatch):
    index = 1 if device == 1 else 0
    c = Q.Cache(n_layers=1, max_requests=2, ctx_capacity=64, hbm_pool_rows=256, budget_tokens=64, ring_tokens=16,
                staging_rows=0, device=None)
    lib, rec = c.L, _Recorder()
    monkeypatch.setattr(api, "_raw_stream", lambda i: 4096 * (i + 1))
    c.device, c.pool, c.L = device, SimpleNamespace(device=SimpleNamespace(index=index)), rec
    try:
        for given, want in ((None, 4096 * (index + 1)), (77, 77)):
            rec.calls.clear()
            c.request_begin(4, stream=given)
            c.request_fork(N.Handle(0, 1), 4, stream=given)
            c.compact(stream=given)
            at = {"qsa_request_begin": 2, "qsa_request_fork": 3, "qsa_cache_compact": 1}
            assert [name for name, _ in rec.calls] == list(at)
            assert [args[at[name]] for name, args in rec.calls] == [want] * 3
    finally:
        c.device, c.L = None, lib


def test_a_cache_without_device_storage_takes_no_stream():
    c = Q.Cache(n_layers=1, max_requests=2, ctx_capacity=64, hbm_pool_rows=256, budget_tokens=64, ring_tokens=16,
                staging_rows=0, device=None)
    h = c.request_begin(4)
    c.request_end(c.request_fork(h, 3))
    c.compact()

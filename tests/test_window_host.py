"""Window and shared-prefix attention, attention weights and eviction on host-only
caches: they need device storage and say so, and the binding checks its arrays
before the library sees them.  No GPU needed."""
import ctypes as C

import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from sparse_attention_decode_qsa_gb300 import _native as N
from tests.test_chunk_host import _cache, _refused


def _heads(rows, dtype=torch.bfloat16):
    return torch.zeros(rows, 16, 128, dtype=dtype)


def test_calls_need_device_storage():
    c = _cache()
    h, p = c.request_begin(100), c.request_begin(50)
    q, out, lse = _heads(3), _heads(3), torch.zeros(3, 16)
    ws = torch.zeros(256, dtype=torch.uint8)
    NO = Q.ERR_NO_DEVICE
    _refused(NO, c.window_attn, [h], [3], 0, 1, q, 4, 16, 0.1, out, lse, workspace=ws)
    _refused(NO, c.shared_attn, [h], [3], 0, 1, p, 50, 0, q, 0.1, out, lse, workspace=ws)
    _refused(NO, c.window_weights, [h], [3], 0, 1, q, lse, 4, 16, 0.1, torch.zeros(1, 100))
    _refused(NO, c.evict, h, torch.zeros(3, 100), 50, workspace=ws)
    with pytest.raises(Q.QsaError):
        c.window_attn_workspace_bytes([h], [3], 0, 1, 4, 16)
    with pytest.raises(Q.QsaError):
        c.shared_attn_workspace_bytes([h], [3], 0, 1, p, 50, 0)
    with pytest.raises(Q.QsaError):
        c.evict_workspace_bytes(h, 50)
    assert c.request_info(h).ctx_len == 100


def test_null_arguments():
    L = N.lib()
    h = N.Handle(0, 1)
    assert L.qsa_window_attn(None, None, None, 0, 1, 0.1, None, None, None, 0, None) == Q.ERR_INVALID_ARG
    assert L.qsa_shared_attn(None, None, h, 0, 0, None, 0.1, None, None, None, 0, None) == Q.ERR_INVALID_ARG
    assert L.qsa_window_weights(None, None, None, None, 0, 1, 0.1, None, 0, 0, None) == Q.ERR_INVALID_ARG
    assert L.qsa_request_evict(None, h, None, 0, 1, 0, 0, None, None, 0, None, 0, None) == Q.ERR_INVALID_ARG
    assert L.qsa_window_attn_workspace_bytes(None, None, 0, 1) == -1
    assert L.qsa_shared_attn_workspace_bytes(None, None, h, 0, 0) == -1
    assert L.qsa_evict_workspace_bytes(None, h, 1) == -1
    c = _cache()
    assert L.qsa_window_attn(c.h, None, None, 0, 1, C.c_float(0.1), None, None, None, 0, None) == Q.ERR_INVALID_ARG


def test_the_binding_checks_types_shapes_and_layouts():
    c = _cache()
    h, p = c.request_begin(100), c.request_begin(50)
    lse, ws = torch.zeros(3, 16), torch.zeros(256, dtype=torch.uint8)
    good = dict(q=_heads(3), out=_heads(3), lse=lse)
    for bad in (dict(q=_heads(3, torch.float16)), dict(q=_heads(2)), dict(out=_heads(3, torch.float32)),
                dict(lse=lse[:, :15]), dict(lse=lse.double()), dict(q=_heads(6)[::2])):
        a = dict(good, **bad)
        with pytest.raises(ValueError):
            c.window_attn([h], [3], 0, 1, a["q"], 4, 16, 0.1, a["out"], a["lse"], workspace=ws)
        with pytest.raises(ValueError):
            c.shared_attn([h], [3], 0, 1, p, 50, 0, a["q"], 0.1, a["out"], a["lse"], workspace=ws)
    with pytest.raises(ValueError):
        c.window_weights([h], [3], 0, 1, good["q"], lse, 4, 16, 0.1, torch.zeros(2, 100))
    with pytest.raises(ValueError):
        c.window_attn([h], [3, 1], 0, 1, good["q"], 4, 16, 0.1, good["out"])
    for w in (torch.zeros(3, 99), torch.zeros(2, 100), torch.zeros(3, 100).double(), torch.zeros(100, 3).t()):
        with pytest.raises(ValueError):
            c.evict(h, w, 50, workspace=ws)


class _Recorder:
    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls[name] = args
            return 0
        return call


def test_numbers_past_32_bits_keep_their_meaning():
    """A window or a number of sinks past 2^31 is all tokens; a length of a prefix
    that does not fit is refused, not cut."""
    c = _cache()
    h, p = c.request_begin(100), c.request_begin(50)
    q, out, lse = _heads(3), _heads(3), torch.zeros(3, 16)
    ws, w = torch.zeros(256, dtype=torch.uint8), torch.zeros(1, 100)
    lib, c.L = c.L, _Recorder()
    most = (1 << 31) - 1
    try:
        for given, want in ((1 << 32, most), (1 << 31, most), ((1 << 40) + 5, most), (most, most), (7, 7), (0, 0)):
            c.window_attn([h], [3], 0, 1, q, given, given, 0.1, out, lse, workspace=ws)
            c.window_attn_workspace_bytes([h], [3], 0, 1, given, given)
            c.window_weights([h], [3], 0, 1, q, lse, given, given, 0.1, w)
            assert c.L.calls["qsa_window_attn"][3:5] == (want, want)
            assert c.L.calls["qsa_window_attn_workspace_bytes"][2:4] == (want, want)
            assert c.L.calls["qsa_window_weights"][4:6] == (want, want)
        for given in (-1, -(1 << 32)):
            c.window_attn([h], [3], 0, 1, q, given, given, 0.1, out, lse, workspace=ws)
            assert all(x < 0 for x in c.L.calls["qsa_window_attn"][3:5])
        c.L.calls.clear()
        for big in ((1 << 32) + 5, 1 << 31, -(1 << 32)):
            for a in ((big, 0), (5, big)):
                with pytest.raises(ValueError):
                    c.shared_attn([h], [3], 0, 1, p, *a, q, 0.1, out, lse, workspace=ws)
                with pytest.raises(ValueError):
                    c.shared_attn_workspace_bytes([h], [3], 0, 1, p, *a)
        assert not c.L.calls
        c.shared_attn([h], [3], 0, 1, p, 50, 7, q, 0.1, out, lse, workspace=ws)
        assert c.L.calls["qsa_shared_attn"][3:5] == (50, 7)
    finally:
        c.L = lib

"""Eviction by attention weight on the GPU against a plain model: which tokens
stay, where their rows, keys, scales and slots go (all equal to the bit), and
what the request is good for afterwards."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q
from tests.test_gpu_chunk import SCALE, Filled, _clean, _queries
from tests.test_gpu_window import FULL, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def _kept(w, keep, first, last):
    """Positions that stay: NaN below everything, ties to the lower position."""
    n = len(w)
    order = sorted(range(first, n - last), key=lambda t: (np.isnan(w[t]), -w[t] if not np.isnan(w[t]) else 0.0, t))
    return sorted(list(range(first)) + order[:keep - first - last] + list(range(n - last, n)))


class Model:
    """One layer of a request: slots, and the bytes of every token."""

    def __init__(self, c, h, layer):
        info = c.request_info(h)
        n = info.ctx_len
        self.c, self.h, self.layer = c, h, layer
        self.base = info.hbm_row_base + layer * info.layer_rows
        self.rows_per_layer = info.layer_rows
        self.slots = c.slot_table[h.index, layer, :n].tolist()
        self.keys = c.index_keys[h.index, layer, :n].cpu()
        self.scales = c.index_scales[h.index, layer, :n].view(torch.int16).cpu()
        self.rows = c.pool[torch.tensor(self.slots, device=c.pool.device)].cpu()

    def evict(self, kept):
        keep = len(kept)
        slots = [self.slots[t] for t in kept]
        used = {s - self.base for s in slots}
        free = [r for r in range(keep) if r not in used]
        for i, s in enumerate(slots):
            if keep <= s - self.base < self.rows_per_layer:
                slots[i] = self.base + free.pop(0)
        self.slots, idx = slots, torch.tensor(kept)
        self.keys, self.scales, self.rows = self.keys[idx], self.scales[idx], self.rows[idx]

    def check(self):
        n = len(self.slots)
        c, h, l = self.c, self.h, self.layer
        assert c.slot_table[h.index, l, :n].tolist() == self.slots
        assert torch.equal(c.index_keys[h.index, l, :n].cpu(), self.keys)
        assert torch.equal(c.index_scales[h.index, l, :n].view(torch.int16).cpu(), self.scales)
        assert torch.equal(c.pool[torch.tensor(self.slots, device=c.pool.device)].cpu(), self.rows)


def _make_weights(kind, layers, n, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "heavy":
        return (2 * torch.randn(layers, n, generator=g)).exp()
    if kind == "ties":
        return torch.randint(0, 4, (layers, n), generator=g).float()
    if kind == "same":
        return torch.zeros(layers, n)
    if kind == "rising":
        return torch.arange(n).float().expand(layers, n).contiguous()
    if kind == "falling":
        return -torch.arange(n).float().expand(layers, n).contiguous()
    if kind == "close":              # differ in the last bits alone
        return (torch.full((layers, n), 1.0).view(torch.int32) + torch.randint(0, 3000, (layers, n), generator=g,
                                                                              dtype=torch.int32)).view(torch.float32)
    w = torch.randn(layers, n, generator=g)
    special = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38])
    pick = torch.randint(0, 2 * len(special), (layers, n), generator=g)
    return torch.where(pick < len(special), special[pick.clamp(max=len(special) - 1)], w)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["heavy", "ties", "same", "rising", "falling", "close", "special"])
@pytest.mark.parametrize("n,keep,first,last", [
    (1, 1, 0, 0), (2, 1, 0, 0), (2, 1, 1, 0), (2, 1, 0, 1), (33, 32, 4, 8), (100, 100, 0, 0), (700, 350, 4, 64),
    (1025, 513, 0, 0), (1500, 7, 3, 4), (1500, 1499, 0, 0), (2000, 900, 900, 0), (2000, 900, 0, 900), (5000, 1234, 1, 1)])
def test_eviction_matches_the_model(fp8, kind, n, keep, first, last):
    f = Filled([n, 20], layers=3, fp8=fp8, seed=n)
    try:
        c, h = f.c, f.hs[0]
        w = _make_weights(kind, 3, n, seed=keep)
        models = [Model(c, h, l) for l in range(3)]
        other = [Model(c, f.hs[1], l) for l in range(3)]
        past = c.index_keys[h.index, :, keep:].clone()
        kept = torch.full((3, keep), -1, dtype=torch.int32, device=f.dev)
        wo = torch.zeros(3, keep + 3, device=f.dev)
        ws = c.evict_workspace_bytes(h, keep)
        guard = torch.full((ws + 4096,), 77, dtype=torch.uint8, device=f.dev)
        c.evict(h, w.to(f.dev), keep, first, last, kept, wo, workspace=guard[:ws])
        torch.cuda.synchronize()
        _clean(c)
        assert c.request_info(h).ctx_len == keep and bool((guard[ws:] == 77).all())
        for l in range(3):
            want = _kept(w[l].numpy(), keep, first, last)
            assert kept[l].tolist() == want
            assert torch.equal(wo[l, :keep].view(torch.int32).cpu(), w[l, want].view(torch.int32))
            models[l].evict(want)
            models[l].check()
            other[l].check()
        assert bool((wo[:, keep:] == 0).all()) and torch.equal(c.index_keys[h.index, :, keep:], past)
    finally:
        f.close()


def test_evictions_between_new_tokens_and_the_attention_over_what_is_left():
    """Rounds of: new tokens, attention, its weights, eviction back to `keep`;
    the attention always sees the tokens that the model holds."""
    keep, grow = 300, 60
    f = Filled([keep], layers=2, seed=5, grow=grow)
    try:
        c, h, dev = f.c, f.hs[0], f.dev
        g = torch.Generator().manual_seed(4)
        for _ in range(4):
            c.advance(h, grow)
            k = torch.randn(2 * grow, 64, generator=g).to(dev)
            kv = torch.randn(2 * grow, 1024, generator=g).bfloat16().view(torch.uint8).to(dev)
            c.append_chunk([h], [grow], 0, 2, k, kv)
            models = [Model(c, h, l) for l in range(2)]
            assert [m.slots[keep:] for m in models] == [[m.base + t for t in range(keep, keep + grow)] for m in models]
            q = _queries(2 * grow, 6, dev)
            out, lse = torch.zeros_like(q), torch.zeros(2 * grow, 16, device=dev)
            c.window_attn([h], [grow], 0, 2, q, 0, FULL, SCALE, out, lse)

            def values(k):
                x = models[k[0]].rows[:k[2] + 1].view(torch.bfloat16).double().view(-1, 2, 4, 128).numpy()
                return x[:, 0], x[:, 1]
            _check([(l, 0, keep + i) for l in range(2) for i in range(grow)], q, out, lse, values)
            w = torch.zeros(2, keep + grow, device=dev)
            c.window_weights([h], [grow], 0, 2, q, lse, 0, FULL, SCALE, w)
            c.evict(h, w, keep, 4, 32)
            for l, m in enumerate(models):
                m.evict(_kept(w[l].cpu().numpy(), keep, 4, 32))
                m.check()
        _clean(c)
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_an_evicted_request_forks_compacts_and_selects(fp8):
    f = Filled([50, 900], layers=2, fp8=fp8, seed=6, spare=2 * 1000, cap=900)
    try:
        c, h, dev = f.c, f.hs[1], f.dev
        w = _make_weights("heavy", 2, 900, 3)
        models = [Model(c, h, l) for l in range(2)]
        c.evict(h, w.to(dev), 401, 4, 16)
        for l, m in enumerate(models):
            m.evict(_kept(w[l].numpy(), 401, 4, 16))
        child = c.request_fork(h, 333)
        for l, m in enumerate(models):
            mc = Model(c, child, l)
            assert torch.equal(mc.rows, m.rows[:333]) and torch.equal(mc.keys, m.keys[:333])
        moved = c.request_info(h).hbm_row_base
        c.request_end(f.hs[0])
        assert c.compact() > 0
        down = moved - c.request_info(h).hbm_row_base
        assert down > 0
        for m in models:
            m.slots = [s - down for s in m.slots]
            m.base -= down
            m.check()
        # a decode step over the kept tokens, all of them within the budget
        q = _queries(1, 3, dev)
        blk, sel = torch.zeros(1, 101, device=dev), torch.zeros(1, 512, dtype=torch.int32, device=dev)
        nsel = torch.zeros(1, dtype=torch.int32, device=dev)
        c.index_score([h], 0, 1, torch.randn(1, 8, 64, device=dev), torch.rand(1, 8, device=dev), blk)
        c.select_c4_topk([h], 0, 1, blk, 2048, sel, nsel)
        out, lse = torch.zeros(1, 16, 128, device=dev), torch.zeros(1, 16, device=dev)
        c.sparse_decode_attn([h], 0, 1, q, sel, nsel, 2048, None, SCALE, out, lse)
        o2, l2 = torch.zeros_like(q), torch.zeros_like(lse)
        c.window_attn([h], [1], 0, 1, q, 0, FULL, SCALE, o2, l2)
        # the same logits in two orders of summation; the outputs differ by the
        # bf16 roundings of window attention (2^-8 of out and of sum p|v| < 6)
        assert nsel.item() == 101 and (lse - l2).abs().max() <= 4e-5
        assert (out - o2.float()).abs().max() <= 2 ** -8 * out.abs().max() + 2 ** -8 * 6
        _clean(c)
    finally:
        f.close()


def test_rows_outside_the_region_stay_and_bad_slots_are_reported():
    f = Filled([600], layers=1, seed=7, spare=40)
    try:
        c, h, dev = f.c, f.hs[0], f.dev
        # tokens 10 and 590 read rows of their own behind the region, 580 shares token 5's
        spare = c.pool.shape[0] - 20
        toks = torch.tensor([10, 590, 580], device=dev)
        base = c.request_info(h).hbm_row_base
        c.pool[spare:spare + 2] = 9
        c.slot_table_set(h, 0, toks, torch.tensor([spare, spare + 1, base + 5], dtype=torch.int32, device=dev))
        m = Model(c, h, 0)
        w = _make_weights("heavy", 1, 600, 3)
        w[0, [10, 590, 580, 5]] = 1e6
        c.evict(h, w.to(dev), 250)
        _clean(c)
        want = _kept(w[0].numpy(), 250, 0, 0)
        m.evict(want)
        m.check()
        assert c.slot_table[h.index, 0, want.index(590)].item() == spare + 1
        c.slot_table[h.index, 0, 7] = -1
        c.slot_table[h.index, 0, 9] = c.pool.shape[0]
        w2 = torch.zeros(1, 250, device=dev)
        c.evict(h, w2, 100, 20)
        assert c.poll_error()[0] == Q.ERR_BAD_SLOT
        assert c.slot_table[h.index, 0, [7, 9]].tolist() == [-1, c.pool.shape[0]]
    finally:
        f.close()


def test_weights_of_one_request_of_a_batch_and_other_streams():
    """Layers of the weights and of the kept weights lie apart; the call runs on a
    stream given or on the current one."""
    f = Filled([400, 380], layers=2, seed=8)
    try:
        c, dev = f.c, f.dev
        w = _make_weights("heavy", 4, 400, 3).to(dev)          # units: layer 0 of both, layer 1 of both
        out = torch.zeros(2, 2, 200, device=dev)
        models = [[Model(c, h, l) for l in range(2)] for h in f.hs]
        torch.cuda.synchronize()
        s = [torch.cuda.Stream() for _ in range(3)]
        with torch.cuda.stream(s[0]):
            c.evict(f.hs[0], w.view(2, 2, 400)[:, 0], 200, 1, 2, weights_out=out[:, 0])
        c.evict(f.hs[1], w.view(2, 2, 400)[:, 1], 199, 1, 2, weights_out=out[:, 1], stream=s[1])
        torch.cuda.synchronize()
        for i, keep in enumerate((200, 199)):
            for l in range(2):
                row = w.view(2, 2, 400)[l, i, :c.ctx_capacity][:[400, 380][i]].cpu()
                want = _kept(row.numpy(), keep, 1, 2)
                models[i][l].evict(want)
                models[i][l].check()
                assert torch.equal(out[l, i, :keep].cpu(), row[want])
        _clean(c)
    finally:
        f.close()


def test_refusals_leave_everything_alone():
    f = Filled([200, 100, 90], [Q.KV_HBM, Q.KV_HOST_RING, Q.KV_HOST], layers=2, seed=2, grow=10)
    try:
        c, dev = f.c, f.dev
        h = f.hs[0]
        models = [Model(c, h, l) for l in range(2)]
        w = torch.rand(2, 200, device=dev)

        def refused(status, *a, **kw):
            with pytest.raises(Q.QsaError) as e:
                c.evict(*a, **kw)
            assert e.value.status == status, e.value
        INV = Q.ERR_INVALID_ARG
        for a in ((0, 0, 0), (201, 0, 0), (-1, 0, 0), (50, 51, 0), (50, 0, 51), (50, 30, 21), (50, -1, 0), (50, 0, -1)):
            refused(INV, h, w, *a)
        refused(INV, f.hs[1], w, 50)
        refused(INV, f.hs[2], w, 50)
        some = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
        with pytest.raises(Q.QsaError):        # (asking for the context already tells)
            c.evict(h.__class__(h.index, h.generation + 1), w, 50, workspace=some)
        refused(INV, h, w, 50, workspace=torch.zeros(64, dtype=torch.uint8, device=dev))
        refused(INV, h, w[:1].expand(2, 200), 50)              # both layers the same weights: stride 0
        for bad in (w[:, :199], w[:1], w.double(), w.cpu(), w.t().contiguous().t()):
            with pytest.raises(ValueError):
                c.evict(h, bad, 50)
        for bad in (torch.zeros(2, 50, device=dev), torch.zeros(2, 49, dtype=torch.int32, device=dev)):
            with pytest.raises(ValueError):
                c.evict(h, w, 50, kept=bad)
        with pytest.raises(ValueError):
            c.evict(h, w, 50, weights_out=torch.zeros(2, 49, device=dev))
        # under capture
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ws = torch.empty(c.evict_workspace_bytes(h, 50), dtype=torch.uint8, device=dev)
        x = torch.zeros(4, device=dev)
        with torch.cuda.graph(g, stream=s):
            x.add_(1)
            refused(INV, h, w, 50, workspace=ws)
        assert c.request_info(h).ctx_len == 200
        for m in models:
            m.check()
        # a kept token cannot be taken back, a newer one can
        c.evict(h, w, 50)
        with pytest.raises(Q.QsaError):
            c.truncate(h, 49)
        c.truncate(h, 50)
        c.advance(h, 5)
        c.truncate(h, 52)
        assert c.request_info(h).ctx_len == 52
        # the slot's next request knows nothing of it
        c.request_end(h)
        h2 = c.request_begin(60, max_ctx=70)
        assert h2.index == h.index
        c.truncate(h2, 3)
        _clean(c)
    finally:
        f.close()


def test_kept_weights_do_not_replace_the_weights_they_are_read_from():
    f = Filled([200, 100, 90], [Q.KV_HBM, Q.KV_HBM, Q.KV_HBM], layers=2, seed=3, grow=10)
    try:
        c, h = f.c, f.hs[0]
        models = [Model(c, h, l) for l in range(2)]
        w = torch.rand(2, 200, device=f.dev)
        before = w.clone()
        with pytest.raises(Q.QsaError) as e:
            c.evict(h, w, 50, weights_out=w)
        assert e.value.status == Q.ERR_INVALID_ARG
        assert c.request_info(h).ctx_len == 200 and torch.equal(w, before)
        for m in models:
            m.check()
    finally:
        f.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_kept_tokens_are_not_stored_again(fp8):
    """The rows of kept tokens are in no order, so that the region's row t may be
    another token's: storing them again is refused, alone, in a chunk that reaches back
    over them and in a batch with others, and nothing changes; new tokens are stored."""
    f = Filled([10, 9], layers=2, fp8=fp8, seed=12, grow=6)
    try:
        c, dev, (h, other) = f.c, f.dev, f.hs
        w = torch.zeros(2, 10)
        w[:, [0, 3, 4, 7, 9]] = 1.0
        models = [Model(c, h, l) for l in range(2)] + [Model(c, other, l) for l in range(2)]
        c.evict(h, w.to(dev), 5)
        for m in models[:2]:
            m.evict([0, 3, 4, 7, 9])
            assert [s - m.base for s in m.slots] == [0, 3, 4, 1, 2]
        g = torch.Generator().manual_seed(2)

        def new(units):
            return (torch.randn(units, 64, generator=g).to(dev),
                    torch.randn(units, 1024, generator=g).bfloat16().view(torch.uint8).to(dev))

        def refused(fn, *a):
            with pytest.raises(Q.QsaError) as e:
                fn(*a)
            assert e.value.status == Q.ERR_INVALID_ARG
            torch.cuda.synchronize()
            for m in models:
                m.check()

        refused(c.append_token, [h], 0, 2, *new(2))
        refused(c.append_token, [other, h], 0, 2, *new(4))
        refused(c.append_chunk, [h], [1], 0, 2, *new(2))
        refused(c.append_chunk, [h, other], [5, 2], 1, 1, *new(7))
        c.advance(h, 3)
        models = [Model(c, h, l) for l in range(2)] + models[2:]
        refused(c.append_chunk, [h], [4], 0, 2, *new(8))
        # from the first new token on, one by one or together, as often as wanted
        for _ in range(2):
            c.append_chunk([h, other], [3, 0], 0, 2, *new(6))
            k, kv = new(2)
            c.append_token([h], 0, 2, k, kv)
            torch.cuda.synchronize()
            for l, m in enumerate(models[:2]):
                old = m.slots[:5]
                now = Model(c, h, l)
                assert now.slots == old + [m.base + t for t in (5, 6, 7)]
                assert torch.equal(now.rows[:5], m.rows[:5]) and torch.equal(now.keys[:5], m.keys[:5])
                assert torch.equal(now.scales[:5], m.scales[:5])
                if not fp8:
                    assert torch.equal(now.rows[7], kv[l].cpu())
            for m in models[2:]:
                m.check()
        # a request whose tokens are not stored here does not matter
        c.append_token([other], 0, 2, *new(2))
        _clean(c)
    finally:
        f.close()


def test_kept_weights_beside_and_inside_the_weights():
    """weights_out as a view into the tensor of the weights: refused where the two
    meet, taken where it has columns or rows of its own."""
    f = Filled([200, 100], layers=2, seed=3)
    try:
        c, h = f.c, f.hs[0]
        models = [Model(c, h, l) for l in range(2)]
        t = torch.rand(4, 260, device=f.dev)
        before = t.clone()
        flat = t.view(-1)
        for out in (t[:2], t[:2, 10:70], t[:2, 199:], t[1:3], t[1:3, 150:], flat[:400].view(2, 200),
                    flat[260 + 199:][:100].view(2, 50)):
            with pytest.raises(Q.QsaError) as e:
                c.evict(h, t[:2, :200], 50, weights_out=out)
            assert e.value.status == Q.ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert c.request_info(h).ctx_len == 200 and torch.equal(t, before)
        for m in models:
            m.check()
        c.evict(h, t[:2, :200], 60, weights_out=t[:2, 200:])           # columns behind
        want = [_kept(before[l, :200].cpu().numpy(), 60, 0, 0) for l in range(2)]
        for l in range(2):
            models[l].evict(want[l])
            models[l].check()
            assert torch.equal(t[l, 200:].cpu(), before[l, want[l]].cpu()) and torch.equal(t[l, :200], before[l, :200])
        c.evict(h, t[:2, 200:], 30, weights_out=t[2:])                 # rows behind
        for l in range(2):
            assert torch.equal(t[2 + l, :30].cpu(), t[l, 200:].cpu()[_kept(t[l, 200:].cpu().numpy(), 30, 0, 0)])
        assert torch.equal(t[2:, 30:], before[2:, 30:])
        _clean(c)
    finally:
        f.close()

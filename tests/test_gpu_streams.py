"""Leases, forks and compactions of the Python binding follow the current
stream, on a cache whose device was given as a number."""
import pytest
import torch

import sparse_attention_decode_qsa_gb300 as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    Q.lib()


def test_pages_of_a_numbered_device_are_ordered_behind_the_current_stream():
    """Rows appended late on a side stream are what a fork and a compaction
    there carry on."""
    n = 500
    c = Q.Cache(n_layers=1, max_requests=4, ctx_capacity=n, hbm_pool_rows=3 * n + 100, budget_tokens=64,
                ring_tokens=16, staging_rows=0, device=0)
    try:
        dev = c.pool.device
        c.pool.zero_()
        side = torch.cuda.Stream(dev)
        busy = torch.empty(1 << 28, dtype=torch.uint8, device=dev)
        kv = torch.randint(0, 256, (n, 2048), dtype=torch.uint8, device=dev)
        k = torch.randn(n, 64, device=dev)
        first = c.request_begin(100)
        h = c.request_begin(n)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(side):
                for _ in range(20):
                    busy.zero_()
                c.append_chunk([h], [n], 0, 1, k, kv)
                child = c.request_fork(h, n)
            side.synchronize()
            assert torch.equal(c.pool[c.slot_table[child.index, 0, :n].long()], kv)
            assert torch.equal(c.index_keys[child.index, 0], c.index_keys[h.index, 0])
            c.request_end(child)
            c.request_end(first)
            with torch.cuda.stream(side):
                for _ in range(20):
                    busy.zero_()
                kv.add_(1)
                c.append_chunk([h], [n], 0, 1, k, kv)
                assert c.compact() == n
                first = c.request_begin(100)
            side.synchronize()
            assert torch.equal(c.pool[c.slot_table[h.index, 0, :n].long()], kv)
            # the request lies in front now: let it move back behind the other
            c.request_end(h)
            with torch.cuda.stream(side):
                c.compact()
                h = c.request_begin(n)
            side.synchronize()
        st, det = c.poll_error()
        assert st == 0, (st, det)
    finally:
        torch.cuda.synchronize()
        c.close()

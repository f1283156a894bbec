"""The exact paged cache at its limits: the most requests that page_tables
takes, and calls of different sizes from two host threads."""
import threading

import pytest
import torch

import nystr_coreset_approximate_b200 as wc
from tests import paged_common as pc

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _many(B):
    """B requests of up to 3 tokens of cache on pages of 2, some that end."""
    ctx = [b % 4 for b in range(B)]
    new = [(1, 2, 0, -1)[b % 5 % 4] for b in range(B)]
    table, at = [], 0
    for c in ctx:
        n = -(-c // 2)
        table.append(list(range(at, at + n)) + [-1] * (3 - n))
        at += n
    ring = list(range(at, at + 4 * B)) + [-1] * at
    return ctx, new, table, ring, 4 * B, sum(max(n, 0) for n in new) + 3


# 12 bytes of shared memory to a request: 48 KB, what a launch gets without asking for more,
# end between 4,071 and 4,072 with the kernel's own few hundred bytes, and at 4,095 without them
@pytest.mark.parametrize("B", [4071, 4072, 4095, 4096, 16384])
def test_tables_of_many_requests(B):
    ctx, new, table, ring, count, T = _many(B)
    want = pc.tables_plain(ctx, new, table, ring, 0, count, 2, T)
    d_table, d_ring = _i32(table), _i32(ring)
    got = wc.page_tables(_i32(ctx), _i32(new), d_table, d_ring, _i32([0, count]), 2, T)
    for name, g, w in zip(("seq_lens", "cu_new", "positions", "slots", "ring"), got, want):
        assert g.tolist() == w, name
    assert d_table.tolist() == want[5] and d_ring.tolist() == want[6]
    assert wc.device_status() == 0


def test_tables_of_two_sizes_from_two_threads():
    """The shared memory a kernel may use is the function's state, not the call's."""
    failed = []

    def calls(B):
        try:
            ctx, new, table, ring, count, T = _many(B)
            args = _i32(ctx), _i32(new), _i32(table), _i32(ring), _i32([0, count]), 2, T
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            for _ in range(1500):
                out = wc.page_tables(*args, stream=stream)
            stream.synchronize()
            assert out[1][-1].item() == T - 3
        except Exception as e:  # noqa: BLE001 - told by the main thread
            failed.append((B, repr(e)))

    threads = [threading.Thread(target=calls, args=(B,)) for B in (16384, 4200, 12000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert wc.device_status() == 0

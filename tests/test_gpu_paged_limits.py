"""The exact paged cache at its limits: the most requests that page_tables
takes, calls of different sizes from two host threads, and tables and rings whose
contents are out of range."""
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


# ------------------------------------------------- ids, lengths and rings that are no such thing
def _bad_call(ctx, new, table, ring, head, count, page=4, T=6):
    d_table, d_ring = _i32(table), _i32(ring)
    got = wc.page_tables(_i32(ctx), _i32(new), d_table, d_ring, _i32([head, count]), page, T)
    out = [g.tolist() for g in got], d_table.tolist(), d_ring.tolist()
    return (*out, wc.device_status(), wc.device_status())


# 2^29 pages of 4 rows are 2^31 slots: the first two wrap to slots of page 0 in 32 bits
@pytest.mark.parametrize("bad", [2 ** 30, 2 ** 30 + 1, 2 ** 29, 2 ** 31 - 1, -1, -5], ids=str)
def test_tables_make_no_slot_of_a_bad_id(bad):
    # cached pages: the last one of request 0 is bad; request 1 is as it should be
    (seq, cu, pos, slots, state), *_, status, again = _bad_call([6, 3], [2, 1], [[3, bad, -1], [5, -1, -1]], [7, 8, 9, -1], 0, 3)
    assert (seq, cu, pos[:3], state) == ([8, 4], [0, 2, 3], [6, 7, 3], [0, 3, 0, 0])
    assert slots == [-1, -1, 23, -1, -1, -1] and (status, again) == (1, 0)
    # a page off the ring
    (seq, _, _, slots, state), table, _, status, again = _bad_call([4, 4], [2, 1], [[3, -1], [5, -1]], [bad, 8, 9, -1], 0, 3)
    assert slots == [-1, -1, 32, -1, -1, -1] and state == [2, 1, 0, 0] and (status, again) == (1, 0)
    assert table == [[3, bad], [5, 8]]


def test_tables_take_the_last_id_whose_slots_fit():
    (_, _, _, slots, _), *_, status, _ = _bad_call([6], [2], [[3, 2 ** 29 - 1]], [7], 0, 1)
    assert slots == [2 ** 31 - 2, 2 ** 31 - 1, -1, -1, -1, -1] and status == 0
    (_, _, _, slots, _), *_, status, _ = _bad_call([1], [1], [[3, -1]], [2 ** 31 - 1], 0, 1, page=1)
    assert slots == [2 ** 31 - 1, -1, -1, -1, -1, -1] and status == 0


def test_tables_report_a_bad_id_that_comes_back():
    (seq, _, _, _, state), _, ring, status, again = _bad_call([6, 1], [-1, 0], [[3, -1, -1], [5, -1, -1]], [7, 8, 9, 0], 1, 2)
    assert seq == [0, 1] and state == [1, 4, 0, 0] and ring == [-1, 8, 9, 3] and (status, again) == (1, 0)


@pytest.mark.parametrize("ctx,new,ring,head,count,what", [
    ([-3, 2], [1, 1], [7, 8], 0, 2, ([1, 3], [7 * 4, 5 * 4 + 2], [1, 1, 0, 0])),  # a length below zero counts as zero
    ([2, 2], [1, 1], [7, 8], 0, 3, ([3, 3], [14, 22], [0, 2, 0, 0])),  # more free pages than the ring has places
    ([2, 2], [1, 1], [7, 8], 0, -1, ([3, 3], [14, 22], [0, 0, 0, 0])),
    ([4, 2], [1, 1], [7, 8], 2, 2, ([5, 3], [28, 22], [1, 1, 0, 0])),  # a first place outside the ring: modulo its size
    ([4, 2], [1, 1], [7, 8], -1, 2, ([5, 3], [32, 22], [0, 1, 0, 0])),
    ([9, 2], [0, 1], [7, 8], 0, 2, ([9, 3], [22], [0, 2, 0, 1])),  # more tokens cached than the row has pages
    ([9, 2], [-1, 1], [7, 8, 0, 0], 0, 2, ([0, 3], [22], [0, 4, 0, 0])),
    ([8, 2], [-1, 1], [7, 8, 0], 0, 2, ([0, 3], [22], [0, 3, 0, 0])),  # more pages come back than the ring has room for
], ids=str)
def test_tables_report_lengths_and_rings_out_of_range(ctx, new, ring, head, count, what):
    (seq, cu, _, slots, state), *_, status, again = _bad_call(ctx, new, [[3, 4], [5, 6]], ring, head, count)
    assert (seq, slots[:cu[-1]], state) == what
    assert (status, again) == (1, 0)


# ----------------------------------------------------------- queries that are overwritten or void
BF, F32 = torch.bfloat16, torch.float32


def _attend(c, **kw):
    return wc.paged_attend(kw.pop("q", c["q"]), c["k_pool"], c["v_pool"], c["d_table"], c["d_lens"], c["d_cu"], 0.17, **kw)


@pytest.mark.parametrize("dtype,d", [(F32, 32), (BF, 32), (F32, 64), (BF, 64), (F32, 128)], ids=str)
def test_attend_in_place_where_units_share_cache_lines(dtype, d):
    """Every key head's unit writes its rows between those that other blocks still read."""
    new = [1, 40, 1, 3, 70, 2]
    c = pc.paged_inputs(41, [300, 40, 2, 90, 700, 65], new, 6, 6, d, 16, dtype, nan=False)
    want = _attend(c)
    ref, _, A, size = pc.attend_plain(c["q"], c["k_pool"], c["v_pool"], c["table"], c["lens"], c["cu"], 0.17, True)
    assert (want.double().cpu() - ref).abs().le(pc.attend_bound(ref, A, size, dtype, d, 700)).all()
    for _ in range(10):
        q = c["q"].clone()
        assert _attend(c, q=q, out=q) is q and torch.equal(q, want)
    assert wc.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("void", [float("nan"), float("inf")])
def test_attend_with_void_queries_behind_the_last_request(dtype, void):
    """A tile of rows may reach past the last request's; what stands there changes nothing."""
    c = pc.paged_inputs(42, [33, 150], [5, 30], 4, 2, 64, 16, dtype, extra_rows=100)
    want = _attend(c, out=torch.zeros_like(c["q"]))
    c["q"][35:] = void
    assert torch.equal(_attend(c, out=torch.zeros_like(c["q"])), want)
    assert (want[35:] == 0).all() and want.isfinite().all()
    assert wc.device_status() == 0


# ------------------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("lens,new,Hq,Hkv,d", [
    ([60001, 20], [1, 1], 4, 2, 64),  # one key head's row cut into pieces over many blocks
    ([3000, 500], [500, 1], 8, 1, 128),  # units of two row tiles
    ([130] * 600, [1] * 600, 2, 1, 64),  # whole units in every block
], ids=["long", "chunk", "short"])
def test_a_block_that_gives_up_is_told_and_spoils_no_other(lens, new, Hq, Hkv, d):
    """The hook lets a wait of the first block run out after 1 ms, its copies and products on their way.  The rows that it
    has a part in stay as they were (no piece of it is joined), all others are as always, and so is the next call."""
    c = pc.paged_inputs(43, lens, new, Hq, Hkv, d, 16, BF, nan=False)
    want_lse, lse = (torch.full(c["q"].shape[:2], 3.25, device="cuda") for _ in range(2))
    want = _attend(c, lse=want_lse)
    assert wc.device_status() == 0
    assert wc.lib().wildcat_test_force_wait_timeout(1_000_000) == 0
    try:
        out = _attend(c, out=torch.full_like(c["q"], 3.25), lse=lse)
        assert wc.device_status() == 5
    finally:
        assert wc.lib().wildcat_test_force_wait_timeout(0) == 0
    untouched = (out == 3.25).all(-1)
    assert torch.equal(untouched, lse == 3.25)
    assert torch.equal(out[~untouched], want[~untouched]) and torch.equal(lse[~untouched], want_lse[~untouched])
    # the first units of the line, and no more than a block's share of them
    units = untouched.view(-1, Hkv, Hq // Hkv).all(-1)
    assert units[0, 0] and units.sum() <= {"60001": 1, "3000": 32, "130": 5}[str(lens[0])]
    again = _attend(c, lse=lse)
    assert torch.equal(again, want) and torch.equal(lse, want_lse) and wc.device_status() == 0


# ------------------------------------------------------------------- turning queries and gradients
@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("d,half", [(64, 32), (34, 14)], ids=str)  # 16 bytes a load, and element by element
def test_write_turns_queries_in_their_place(dtype, d, half):
    gen = torch.Generator(device="cuda").manual_seed(d)
    T, Hq, Hkv, page = 45, 6, 2, 8
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dtype)
    slots = torch.randperm(8 * page, generator=gen, device="cuda")[:T].to(torch.int32)
    slots[7] = -1  # not written, but its queries are turned
    pos = torch.randint(0, 9000, (2, T), generator=gen, device="cuda").to(torch.int32)
    turn = dict(positions=pos, inv_freq=torch.rand(half, generator=gen, device="cuda", dtype=torch.float64), sections=(half - 5, 5))
    pools = [torch.zeros(8, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(4)]
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    want = wc.paged_write(k, v, slots, *pools[:2], q=q, **turn)
    rest = qkv[:, Hq:].clone()
    assert wc.paged_write(k, v, slots, *pools[2:], q=q, out=q, **turn) is q
    assert torch.equal(q, want) and torch.equal(qkv[:, Hq:], rest)
    assert torch.equal(pools[2], pools[0]) and torch.equal(pools[3], pools[1])
    assert wc.device_status() == 0


def test_rotary_and_its_backward_in_an_autograd_function():
    """What the documentation tells a program that trains to do."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(9, 3, 32, generator=gen, device="cuda", requires_grad=True)
    dy = torch.randn(9, 3, 32, generator=gen, device="cuda")
    pos = torch.randint(0, 500, (1, 9), generator=gen, device="cuda").to(torch.int32)
    freq = torch.rand(16, generator=gen, device="cuda", dtype=torch.float64)

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return wc.rotary(x, pos, freq, (16,))

        @staticmethod
        def backward(ctx, dy):
            return wc.rotary_backward(dy, pos, freq, (16,))

    assert not wc.rotary(x, pos, freq, (16,)).requires_grad
    (grad,) = torch.autograd.grad((Turn.apply(x) * dy).sum(), x)
    ref, size = pc.rotary_plain(dy, pos, freq, (16,), back=True)
    assert (grad.double().cpu() - ref).abs().le(pc.rotary_bound(ref, size, F32)).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_values_do_not_depend_on_the_layout(dtype, interleaved):
    """The same rows in tensors that take 16 bytes a load and in tensors that do not, alone and beside a pool that does
    not: bit for bit the same."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    T, H, d, half = 200, 3, 128, 64
    x = torch.randn(T, H, d, generator=gen, device="cuda").to(dtype)
    odd = torch.zeros(T, H, d + 1, dtype=dtype, device="cuda")[..., 1:].copy_(x)
    pos = torch.randint(0, 100000, (2, T), generator=gen, device="cuda").to(torch.int32)
    turn = dict(positions=pos, inv_freq=torch.rand(half, generator=gen, device="cuda", dtype=torch.float64), sections=(40, 24),
                interleaved=interleaved)
    want = wc.rotary(x, **turn)
    assert torch.equal(wc.rotary(odd, **turn), want)
    assert torch.equal(wc.rotary_backward(odd, **turn), wc.rotary_backward(x, **turn))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    for wide in (0, 1):
        pools = [torch.zeros(T // 8, H, 8, d + wide, dtype=dtype, device="cuda")[..., wide:] for _ in range(2)]
        assert torch.equal(wc.paged_write(x, x, slots, *pools, q=x, **turn), want)
        assert torch.equal(pools[0].transpose(1, 2).reshape(T, H, d), want)
        assert torch.equal(pools[1].transpose(1, 2).reshape(T, H, d), x)


@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("cu", [[0, 2, 9], [-3, 2, 4], [0, 2, 2 ** 31 - 1], [-(2 ** 31), 2, 4]], ids=str)
def test_attend_cuts_rows_to_the_queries(dtype, cu):
    """Rows of new tokens that no query stands for: the others as if they were not there, and the device status says so."""
    c = pc.paged_inputs(44, [50, 90], [2, 2], 4, 2, 64, 16, dtype)
    want = _attend(c)
    assert wc.device_status() == 0
    assert torch.equal(_attend(dict(c, d_cu=_i32(cu))), want)
    assert wc.device_status() == 1 and wc.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF], ids=str)
def test_attend_negative_lengths_are_empty(dtype):
    c = pc.paged_inputs(45, [0, 90], [1, 2], 4, 2, 64, 16, dtype)
    want = _attend(c)
    assert wc.device_status() == 0
    assert torch.equal(_attend(dict(c, d_lens=_i32([-7, 90]))), want) and (want[0] == 0).all()
    assert wc.device_status() == 1 and wc.device_status() == 0


def test_tables_of_as_many_pages_as_32_bits_hold():
    """One request of 2^31 - 1 pages ends (a table and a ring of 8.6 GB each)."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    table = torch.arange(n, dtype=torch.int32, device="cuda").flip(0)[None]
    ring = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    seq, cu, _, slots, state = wc.page_tables(_i32([n]), _i32([-1]), table, ring, _i32([n - 5, 0]), 1, 148 * 512)
    assert (seq.tolist(), cu.tolist(), state.tolist()) == ([0], [0, 0], [n - 5, n, 0, 0]) and (slots == -1).all()
    assert torch.equal(ring[-5:], table[0, :5]) and torch.equal(ring[:-5], table[0, 5:])
    assert wc.device_status() == 0
    del table, ring, slots
    torch.cuda.empty_cache()

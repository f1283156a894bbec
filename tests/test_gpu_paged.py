"""The exact paged cache on the GPU: page_tables, rotary, paged_write and
paged_attend against plain forms in 64 bits, where they can go wrong."""
import math
import random

import pytest
import torch

import nystr_coreset_approximate_b200 as wc
from tests import paged_common as pc

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page tables
def _tables_case(seed, B, page, most, W, P, count, kinds):
    rng = random.Random(seed)
    ctx = [rng.choice([0, 1, page, page - 1, rng.randint(0, most)]) for _ in range(B)]
    ctx = [min(c, W * page) for c in ctx]
    new = [rng.choice(kinds) for _ in range(B)]
    ids = rng.sample(range(P), P)
    table, at = [], 0
    for c in ctx:
        n = -(-c // page)
        table.append([ids[(at + i) % P] for i in range(n)] + [-1] * (W - n))
        at += n
    ring = rng.sample(range(P), P)
    return ctx, new, table, ring, rng.randrange(P), count


def _tables_check(ctx, new, table, ring, head, count, page, T, pad=0):
    want = pc.tables_plain(ctx, new, table, ring, head, count, page, T)
    W = len(table[0])
    wide = torch.full((len(ctx), W + pad), -7, dtype=torch.int32, device="cuda")
    d_table = wide[:, :W]
    d_table.copy_(_i32(table))
    d_ring = _i32(ring)
    args = _i32(ctx), _i32(new), d_table, d_ring, _i32([head, count])
    for _ in range(2):  # the same inputs again: the same outputs
        got = wc.page_tables(*args, page, T)
        for name, g, w in zip(("seq_lens", "cu_new", "positions", "slots", "ring"), got, want):
            assert g.tolist() == w, name
        assert d_table.tolist() == want[5]
        assert d_ring.tolist() == want[6]
        assert (wide[:, W:] == -7).all()


@pytest.mark.parametrize("B,page,most,W,P,count,kinds", [
    (1, 16, 40, 8, 30, 30, [1]),
    (7, 1, 9, 40, 300, 90, [0, 1, 2, 5]),
    (33, 16, 200, 40, 2000, 900, [1, 1, 1, 40, -1]),
    (600, 8, 60, 20, 9000, 3000, [0, 1, 1, 30, -1, -5]),
    (1500, 128, 700, 9, 20000, 9000, [1, 200, -1]),
], ids=str)
def test_tables(B, page, most, W, P, count, kinds):
    case = _tables_case(B, B, page, most, W, P, count, kinds)
    T = sum(max(n, 0) for n in case[1])
    _tables_check(*case, page, T + 5, pad=3)


def test_tables_where_pages_run_out():
    # needs 2, 0, 3, 1, 0 pages of 3: the third does not advance, nor does the fourth behind it
    page = 4
    ctx, new = [4, 5, 0, 8, 2], [8, 3, 12, 1, 1]
    table = [[9, -1, -1], [8, 7, -1], [-1, -1, -1], [6, 5, -1], [4, -1, -1]]
    _tables_check(ctx, new, table, [3, 2, 1, 0, 10, 11], 4, 3, page, 25)


def test_tables_where_a_row_or_the_outputs_are_full():
    page = 4
    ctx, new = [4, 12, 1, 0, 3], [1, 1, 2, 9, 1]
    table = [[9, -1, -1], [8, 7, 6], [5, -1, -1], [-1, -1, -1], [4, -1, -1]]
    _tables_check(ctx, new, table, [3, 2, 1, 0, 10, 11], 2, 6, page, 14)
    _tables_check(ctx, new, table, [3, 2, 1, 0, 10, 11], 2, 6, page, 6)
    _tables_check(ctx, new, table, [3, 2, 1, 0, 10, 11], 2, 0, page, 0)


def test_tables_without_requests():
    out = wc.page_tables(_i32([]), _i32([]), torch.zeros(0, 4, dtype=torch.int32, device="cuda"), _i32([5, 6]), _i32([1, 1]), 16, 3)
    assert [o.tolist() for o in out] == [[], [0], [0, 0, 0], [-1, -1, -1], [1, 1, 0, 0]]


# ----------------------------------------------------------------------- rotary
def _freqs(half, base=10000.0):
    return torch.tensor([base ** (-i / half) for i in range(half)], dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,d,sections,interleaved", [
    (1, 1, 64, (32,), False),
    (300, 3, 128, (16, 24, 24), False),
    (77, 5, 128, (16, 24, 24), True),
    (40, 2, 128, (10, 10, 12), False),  # 64 of 128 columns turned
    (40, 2, 128, (16, 16, 8, 8), True),  # 96 of 128
    (9, 3, 96, (20, 20), False),  # sections that are no multiple of a load
    (9, 3, 34, (7, 0, 9), False),  # rows of 34: element by element
    (9, 3, 34, (7, 0, 9), True),
    (5, 1, 2, (1,), True),
    (3, 70, 256, (128,), False),
], ids=str)
@pytest.mark.parametrize("back", [False, True])
def test_rotary(dtype, T, H, d, sections, interleaved, back):
    gen = torch.Generator(device="cuda").manual_seed(T * d + back)
    x = torch.randn(T, H, d, generator=gen, device="cuda").to(dtype)
    pos = torch.randint(-1000, 1 << 20, (len(sections), T), generator=gen, device="cuda").to(torch.int32)
    pos[:, 0] = torch.tensor([2 ** 31 - 1, -(2 ** 31), 0, 1])[: len(sections)]
    freq = _freqs(sum(sections))
    turn = wc.rotary_backward if back else wc.rotary
    y = turn(x, pos, freq, sections, interleaved=interleaved)
    ref, size = pc.rotary_plain(x, pos, freq, sections, interleaved, back)
    assert (y.double().cpu() - ref).abs().le(pc.rotary_bound(ref, size, dtype)).all()
    rot = 2 * sum(sections)
    assert torch.equal(y[..., rot:], x[..., rot:])
    turn(x, pos, freq, sections, interleaved=interleaved, out=x)  # in place
    assert torch.equal(x, y)


def test_rotary_strides_and_one_axis():
    gen = torch.Generator(device="cuda").manual_seed(3)
    big = torch.randn(6, 50, 3 * 64 + 1, generator=gen, device="cuda")
    freq, pos = _freqs(32), torch.arange(50, dtype=torch.int32, device="cuda") * 1000
    for x in (big[..., 64:128].transpose(0, 1), big[..., 1:65].transpose(0, 1), big[::2, :, 128:192].transpose(0, 1)):
        ref, size = pc.rotary_plain(x, pos, freq, (32,))
        assert (wc.rotary(x, pos, freq, (32,)).double().cpu() - ref).abs().le(pc.rotary_bound(ref, size, F32)).all()
    # positions whose axes lie apart in a wider tensor
    wide = torch.randint(0, 99, (3, 80), generator=gen, device="cuda").to(torch.int32)
    x = big[..., :64].transpose(0, 1)
    assert torch.equal(wc.rotary(x, wide[:, 7:57], freq, (8, 12, 12)), wc.rotary(x, wide[:, 7:57].contiguous(), freq, (8, 12, 12)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_gradient_against_differences(interleaved):
    """The map is linear, so a difference quotient is exact but for rounding:
    with steps of 1, sums of |y| below 8 and 2^-22 per turned value."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(3, 2, 16, generator=gen, device="cuda")
    dy = torch.randn(3, 2, 16, generator=gen, device="cuda")
    pos = torch.randint(0, 5000, (2, 3), generator=gen, device="cuda").to(torch.int32)
    freq = _freqs(7)
    f = lambda t: (wc.rotary(t, pos, freq, (3, 4), interleaved=interleaved).double() * dy.double()).sum().item()  # noqa: E731
    grad = wc.rotary_backward(dy, pos, freq, (3, 4), interleaved=interleaved)
    for t, h, c in [(0, 0, 0), (1, 1, 5), (2, 0, 13), (2, 1, 15), (1, 0, 7)]:
        step = torch.zeros_like(x)
        step[t, h, c] = 1
        assert abs(f(x + step) - f(x - step) - 2 * grad[t, h, c].item()) < 96 * 4 * 2.0 ** -20


def test_rotary_of_nothing():
    x = torch.empty(0, 4, 64, device="cuda")
    assert wc.rotary(x, torch.empty(1, 0, dtype=torch.int32, device="cuda"), _freqs(32), (32,)).shape == (0, 4, 64)


# ----------------------------------------------------------------------- writes
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,d,page,layout,turned", [
    (1, 4, 1, 64, 16, "head", True),
    (130, 7, 1, 128, 16, "token", True),
    (50, 6, 3, 34, 5, "head", True),
    (70, 2, 2, 128, 32, "token", False),
], ids=str)
def test_write(dtype, T, Hq, Hkv, d, page, layout, turned):
    gen = torch.Generator(device="cuda").manual_seed(T)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dtype)
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    pages = -(-T // page) + 4
    shape = (pages, Hkv, page, d) if layout == "head" else (pages, page, Hkv, d)
    pools = [torch.randn(shape, generator=gen, device="cuda").to(dtype) for _ in range(2)]
    if layout == "token":
        pools = [p.transpose(1, 2) for p in pools]
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:T].to(torch.int32)
    if T > 4:
        slots[[0, 3]] = -1
    half = d // 2 if d % 4 == 0 else d // 2 - 3
    sections = (half - 2 * (half // 3), half // 3, half // 3)
    pos = torch.randint(0, 30000, (3, T), generator=gen, device="cuda").to(torch.int32)
    freq = _freqs(half)
    want = [p.clone() for p in pools]
    tk = wc.rotary(k, pos, freq, sections) if turned else k
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want[0][s // page, :, s % page] = tk[t]
            want[1][s // page, :, s % page] = v[t]
    if turned:
        got = wc.paged_write(k, v, slots, *pools, q=q, positions=pos, inv_freq=freq, sections=sections)
        assert torch.equal(got, wc.rotary(q, pos, freq, sections))
    else:
        assert wc.paged_write(k, v, slots, *pools) is None
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])
    assert wc.device_status() == 0


def test_write_skips_slots_past_the_pool():
    k = torch.ones(3, 2, 64, device="cuda")
    pools = [torch.zeros(2, 2, 4, 64, device="cuda") for _ in range(2)]
    wc.paged_write(k, k, _i32([7, 8, 2 ** 31 - 1]), *pools)
    assert wc.device_status() == 1
    assert pools[0].sum() == 128 and (pools[1][1, :, 3] == 1).all()
    assert wc.device_status() == 0


# -------------------------------------------------------------------- attention
def _attend(c, beta, causal=True, lse=None, out=None, **kw):
    return wc.paged_attend(c["q"], c["k_pool"], c["v_pool"], c["d_table"], c["d_lens"], c["d_cu"], beta, causal=causal, lse=lse, out=out, **kw)


def _attend_check(c, beta, causal=True):
    q = c["q"]
    d, dtype = q.shape[2], q.dtype
    fill = torch.full(q.shape, 3.25, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:2], 3.25, device="cuda")
    out = _attend(c, beta, causal, lse, fill)
    assert out is fill
    T = c["cu"][-1]
    ref, rlse, A, size = pc.attend_plain(q, c["k_pool"], c["v_pool"], c["table"], c["lens"], c["cu"], beta, causal, beyond=torch.full_like(q, 3.25))
    keys = max(c["lens"] + [1])
    off = (out.double().cpu() - ref).abs()
    assert not off.isnan().any()
    assert off.le(pc.attend_bound(ref, A, size, dtype, d, keys)).all(), off.max()
    assert (out[T:] == 3.25).all() and (lse[T:] == 3.25).all()
    seen = rlse[:T].isfinite()
    got = lse[:T].double().cpu()
    assert torch.equal(got.isinf(), ~seen) and not got.isnan().any()
    # a log of sums: relative errors of the exponentials, and its own float32 rounding
    slack = 2 * (2 * (d + 4) * 2.0 ** -24 * size[:T, :, 0] + 2.0 ** -21) + (keys + 16) * 2.0 ** -24 + 2.0 ** -22 * rlse[:T].abs()
    assert (got - rlse[:T])[seen].abs().le(slack[seen]).all()
    assert wc.device_status() == 0
    assert torch.equal(_attend(c, beta, causal, None, fill.clone()), out)  # the same in every run


SHAPES = [  # (lengths, new tokens)
    ([1], [1]),
    ([130, 1, 64], [1, 1, 1]),
    ([128, 129, 255, 256, 257], [1, 1, 2, 1, 3]),
    ([300], [300]),
    ([500, 40, 0, 7], [70, 40, 0, 1]),
    ([0, 3, 200], [2, 5, 33]),  # rows that see nothing: more new tokens than positions
    ([1030, 700], [19, 150]),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d,page", [(4, 2, 64, 16), (7, 1, 128, 32), (3, 3, 128, 8), (2, 1, 32, 16), (5, 1, 64, 3), (2, 2, 64, 256)], ids=str)
@pytest.mark.parametrize("lens,new", SHAPES, ids=str)
def test_attend(dtype, Hq, Hkv, d, page, lens, new):
    c = pc.paged_inputs(sum(lens) + d, lens, new, Hq, Hkv, d, page, dtype, extra_rows=2)
    _attend_check(c, 1.0 / math.sqrt(d))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,new", [([77, 5, 200], [130, 1, 300]), ([0, 140], [3, 40]), ([1, 1], [1, 260])], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_attend_over_an_encoders_states(dtype, lens, new, d):
    c = pc.paged_inputs(5, lens, new, 4, 4, d, 16, dtype, extra_rows=1)
    _attend_check(c, 1.0 / math.sqrt(d), causal=False)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_sharp_rows(dtype):
    """Scores that grow along the keys, over a wide range: the running maximum
    is raised at every tile, and exponentials underflow."""
    c = pc.paged_inputs(8, [900, 300], [140, 1], 4, 2, 64, 16, dtype)
    grow = torch.linspace(0.1, 4, 1200, device="cuda")
    for b, L in enumerate(c["lens"]):
        for x in range(L):
            c["k_pool"][c["table"][b][x // 16], :, x % 16] *= grow[x]
    _attend_check(c, 0.7)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_strided(dtype):
    """Queries and outputs that are views of wider rows, and pools that hold a
    token's heads together."""
    c = pc.paged_inputs(9, [260, 33], [70, 5], 6, 2, 64, 16, dtype, layout="token")
    T = c["cu"][-1]
    wide = torch.zeros(T, 6 + 4, 3 * 64, dtype=dtype, device="cuda")
    wide[:, 2:8, 64:128] = c["q"]
    q, plain = wide[:, 2:8, 64:128], _attend(c, 0.125)
    ref, _, A, size = pc.attend_plain(c["q"], c["k_pool"], c["v_pool"], c["table"], c["lens"], c["cu"], 0.125, True)
    for out in (torch.zeros(T, 12, 64, dtype=dtype, device="cuda")[:, ::2], torch.zeros(T, 6, 65, dtype=dtype, device="cuda")[..., 1:]):
        got = _attend(dict(c, q=q), 0.125, out=out)
        off = (got.double().cpu() - ref).abs()
        assert off.le(pc.attend_bound(ref, A, size, dtype, 64, 260)).all()
    odd = torch.zeros(T, 6, 67, dtype=dtype, device="cuda")[..., 3:]
    odd.copy_(c["q"])
    off = (_attend(dict(c, q=odd), 0.125).double().cpu() - ref).abs()
    assert off.le(pc.attend_bound(ref, A, size, dtype, 64, 260)).all()
    assert torch.equal(_attend(dict(c, q=q), 0.125), plain)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_page_ids_outside_the_pool(dtype):
    """Such pages read as zeros, and the device status says so."""
    c = pc.paged_inputs(10, [100, 50], [3, 1], 2, 1, 64, 16, dtype, nan=False)
    pages = c["k_pool"].shape[0]
    bad = c["d_table"].clone()
    bad[0, 2], bad[1, 0] = pages, -1
    zero = [torch.cat([p, torch.zeros_like(p[:1])]) for p in (c["k_pool"], c["v_pool"])]
    table = [list(r) for r in c["table"]]
    table[0][2] = table[1][0] = pages
    ref, _, A, size = pc.attend_plain(c["q"], *zero, table, c["lens"], c["cu"], 0.125, True)
    got = _attend(dict(c, d_table=bad), 0.125)
    assert (got.double().cpu() - ref).abs().le(pc.attend_bound(ref, A, size, dtype, 64, 100)).all()
    assert wc.device_status() == 1 and wc.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_lengths_past_the_table(dtype):
    c = pc.paged_inputs(11, [64, 40], [2, 2], 2, 1, 64, 16, dtype, W=4)
    want = _attend(c, 0.125)
    got = _attend(dict(c, d_lens=_i32([5000, 40])), 0.125)
    assert torch.equal(got, want)
    assert wc.device_status() == 1 and wc.device_status() == 0


def test_attend_of_nothing():
    c = pc.paged_inputs(12, [5], [1], 2, 1, 64, 16, BF)
    assert wc.paged_attend(c["q"][:0], c["k_pool"], c["v_pool"], c["d_table"], c["d_lens"], _i32([0, 0]), 0.125).shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_long_context_and_many_requests(dtype):
    """One request over the whole GPU, then more requests than blocks."""
    for lens, new in (([9001], [1]), ([9001], [5]), ([17 + 3 * (i % 50) for i in range(400)], [1 + i % 2 for i in range(400)])):
        c = pc.paged_inputs(len(lens), lens, new, 2, 1, 64, 16, dtype, nan=False)
        _attend_check(c, 0.125)


# --------------------------------------------------------------- the whole step
def _serve(dtype, d, steps, seed, run=None):
    """Requests that come, grow by a chunk and then by single tokens, and end;
    returns the outputs and what dense attention says."""
    Hq, Hkv, page, B, P = 4, 2, 16, 5, 120
    gen = torch.Generator(device="cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((B, 30), -1, **i32)
    ring = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    state = torch.tensor([0, P], **i32)
    lens = torch.zeros(B, **i32)
    k_pool, v_pool = (torch.full((P, Hkv, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2))
    freq, sections = _freqs(d // 2), (d // 4, d // 8, d // 8)
    seen = [[] for _ in range(B)]
    for new in steps:
        T = sum(max(n, 0) for n in new) + 2
        qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen, device="cuda").to(dtype)
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        lens, cu, pos, slots, state = wc.page_tables(lens, _i32(new), table, ring, state, page, T)
        pos3 = torch.stack([pos, pos % 7, pos // 7])
        tq = wc.paged_write(k, v, slots, k_pool, v_pool, q=q, positions=pos3, inv_freq=freq, sections=sections)
        got = wc.paged_attend(tq, k_pool, v_pool, table, lens, cu, 1 / math.sqrt(d))
        tk = wc.rotary(k, pos3, freq, sections)
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                seen[b] = []
            for i in range(max(n, 0)):
                seen[b].append((tk[at + i].double(), v[at + i].double()))
            if n > 0:
                K, V = (torch.stack([x[j] for x in seen[b]]).repeat_interleave(Hq // Hkv, 1) for j in (0, 1))
                s = torch.einsum("ihd,jhd->hij", tq[at:at + n].double(), K) / math.sqrt(d)
                L = len(seen[b])
                s = s.masked_fill(torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None], -math.inf)
                p = s.softmax(-1)
                ref = torch.einsum("hij,jhd->ihd", p, V).cpu()
                A = torch.einsum("hij,jhd->ihd", p, V.abs()).cpu()
                size = torch.full((1, 1, 1), 4.0 * d / math.sqrt(d), dtype=torch.float64)
                off = (got[at:at + n].double().cpu() - ref).abs()
                assert off.le(pc.attend_bound(ref, A, size, dtype, d, L)).all()
                at += n
        assert lens.tolist() == [len(x) for x in seen]
    assert state.tolist()[1] == P - sum(-(-len(x) // page) for x in seen)
    assert wc.device_status() == 0


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64)], ids=["bf16-64", "bf16-128", "f32-64"])
def test_serving_steps(dtype, d):
    _serve(dtype, d, [[40, 0, 3, 0, 0], [1, 70, 1, 0, 200], [1, 1, -1, 16, 1], [-1, 33, 90, 1, 1], [17, 1, 1, -1, 1], [1, 1, 1, 5, 1]], 1)


def _step_state(seed, dtype=BF):
    c = pc.paged_inputs(seed, [300, 90, 17], [1, 1, 1], 4, 2, 64, 16, dtype, nan=False)
    c["kv"] = torch.randn(3, 4, 64, device="cuda").to(dtype)
    return c


def test_a_captured_step_follows_its_inputs():
    """Two graphs that share a workspace and run after one another, replayed
    with other lengths and values than they were captured with."""
    c = _step_state(21)
    ring, table = torch.arange(50, 90, dtype=torch.int32, device="cuda"), torch.cat([c["d_table"], torch.full((3, 4), -1, dtype=torch.int32, device="cuda")], 1)
    pools = [torch.cat([p, torch.zeros(100 - p.shape[0], *p.shape[1:], dtype=p.dtype, device="cuda")]) for p in (c["k_pool"], c["v_pool"])]
    freq = _freqs(32)
    ctx, new, state = _i32([299, 89, 16]), _i32([1, 1, 1]), _i32([0, 40])
    q, kv = c["q"].clone(), c["kv"].clone()

    def step():
        lens, cu, pos, slots, out = wc.page_tables(ctx, new, table, ring, state, 16, 3)
        tq = wc.paged_write(kv[:, :2], kv[:, 2:], slots, *pools, q=q, positions=pos, inv_freq=freq, sections=(32,))
        return wc.paged_attend(tq, *pools, table, lens, cu, 0.125), lens, out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=graphs[0][0].pool() if graphs else None):
            res = step()
        graphs.append((graph, res))
    for k in range(4):
        with torch.no_grad():
            ctx.copy_(_i32([200 + 16 * k, 80 + k, 5 * k]))
            q.normal_()
            kv.normal_()
        saved = [p.clone() for p in pools], table.clone()
        graph, res = graphs[k % 2]
        graph.replay()
        got = [x.clone() for x in res]
        after = [p.clone() for p in pools]
        for p, s in zip(pools, saved[0]):
            p.copy_(s)
        table.copy_(saved[1])
        want = step()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
        assert all(torch.equal(a, p) for a, p in zip(after, pools))
    assert wc.device_status() == 0


def test_calls_on_two_streams_at_once():
    cases = [pc.paged_inputs(31 + i, [2000 + 300 * i, 700], [1 + 80 * i, 1], 4, 2, 64, 16, BF, nan=False) for i in range(2)]
    want = [_attend(c, 0.125) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(_attend(cases[i], 0.125, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


# ------------------------------------------------------------ more that can go wrong
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,page", [(130, 1, 16), (33, 1, 128), (128, 1, 8), (48, 2, 64)], ids=str)
def test_attend_wide_groups(dtype, Hq, Hkv, page):
    """More query heads to a key head than a tile has rows, and numbers that do not divide it."""
    _attend_check(pc.paged_inputs(Hq, [150, 300, 2], [3, 9, 1], Hq, Hkv, 64, page, dtype, extra_rows=1), 0.125)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_more_requests_than_threads(dtype):
    """Requests without new tokens among them, and some without anything."""
    rng = random.Random(5)
    lens = [rng.choice([0, 1, 15, 16, 17, 60]) for _ in range(1300)]
    new = [rng.choice([0, 0, 1, 2]) for _ in range(1300)]
    _attend_check(pc.paged_inputs(13, lens, new, 2, 1, 64, 16, dtype), 0.125)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_long_chunks_beside_short_ones(dtype, causal):
    """Many row tiles to a request, most of whose rows see nothing (causal: 900 new tokens of 260)."""
    _attend_check(pc.paged_inputs(14, [260, 700, 33], [900, 700, 1], 5, 1, 64, 32, dtype), 0.125, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 100])
def test_attend_scores_that_leap(d, new):
    """A key every few tiles scores far above all before it, so that exponentials with the maximum of the tiles before
    overflow; in between they vanish."""
    c = pc.paged_inputs(15, [1500], [new], 4, 2, d, 16, BF)
    for x in (140, 141, 400, 900, 1290, 1399):
        c["k_pool"][c["table"][0][x // 16], :, x % 16] *= 1 + x / 50
    _attend_check(c, 2.0)


def test_attend_broadcast_queries_and_one_pool():
    """Every token with the same queries (a stride of zero), keys that are their own values."""
    c = pc.paged_inputs(16, [90, 40], [3, 2], 4, 2, 64, 16, BF)
    same = dict(c, q=c["q"][:1].expand(5, 4, 64), v_pool=c["k_pool"])
    _attend_check(same, 0.125)
    _attend_check(dict(same, q=same["q"].contiguous()), 0.125)


def test_what_a_page_shared_by_two_requests_holds():
    """A prefix that two requests share: the same pages in both rows of the table."""
    c = pc.paged_inputs(17, [64, 100], [1, 1], 4, 2, 64, 16, BF)
    c["table"][1][:3] = c["table"][0][:3]
    c["d_table"] = _i32(c["table"])
    _attend_check(c, 0.125)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_write_and_rotary_on_another_stream(dtype):
    side = torch.cuda.Stream()
    x = torch.randn(50, 4, 64, device="cuda").to(dtype)
    pos, freq = torch.arange(50, dtype=torch.int32, device="cuda"), _freqs(32)
    pools = [torch.zeros(8, 4, 16, 64, device="cuda", dtype=dtype) for _ in range(4)]
    slots = torch.randperm(128, device="cuda")[:50].to(torch.int32)
    want = wc.rotary(x, pos, freq, (32,))
    wc.paged_write(x, x, slots, pools[0], pools[1], positions=pos, inv_freq=freq, sections=(32,))
    torch.cuda.synchronize()
    got = wc.rotary(x, pos, freq, (32,), stream=side)
    wc.paged_write(x, x, slots, pools[2], pools[3], positions=pos, inv_freq=freq, sections=(32,), stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_without_new_tokens(dtype):
    """Requests that bring none, and rows behind the last one."""
    c = pc.paged_inputs(18, [40, 0, 5], [0, 0, 0], 2, 1, 64, 16, dtype, extra_rows=4)
    _attend_check(c, 0.125)


def test_attend_pools_without_pages():
    """Nothing cached at all: zeros, and the logs of empty sums."""
    q = torch.randn(3, 2, 64, device="cuda").to(BF)
    pool = torch.zeros(0, 1, 16, 64, device="cuda", dtype=BF)
    lse = torch.zeros(3, 2, device="cuda")
    out = wc.paged_attend(q, pool, pool, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), _i32([0, 0]), _i32([0, 1, 3]), 0.125, lse=lse)
    assert (out == 0).all() and (lse == -math.inf).all() and wc.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attend_infinities_behind_the_length(dtype):
    """What a page holds past a request's length does not matter, infinities of either sign among it."""
    c = pc.paged_inputs(19, [37, 130], [5, 1], 4, 2, 64, 16, dtype)
    want = _attend(c, 0.125)
    for p in (c["k_pool"], c["v_pool"]):
        p[p.isnan()] = -math.inf
    assert torch.equal(_attend(c, 0.125), want)
    for p in (c["k_pool"], c["v_pool"]):
        p[p.isinf()] = math.inf
    assert torch.equal(_attend(c, 0.125), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,new", [([300, 40], [300, 1]), ([5000, 2000, 9], [1, 1, 1])], ids=str)
def test_attend_in_place(dtype, lens, new):
    """O over Q: other blocks may still hold parts of a row's work when its first result is written."""
    c = pc.paged_inputs(20, lens, new, 4, 2, 64, 16, dtype, nan=False)
    want = _attend(c, 0.125)
    for _ in range(5):
        q = c["q"].clone()
        assert _attend(dict(c, q=q), 0.125, out=q) is q and torch.equal(q, want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 32), (2, 1, 64), (3, 1, 128), (4, 1, 64), (5, 1, 128)], ids=str)
def test_attend_few_rows_in_odd_pages(dtype, Hq, Hkv, d):
    """Units of one to five rows, also two tokens of two heads, over pages that divide nothing."""
    _attend_check(pc.paged_inputs(21, [700, 1, 65, 130], [1, 1, 2, 1], Hq, Hkv, d, 7, dtype), 1 / math.sqrt(d))

"""What the paged-cache entry points refuse, on the host and before any CUDA
call, and the plain forms of their tests against simpler statements."""
import ctypes
import math

import pytest
import torch

import nystr_coreset_approximate_b200 as wc
from tests import paged_common as pc

FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
OTHER = ctypes.c_void_p(1 << 21)


def _longs(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _ints(*v):
    return (ctypes.c_int * len(v))(*v)


def _call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(wc.lib(), fn)(*a.values())


TABLES = dict(ctx=FAKE, new=FAKE, B=4, table=FAKE, stride=8, W=8, ring=OTHER, P=64, state=FAKE, page=16, T=10, seq=OTHER, cu=OTHER,
              pos=OTHER, slots=OTHER, out=OTHER, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(B=16385), 2), (dict(W=-1), 1), (dict(T=-1), 1), (dict(page=0), 1), (dict(P=0), 1), (dict(stride=7), 1),
    (dict(P=1 << 28), 2), (dict(P=1 << 31, page=1), 2), (dict(T=1 << 31), 2), (dict(W=1 << 31, stride=1 << 31), 2),
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(ring=None), 1), (dict(state=None), 1), (dict(seq=None), 1),
    (dict(cu=None), 1), (dict(pos=None), 1), (dict(slots=None), 1), (dict(out=None), 1),
    (dict(seq=FAKE), 1), (dict(out=FAKE), 1), (dict(ring=FAKE), 1),
], ids=str)
def test_page_tables_refuses(kw, code):
    assert _call("wildcat_page_tables", TABLES, kw) == code
    assert wc.lib().wildcat_last_error().startswith(b"wildcat_page_tables")


ROTARY = dict(x=FAKE, xt=256, xh=64, dtype=1, T=5, H=4, d=64, pos=FAKE, ps=5, freq=FAKE, sections=_ints(16, 8, 8), axes=3, inter=0,
              back=0, out=OTHER, ot=256, oh=64, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 1), (dict(T=-1), 1), (dict(T=1 << 31), 2), (dict(H=-1), 1), (dict(H=65536), 2), (dict(d=63), 2), (dict(d=0), 2),
    (dict(d=1026), 2), (dict(axes=0), 1), (dict(axes=5), 1), (dict(sections=None), 1), (dict(sections=_ints(16, 8, 9)), 1),
    (dict(sections=_ints(0, 0, 0)), 1), (dict(sections=_ints(16, -8, 8)), 1), (dict(sections=_ints(2 ** 31 - 1, 2 ** 31 - 1, 34)), 1),
    (dict(pos=None), 1), (dict(freq=None), 1), (dict(ps=-1), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(xt=-256), 1),
    (dict(ot=63), 1), (dict(oh=63), 1), (dict(x=ctypes.c_void_p(1001)), 1), (dict(out=FAKE, ot=512), 1), (dict(out=FAKE, oh=128, ot=512), 1),
], ids=lambda k: str(k)[:40])
def test_rotary_refuses(kw, code):
    assert _call("wildcat_rotary", ROTARY, kw) == code


WRITE = dict(k=FAKE, kt=128, kh=64, v=FAKE, vt=128, vh=64, slots=FAKE, dtype=1, T=5, Hkv=2, d=64, kp=OTHER, ks=_longs(2048, 1024, 64),
             vp=OTHER, vs=_longs(2048, 1024, 64), pages=10, page=16, pos=FAKE, ps=5, freq=FAKE, sections=_ints(32), axes=1, inter=0,
             q=FAKE, qt=256, qh=64, Hq=4, qo=OTHER, qot=256, qoh=64, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), 1), (dict(T=-1), 1), (dict(d=7), 2), (dict(Hkv=0), 1), (dict(Hq=-1), 1), (dict(pages=-1), 1), (dict(page=0), 1),
    (dict(pages=1 << 27), 2), (dict(Hkv=65536), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(kp=None), 1),
    (dict(vp=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(qo=None), 1), (dict(kt=-1), 1), (dict(vh=-1), 1), (dict(qt=-1), 1),
    (dict(ks=_longs(0, 1024, 64)), 1), (dict(ks=_longs(2048, 0, 64)), 1), (dict(vs=_longs(2048, 1024, 32)), 1), (dict(qot=32), 1),
    (dict(qoh=0), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(axes=0), 1), (dict(qo=FAKE, qot=512), 1),
    (dict(v=ctypes.c_void_p(4097)), 1),
], ids=lambda k: str(k)[:40])
def test_paged_write_refuses(kw, code):
    assert _call("wildcat_paged_write", WRITE, kw) == code


def _attend_defaults():
    n = int(wc.lib().wildcat_paged_attend_workspace_size(3, 64))
    return dict(q=FAKE, qt=256, qh=64, kp=FAKE, ks=_longs(2048, 1024, 64), vp=FAKE, vs=_longs(2048, 1024, 64), pages=10, page=16, dtype=1,
                T=5, Hq=4, Hkv=2, d=64, table=FAKE, stride=4, W=4, lens=FAKE, cu=FAKE, B=3, beta=0.125, causal=1, out=OTHER, ot=256, oh=64,
                lse=None, ws=FAKE, n=n, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 1), (dict(d=96), 2), (dict(beta=0.0), 1), (dict(beta=math.inf), 1), (dict(B=-1), 1), (dict(B=65536), 2), (dict(T=-1), 1),
    (dict(W=-1), 1), (dict(stride=3), 1), (dict(page=0), 1), (dict(pages=-1), 1), (dict(pages=1 << 27), 2), (dict(Hkv=0), 1),
    (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=65538), 2), (dict(T=1 << 30), 2), (dict(W=1 << 31, stride=1 << 31), 2), (dict(q=None), 1),
    (dict(kp=None), 1), (dict(vp=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(cu=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(qt=-1), 1), (dict(ks=_longs(2048, -1, 64)), 1), (dict(ot=10), 1),
    (dict(oh=10), 1), (dict(out=FAKE, ot=512), 1), (dict(out=FAKE, ot=512, oh=128), 1), (dict(ws=ctypes.c_void_p((1 << 20) + 64)), 4), (dict(n=4096), 4), (dict(q=ctypes.c_void_p(4097)), 1),
], ids=lambda k: str(k)[:40])
def test_paged_attend_refuses(kw, code):
    assert _call("wildcat_paged_attend", _attend_defaults(), kw) == code


def test_nothing_to_do_is_no_call():
    assert _call("wildcat_rotary", ROTARY, dict(T=0)) == 0
    assert _call("wildcat_rotary", ROTARY, dict(H=0)) == 0
    assert _call("wildcat_paged_write", WRITE, dict(T=0)) == 0
    assert _call("wildcat_paged_attend", _attend_defaults(), dict(T=0)) == 0
    assert _call("wildcat_paged_attend", _attend_defaults(), dict(B=0)) == 0


def test_workspace_holds_two_pieces_of_every_block():
    small, large = (int(wc.lib().wildcat_paged_attend_workspace_size(B, 128)) for B in (1, 60000))
    assert 2 * 148 * 256 * 130 * 4 <= small <= large < small + 60000 * 17 + 4096
    assert wc.lib().wildcat_paged_attend_workspace_size(-1, 64) == 0


def test_the_binding_refuses_on_the_host():
    i32 = dict(dtype=torch.int32)
    x, pool = torch.zeros(5, 2, 64), torch.zeros(3, 2, 16, 64)
    pos, freq, lens, cu, table = torch.zeros(1, 5, **i32), torch.zeros(32, dtype=torch.float64), torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(2, 3, **i32)
    for call in (
        lambda: wc.rotary(x, pos, freq, (32,)),  # not on the GPU
        lambda: wc.rotary(x[0], pos, freq, (32,)),
        lambda: wc.rotary(x, pos, freq, (16, 16)),
        lambda: wc.rotary(x, pos, freq, (16,)),
        lambda: wc.rotary(x, pos[:, :4], freq, (32,)),
        lambda: wc.paged_write(x, x[:4], lens, pool, pool),
        lambda: wc.paged_write(x, x, lens, pool, pool),
        lambda: wc.paged_write(x, x, lens, pool, pool[:2]),
        lambda: wc.paged_write(x, x, torch.zeros(5, **i32), pool, pool, q=x),
        lambda: wc.paged_write(x, x, torch.zeros(5, **i32), pool, pool, out=x),
        lambda: wc.paged_write(x, x, torch.zeros(5, **i32), pool, pool, positions=pos),
        lambda: wc.paged_attend(x, pool[..., :32], pool[..., :32], table, lens, cu, 0.1),
        lambda: wc.paged_attend(x, pool, pool, table, lens, cu[:2], 0.1),
        lambda: wc.paged_attend(x, pool, pool, table[:1], lens, cu, 0.1),
        lambda: wc.paged_attend(x, pool, pool, table, lens, cu, 0.1, lse=torch.zeros(5, 3)),
        lambda: wc.page_tables(lens, lens[:1], table, lens, lens, 16, 4),
        lambda: wc.page_tables(lens, lens, table[0], lens, lens, 16, 4),
        lambda: wc.page_tables(lens, lens, table, lens, lens, 16, -1),
        lambda: wc.page_tables(lens, lens, table, lens, lens[:1], 16, 4),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: wc.rotary(x.half(), pos, freq, (32,)),
        lambda: wc.paged_write(x, x, torch.zeros(5, **i32), pool.bfloat16(), pool.bfloat16()),
        lambda: wc.paged_attend(x.bfloat16(), pool, pool, table, lens, cu, 0.1),
    ):
        with pytest.raises(TypeError):
            call()


def test_plain_rotary_turns_complex_numbers():
    x, pos, freq = torch.randn(7, 2, 12), torch.randint(-50, 50, (2, 7)), torch.rand(5, dtype=torch.float64)
    for inter in (False, True):
        y, _ = pc.rotary_plain(x, pos, freq, (3, 2), inter)
        back, _ = pc.rotary_plain(y, pos, freq, (3, 2), inter, True)
        assert torch.allclose(back, x.double(), atol=1e-12) and torch.equal(y[..., 10:], x[..., 10:].double())
        lo, hi = (x[..., 0:10:2], x[..., 1:10:2]) if inter else (x[..., :5], x[..., 5:10])
        u, v = (y[..., 0:10:2], y[..., 1:10:2]) if inter else (y[..., :5], y[..., 5:10])
        angle = torch.cat([pos[:1].expand(3, 7), pos[1:].expand(2, 7)]).double().T * freq
        z = torch.complex(lo.double(), hi.double()) * torch.exp(1j * angle)[:, None]
        assert torch.allclose(torch.complex(u, v), z, atol=1e-12)


def test_plain_tables_hand_out_and_take_back():
    seq, cu, pos, slots, state, table, ring = pc.tables_plain([3, 4, 5], [2, -1, 0], [[6, -1], [7, -1], [8, 9]], [1, 2, 3, 0], 3, 2, 4, 3)
    assert (seq, cu, pos, slots) == ([5, 0, 5], [0, 2, 2, 2], [3, 4, 0], [27, 0, -1])
    assert table == [[6, 0], [7, -1], [8, 9]] and ring == [1, 7, 3, 0] and state == [0, 2, 0, 0]

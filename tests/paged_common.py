"""Plain forms of the paged-cache operators, in 64 bits on the CPU, and the
inputs their tests use."""
import math
import random

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def tables_plain(ctx, new, table, ring, head, count, page, max_tokens):
    """One request after the other, one token after the other."""
    table, ring = [list(r) for r in table], list(ring)
    B, W, P = len(ctx), len(table[0]) if table else 0, len(ring)
    seq, cu, pos, slots = [], [0], [0] * max_tokens, [-1] * max_tokens
    asked = taken = refused = 0
    given = []
    for b in range(B):
        have = -(-ctx[b] // page)
        n = max(new[b], 0)
        start = cu[-1]
        cu.append(start + n)
        for i in range(n):
            if start + i < max_tokens:
                pos[start + i] = ctx[b] + i
        if new[b] < 0:
            given += table[b][:have]
            seq.append(0)
            continue
        want = -(-(ctx[b] + n) // page)
        if want > W or start + n > max_tokens:
            refused += 1
            seq.append(ctx[b])
            continue
        need = want - have
        if need and asked + need > count:
            asked += need
            refused += 1
            seq.append(ctx[b])
            continue
        for k in range(need):
            table[b][have + k] = ring[(head + asked + k) % P]
        asked += need
        taken += need
        seq.append(ctx[b] + n)
        for i in range(n):
            x = ctx[b] + i
            p = table[b][x // page]
            slots[start + i] = p * page + x % page if p >= 0 else -1
    for j, p in enumerate(given):
        ring[(head + count + j) % P] = p
    state = [(head + taken) % P, count - taken + len(given), asked - taken, refused]
    return seq, cu, pos, slots, state, table, ring


def rotary_plain(x, positions, inv_freq, sections, interleaved=False, back=False):
    """(turned x, the pairs' |a| + |b| laid out like x) in float64."""
    x = x.double().cpu()
    positions = positions.cpu().double()
    if positions.dim() == 1:
        positions = positions[None]
    half = inv_freq.numel()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    angle = positions[axis].T * inv_freq.cpu()  # [T, half]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    if back:
        sin = -sin
    lo = torch.arange(half) * 2 if interleaved else torch.arange(half)
    hi = lo + 1 if interleaved else lo + half
    a, b = x[..., lo], x[..., hi]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., lo], y[..., hi] = a * cos - b * sin, b * cos + a * sin
    size[..., lo] = size[..., hi] = a.abs() + b.abs()
    return y, size


def rotary_bound(ref, size, dtype):
    """One rounding to dtype; before it float32: the angle's fraction of a turn
    is rounded to float32 (2 pi 2^-25 radians and the argument's own error in
    64 bits, below 2^-21 up to positions of 2^31), sine and cosine and the
    three operations of a pair some 2^-24 each."""
    return EPS[dtype] * ref.abs() * 1.01 + 2.0 ** -20 * size


def attend_plain(q, k_pool, v_pool, table, lens, cu, beta, causal, beyond=None):
    """(O, lse, A) in float64, A = sum p |v| / sum p and the largest sum of |q||k|."""
    T, Hq, d = q.shape
    _, H, page, _ = k_pool.shape
    g = Hq // H
    q, kp, vp = q.double().cpu(), k_pool.double().cpu(), v_pool.double().cpu()
    O = torch.zeros(T, Hq, d, dtype=torch.float64) if beyond is None else beyond.double().cpu().clone()
    A = torch.zeros(T, Hq, d, dtype=torch.float64)
    size = torch.zeros(T, Hq, 1, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    for b, L in enumerate(lens):
        lo, n = cu[b], cu[b + 1] - cu[b]
        ids = torch.tensor([table[b][j // page] for j in range(L)], dtype=torch.long)
        at = torch.arange(L) % page
        K, V = kp[ids, :, at], vp[ids, :, at]  # [L, H, d]
        for i in range(n):
            end = max(0, min(L, L - n + i + 1 if causal else L))
            O[lo + i] = 0
            if end == 0:
                continue
            for h in range(Hq):
                k, v = K[:end, h // g], V[:end, h // g]
                s = beta * (k @ q[lo + i, h])
                m = s.max()
                p = (s - m).exp()
                O[lo + i, h] = p @ v / p.sum()
                A[lo + i, h] = p @ v.abs() / p.sum()
                size[lo + i, h] = beta * (k.abs() @ q[lo + i, h].abs()).max()
                lse[lo + i, h] = m + p.sum().log()
    return O, lse, A, size


def attend_bound(ref, A, size, dtype, d, keys):
    """A score is a float32 sum of d products, scaled: off by at most
    (d + 4) 2^-24 sum |q||k| beta, and an exponential by twice that (its own and
    the row's maximum) and 2^-21; numerator and denominator both carry it.  The
    float32 sums over the keys add (keys + 16) 2^-24 each.  In bf16 each
    exponential is rounded once for the product with V (2^-8); the result is
    rounded once to its type."""
    f32 = 2.0 ** -24
    rel = 2 * (2 * (d + 4) * f32 * size + 2.0 ** -21) + 2 * (keys + 16) * f32
    if dtype == torch.bfloat16:
        rel = rel + 2.0 ** -8
    return (rel * A + EPS[dtype] * ref.abs()) * 1.01 + 1e-30


def paged_inputs(seed, lens, new, Hq, Hkv, d, page, dtype, *, layout="head", spare=3, nan=True, extra_rows=0, W=None):
    """A cache whose pages lie in random order, with NaN wherever no request has
    a token; queries of `new` tokens (and extra_rows behind them)."""
    gen = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.sample(range(pages), pages)
    W = max(need + [1]) + 1 if W is None else W
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (W - n))
        at += n
    shape = (pages, Hkv, page, d) if layout == "head" else (pages, page, Hkv, d)
    pools = []
    for _ in range(2):
        pool = torch.full(shape, math.nan) if nan else torch.zeros(shape)
        view = pool if layout == "head" else pool.transpose(1, 2)
        for b, n in enumerate(lens):
            for x in range(n):
                view[table[b][x // page], :, x % page] = torch.randn(Hkv, d, generator=gen)
        pool = pool.to(dtype).cuda()
        pools.append(pool if layout == "head" else pool.transpose(1, 2))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1] + extra_rows, Hq, d, generator=gen).to(dtype).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(q=q, k_pool=pools[0], v_pool=pools[1], table=table, lens=list(lens), cu=cu,
                d_table=torch.tensor(table, **i32).view(len(lens), W), d_lens=torch.tensor(list(lens), **i32),
                d_cu=torch.tensor(cu, **i32))

"""What the paged-cache operators are measured on: their cases, inputs, plain forms and exact values.

Four operators that a serving program runs in this order at every step:

  tables   page_tables: the step's slots, positions and pages from the requests' lengths
  rotary   rotary / rotary_backward: rotary positions with several axes
  write    paged_write: keys (rotated where positions are given) and values into the cache, queries rotated beside them
  attend   paged_attend: the step's tokens over the paged cache

A case's lengths come from the case alone, its values and page orders from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 64 requests: one token each, now and then a new page
        dict(name="tables_decode", op="tables", B=64, page=16, ctx=8000, chunk=0, chunks=0, done=2, mix=1),
        # a large step: 1,000 requests, some of them bring prompts, some end and give their pages back
        dict(name="tables_mixed", op="tables", B=1000, page=16, ctx=4000, chunk=700, chunks=90, done=40, mix=2),
        # queries of the 56 x 56 image workload (32 heads of 64), rows and columns as two axes
        dict(name="rotary_image", op="rotary", dtype="bf16", T=3136, H=32, d=64, axes=2, part=64, pairs=0, back=0),
        # gradients of a video's queries: time, height and width, 24 frames of 36 x 36, one partial rotation
        dict(name="rotary_video_back", op="rotary", dtype="f32", T=31104, H=16, d=128, axes=3, part=96, pairs=1, back=1),
        # one decoding step of 64 requests: 64 tokens into the cache
        dict(name="write_decode", op="write", dtype="bf16", T=64, Hq=32, Hkv=8, d=128, axes=1, page=16, pages=4096),
        # a prompt with images in it (time, height, width), an odd number of tokens, seven queries to a key head
        dict(name="write_prompt", op="write", dtype="bf16", T=16383, Hq=28, Hkv=4, d=128, axes=3, page=32, pages=2048),
        # the smallest serving step: three short requests, one token each
        dict(name="attend_few", op="attend", dtype="bf16", B=3, Hq=32, Hkv=8, d=128, page=16, low=300, ctx=1000, chunk=1, chunks=0, causal=1, mix=3),
        # decoding at the key-value-cache workload's length: 32 requests of up to 32,768 tokens
        dict(name="attend_decode_long", op="attend", dtype="bf16", B=32, Hq=32, Hkv=8, d=128, page=16, low=20000, ctx=32768, chunk=1, chunks=0, causal=1, mix=4),
        # a chunk of a long prompt behind 30,001 cached tokens
        dict(name="attend_chunk_long", op="attend", dtype="bf16", B=1, Hq=32, Hkv=8, d=128, page=64, low=32049, ctx=32049, chunk=2048, chunks=1, causal=1, mix=5),
        # a chunk of a prompt beside decoding requests of all lengths, seven queries to a key head
        dict(name="attend_mixed", op="attend", dtype="bf16", B=24, Hq=28, Hkv=4, d=128, page=16, low=1, ctx=8000, chunk=333, chunks=2, causal=1, mix=6),
        # an image's 4,096 positions over an encoder's cached states (the image workload's 64 x 64 tokens, heads of 64)
        dict(name="attend_cross", op="attend", dtype="bf16", B=4, Hq=16, Hkv=16, d=64, page=32, low=77, ctx=700, chunk=4096, chunks=4, causal=0, mix=7),
        # single precision: short chunks over short contexts
        dict(name="attend_f32", op="attend", dtype="f32", B=4, Hq=8, Hkv=4, d=64, page=16, low=100, ctx=3000, chunk=200, chunks=2, causal=1, mix=8),
    ]


def _between(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "write", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 30)
    if op == "tables":
        B = _between(rng, 1, 1000)
        return dict(op=op, B=B, page=rng.choice([8, 16, 32, 64, 128]), ctx=_between(rng, 16, 8000), chunk=_between(rng, 2, 700),
                    chunks=rng.randint(0, max(1, B // 10)), done=rng.randint(0, B // 8), mix=mix)
    if op == "rotary":
        d, axes = rng.choice([64, 128]), rng.randint(1, 4)
        part = rng.choice([d, d // 2, d - 32]) if axes < 3 else d
        T, H = _between(rng, 1, 31000), _between(rng, 1, 32)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=max(1, min(T, 31104 * 16 * 128 // (H * d))), H=H, d=d, axes=axes, part=part,
                    pairs=rng.randint(0, 1), back=rng.randint(0, 1))
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    Hkv, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    if op == "write":
        T = min(_between(rng, 1, 16000), 16000 * 36 // ((g + 1) * Hkv))
        return dict(op=op, dtype=dtype, T=T, Hq=g * Hkv, Hkv=Hkv, d=d, axes=rng.randint(0, 3), page=page, pages=-(-2 * T // page) + 64)
    kind = rng.choice(["decode", "chunk", "mixed", "cross"])
    B = {"decode": _between(rng, 1, 64), "chunk": rng.randint(1, 4), "mixed": _between(rng, 2, 24), "cross": rng.randint(1, 8)}[kind]
    chunk = {"decode": rng.choice([1, 1, 1, 2, 4]), "chunk": _between(rng, 16, 2048), "mixed": _between(rng, 16, 333), "cross": _between(rng, 16, 2048)}[kind]
    most = 1 << (28 if dtype == "bf16" else 24)  # scores of the padded plain form; single precision runs on fewer units
    cached = (1 << 30) // (B * Hkv * d * (2 if dtype == "bf16" else 4))
    ctx = max(1, min(_between(rng, 64, 32768 if kind != "cross" else 2000), most // (B * g * Hkv * chunk), cached))
    return dict(op=op, dtype=dtype, B=B, Hq=g * Hkv, Hkv=Hkv, d=d, page=page, low=rng.choice([1, max(1, ctx // 2)]), ctx=ctx, chunk=chunk,
                chunks={"decode": B, "chunk": B, "mixed": rng.randint(1, 2), "cross": B}[kind], causal=int(kind != "cross"), mix=mix)


# --------------------------------------------------------------------------- lengths and inputs
def _lengths(case):
    """The requests' cached and new lengths: (contexts, new tokens; -1 for a request that ends)."""
    rng = random.Random(case["mix"])
    B = case["B"]
    if case["op"] == "tables":
        ctx = [_between(rng, 1, case["ctx"]) for _ in range(B)]
        new = [1] * B
        order = rng.sample(range(B), B)
        for b in order[: case["chunks"]]:
            ctx[b], new[b] = rng.choice([0, ctx[b]]), _between(rng, 1, case["chunk"])
        for b in order[case["chunks"] : case["chunks"] + case["done"]]:
            new[b] = -1
        return ctx, new
    total = [rng.randint(case["low"], max(case["low"], case["ctx"])) for _ in range(B)]
    total[rng.randrange(B)] = case["ctx"]
    new = [1] * B
    for b in rng.sample(range(B), case["chunks"]):
        new[b] = case["chunk"] if case["chunks"] == 1 else rng.randint(max(1, case["chunk"] * 3 // 4), case["chunk"])
    if case["causal"]:
        return total, new
    return [t - n for t, n in zip(total, new)], new  # over an encoder's states: `total` of them, whatever the queries' number


def _sections(half, axes):
    """The rotated pairs of each axis: the first axis takes what the others leave."""
    other = half // axes
    return (half - other * (axes - 1),) + (other,) * (axes - 1)


def _inv_freq(half):
    return torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _positions(gen, axes, T):
    """Positions of a prompt: the first axis runs far (a long cache), the others over an image's rows and columns."""
    start = torch.randint(0, 100000, (), generator=gen, device=DEV)
    first = start + torch.arange(T, device=DEV)
    rest = torch.randint(0, 64, (max(0, axes - 1), T), generator=gen, device=DEV)
    return torch.cat([first[None], rest]).to(torch.int32)


def _spread_tables(gen, lens, page, W, pages):
    """Block tables [B, W] that hand out random pages, -1 where a request has none."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))] if len(need) < 64 else _before(need), device=DEV)
    at = first[:, None] + torch.arange(W, device=DEV)[None]
    return torch.where(torch.arange(W, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None], order[at.clamp(max=pages - 1)], -1), order, sum(need)


def _before(v):
    total, out = 0, []
    for x in v:
        out.append(total)
        total += x
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + 17)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=TYPES[case["dtype"]])

    if op == "tables":
        ctx, new = _lengths(case)
        page = case["page"]
        last = [c + max(n, 0) for c, n in zip(ctx, new)]
        W = max(-(-x // page) for x in last) + 3
        pages = sum(-(-x // page) for x in last) + 50
        table, order, used = _spread_tables(gen, ctx, page, W, pages)
        ring = torch.zeros(pages, dtype=torch.int32, device=DEV)
        head = int(torch.randint(0, pages, (), generator=gen, device=DEV))
        free = order[used:]
        ring[(head + torch.arange(pages - used, device=DEV)) % pages] = free
        tokens = sum(max(n, 0) for n in new)
        return dict(case=case, ctx=_ints(ctx), new=_ints(new), table=table, ring=ring, state=_ints([head, pages - used]), tokens=-(-tokens // 64) * 64)
    if op == "rotary":
        half = case["part"] // 2
        return dict(case=case, x=normal(case["T"], case["H"], case["d"]), positions=_positions(gen, case["axes"], case["T"]),
                    inv_freq=_inv_freq(half), sections=_sections(half, case["axes"]))
    if op == "write":
        T, Hq, Hkv, d, page = (case[k] for k in ("T", "Hq", "Hkv", "d", "page"))
        qkv = normal(T, Hq + 2 * Hkv, d)  # one projection's output: queries, keys and values are views of it
        slots = torch.randperm(case["pages"] * page, generator=gen, device=DEV)[:T].to(torch.int32)
        axes = case["axes"]
        return dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq : Hq + Hkv], v=qkv[:, Hq + Hkv :], slots=slots,
                    k_pool=normal(case["pages"], Hkv, page, d), v_pool=normal(case["pages"], Hkv, page, d),
                    positions=_positions(gen, axes, T) if axes else None, inv_freq=_inv_freq(d // 2) if axes else None,
                    sections=_sections(d // 2, axes) if axes else None)
    ctx, new = _lengths(case)
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    lens = ctx if case["causal"] else [c + n for c, n in zip(ctx, new)]
    lens = [max(c, n) for c, n in zip(lens, new)] if case["causal"] else lens
    W = max(-(-x // page) for x in lens)
    pages = sum(-(-x // page) for x in lens) + 7
    table, _, _ = _spread_tables(gen, lens, page, W, pages)
    cu = _before(new) + [sum(new)]
    k_pool, v_pool = normal(pages, Hkv, page, d), normal(pages, Hkv, page, d)
    k_pool += 0.5 * normal(1, Hkv, 1, d)  # keys and values around a mean of their head
    v_pool += 0.5 * normal(1, Hkv, 1, d)
    return dict(case=case, q=normal(sum(new), case["Hq"], d), k_pool=k_pool, v_pool=v_pool, table=table, lens=_ints(lens), cu=_ints(cu),
                most=max(new), beta=1.0 / math.sqrt(d))


# --------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "rotary": _own_rotary, "write": _own_write, "attend": _own_attend}[op](state)
    return {"tables": _plain_tables, "rotary": _plain_rotary, "write": _plain_write, "attend": _plain_attend}[op](state)


def _own_tables(s):
    import nystr_coreset_approximate_b200 as wc

    seq_lens, cu_new, positions, slots, ring_state = wc.page_tables(s["ctx"], s["new"], s["table"], s["ring"], s["state"], s["case"]["page"], s["tokens"])
    return dict(seq_lens=seq_lens, cu_new=cu_new, positions=positions, slots=slots, ring_state=ring_state, table=s["table"], ring=s["ring"])


def _own_rotary(s):
    import nystr_coreset_approximate_b200 as wc

    turn = wc.rotary_backward if s["case"]["back"] else wc.rotary
    return turn(s["x"], s["positions"], s["inv_freq"], s["sections"], interleaved=bool(s["case"]["pairs"]))


def _own_write(s):
    import nystr_coreset_approximate_b200 as wc

    if s["positions"] is None:
        wc.paged_write(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"])
        return dict(k_pool=s["k_pool"], v_pool=s["v_pool"])
    q = wc.paged_write(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], q=s["q"], positions=s["positions"], inv_freq=s["inv_freq"],
                       sections=s["sections"])
    return dict(q=q, k_pool=s["k_pool"], v_pool=s["v_pool"])


def _own_attend(s):
    import nystr_coreset_approximate_b200 as wc

    return wc.paged_attend(s["q"], s["k_pool"], s["v_pool"], s["table"], s["lens"], s["cu"], s["beta"], causal=bool(s["case"]["causal"]))


# --------------------------------------------------------------------------- plain forms
def _plain_tables(s):
    page, tokens, table, ring = s["case"]["page"], s["tokens"], s["table"], s["ring"]
    ctx, new = s["ctx"].long(), s["new"].long()
    B, W = table.shape
    P = ring.numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    ends, fresh = new < 0, new.clamp(min=0)
    cu = torch.cat([fresh.new_zeros(1), fresh.cumsum(0)])
    have, want = (ctx + page - 1) // page, (ctx + fresh + page - 1) // page
    # a request gets all the pages that it needs, or it does not advance
    fits = ~ends & (want <= W) & (cu[1:] <= tokens)
    need = torch.where(fits, want - have, 0)
    first = need.cumsum(0) - need
    granted = fits & ((need == 0) | (first + need <= count))
    need = torch.where(granted, need, 0)
    seq = torch.where(ends, 0, torch.where(granted, ctx + fresh, ctx))
    # new pages, request by request, off the ring's head
    col = torch.arange(W, device=DEV)[None]
    takes = (col >= have[:, None]) & (col < (have + need)[:, None])
    table.copy_(torch.where(takes, ring[(head + first[:, None] + col - have[:, None]) % P], table))
    # the pages of requests that end, to the ring's tail
    gives = torch.where(ends, have.clamp(max=W), 0)
    back = ends[:, None] & (col < gives[:, None])
    ring[((head + count + (gives.cumsum(0) - gives)[:, None] + col) % P)[back]] = table[back]
    # the tokens
    t = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    live = t < cu[-1]
    pos = torch.where(live, ctx[b] + t - cu[b], 0)
    at = table[b, (pos // page).clamp(max=W - 1)].long()
    slots = torch.where(live & granted[b] & (at >= 0), at * page + pos % page, -1)
    taken, asked = need.sum(), torch.where(fits, want - have, 0).sum()
    ring_state = torch.stack([(head + taken) % P, count - taken + gives.sum(), asked - taken, (~ends & ~granted).sum()])
    as32 = torch.int32
    return dict(seq_lens=seq.to(as32), cu_new=cu.to(as32), positions=pos.to(as32), slots=slots.to(as32), ring_state=ring_state.to(as32), table=table, ring=ring)


def _turned(x, positions, inv_freq, sections, pairs, sign):
    """x [T, H, d] with its first 2 * half columns rotated; angles in 64 bits (positions run far), the rest in 32."""
    half = inv_freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV), torch.tensor(sections, device=DEV), output_size=half)
    angle = positions.double()[axis].T * inv_freq
    cos, sin = angle.cos().float()[:, None], (sign * angle.sin()).float()[:, None]
    y = x.float()
    part = y[..., : 2 * half]
    a, b = (part[..., 0::2], part[..., 1::2]) if pairs else (part[..., :half], part[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([part, y[..., 2 * half :]], -1).to(x.dtype)


def _plain_rotary(s):
    return _turned(s["x"], s["positions"], s["inv_freq"], s["sections"], s["case"]["pairs"], -1 if s["case"]["back"] else 1)


def _plain_write(s):
    slots, page = s["slots"].long(), s["case"]["page"]
    k, q, told = s["k"], None, s["positions"] is not None
    if told:
        k = _turned(k, s["positions"], s["inv_freq"], s["sections"], 0, 1)
        q = _turned(s["q"], s["positions"], s["inv_freq"], s["sections"], 0, 1)
    keep = slots >= 0
    at = slots[keep]
    s["k_pool"][at // page, :, at % page] = k[keep]
    s["v_pool"][at // page, :, at % page] = s["v"][keep]
    out = dict(k_pool=s["k_pool"], v_pool=s["v_pool"])
    return dict(q=q, **out) if told else out


def _plain_attend(s):
    q, table, lens, cu = s["q"], s["table"].long().clamp(min=0), s["lens"].long(), s["cu"].long()
    (B, W), (P, H, page, d) = table.shape, s["k_pool"].shape
    g, m = q.shape[1] // H, s["most"]
    n = cu[1:] - cu[:-1]
    i = torch.arange(m, device=DEV)
    there = i[None] < n[:, None]
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    Q = q[rows].float().view(B, m, H, g, d).permute(0, 2, 3, 1, 4).reshape(B, H, g * m, d)
    K = s["k_pool"][table].float().permute(0, 2, 1, 3, 4).reshape(B, H, W * page, d)
    V = s["v_pool"][table].float().permute(0, 2, 1, 3, 4).reshape(B, H, W * page, d)
    j = torch.arange(W * page, device=DEV)
    V = V * (j < lens[:, None])[:, None, :, None]
    end = lens[:, None] - n[:, None] + i + 1 if s["case"]["causal"] else lens[:, None].expand(B, m)
    seen = j < end[:, :, None]
    S = torch.matmul(Q, K.transpose(-1, -2)).view(B, H, g, m, W * page)
    S = torch.where(seen[:, None, None], S * s["beta"], -math.inf)
    top = S.amax(-1, keepdim=True)
    E = torch.exp(S - torch.where(torch.isinf(top), 0.0, top)).view(B, H, g * m, W * page)
    O = torch.matmul(E, V) / E.sum(-1, keepdim=True).clamp(min=1e-30)
    return O.view(B, H, g, m, d).permute(0, 3, 1, 2, 4).reshape(B, m, H * g, d)[there].to(q.dtype)


# --------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "tables":
        ctx, new = _lengths(case)
        page = case["page"]
        tokens = -(-sum(max(n, 0) for n in new) // 64) * 64
        moved = sum(-(-c // page) if n < 0 else -(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        return dict(bytes=4 * (4 * case["B"] + 2 * tokens + 2 * moved + 8), flops=0)
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    if op == "rotary":
        n = case["T"] * case["H"]
        return dict(bytes=2 * n * case["d"] * size + 4 * case["axes"] * case["T"], flops=3 * n * case["part"])
    if op == "write":
        heads = 2 * case["Hkv"] + (case["Hq"] if case["axes"] else 0)
        turned = case["Hq"] + case["Hkv"] if case["axes"] else 0
        return dict(bytes=2 * case["T"] * heads * case["d"] * size + 4 * (1 + case["axes"]) * case["T"], flops=3 * case["T"] * turned * case["d"])
    ctx, new = _lengths(case)
    if case["causal"]:
        lens = [max(c, n) for c, n in zip(ctx, new)]
        pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, new))
    else:
        lens = [c + n for c, n in zip(ctx, new)]
        pairs = sum(n * L for L, n in zip(lens, new))
    cached = sum(lens) * case["Hkv"] * 2 + sum(new) * case["Hq"] * 2
    return dict(bytes=cached * case["d"] * size + 4 * sum(-(-L // case["page"]) for L in lens), flops=4 * case["d"] * case["Hq"] * pairs)


# --------------------------------------------------------------------------- exact values, in 64 bits
def _exact_turned(x, positions, inv_freq, sections, pairs, back):
    """Each pair (a, b) as the complex number a + ib, turned by its angle."""
    T, H, _ = x.shape
    half = inv_freq.numel()
    x = x.double()
    out = x.clone()
    start = 0
    for a, n in enumerate(sections):
        for i in range(start, start + n):
            lo, hi = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            angle = positions[a].double() * inv_freq[i]
            turn = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
            z = torch.complex(x[:, :, lo], x[:, :, hi]) * turn
            out[:, :, lo], out[:, :, hi] = z.real, z.imag
        start += n
    return out


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None  # whole numbers: they are compared as they are
    s = prepare(case, seed)
    if op == "rotary":
        return _exact_turned(s["x"], s["positions"], s["inv_freq"], s["sections"], case["pairs"], case["back"])
    if op == "write":
        told = s["positions"] is not None
        turn = (lambda x: _exact_turned(x, s["positions"], s["inv_freq"], s["sections"], 0, 0)) if told else (lambda x: x.double())
        page, slots = case["page"], s["slots"].long()
        P, H, _, d = s["k_pool"].shape
        pools = {}
        for name, rows in (("k_pool", turn(s["k"])), ("v_pool", s["v"].double())):
            flat = s[name].double().transpose(1, 2).reshape(P * page, H, d)
            flat[slots] = rows
            pools[name] = flat.view(P, page, H, d).transpose(1, 2)
        return dict(q=turn(s["q"]), **pools) if told else pools
    q, cu, lens, table = s["q"].double(), s["cu"].tolist(), s["lens"].tolist(), s["table"]
    T, Hq, d = q.shape
    _, H, page, _ = s["k_pool"].shape
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=DEV)
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if L == 0 or n == 0:
            continue
        at = table[b, : -(-L // page)].long()
        end = torch.arange(L - n + 1, L + 1, device=DEV) if case["causal"] else torch.full((n,), L, device=DEV)
        hidden = torch.arange(L, device=DEV)[None] >= end[:, None]
        for h in range(H):
            K, V = (s[name][at, h].reshape(-1, d)[:L].double() for name in ("k_pool", "v_pool"))
            for x in range(h * (Hq // H), (h + 1) * (Hq // H)):
                logit = (q[cu[b] : cu[b + 1], x] @ K.T * s["beta"]).masked_fill(hidden, -math.inf)
                out[cu[b] : cu[b + 1], x] = torch.softmax(logit, -1) @ V
    return out

"""The operators of cached user histories, as cases that can be timed and compared.

A user's history is cached in 4 bits and paged; the candidates (or the user's own next tokens) attend over
it.  Four operators carry that: the page tables of a batch, rotary positions of its queries and keys, the
write of new keys and values into the cache (with the read of cached rows), and the attention over it.
``own`` selects the framework's kernels; otherwise ``run`` computes the same in elementary torch operations.

The cache holds one tile of bytes for each (page of 64 tokens, key/value head), 68 * head_dim bytes:
    K codes   [64 tokens][head_dim/2]        byte c: element 2c in the low 4 bits, 2c+1 in the high ones
    V codes   [head_dim/2][64 tokens]        byte (c, token): elements 2c and 2c+1 of that token
    K scales  [head_dim/32][64]              token t stands at 16*(t//16) + 4*(t%4) + (t//4)%4
    V scales  [head_dim/32][64 tokens]
A code is a sign, two exponent bits and one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6.  32 neighbouring
elements of one token share a scale 2^(byte-127), the smallest power of two (between 2^-125 and 2^125)
that keeps the largest of them at 6 or below.
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # The next token of a ranking request's 59 users: the tables of one small step.
        dict(name="tables-step-59", op="tables", requests=59, tokens=59, longest=4096, leaving=0, spare=5),
        # A large server's step: histories that arrive, grow and leave at once, odd counts.
        dict(name="tables-batch-4096", op="tables", requests=4096, tokens=65000, longest=2048, leaving=255, spare=536),
        # One new token for each of 15 users, every element of a head rotated.
        dict(name="rope-step-15", op="rope", tokens=15, heads=4, kv_heads=4, dim=128, rot=128, layout="half", dtype="bf16", far=4096, scaling="none", backward=False),
        # Long histories taken in at once: frequencies stretched for far positions, shared key heads.
        dict(name="rope-intake-16381", op="rope", tokens=16381, heads=32, kv_heads=8, dim=128, rot=128, layout="half", dtype="bf16", far=1000000, scaling="bands", backward=False),
        # Training: the gradients of a part-rotated head with neighbouring pairs, in 32 bits.
        dict(name="rope-gradient-f32", op="rope", tokens=4097, heads=16, kv_heads=4, dim=64, rot=48, layout="interleaved", dtype="f32", far=30000, scaling="linear", backward=True),
        # One new token for each of 59 users goes into the cache.
        dict(name="write-step-59", op="write", tokens=59, users=59, kv_heads=4, dim=128, dtype="bf16"),
        # Histories are taken in: many pages at once, runs that start and end inside a page.
        dict(name="write-intake-16381", op="write", tokens=16381, users=23, kv_heads=8, dim=128, dtype="bf16"),
        # A ragged intake in 32 bits, small heads.
        dict(name="write-ragged-f32", op="write", tokens=1027, users=15, kv_heads=3, dim=64, dtype="f32"),
        # The smallest call: one query token for each of 15 users over about a thousand cached tokens.
        dict(name="attend-step-15", op="attend", users=15, candidates=15, per_user=1, heads=4, kv_heads=4, queries=1, dim=128, longest=1024, shortest=0, causal=False, shuffled=False),
        # One query token each over long histories, shared key heads: the cache's bytes are what counts.
        dict(name="attend-step-long", op="attend", users=26, candidates=26, per_user=1, heads=32, kv_heads=8, queries=1, dim=128, longest=32000, shortest=500, causal=False, shuffled=False),
        # Ranking: 1024 candidates with 64 query tokens each against 15 users' histories (70:1).
        dict(name="attend-targets-70to1", op="attend", users=15, candidates=1024, per_user=69, heads=4, kv_heads=4, queries=64, dim=128, longest=1024, shortest=777, causal=False, shuffled=False),
        # The users' own new tokens, each seeing the history up to itself: ragged, causal, small heads.
        dict(name="attend-intake-causal", op="attend", users=23, candidates=4001, per_user=174, heads=16, kv_heads=4, queries=1, dim=64, longest=4096, shortest=300, causal=True, shuffled=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "write", "attend", "attend"])
    if op == "tables":
        requests = _spread(rng, 1, 4096)
        return dict(op=op, requests=requests, tokens=_spread(rng, requests, 64000), longest=_spread(rng, 16, 2048),
                    leaving=rng.randrange(0, max(1, requests // 4)), spare=rng.randrange(0, 500))
    if op == "rope":
        kv = rng.choice([1, 2, 3, 4, 8])
        dim = rng.choice([64, 80, 128])
        return dict(op=op, tokens=_spread(rng, 1, 16000), heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim - 16]), layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), far=_spread(rng, 64, 1000000),
                    scaling=rng.choice(["none", "linear", "bands"]), backward=rng.random() < 0.4)
    if op == "write":
        users = _spread(rng, 1, 60)
        return dict(op=op, tokens=_spread(rng, users, 16000), users=users, kv_heads=rng.choice([1, 2, 3, 4, 8]),
                    dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    kv = rng.choice([1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128])
    kind = rng.choice(["step", "step", "targets", "causal"])
    users = _spread(rng, 1, 26)
    if kind == "step":
        longest = _spread(rng, 1, 30000)
        return dict(op="attend", users=users, candidates=users, per_user=1, heads=kv * group, kv_heads=kv, queries=1,
                    dim=dim, longest=longest, shortest=rng.randrange(0, longest + 1), causal=False, shuffled=False)
    longest = _spread(rng, 60, 4000)
    if kind == "targets":
        per = _spread(rng, 1, 60)
        return dict(op="attend", users=min(users, 15), candidates=min(users, 15) * per, per_user=per, heads=kv * min(group, 2),
                    kv_heads=kv, queries=rng.choice([1, 5, 16, 33, 64]), dim=dim, longest=min(longest, 1024),
                    shortest=rng.randrange(0, 60), causal=False, shuffled=rng.random() < 0.5)
    per = min(_spread(rng, 1, 180), longest)
    return dict(op="attend", users=users, candidates=users * per - rng.randrange(0, per), per_user=per, heads=kv * min(group, 4),
                kv_heads=kv, queries=1, dim=dim, longest=longest, shortest=per, causal=True, shuffled=rng.random() < 0.3)


# ---- inputs --------------------------------------------------------------------------------


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _paged(g, lens, width, pages):
    """A block table [users, width] whose used entries are distinct pages in random order; the others are -1."""
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    need = (lens + PAGE - 1) // PAGE
    at = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    used = col < need[:, None]
    return torch.where(used, order[torch.where(used, at[:, None] + col, 0)], -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return globals()["_prepare_" + case["op"]](dict(case), g)


def _prepare_tables(case, g):
    n = case["requests"]
    lens = _lengths(g, n, 0, case["longest"])
    leave = torch.zeros(n, dtype=torch.bool, device=DEV)
    leave[torch.randperm(n, generator=g, device=DEV)[:case["leaving"]]] = True
    stay = max(1, n - case["leaving"])
    counts = torch.full((n,), max(1, case["tokens"] // stay), dtype=torch.int32, device=DEV)
    if case["tokens"] > 2 * stay:   # ragged arrivals; a step gives each request one token
        counts = (torch.rand(n, generator=g, device=DEV) * 2 * case["tokens"] / stay * 0.94).to(torch.int32)
        counts = torch.where(torch.cumsum(counts, 0) <= case["tokens"], counts, 0)
    counts = torch.where(leave, -1, counts).to(torch.int32)
    width = (case["longest"] + case["tokens"] // stay * 2 + 2) // PAGE + 2
    held = int(((lens + PAGE - 1) // PAGE).sum())
    pages = n * (-(-case["longest"] // PAGE) + 1) + -(-case["tokens"] // PAGE) + 7
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    need = (lens + PAGE - 1) // PAGE
    at = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    used = col < need[:, None]
    table = torch.where(used, order[torch.where(used, at[:, None] + col, 0)], -1).to(torch.int32)
    ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    head = pages - 3   # the free pages wrap round the ring's end
    ring[(head + torch.arange(pages - held, device=DEV)) % pages] = order[held:]
    state = torch.tensor([head, pages - held, 0, 0], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    return dict(case=case, lens=lens, counts=counts, table=table, ring=ring, state=state, status=status,
                capacity=case["tokens"] + case["spare"])


def _frequencies(case):
    """theta^(-2i/rot) in 64 bits, stretched for far positions; and the factor on cos and sin."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        f = f / 4.0
    if case["scaling"] == "bands":
        # Wavelengths past 8192 are stretched by 8, those below 2048 are kept, with a ramp between.
        ramp = ((8192 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * ramp + f / 8.0 * (1 - ramp)
        return f.to(DEV), 1.2079
    return f.to(DEV), 1.0


def _prepare_rope(case, g):
    t, h, kv, dim = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    qkv = torch.randn(t, h + 2 * kv, dim, generator=g, device=DEV).to(_dtype(case))
    positions = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
    freq, factor = _frequencies(case)
    return dict(case=case, q=qkv[:, :h], k=qkv[:, h:h + kv], positions=positions, freq=freq, factor=factor)


def _prepare_write(case, g):
    t, users, kv, dim = case["tokens"], case["users"], case["kv_heads"], case["dim"]
    kvs = torch.randn(2, t, kv, dim, generator=g, device=DEV)
    kvs = kvs * torch.exp(torch.randn(2, t, kv, dim // 32, 1, generator=g, device=DEV)).expand(-1, -1, -1, -1, 32).reshape(kvs.shape)
    kvs = kvs.to(_dtype(case))
    # Each user's run of new tokens starts somewhere inside a page and goes on over its pages.
    run = -(-t // users)
    start = _lengths(g, users, 0, 200).long()
    width = (200 + run + PAGE) // PAGE
    pages = users * width + 3
    table = torch.randperm(pages, generator=g, device=DEV)[:users * width].reshape(users, width)
    row = torch.arange(t, device=DEV)
    pos = start[row // run] + row % run
    slots = (table[row // run, pos // PAGE] * PAGE + pos % PAGE).to(torch.int32)
    tiles = torch.zeros(pages, kv, 68 * dim, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    return dict(case=case, k=kvs[0], v=kvs[1], slots=slots, tiles=tiles, status=status)


def _prepare_attend(case, g):
    users, cand, dim, kv = case["users"], case["candidates"], case["dim"], case["kv_heads"]
    lens = _lengths(g, users, case["shortest"], case["longest"])
    width = (case["longest"] + PAGE - 1) // PAGE + 1
    pages = int(((lens + PAGE - 1) // PAGE).sum()) + 5
    table = _paged(g, lens, width, pages)
    tiles = torch.randint(0, 256, (pages, kv, 68 * dim), generator=g, device=DEV, dtype=torch.uint8)
    # Scales of unit-sized values: 2^-2 to 2^0.
    tiles[:, :, 64 * dim:] = torch.randint(125, 128, (pages, kv, 4 * dim), generator=g, device=DEV, dtype=torch.uint8)
    per = case["per_user"]
    mapping = (torch.arange(cand, device=DEV) // per).to(torch.int32)
    positions = None
    if case["causal"]:
        n_new = torch.bincount(mapping.long(), minlength=users)
        rank = torch.arange(cand, device=DEV) - mapping * per
        positions = (lens[mapping.long()] - n_new[mapping.long()] + rank).to(torch.int32)
    if case["shuffled"]:
        order = torch.randperm(cand, generator=g, device=DEV)
        mapping, positions = mapping[order], None if positions is None else positions[order]
    q = torch.randn(cand, case["heads"], case["queries"], dim, generator=g, device=DEV).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    return dict(case=case, q=q, tiles=tiles, table=table, lens=lens, map=mapping, positions=positions, status=status)


# ---- one pass ------------------------------------------------------------------------------


def run(state):
    if own:
        return globals()["_own_" + state["case"]["op"]](state)
    return globals()["_plain_" + state["case"]["op"]](state)


def _own_tables(s):
    from broadcast_gemm_amd import history

    t = history.kv_tables(s["counts"], s["lens"], s["table"], s["ring"], s["state"], s["capacity"], s["status"])
    return dict(slots=t.slots, positions=t.positions, rows=t.rows, starts=t.starts, lens=t.lens, free=t.state[:2],
                table=s["table"], ring=s["ring"])


def _own_rope(s):
    from broadcast_gemm_amd import history

    c = s["case"]
    q, k = history.rope(s["q"], s["k"], s["positions"], s["freq"], layout=c["layout"], factor=s["factor"], inverse=c["backward"])
    return dict(q=q, k=k)


def _own_write(s):
    from broadcast_gemm_amd import history

    history.kv4_write(s["k"], s["v"], s["slots"], s["tiles"], s["status"])
    k, v = history.kv4_read(s["slots"], s["tiles"], s["status"], dtype=s["k"].dtype)
    return dict(k=k, v=v)


def _own_attend(s):
    from broadcast_gemm_amd import history

    return history.kv4_attention(s["q"], s["tiles"], s["table"], s["lens"], s["map"], s["status"], positions=s["positions"])


def _plain_tables(s):
    lens, counts, table, ring = s["lens"].long(), s["counts"].long(), s["table"], s["ring"]
    n_pages, head, free = ring.numel(), s["state"][0].long(), s["state"][1].long()
    new = counts.clamp(min=0)
    ends = torch.cumsum(new, 0)
    have = (lens + PAGE - 1) // PAGE
    take = torch.where(counts >= 0, (lens + new + PAGE - 1) // PAGE - have, 0)
    leave = torch.where(counts < 0, have, 0)
    take_at, leave_at = torch.cumsum(take, 0) - take, torch.cumsum(leave, 0) - leave
    col = torch.arange(table.shape[1], device=DEV)
    fresh = (col >= have[:, None]) & (col < (have + take)[:, None])
    taken = ring[torch.where(fresh, head + take_at[:, None] + col - have[:, None], 0) % n_pages]
    gone = col < leave[:, None]
    # The page of a leaving request goes behind the free ones; the extra place takes what does not leave.
    to = torch.where(gone, (head + free + leave_at[:, None] + col) % n_pages, n_pages)
    ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, to.reshape(-1), table.reshape(-1))[:n_pages])
    table.copy_(torch.where(fresh, taken, table))
    t = torch.arange(s["capacity"], device=DEV)
    row = torch.searchsorted(ends, t, right=True)
    live = t < ends[-1]
    row = torch.where(live, row, 0)
    pos = lens[row] + t - (ends - new)[row]
    slot = table[row, torch.where(live, pos // PAGE, 0)] * PAGE + pos % PAGE
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(slots=i32(torch.where(live, slot, -1)), positions=i32(torch.where(live, pos, -1)), rows=i32(torch.where(live, row, -1)),
                starts=i32(torch.cat([ends.new_zeros(1), ends])), lens=i32(torch.where(counts < 0, 0, lens + new)),
                free=i32(torch.stack([(head + take.sum()) % n_pages, free - take.sum() + leave.sum()])), table=table, ring=ring)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    if c["backward"]:
        sin = -sin

    def turn(x):
        y = x.float()
        r, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        a, b = r.chunk(2, -1) if c["layout"] == "half" else (r[..., 0::2], r[..., 1::2])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([r, rest], -1).to(x.dtype)

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _power(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x):
    """x [..., dim] as codes [..., dim] and scale bytes [..., dim/32]."""
    y = x.float().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    mant, ex = torch.frexp(top)
    e = ex - 3 + (mant > 0.75).to(torch.int32)
    e = torch.where(top > 0, e, -125).clamp(-125, 125)
    y = y * _power(-e)[..., None]
    a = y.abs()
    code = torch.signbit(y).to(torch.uint8) * 8
    for edge, tie in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):   # ties to the even code
        code += ((a >= edge) if tie else (a > edge)).to(torch.uint8)
    return code.flatten(-2), (e + 127).to(torch.uint8)


def _scale_place(t):
    return 16 * (t // 16) + 4 * (t % 4) + (t // 4) % 4


def _parts(tiles):
    """K codes [.., 64, dim/2], V codes [.., dim/2, 64], K scales and V scales [.., dim/32, 64]: views of the tiles."""
    dim = tiles.shape[-1] // 68
    k, v, ks, vs = tiles.split([32 * dim, 32 * dim, 2 * dim, 2 * dim], -1)
    return k.unflatten(-1, (64, dim // 2)), v.unflatten(-1, (dim // 2, 64)), ks.unflatten(-1, (dim // 32, 64)), vs.unflatten(-1, (dim // 32, 64))


def _values(codes, scales):
    """Bytes [..., dim/2] and scale bytes [..., dim/32] as 32-bit values [..., dim]."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=DEV)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    x = level[both.to(torch.int32)]
    return (x.unflatten(-1, (-1, 32)) * _power(scales.to(torch.int32) - 127)[..., None]).flatten(-2)


def _plain_write(s):
    page, t = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    kc, vc, ks, vs = _parts(s["tiles"])
    for x, codes, scales, place in ((s["k"], kc, ks, _scale_place(t)), (s["v"], vc.transpose(-1, -2), vs, t)):
        c, e = _codes(x)
        codes[page, :, t] = c[..., 0::2] | (c[..., 1::2] << 4)
        scales.transpose(-1, -2)[page, :, place] = e
    k = _values(kc[page, :, t], ks.transpose(-1, -2)[page, :, _scale_place(t)])
    v = _values(vc.transpose(-1, -2)[page, :, t], vs.transpose(-1, -2)[page, :, t])
    return dict(k=k.to(s["k"].dtype), v=v.to(s["k"].dtype))


def _plain_attend(s):
    c = s["case"]
    users, kv, per, lq, dim = c["users"], c["kv_heads"], c["per_user"], c["queries"], c["dim"]
    group = c["heads"] // kv
    kc, vc, ks, vs = _parts(s["tiles"][s["table"].clamp(min=0).long()])     # [users, width, kv, ...]
    place = _scale_place(torch.arange(PAGE, device=DEV))
    k = _values(kc, ks.transpose(-1, -2)[..., place, :]).transpose(1, 2).flatten(2, 3)          # [users, kv, keys, dim]
    v = _values(vc.transpose(-1, -2), vs.transpose(-1, -2)).transpose(1, 2).flatten(2, 3)
    keys = k.shape[2]
    # Candidates go beside their user's others: row `rank` of the user's `per` rows.
    m = s["map"].long()
    order = torch.argsort(m, stable=True)
    grouped = m[order]
    rank = torch.empty_like(m)
    rank[order] = torch.arange(m.numel(), device=DEV) - torch.searchsorted(grouped, grouped)
    q = s["q"].new_zeros(users, per, kv, group, lq, dim, dtype=torch.float32)
    q[m, rank] = s["q"].float().unflatten(1, (kv, group))
    q = q.permute(0, 2, 1, 3, 4, 5).reshape(users, kv, per * group * lq, dim)
    limit = s["lens"].long()[:, None].expand(users, per).contiguous()
    if s["positions"] is not None:
        limit[m, rank] = torch.minimum(limit[m, rank], s["positions"].long() + 1)
    seen = torch.arange(keys, device=DEV) < limit.repeat_interleave(group * lq, 1)[:, None, :, None]
    score = torch.where(seen, (q @ k.transpose(-1, -2)) * dim ** -0.5, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, 1.0)   # a row that sees nothing is zero
    o = o.reshape(users, kv, per, group, lq, dim).permute(0, 2, 1, 3, 4, 5)[m, rank]
    return o.flatten(1, 2).to(torch.bfloat16)


# ---- what a pass cannot do without ---------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "tables":
        n, t = case["requests"], case["tokens"] + case["spare"]
        return dict(bytes=4 * (2 * n + n + n + 1 + 3 * t + 2 * (t // PAGE + n)), flops=0)
    if op == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return dict(bytes=n * case["dim"] * size * 2 + case["tokens"] * 4, flops=n * case["rot"] * 3)
    if op == "write":
        size = 2 if case["dtype"] == "bf16" else 4
        n = 2 * case["tokens"] * case["kv_heads"] * case["dim"]
        return dict(bytes=n * size * 2 + 2 * n * 17 // 32 + case["tokens"] * 8, flops=n * 3)
    keys = case["users"] * (case["longest"] + case["shortest"]) / 2
    rows = case["candidates"] * case["heads"] * case["queries"]
    cache = keys * case["kv_heads"] * case["dim"] * 17 / 16
    seen = (case["longest"] + case["shortest"]) / 2 - (case["per_user"] / 2 if case["causal"] else 0)
    return dict(bytes=cache + rows * case["dim"] * 4, flops=rows * seen * case["dim"] * 4)


# ---- the definitions in 64 bits, on the same inputs ----------------------------------------


def exact(case, seed):
    f = globals().get("_exact_" + case["op"])
    return None if f is None else f(prepare(case, seed))


def _exact_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    i = torch.arange(half, device=DEV)
    at = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
    way = -1.0 if c["backward"] else 1.0
    z = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=DEV), way * s["positions"].double()[:, None, None] * s["freq"])
    out = {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        turned = torch.complex(x[..., at[0]], x[..., at[1]]) * z
        x[..., at[0]], x[..., at[1]] = turned.real, turned.imag
        out[name] = x
    return out


def _exact_write(s):
    grid = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    out = {}
    for name in ("k", "v"):
        x = s[name].double().unflatten(-1, (-1, 32))
        top = x.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 6))
        e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 3 * torch.exp2(e), e - 1, e)).clamp(-125, 125)
        y = x.abs() / torch.exp2(e)
        up = torch.searchsorted(grid, y.contiguous()).clamp(max=7)          # the first level at or above
        lo = (up - 1).clamp(min=0)
        to_up, to_lo = grid[up] - y, y - grid[lo]
        pick = torch.where((to_up < to_lo) | ((to_up == to_lo) & (up % 2 == 0)), up, lo)
        out[name] = (torch.sign(x) * grid[pick] * torch.exp2(e)).flatten(-2)
    return out


def _exact_attend(s):
    c = s["case"]
    dim, kv, group = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    signed = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=DEV)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lens, m = s["lens"].tolist(), s["map"]
    token = torch.arange(PAGE, device=DEV)
    for u, n in enumerate(lens):
        mine = (m == u).nonzero().flatten()
        if n == 0 or mine.numel() == 0:
            continue
        tiles = s["tiles"][s["table"][u, :-(-n // PAGE)].long()]             # [pages, kv, bytes]
        b = 64 * dim
        raw_k = tiles[..., :32 * dim].reshape(-1, kv, 64, dim // 2)
        raw_v = tiles[..., 32 * dim:b].reshape(-1, kv, dim // 2, 64).permute(0, 1, 3, 2)
        e_k = tiles[..., b:b + 2 * dim].reshape(-1, kv, dim // 32, 64)[..., _scale_place(token)].permute(0, 1, 3, 2)
        e_v = tiles[..., b + 2 * dim:].reshape(-1, kv, dim // 32, 64).permute(0, 1, 3, 2)
        full = []
        for raw, e in ((raw_k, e_k), (raw_v, e_v)):
            x = torch.empty(*raw.shape[:-1], dim, dtype=torch.float64, device=DEV)
            x[..., 0::2], x[..., 1::2] = signed[(raw % 16).long()], signed[(raw // 16).long()]
            x = x * torch.exp2(e.double() - 127).repeat_interleave(32, -1)
            full.append(x.permute(1, 0, 2, 3).reshape(kv, -1, dim)[:, :n])
        k, v = full
        q = s["q"][mine].double().reshape(-1, kv, group, c["queries"], dim).permute(1, 0, 2, 3, 4)
        shape = q.shape
        score = q.reshape(kv, -1, dim) @ k.transpose(-1, -2) / math.sqrt(dim)
        if s["positions"] is not None:
            past = s["positions"][mine].long().repeat_interleave(group * c["queries"])
            score.masked_fill_(torch.arange(n, device=DEV)[None] > past[:, None], float("-inf"))
        o = torch.softmax(score, -1).nan_to_num(0.0) @ v
        out[mine] = o.reshape(shape).permute(1, 0, 2, 3, 4).reshape(-1, c["heads"], c["queries"], dim)
    return out

"""The operators that train target attention, as cases that can be timed and compared.

The queries of a candidate attend over the keys and values of its user, which all candidates of the user share.
Three operators carry its training: the attention with the statistics that its gradient needs (``attend``), a
training step of it, forward and backward (``step``), and dropout from a counter-based generator, which acts on the
attention's weights and, alone, on activations (``dropout``).  ``own`` selects the framework's kernels; otherwise
``run`` computes the same in elementary torch operations.

Query l of head h of candidate b, with u = map[b] and shared head h // group, sees the tokens t < lens[u] with
t <= positions[b, l] where positions are given.  Candidates whose map entry is -1 are padding: rows of zeros.

Random numbers: a Philox generator of four 32-bit words and 7 rounds (Salmon, Moraes, Dror, Shaw 2011), key = the
seed, last counter word = the offset.  On weights, the counter (2 (t // 32) + (t // 4) % 2, b L_q + l, h, offset)
decides 16 tokens: token t has byte t % 4 of word (t % 32) // 8, and stays where that is at least round(256 p).  On
activations, the counter (n // 8 low, n // 8 high, 2^32 - 1, offset) decides elements 8 (n // 8) .. + 7, 16 bits each
in order; an element stays where they are at least round(65536 p).  What stays is divided by the share that stays.
"""
import math

import torch

own = False

DEV = "cuda"


def _attend(name, op, users, candidates, heads, kv_heads, queries, dim, keys, shortest, causal=False, dropout=0.0, shuffled=False, skewed=False,
            padding=0):
    return dict(name=name, op=op, users=users, candidates=candidates, heads=heads, kv_heads=kv_heads, queries=queries, dim=dim, keys=keys,
                shortest=shortest, causal=causal, dropout=dropout, shuffled=shuffled, skewed=skewed, padding=padding)


def listed():
    return [
        # The smallest call: a few candidates of a few users, one query each, short histories.
        _attend("attend-small", "attend", 4, 37, 4, 4, 1, 128, 130, 20),
        # Ranking batch of 1024 candidates, 64 queries each, 15 users (70:1).
        _attend("attend-targets-70to1", "attend", 15, 1024, 4, 4, 64, 128, 1024, 777),
        # Few rows over long histories, shared heads.
        _attend("attend-long", "attend", 2, 48, 8, 2, 1, 128, 32000, 20001),
        # A training batch in time order: each candidate sees its user's history up to itself; dropout; users without history.
        _attend("attend-causal-dropout", "attend", 59, 4096, 16, 4, 1, 64, 2048, 0, causal=True, dropout=0.1, shuffled=True, padding=5),
        # A small training step: latency counts.
        _attend("step-small", "step", 3, 50, 4, 2, 1, 64, 200, 90, dropout=0.1),
        # The ranking batch as a training step.
        _attend("step-targets-70to1", "step", 15, 1024, 4, 4, 64, 128, 1024, 777),
        # The small batch ratio (10:1) with dropout, odd numbers of queries and keys.
        _attend("step-10to1-dropout", "step", 26, 256, 8, 8, 33, 64, 1023, 300, dropout=0.2, shuffled=True),
        # One query each in time order, shared heads, most candidates with one user.
        _attend("step-causal-skewed", "step", 23, 8001, 16, 4, 1, 128, 1500, 64, causal=True, shuffled=True, skewed=True, padding=3),
        # The smallest activations: one request's user embeddings.
        dict(name="dropout-small", op="dropout", n=15 * 160, dtype="bf16", p=0.1, residual=False),
        # The LCE's output of the ranking batch, 1024 candidates of 96 x 160, added to the residual stream.
        dict(name="dropout-residual", op="dropout", n=1024 * 96 * 160, dtype="bf16", p=0.1, residual=True),
        # A gradient in 32 bits, an odd number of elements (4096 candidates of 96 x 160, and 3).
        dict(name="dropout-gradient-f32", op="dropout", n=4096 * 96 * 160 + 3, dtype="f32", p=0.25, residual=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "step", "step", "dropout"])
    if op == "dropout":
        return dict(op=op, n=_spread(rng, 1, 60_000_000), dtype=rng.choice(["bf16", "f32"]), p=rng.choice([0.05, 0.1, 0.3, 0.5]),
                    residual=rng.random() < 0.5)
    kv = rng.choice([1, 2, 3, 4])
    group = rng.choice([1, 1, 2, 3, 4])
    dim = rng.choice([64, 128])
    users = _spread(rng, 1, 60)
    queries = rng.choice([1, 1, 5, 16, 33, 64])
    keys = _spread(rng, 40, 30000 if queries == 1 and users < 8 else 2000)
    # At most the work of the ranking batch.
    most = max(users, min(9000, int(1.3e8 / (128 * keys * kv * group * queries) * 128 * 2)))
    candidates = _spread(rng, users, max(users, most))
    return _attend(None, op, users, candidates, kv * group, kv, queries, dim, keys, rng.randrange(24, keys + 1), causal=rng.random() < 0.3,
                   dropout=rng.choice([0.0, 0.0, 0.1, 0.3]), shuffled=rng.random() < 0.5, skewed=users <= 20 and rng.random() < 0.3,
                   padding=rng.choice([0, 0, 2]) if candidates > users + 2 else 0)


# ---- inputs --------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = torch.randint(0, 1 << 62, (2,), generator=g, device=DEV) & torch.tensor([-1, 0xFFFFFF], device=DEV)
    if case["op"] == "dropout":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.randn(case["n"], generator=g, device=DEV).to(dtype)
        r = torch.randn(case["n"], generator=g, device=DEV).to(dtype) if case["residual"] else None
        return dict(case=case, x=x, residual=r, rng=rng)
    users, cand, dim, keys = case["users"], case["candidates"], case["dim"], case["keys"]
    b = torch.arange(cand, device=DEV)
    if case["skewed"]:   # two thirds of the candidates belong to user 0
        m = torch.where(b < 2 * cand // 3, 0, b % users)
    else:
        m = b * users // cand
    if case["padding"]:
        m[cand - case["padding"]:] = -1
    if case["shuffled"]:
        m = m[torch.randperm(cand, generator=g, device=DEV)]
    lens = torch.randint(case["shortest"], keys + 1, (users,), generator=g, device=DEV)
    positions = None
    if case["causal"]:   # places in the user's history, most of them within it
        positions = (torch.rand(cand, case["queries"], generator=g, device=DEV) * (lens[m.clamp(min=0)] * 1.1)[:, None]).to(torch.int32)
    bf = lambda *shape: torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    s = dict(case=case, q=bf(cand, case["heads"], case["queries"], dim), k=bf(users, case["kv_heads"], keys, dim),
             v=bf(users, case["kv_heads"], keys, dim), map=m.to(torch.int32), lens=lens.to(torch.int32), positions=positions, rng=rng,
             status=torch.zeros(1, dtype=torch.int32, device=DEV), most=int(torch.bincount(m.clamp(min=0), minlength=users).max()))
    if case["op"] == "step":
        s["do"] = bf(*s["q"].shape)
    return s


# ---- one pass ------------------------------------------------------------------------------


def run(state):
    if own:
        return globals()["_own_" + state["case"]["op"]](state)
    return globals()["_plain_" + state["case"]["op"]](state)


def _own_attend(s):
    from broadcast_gemm_amd import training

    O, lse = training.attention(s["q"], s["k"], s["v"], s["map"], s["status"], lens=s["lens"], positions=s["positions"],
                                dropout=s["case"]["dropout"], rng=s["rng"])
    return dict(O=O, lse=lse)


def _own_step(s):
    from broadcast_gemm_amd import training

    how = dict(lens=s["lens"], positions=s["positions"], dropout=s["case"]["dropout"], rng=s["rng"])
    O, lse = training.attention(s["q"], s["k"], s["v"], s["map"], s["status"], **how)
    dQ, dK, dV = training.attention_backward(s["do"], s["q"], s["k"], s["v"], O, lse, s["map"], s["status"], **how)
    return dict(O=O, dQ=dQ, dK=dK, dV=dV)


def _own_dropout(s):
    from broadcast_gemm_amd import training

    return training.dropout(s["x"], s["case"]["p"], s["rng"], residual=s["residual"])


_LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, seed):
    """Four words of the generator, in int64 tensors; products wrap, and their bits 32 to 63 are the high word all the same."""
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c0, c1, c2, c3


def _kept(s, row, head, keys):
    """Which weights [..., keys] stay, for rows given by their number b L_q + l and head [...]."""
    call = torch.arange(-(-keys // 32) * 2, device=DEV)
    words = _philox(call, row[..., None], head[..., None], s["rng"][1] & _LOW, s["rng"][0])
    edge = round(256 * s["case"]["dropout"])
    words = torch.stack([w.expand(*row.shape, call.numel()) for w in words], -1).unflatten(-2, (-1, 2)).transpose(-1, -2)   # [.., 32s, word, half]
    return torch.stack([((words >> (8 * i)) & 255) >= edge for i in range(4)], -1).flatten(-4)[..., :keys]


def _weights(s):
    """Rows beside their user's others: q [users, kv, rows, dim], the weights and lse there, what stays, and how rows go there and back."""
    c = s["case"]
    users, kv, lq, dim, per, keys = c["users"], c["kv_heads"], c["queries"], c["dim"], s["most"], c["keys"]
    group, cand = c["heads"] // kv, c["candidates"]
    m = s["map"].long()
    order = torch.argsort(m, stable=True)
    grouped = m[order]
    rank = torch.empty_like(m)
    rank[order] = torch.arange(cand, device=DEV) - torch.searchsorted(grouped, grouped)
    # Padding goes to a place of its own behind the last user.
    to = torch.where(m >= 0, m * per + rank, users * per)

    def there(x):   # [cand, heads, lq, ...] -> [users, kv, per * group * lq, ...]
        y = x.new_zeros(users * per + 1, *x.shape[1:], dtype=torch.float32 if x.is_floating_point() else x.dtype)
        y[to] = x.to(y.dtype)
        y = y[:-1].unflatten(0, (users, per)).unflatten(2, (kv, group))
        return y.transpose(1, 2).flatten(2, 4)

    def back(x):
        y = x.unflatten(2, (per, group, lq)).transpose(1, 2).flatten(2, 3).flatten(0, 1)
        return torch.cat([y, torch.zeros_like(y[:1])])[to]

    limit = s["lens"].long().clamp(0, keys)[m.clamp(min=0)][:, None, None].expand(cand, c["heads"], lq)
    if s["positions"] is not None:
        limit = torch.minimum(limit, s["positions"].long()[:, None] + 1)
    q, k = there(s["q"]), s["k"].float()
    seen = torch.arange(keys, device=DEV) < there(limit.contiguous())[..., None]
    score = torch.where(seen, q @ k.transpose(-1, -2) * dim ** -0.5, float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    p = p / torch.where(total > 0, total, 1.0)   # a row that sees nothing is zero
    z = None
    if c["dropout"]:
        row = (torch.arange(cand, device=DEV)[:, None] * lq + torch.arange(lq, device=DEV))[:, None].expand(cand, c["heads"], lq)
        head = torch.arange(c["heads"], device=DEV)[:, None].expand(cand, c["heads"], lq)
        z = _kept(s, there(row.contiguous()), there(head.contiguous()), keys).to(torch.float32) * (256 / (256 - round(256 * c["dropout"])))
    return q, p, lse, z, there, back


def _plain_attend(s):
    _, p, lse, z, _, back = _weights(s)
    o = (p if z is None else p * z) @ s["v"].float()
    lse = torch.where(s["map"][:, None, None] >= 0, back(lse), float("-inf"))
    return dict(O=back(o).to(torch.bfloat16), lse=lse)


def _plain_step(s):
    scale = s["case"]["dim"] ** -0.5
    q, p, _, z, there, back = _weights(s)
    k, v, do = s["k"].float(), s["v"].float(), there(s["do"])
    pz = p if z is None else p * z
    dp = do @ v.transpose(-1, -2)
    dp = dp if z is None else dp * z
    ds = p * (dp - (p * dp).sum(-1, keepdim=True))
    bf = lambda x: x.to(torch.bfloat16)  # noqa: E731
    return dict(O=bf(back(pz @ v)), dQ=bf(back(ds @ k * scale)), dK=bf(ds.transpose(-1, -2) @ q * scale), dV=bf(pz.transpose(-1, -2) @ do))


def _plain_dropout(s):
    x, edge = s["x"], round(65536 * s["case"]["p"])
    call = torch.arange(-(-x.numel() // 8), device=DEV)
    words = torch.stack(_philox(call & _LOW, call >> 32, _LOW, s["rng"][1] & _LOW, s["rng"][0]), -1)
    kept = (torch.stack([words & 0xFFFF, words >> 16], -1) >= edge).flatten()[:x.numel()]
    y = torch.where(kept, x.float() * (65536 / (65536 - edge)), 0.0)
    return (y if s["residual"] is None else s["residual"].float() + y).to(x.dtype)


# ---- what a pass cannot do without ---------------------------------------------------------


def work(case):
    if case["op"] == "dropout":
        return dict(bytes=case["n"] * (2 if case["dtype"] == "bf16" else 4) * (3 if case["residual"] else 2), flops=2 * case["n"])
    c = case
    rows = (c["candidates"] - c["padding"]) * c["heads"] * c["queries"]
    seen = (c["keys"] + c["shortest"]) / 2
    cache = c["users"] * c["kv_heads"] * seen * c["dim"] * 2
    seen = seen * 0.55 if c["causal"] else seen
    if c["op"] == "attend":
        return dict(bytes=2 * cache + rows * (4 * c["dim"] + 4), flops=4 * rows * seen * c["dim"])
    return dict(bytes=4 * cache + rows * 8 * c["dim"], flops=14 * rows * seen * c["dim"])


# ---- the definitions in 64 bits, on the same inputs ----------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_dropout(s) if case["op"] == "dropout" else _exact_attention(s)


def _times(a, b):
    """High and low word of the product of 32-bit numbers, by halves."""
    a1, a0, b1, b0 = a // 65536, a % 65536, b // 65536, b % 65536
    mid = a1 * b0 + (a0 * b0) // 65536
    mid2 = a0 * b1 + mid % 65536
    return a1 * b1 + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (a0 * b0) % 65536


def _bytes_of(counter, rng):
    """The 16 bytes, in order, that the generator gives for counters [..., 4]: the definition, round by round."""
    seed, offset = rng.tolist()
    x = [counter[..., i] for i in range(3)] + [torch.full_like(counter[..., 0], offset % 2 ** 32)]
    for r in range(7):
        keys = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        h0, l0 = _times(x[0], 0xD2511F53)
        h1, l1 = _times(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ keys[0], l1, h0 ^ x[3] ^ keys[1], l0]
    return torch.stack([w // 256 ** i % 256 for w in x for i in range(4)], -1)


def _exact_dropout(s):
    n, p = s["x"].numel(), s["case"]["p"]
    call = torch.arange((n + 7) // 8, device=DEV)
    b = _bytes_of(torch.stack([call % 2 ** 32, call // 2 ** 32, torch.full_like(call, 2 ** 32 - 1)], -1), s["rng"])
    stays = (b[:, 0::2] + 256 * b[:, 1::2]).reshape(-1)[:n] >= round(65536 * p)
    y = s["x"].double() * stays / (1 - round(65536 * p) / 65536)
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_attention(s):
    c = s["case"]
    heads, kv, lq, dim, step = c["heads"], c["kv_heads"], c["queries"], c["dim"], c["op"] == "step"
    group, edge = heads // kv, round(256 * c["dropout"])
    O = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    dQ, dK, dV = torch.zeros_like(O), torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["k"].shape, dtype=torch.float64, device=DEV)
    for u, n in enumerate(s["lens"].tolist()):
        mine = (s["map"] == u).nonzero().flatten()
        if n == 0 or mine.numel() == 0:
            continue
        token = torch.arange(n, device=DEV)
        past = torch.full((mine.numel(), lq), n - 1, device=DEV)
        if s["positions"] is not None:
            past = s["positions"][mine].long().clamp(max=n - 1)
        for h in range(heads):
            q = s["q"][mine, h].double().reshape(-1, dim).requires_grad_(step)
            k, v = (s[x][u, h // group, :n].double().requires_grad_(step) for x in ("k", "v"))
            with torch.set_grad_enabled(step):
                score = (q @ k.T / math.sqrt(dim)).masked_fill(token > past.reshape(-1, 1), -math.inf)
                l = torch.logsumexp(score, -1)
                w = torch.exp(score - l[:, None])
                if edge:
                    row = (mine[:, None] * lq + torch.arange(lq, device=DEV)).reshape(-1, 1).expand(-1, n)
                    call = torch.arange(2 * (-(-n // 32)), device=DEV).expand(row.shape[0], -1)
                    b = _bytes_of(torch.stack([call, row[:, :1].expand_as(call), torch.full_like(call, h)], -1), s["rng"]).to(torch.uint8)
                    at = (2 * (token // 32) + token // 4 % 2) * 16 + 4 * (token % 32 // 8) + token % 4
                    w = w * (b.flatten(1)[:, at] >= edge) / (1 - edge / 256)
                o = w @ v
            O[mine, h], lse[mine, h] = o.detach().reshape(-1, lq, dim), l.detach().reshape(-1, lq)
            if step:
                dq, dk, dv = torch.autograd.grad(o, (q, k, v), s["do"][mine, h].double().reshape(-1, dim))
                dQ[mine, h] = dq.reshape(-1, lq, dim)
                dK[u, h // group, :n] += dk
                dV[u, h // group, :n] += dv
    return dict(O=O, dQ=dQ, dK=dK, dV=dV) if step else dict(O=O, lse=lse)

"""Plain 64-bit forms of attention's training and of dropout, on the CPU, for their tests, with bounds on what the
kernels may be off."""
import numpy as np

U24 = 2.0 ** -24            # half a step of float32
B8 = 2.0 ** -8              # half a step of bf16


def philox(counter, key, rounds=7):
    """Words [..., 4] of the generator for counters [..., 4] (uint64 arrays of 32-bit values)."""
    c = [np.asarray(x, np.uint64) for x in np.moveaxis(np.asarray(counter, np.uint64), -1, 0)]
    k = [np.uint64(int(key) & 0xFFFFFFFF), np.uint64((int(key) >> 32) & 0xFFFFFFFF)]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ k[0], b & low, (a >> half) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, -1)


def weights_kept(rows, head, keys, p, rng):
    """[rows, keys] of truth: which weights of the queries numbered b L_q + l stay."""
    t = np.arange(keys)
    n = 2 * (-(-keys // 32))
    counter = np.zeros((len(rows), n, 4), np.uint64)
    counter[..., 0] = np.arange(n)
    counter[..., 1] = np.asarray(rows)[:, None]
    counter[..., 2] = head
    counter[..., 3] = int(rng[1]) & 0xFFFFFFFF
    words = philox(counter, rng[0])
    word = words[:, 2 * (t // 32) + (t // 4) % 2, (t % 32) // 8]
    return ((word >> (8 * (t % 4)).astype(np.uint64)) & np.uint64(255)) >= round(256 * p)


def elements_kept(n, p, rng):
    counter = np.zeros((-(-n // 8), 4), np.uint64)
    counter[:, 0] = np.arange(len(counter)) & 0xFFFFFFFF
    counter[:, 1] = np.arange(len(counter)) >> 32
    counter[:, 2] = 0xFFFFFFFF
    counter[:, 3] = int(rng[1]) & 0xFFFFFFFF
    words = philox(counter, rng[0])
    return np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(-1)[:n] >= round(65536 * p)


def attention(Q, K, V, mp, lens=None, positions=None, scale=0.0, dropout=0.0, rng=None, dO=None):
    """By definition, in float64 arrays: a dict of O, lse and, with dO, dQ, dK, dV; and under "off" how far a kernel may be from each:

    a score by (dim + 4) 2^-24 of the sum of its products' sizes (a float32 sum of exact products, the scale, the exponent's
    argument), a weight by that and 2^-21 (exp2, the row's sum) and, where it is an operand, by half a step of bf16; dP like a score; D
    by what O is off, taken with dO; sums by the number of their terms times 2^-24.  Outputs round once more (``within``)."""
    B_c, H_q, L_q, dim = Q.shape
    B_u, H_kv, L_kv, _ = K.shape
    scale = scale or dim ** -0.5
    edge = round(256 * dropout)
    out = dict(O=np.zeros_like(Q), lse=np.full(Q.shape[:3], -np.inf))
    off = dict(O=np.zeros_like(Q), lse=np.zeros(Q.shape[:3]))
    if dO is not None:
        for n, x in (("dQ", Q), ("dK", K), ("dV", V)):
            out[n], off[n] = np.zeros_like(x), np.zeros_like(x)
    for b in range(B_c):
        u = int(mp[b])
        if not 0 <= u < B_u:
            continue
        n_u = L_kv if lens is None else min(max(int(lens[u]), 0), L_kv)
        for h in range(H_q):
            k, v = K[u, h // (H_q // H_kv), :n_u], V[u, h // (H_q // H_kv), :n_u]
            limit = np.full(L_q, n_u) if positions is None else np.clip(positions[b].astype(np.int64) + 1, 0, n_u)
            live = limit > 0
            if not live.any():
                continue
            q = Q[b, h][live]
            seen = np.arange(n_u) < limit[live][:, None]
            s = np.where(seen, scale * (q @ k.T), -np.inf)
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(-1, keepdims=True)
            p = e / total
            z = np.ones_like(p)
            if edge:
                z = weights_kept(b * L_q + np.flatnonzero(live), h, n_u, dropout, rng) * (256 / (256 - edge))
            o = (p * z) @ v
            # Each weight's score, and that of the row's largest.
            s_off = np.where(seen, scale * (np.abs(q) @ np.abs(k).T), 0.0)
            s_off = (dim + 4) * U24 * (s_off + s_off.max(-1, keepdims=True))
            rel = s_off + 2.0 ** -21 + n_u * U24
            o_off = (p * z * (B8 + 2 * rel)) @ np.abs(v)
            out["O"][b, h][live], off["O"][b, h][live] = o, o_off
            out["lse"][b, h][live] = (top + np.log(total))[:, 0]
            off["lse"][b, h][live] = rel.max(-1) + 4 * U24 * np.abs((top + np.log(total))[:, 0])
            if dO is None:
                continue
            g = dO[b, h][live]
            dp = (g @ v.T) * z
            dp_off = (dim + 4) * U24 * (np.abs(g) @ np.abs(v).T) * z
            d = (g * o).sum(-1, keepdims=True)
            d_off = (np.abs(g) * (o_off + B8 * (np.abs(o) + o_off))).sum(-1, keepdims=True) + (p * (2 * rel * np.abs(dp) + dp_off)).sum(-1, keepdims=True)
            d_off += (dim + n_u) * U24 * (np.abs(g * o).sum(-1, keepdims=True) + (p * np.abs(dp)).sum(-1, keepdims=True))
            ds = p * (dp - d)
            ds_off = p * ((B8 + 2 * rel) * np.abs(dp - d) + (1 + B8 + 2 * rel) * (dp_off + d_off))
            hk = h // (H_q // H_kv)
            rows = B_c * L_q * U24   # dK and dV sum over these
            out["dQ"][b, h][live] = scale * ds @ k
            off["dQ"][b, h][live] = scale * (ds_off + n_u * U24 * np.abs(ds)) @ np.abs(k)
            out["dK"][u, hk, :n_u] += scale * ds.T @ q
            off["dK"][u, hk, :n_u] += scale * (ds_off + rows * np.abs(ds)).T @ np.abs(q)
            out["dV"][u, hk, :n_u] += (p * z).T @ g
            off["dV"][u, hk, :n_u] += (p * z * (B8 + 2 * rel + rows)).T @ np.abs(g)
    out["off"] = off
    return out


def within(got, want, off, half_step):
    """Whether every value is within its bound and one rounding to the output's type; and the largest share of the bound."""
    bound = off * (1 + half_step) + half_step * np.abs(want) + 1e-37
    share = np.abs(got - want) / bound
    return bool((share <= 1).all()), float(np.nan_to_num(share, nan=np.inf).max(initial=0.0))

"""Plain 64-bit forms of the cached-history operators, on the CPU, for their tests."""
import math

import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
PAGE = 64


def half_step(dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def scale_place(t):
    return 16 * (t // 16) + 4 * (t % 4) + (t // 4) % 4


def encode(x):
    """x [..., dim] float64 (finite) -> codes [..., dim] and scale bytes [..., dim/32] by definition."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(y).max(-1)
    e = np.full(top.shape, -125)
    for ex in range(-125, 125):                  # the smallest exponent that keeps the largest value at 6 or below
        e = np.where(top > 6.0 * 2.0 ** ex, ex + 1, e)
    a = np.minimum(np.abs(y) / 2.0 ** e[..., None].astype(float), 6.0)
    d = np.abs(a[..., None] - LEVELS)
    near = d.min(-1, keepdims=True)
    tied = d == near                              # two levels at a tie: the even code
    pick = np.where(tied & (np.arange(8) % 2 == 0), 2, np.where(tied, 1, 0)).argmax(-1)
    code = pick + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), (e + 127).astype(np.uint8)


def decode(codes, scales):
    x = np.where(codes >= 8, -1.0, 1.0) * LEVELS[codes & 7]
    return (x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32) * 2.0 ** (scales[..., None].astype(float) - 127)).reshape(x.shape)


def put(tiles, k, v, slots):
    """Write rows into tiles (numpy uint8 [pages, H, 68*dim]) at their slots."""
    dim = tiles.shape[2] // 68
    for r, slot in enumerate(slots):
        if slot < 0:
            continue
        page, t = divmod(int(slot), PAGE)
        kc, ks = encode(k[r])
        vc, vs = encode(v[r])
        for h in range(tiles.shape[1]):
            w = tiles[page, h]
            w[t * dim // 2:(t + 1) * dim // 2] = kc[h, 0::2] | (kc[h, 1::2] << 4)
            w[32 * dim:64 * dim].reshape(dim // 2, 64)[:, t] = vc[h, 0::2] | (vc[h, 1::2] << 4)
            w[64 * dim:66 * dim].reshape(dim // 32, 64)[:, scale_place(t)] = ks[h]
            w[66 * dim:].reshape(dim // 32, 64)[:, t] = vs[h]


def put_all(tiles, k, v, slots):
    """``put`` for distinct slots, all rows at once."""
    n, H, size = tiles.shape
    dim = size // 68
    live = slots >= 0
    page, t = np.divmod(slots[live].astype(int), PAGE)
    for x, codes, scales, place in ((k, tiles[..., :32 * dim].reshape(n, H, 64, dim // 2).swapaxes(2, 3), tiles[..., 64 * dim:66 * dim], scale_place(t)),
                                    (v, tiles[..., 32 * dim:64 * dim].reshape(n, H, dim // 2, 64), tiles[..., 66 * dim:], t)):
        scales = scales.reshape(n, H, dim // 32, 64)
        assert np.shares_memory(codes, tiles) and np.shares_memory(scales, tiles)
        c, s = encode(x[live])
        codes[page, :, :, t] = c[..., 0::2] | (c[..., 1::2] << 4)
        scales[page, :, :, place] = s


def rows_of(tiles):
    """K and V values [pages, H, 64, dim] float64 that tiles hold."""
    n, H, size = tiles.shape
    dim = size // 68
    t = np.arange(64)
    kb = tiles[..., :32 * dim].reshape(n, H, 64, dim // 2)
    vb = tiles[..., 32 * dim:64 * dim].reshape(n, H, dim // 2, 64).swapaxes(2, 3)
    ks = tiles[..., 64 * dim:66 * dim].reshape(n, H, dim // 32, 64)[..., scale_place(t)].swapaxes(2, 3)
    vs = tiles[..., 66 * dim:].reshape(n, H, dim // 32, 64).swapaxes(2, 3)
    out = []
    for b, s in ((kb, ks), (vb, vs)):
        codes = np.empty((n, H, 64, dim), np.uint8)
        codes[..., 0::2], codes[..., 1::2] = b & 15, b >> 4
        out.append(decode(codes, s))
    return out


def attend(Q, k, v, table, lens, mp, positions, scale=None):
    """O [B_c, H_q, L_q, dim] float64 and an elementwise bound on the kernel's error before its last rounding.

    k, v [pages, H, 64, dim] float64 of the cache's pages.  The kernel's own steps, per row with weights
    p_t: the weights reach the products as bf16, numerator and sum alike (each off by at most half a step h of
    bf16, so their quotient by 2 h of A = sum p|v| / sum p); scores are float32 sums of dim products
    (dim 2^-24 of scale * sum |q||k|) times a float32 constant (2^-23 of the score), which a weight takes over
    twice (score and maximum), and its exp2 adds 2^-22; float32 sums over the tokens and splits add
    (tokens + 16) 2^-24.  All act on A."""
    B_c, H_q, L_q, dim = Q.shape
    H = k.shape[1]
    G = H_q // H
    scale = dim ** -0.5 if scale is None else scale
    O = np.zeros(Q.shape)
    bound = np.zeros(Q.shape)
    for b in range(B_c):
        u = b if mp is None else int(mp[b])
        if not 0 <= u < len(lens):
            continue
        n = int(lens[u])
        if n == 0:
            continue
        pages = table[u][:-(-n // PAGE)]
        K = k[pages].transpose(1, 0, 2, 3).reshape(H, -1, dim)[:, :n]
        V = v[pages].transpose(1, 0, 2, 3).reshape(H, -1, dim)[:, :n]
        for hq in range(H_q):
            for l in range(L_q):
                m = n if positions is None else min(n, max(0, int(positions[b, l]) + 1))
                if m == 0:
                    continue
                q, Kh, Vh = Q[b, hq, l], K[hq // G, :m], V[hq // G, :m]
                s = scale * (Kh @ q)
                p = np.exp(s - s.max())
                p /= p.sum()
                O[b, hq, l] = p @ Vh
                A = p @ np.abs(Vh)
                size = scale * (np.abs(Kh) @ np.abs(q)).max()
                bound[b, hq, l] = A * (2 * half_step(torch.bfloat16) + 2 * (size * (dim * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -22)
                                       + (m + 16) * 2.0 ** -24)
    return O, bound


def turn(x, positions, freq, layout, factor=1.0, inverse=False):
    """x [T, H, dim] float64 turned by positions (ints) times freq (float64), and a bound on the kernel's error.

    The kernel's angle in turns is off by 3 half steps of float64 of the unreduced angle, plus half a step of
    float32 at most 2^-26 turns after the reduction; sine and cosine and the rotation in float32 add at most 6
    half steps of float32 of |a| + |b|.  This form's own angle is off by 2 half steps of float64."""
    rot = 2 * len(freq)
    angle = positions[:, None].astype(float) * freq
    c, s = np.cos(angle)[:, None] * factor, np.sin(angle)[:, None] * factor * (-1 if inverse else 1)
    at = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y, bound = x.copy(), np.zeros(x.shape)
    a, b = x[..., at[0]], x[..., at[1]]
    y[..., at[0]], y[..., at[1]] = a * c - b * s, a * s + b * c
    size = (np.abs(a) + np.abs(b)) * abs(factor)
    off = size * ((5 * 2.0 ** -53 * np.abs(angle) + 2 * math.pi * 2.0 ** -26)[:, None] + 6 * 2.0 ** -24)
    bound[..., at[0]] = bound[..., at[1]] = off
    return y, bound


def tables(counts, lens, table, ring, head, free, capacity, P=PAGE):
    """One step by the definition, one token after the other: (slots, positions, rows, starts, lens, head, free) with
    table and ring changed in place; None if the step does not fit (nothing changed)."""
    N, width = len(ring), table.shape[1]
    new = [max(0, int(c)) for c in counts]
    need = [-(-(int(n) + c) // P) - -(-int(n) // P) for n, c in zip(lens, new)]
    if sum(new) > capacity or sum(need) > free or any(int(n) + c > width * P for n, c in zip(lens, new)):
        return None
    slots, positions, rows = (np.full(capacity, -1, np.int32) for _ in range(3))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = np.array([0 if c < 0 else n + c for n, c in zip(lens, counts)], np.int32)
    at, tail, t = head, head + free, 0
    gone = []
    for i, (n, c) in enumerate(zip(lens, counts)):
        n = int(n)
        if c < 0:
            gone += [table[i, p] for p in range(-(-n // P))]
            continue
        for pos in range(n, n + int(c)):
            if pos % P == 0:
                table[i, pos // P] = ring[at % N]
                at += 1
            slots[t], positions[t], rows[t] = table[i, pos // P] * P + pos % P, pos, i
            t += 1
    for j, page in enumerate(gone):
        ring[(tail + j) % N] = page
    return slots, positions, rows, starts, out, at % N, free - (at - head) + len(gone)

"""Cached user histories: target attention for users whose keys and values are kept between requests.

``FaPlan`` attends over dense K and V that the caller holds per request.  Here a user's history lives in a
cache of 4-bit codes, in pages of 64 tokens that a block table names; it grows by tokens and has a length of
its own.  The calls bind the C ABI (``ikbo_kv_*``, ``ikbo_rope``, ``ikbo_kv4_*`` in ``include/ikbo.h``, which
states formulas and layouts); every step runs in the library's HIP kernels, there is no CPU path.

    t = kv_tables(counts, lens, table, ring, state, capacity, status)     # pages, slots, positions, rows of a step
    q, k = rope(q, k, t.positions, freq)                                  # rotary positions (rope_frequencies)
    kv4_write(k, v, t.slots, tiles, status)                               # into the cache
    O = kv4_attention(Q, tiles, table, t.lens, map, status)               # candidates over their users' histories

``UserHistories`` owns the cache and its tables and runs these in order.

Buffers.  Nothing is kept between calls: outputs and the attention's workspace come from torch's allocator on
the stream the call runs on (the current one, or ``stream``), so calls on several streams or devices, and
captured graphs, share nothing but the tensors they are given.  Conditions that only the device sees set bits of
``status`` (an int32 tensor of one element, zeroed once); ``kv_status`` waits, returns and clears them.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import IKBO_ERR_INVALID_ARG, IKBO_OK, IkboError, lib

PAGE = 64                  # tokens per page of the 4-bit cache
MAX_USERS = 4096
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class _TablesArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("counts", "lens", "lens_out", "block_table", "ring", "state", "state_out", "slots", "positions",
                                    "rows", "starts", "status")]
                + [("table_stride", _i64)] + [(n, _i32) for n in ("B_u", "max_pages", "num_pages", "page_size", "capacity")])


class _RopeArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "q_out", "k_out", "positions", "freq")]
                + [(n, _i64) for n in ("q_token", "q_head", "k_token", "k_head", "q_out_token", "q_out_head", "k_out_token", "k_out_head")]
                + [(n, _i32) for n in ("T", "H_q", "H_k", "head_dim", "rot_dim", "layout", "dtype", "inverse")]
                + [("factor", ctypes.c_float)])


class _RowsArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("k", "v", "slots", "tiles", "status")]
                + [(n, _i64) for n in ("k_token", "k_head", "v_token", "v_head")]
                + [(n, _i32) for n in ("T", "H_kv", "head_dim", "num_pages", "dtype")])


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("Q", "O", "tiles", "block_table", "lens", "map", "positions", "status", "workspace")]
                + [(n, _i64) for n in ("workspace_bytes", "q_cand", "q_head", "q_query", "o_cand", "o_head", "o_query", "table_stride")]
                + [(n, _i32) for n in ("B_u", "B_c", "H_q", "H_kv", "L_q", "head_dim", "max_pages", "num_pages")]
                + [("scale", ctypes.c_float)])


def _check(status: int, what: str) -> None:
    if status != IKBO_OK:
        raise IkboError(status, what)


@contextlib.contextmanager
def _on_device_and_stream(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            with torch.cuda.stream(s):
                yield s.cuda_stream


def _run(device, stream, call):
    """call(stream handle) with ``device`` current and allocations on the stream."""
    if stream is None and torch.cuda.current_device() == device.index:
        return call(torch.cuda.current_stream().cuda_stream)
    with _on_device_and_stream(device, stream) as handle:
        return call(handle)


def _ints(device, **tensors) -> None:
    for name, t in tensors.items():
        if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor on {device}")


def _table(device, table) -> None:
    if table.dtype != torch.int32 or table.device != device or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"the block table must be an int32 tensor [users, pages] with contiguous rows on {device}")


def _status(device, status) -> None:
    if status.dtype != torch.int32 or status.device != device or status.numel() != 1:
        raise ValueError(f"status must be an int32 tensor of one element on {device}")


def _shapes(ok: bool, what: str) -> None:
    if not ok:
        raise IkboError(IKBO_ERR_INVALID_ARG, what)


def _device(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return t.device


def kv_status(status, stream=None) -> int:
    """Wait for the stream, then return and clear the condition recorded in ``status`` (an IKBO_* code)."""
    device = _device(status)
    _status(device, status)
    return _run(device, stream, lambda s: lib().ikbo_kv_status(status.data_ptr(), s))


class StepTables(NamedTuple):
    slots: torch.Tensor        # [capacity] page * page_size + offset, -1 behind the last token
    positions: torch.Tensor    # [capacity] place in the history, -1 behind the last token
    rows: torch.Tensor         # [capacity] the token's request, -1 behind the last token
    starts: torch.Tensor       # [B_u + 1] the requests' first rows
    lens: torch.Tensor         # [B_u] lengths after the step
    state: torch.Tensor        # [4] ring head and free pages after the step


def kv_tables(counts, lens, block_table, ring, state, capacity: int, status, page_size: int = PAGE, in_place: bool = False,
              out: Optional[StepTables] = None, stream=None) -> StepTables:
    """Page tables, slots, positions and rows of one step (``ikbo_kv_tables``).

    ``block_table`` and ``ring`` are updated in place; ``lens`` and ``state`` too if ``in_place``, otherwise new
    tensors hold them after the step.  ``out`` may supply the result's tensors (then they are what is written)."""
    device = _device(lens)
    _ints(device, counts=counts, lens=lens, ring=ring, state=state)
    _table(device, block_table)
    _status(device, status)
    B = lens.numel()
    _shapes(counts.numel() == B and block_table.shape[0] == B and state.numel() == 4, "inconsistent shapes")

    def call(s):
        if out is None:
            rows = torch.empty((3, capacity), dtype=torch.int32, device=device)
            new = (lens, state) if in_place else (torch.empty_like(lens), torch.empty_like(state))
            t = StepTables(rows[0], rows[1], rows[2], torch.empty(B + 1, dtype=torch.int32, device=device), *new)
        else:
            t = StepTables(*out)
            _ints(device, slots=t.slots, positions=t.positions, rows=t.rows, starts=t.starts, lens_out=t.lens, state_out=t.state)
            _shapes(all(x.numel() == capacity for x in t[:3]) and t.starts.numel() == B + 1 and t.lens.numel() == B
                    and t.state.numel() == 4, "out has other shapes")
        args = _TablesArgs(counts.data_ptr(), lens.data_ptr(), t.lens.data_ptr(), block_table.data_ptr(), ring.data_ptr(), state.data_ptr(),
                           t.state.data_ptr(), t.slots.data_ptr(), t.positions.data_ptr(), t.rows.data_ptr(), t.starts.data_ptr(),
                           status.data_ptr(), block_table.stride(0), B, block_table.shape[1], ring.numel(), page_size, capacity)
        _check(lib().ikbo_kv_tables(ctypes.byref(args), s), "ikbo_kv_tables")
        return t

    return _run(device, stream, call)


def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: Optional[dict] = None, device="cuda") -> Tuple[torch.Tensor, float]:
    """Radians per position of the rot_dim/2 pairs, theta^(-2i/rot_dim) in float64, and the factor on cos and sin.

    ``scaling`` stretches them for contexts longer than the trained one, by ``factor``:
      {"kind": "linear", "factor": s}      every frequency divided by s
      {"kind": "theta", "factor": s}       theta times s^(rot_dim/(rot_dim-2)): the slowest pair is divided by s
      {"kind": "turns", "factor": s, "context": n, "low": a, "high": b}
            pairs that turn more than b times over n trained positions are kept, those below a turns divided by s,
            with a ramp linear in the number of turns between
      {"kind": "pairs", "factor": s, "context": n, "low": a, "high": b}
            the same ends, with a ramp linear in the pair's index (ends rounded outwards to whole pairs)
    An "attention" entry is the factor on cos and sin; "pairs" defaults to 0.1 ln(s) + 1, the others to 1."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    kind = scaling["kind"] if scaling else "none"
    s = float(scaling["factor"]) if scaling else 1.0
    if not s > 0 or not theta > 0:
        raise ValueError("theta and the scaling factor must be positive")
    if kind == "theta":
        if rot_dim < 4:
            raise ValueError("theta scaling needs rot_dim >= 4")
        theta = theta * s ** (rot_dim / (rot_dim - 2))
    f = float(theta) ** (-i / rot_dim)
    factor = 1.0
    if kind == "linear":
        f = f / s
    elif kind in ("turns", "pairs"):
        n, low, high = float(scaling["context"]), float(scaling["low"]), float(scaling["high"])
        if not 0 < low < high or not n > 0:
            raise ValueError("scaling needs context > 0 and 0 < low < high")
        if kind == "turns":
            keep = ((n * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        else:
            def pair(turns):   # the (fractional) pair that turns this often over the context
                return rot_dim * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(theta))
            first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot_dim - 1)
            keep = 1 - ((i / 2 - first) / max(last - first, 1e-3)).clamp(0, 1)
            factor = 0.1 * math.log(s) + 1 if s > 1 else 1.0
        f = f * keep + f / s * (1 - keep)
    elif kind not in ("none", "theta"):
        raise ValueError(f"unknown scaling kind {kind!r}")
    if scaling and scaling.get("attention") is not None:
        factor = float(scaling["attention"])
    return f.to(device), factor


def _heads(name, t, device, dtype, T, dim) -> None:
    if t.dtype != dtype or t.device != device or t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be a {dtype} tensor [tokens, heads, head_dim] with contiguous heads on {device}")
    _shapes(t.shape[0] == T and t.shape[2] == dim, f"{name}: inconsistent shape")


def _spans(t) -> Tuple[int, int]:
    """First and last byte address that a tensor's elements take."""
    if t.numel() == 0:
        return 0, -1
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size() - 1


def _distinct(name, t) -> None:
    """Refuse an output whose elements share memory (an expanded or otherwise folded tensor)."""
    at = 0
    for stride, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride <= at:
            raise ValueError(f"{name}: elements of an output must not overlap")
        at += stride * (n - 1)


def rope(q, k, positions, freq, layout: str = "half", factor: float = 1.0, inverse: bool = False, out=None, stream=None):
    """Rotary positions of q [T, H_q, head_dim] and k [T, H_k, head_dim] (either may be None): (q, k) turned.

    ``freq`` [rot_dim/2] is float64 on the GPU (``rope_frequencies``); elements from rot_dim on are copied.
    ``inverse`` turns back, with the same factor: the gradient.  ``out`` may be (q, k) themselves or other tensors
    that do not overlap the inputs."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("rope needs q or k")
    device, dtype = _device(x), x.dtype
    if dtype not in _DTYPES:
        raise ValueError("q and k must be bfloat16 or float32")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    T, dim = x.shape[0], x.shape[-1]
    _ints(device, positions=positions)
    if freq.dtype != torch.float64 or freq.device != device or not freq.is_contiguous():
        raise ValueError(f"freq must be a contiguous float64 tensor on {device}")
    _shapes(positions.shape == (T,) and freq.dim() == 1, "inconsistent shapes")
    given = [t for t in (q, k) if t is not None]
    for t in given:
        _heads("q and k", t, device, dtype, T, dim)

    def call(s):
        if out is None:
            res = [None if t is None else torch.empty(t.shape, dtype=dtype, device=device) for t in (q, k)]
        else:
            res = list(out)
            _shapes(len(res) == 2, "out must be (q, k)")
            for t, o in zip((q, k), res):
                if (t is None) != (o is None):
                    raise ValueError("out must hold the outputs of the tensors that are given")
                if t is None:
                    continue
                _heads("out", o, device, dtype, T, dim)
                _shapes(o.shape == t.shape, "out: inconsistent shape")
                _distinct("out", o)
            outs = [o for o in res if o is not None]
            for o in outs:
                a = _spans(o)
                for t in given:
                    if o.data_ptr() == t.data_ptr() and o.stride() == t.stride() and o.shape == t.shape:
                        continue
                    b = _spans(t)
                    if a[0] <= b[1] and b[0] <= a[1] and not _interleaved(o, t):
                        raise ValueError("an output overlaps an input that it is not")
            if len(outs) == 2:
                a, b = _spans(outs[0]), _spans(outs[1])
                if a[0] <= b[1] and b[0] <= a[1] and not _interleaved(*outs):
                    raise ValueError("the outputs overlap")
        qs, ks, qo, ko = (t.stride() if t is not None else (0, 0, 1) for t in (q, k, res[0], res[1]))
        ptr = [0 if t is None else t.data_ptr() for t in (q, k, res[0], res[1])]
        args = _RopeArgs(*ptr, positions.data_ptr(), freq.data_ptr(), qs[0], qs[1], ks[0], ks[1], qo[0], qo[1], ko[0], ko[1],
                         T, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], dim, 2 * freq.numel(),
                         ROPE_LAYOUTS[layout], _DTYPES[dtype], int(bool(inverse)), float(factor))
        _check(lib().ikbo_rope(ctypes.byref(args), s), "ikbo_rope")
        return res[0], res[1]

    return _run(device, stream, call)


def _interleaved(a, b) -> bool:
    """Whether two tensors [T, H, dim] are different heads of one tensor: same token stride, and the heads of a token
    lie within it without meeting."""
    st = a.stride(0)
    if b.stride(0) != st or a.shape[0] <= 1 or st <= 0:
        return False
    size = a.element_size()
    lo, hi = (a, b) if a.data_ptr() <= b.data_ptr() else (b, a)
    within = [(t.shape[1] - 1) * t.stride(1) + t.shape[2] for t in (lo, hi)]
    gap = hi.data_ptr() - lo.data_ptr()
    return gap % size == 0 and within[0] <= gap // size and gap // size + within[1] <= st


def _tiles(device, tiles):
    if tiles.dtype != torch.uint8 or tiles.device != device or tiles.dim() != 3 or not tiles.is_contiguous():
        raise ValueError(f"tiles must be a contiguous uint8 tensor [pages, heads, 68 * head_dim] on {device}")
    _shapes(tiles.shape[2] % 68 == 0, "tiles: the last dimension must be 68 * head_dim")
    return tiles.shape[0], tiles.shape[1], tiles.shape[2] // 68


def kv4_write(k, v, slots, tiles, status, stream=None) -> None:
    """Put the rows k, v [T, H_kv, head_dim] (bf16 or float32) into the cache at their slots (``ikbo_kv4_write``)."""
    device = _device(k)
    pages, H, dim = _tiles(device, tiles)
    if k.dtype not in _DTYPES:
        raise ValueError("k and v must be bfloat16 or float32")
    T = slots.numel()
    _ints(device, slots=slots)
    _status(device, status)
    for name, t in (("k", k), ("v", v)):
        _heads(name, t, device, k.dtype, T, dim)
        _shapes(t.shape[1] == H, f"{name}: heads differ from the cache's")
    args = _RowsArgs(k.data_ptr(), v.data_ptr(), slots.data_ptr(), tiles.data_ptr(), status.data_ptr(), k.stride(0), k.stride(1),
                     v.stride(0), v.stride(1), T, H, dim, pages, _DTYPES[k.dtype])
    _run(device, stream, lambda s: _check(lib().ikbo_kv4_write(ctypes.byref(args), s), "ikbo_kv4_write"))


def kv4_read(slots, tiles, status, dtype=torch.bfloat16, out=None, stream=None):
    """The values of the cached rows at the slots: (k, v) [T, H_kv, head_dim] (``ikbo_kv4_read``).

    Rows of a slot of -1 are left as they were (unspecified without ``out``)."""
    device = _device(tiles)
    pages, H, dim = _tiles(device, tiles)
    _ints(device, slots=slots)
    _status(device, status)
    T = slots.numel()

    def call(s):
        if out is None:
            if dtype not in _DTYPES:
                raise ValueError("dtype must be bfloat16 or float32")
            res = tuple(torch.empty((T, H, dim), dtype=dtype, device=device) for _ in range(2))
        else:
            res = tuple(out)
            _shapes(len(res) == 2, "out must be (k, v)")
            if res[0].dtype not in _DTYPES:
                raise ValueError("out must be bfloat16 or float32")
            for t in res:
                _heads("out", t, device, res[0].dtype, T, dim)
                _shapes(t.shape[1] == H, "out: heads differ from the cache's")
                _distinct("out", t)
        k, v = res
        args = _RowsArgs(k.data_ptr(), v.data_ptr(), slots.data_ptr(), tiles.data_ptr(), status.data_ptr(), k.stride(0), k.stride(1),
                         v.stride(0), v.stride(1), T, H, dim, pages, _DTYPES[k.dtype])
        _check(lib().ikbo_kv4_read(ctypes.byref(args), s), "ikbo_kv4_read")
        return res

    return _run(device, stream, call)


def kv4_attention(Q, tiles, block_table, lens, mp, status, positions=None, scale: float = 0.0, out=None, stream=None):
    """O = softmax(scale Q K[map]^T) V[map] over the cached histories (``ikbo_kv4_attention``).

    Q [B_c, H_q, L_q, head_dim] bf16 (or [B_c, H_q, head_dim]: one query each), any strides that are multiples of 8;
    ``mp`` [B_c] int32, or None where candidate b belongs to user b; -1 entries are padding.  ``positions`` [B_c, L_q]
    (or [B_c]) int32 limits each query to tokens up to its position.  O has Q's shape; the rows of padding are left as
    they were (unspecified without ``out``)."""
    device = _device(Q)
    pages, H, dim = _tiles(device, tiles)
    if Q.dtype != torch.bfloat16 or Q.dim() not in (3, 4) or (Q.shape[-1] > 1 and Q.stride(-1) != 1):
        raise ValueError("Q must be a bfloat16 tensor [B_c, H_q, L_q, head_dim] or [B_c, H_q, head_dim] with contiguous heads")
    _table(device, block_table)
    _ints(device, lens=lens)
    _status(device, status)
    B_c, H_q, L_q = Q.shape[0], Q.shape[1], Q.shape[2] if Q.dim() == 4 else 1
    B_u = lens.numel()
    _shapes(Q.shape[-1] == dim and block_table.shape[0] == B_u, "inconsistent shapes")
    if mp is not None:
        _ints(device, map=mp)
        _shapes(mp.shape == (B_c,), "map: inconsistent shape")
    if positions is not None:
        _ints(device, positions=positions)
        _shapes(positions.numel() == B_c * L_q, "positions: inconsistent shape")
    need = lib().ikbo_kv4_attention_workspace(B_u, B_c, H_q, H, L_q, dim, block_table.shape[1])
    if need < 0:
        raise IkboError(int(need), "ikbo_kv4_attention")

    def strides(t):
        return (t.stride(0), t.stride(1), t.stride(2)) if t.dim() == 4 else (t.stride(0), t.stride(1), 0)

    def call(s):
        if out is None:
            o = torch.empty(Q.shape, dtype=Q.dtype, device=device)
        else:
            o = out
            if o.dtype != Q.dtype or o.device != device or o.shape != Q.shape or (dim > 1 and o.stride(-1) != 1):
                raise ValueError("out must be a bfloat16 tensor shaped like Q with contiguous heads")
            _distinct("out", o)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        args = _AttentionArgs(Q.data_ptr(), o.data_ptr(), tiles.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
                              0 if mp is None else mp.data_ptr(), 0 if positions is None else positions.data_ptr(), status.data_ptr(),
                              ws.data_ptr(), need, *strides(Q), *strides(o), block_table.stride(0), B_u, B_c, H_q, H, L_q, dim,
                              block_table.shape[1], pages, float(scale))
        _check(lib().ikbo_kv4_attention(ctypes.byref(args), s), "ikbo_kv4_attention")
        return o

    return _run(device, stream, call)


class UserHistories:
    """The cached histories of up to ``users`` users: 4-bit tiles, block table, lengths and the ring of free pages.

        h = UserHistories(users, max_tokens, num_pages, H_kv, head_dim, rot_dim=head_dim)
        h.append(k, v, counts)                        # counts[u] new tokens per user, -1: the user leaves
        O = h.attend(Q, map, positions=positions)     # candidates, or the users' own queries with causal=True
        h.check()                                     # waits; IKBO_OK or what a step recorded

    With ``rot_dim`` keys are stored turned by their positions, and queries are turned by theirs.  ``append`` updates
    tables and lengths in place, so captured steps can be replayed; one object serves one stream at a time."""

    def __init__(self, users: int, max_tokens: int, num_pages: int, H_kv: int, head_dim: int, rot_dim: int = 0,
                 theta: float = 10000.0, scaling: Optional[dict] = None, layout: str = "half", device="cuda"):
        if not 1 <= users <= MAX_USERS:
            raise ValueError(f"users must be between 1 and {MAX_USERS}")
        if head_dim not in (64, 128) or H_kv < 1 or num_pages < 1 or max_tokens < 1:
            raise ValueError("head_dim must be 64 or 128; H_kv, num_pages and max_tokens positive")
        if rot_dim and (rot_dim % 2 or not 2 <= rot_dim <= head_dim):
            raise ValueError("rot_dim must be even and at most head_dim")
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
        i32 = dict(dtype=torch.int32, device=device)
        self.tiles = torch.zeros((num_pages, H_kv, 68 * head_dim), dtype=torch.uint8, device=device)
        self.table = torch.full((users, -(-max_tokens // PAGE)), -1, **i32)
        self.lens = torch.zeros(users, **i32)
        self.ring = torch.arange(num_pages, **i32)
        self.state = torch.tensor([0, num_pages, 0, 0], **i32)
        self.status = torch.zeros(1, **i32)
        self.layout = layout
        self.freq, self.factor = rope_frequencies(rot_dim, theta, scaling, device) if rot_dim else (None, 1.0)

    def append(self, k, v, counts, stream=None) -> StepTables:
        """Take in one step: rows k, v [T, H_kv, head_dim] hold the users' new tokens one user after the other
        (``counts`` [users] int32 of them; rows behind the last are padding)."""
        t = kv_tables(counts, self.lens, self.table, self.ring, self.state, k.shape[0], self.status, in_place=True, stream=stream)
        if self.freq is not None:
            k = rope(None, k, t.positions, self.freq, layout=self.layout, factor=self.factor, stream=stream)[1]
        kv4_write(k, v, t.slots, self.tiles, self.status, stream=stream)
        return t

    def attend(self, Q, mp=None, positions=None, causal: bool = False, scale: float = 0.0, out=None, stream=None):
        """Attention of Q [B_c, H_q, L_q, head_dim] (or [B_c, H_q, head_dim]) over the users' histories.

        ``positions`` [B_c, L_q] (or [B_c]) says where the queries stand: they are turned by it (``rot_dim``), and with
        ``causal`` see tokens up to it only."""
        if positions is None and (causal or self.freq is not None):
            raise ValueError("positions are needed for causal attention and for rotary queries")
        if self.freq is not None:
            q = Q.transpose(1, 2) if Q.dim() == 4 else Q          # [.., heads, head_dim], tokens first
            turned = rope(q.reshape(-1, *q.shape[-2:]), None, positions.reshape(-1), self.freq, layout=self.layout,
                          factor=self.factor, stream=stream)[0].view(q.shape)
            Q = turned.transpose(1, 2) if Q.dim() == 4 else turned
        return kv4_attention(Q, self.tiles, self.table, self.lens, mp, self.status, positions=positions if causal else None,
                             scale=scale, out=out, stream=stream)

    def check(self, stream=None) -> int:
        """Wait, then return and clear the condition that a step recorded."""
        return kv_status(self.status, stream)

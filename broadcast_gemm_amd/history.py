"""Cached user histories: target attention for users whose keys and values are kept between requests.

``FaPlan`` attends over dense K and V that the caller holds per request.  Here a user's history lives in a
cache of 4-bit codes, in pages of 64 tokens that a block table names; it grows by tokens and has a length of
its own.  The calls bind the C ABI (``ikbo_kv_*``, ``ikbo_rope``, ``ikbo_kv4_*`` in ``include/ikbo.h``, which
states formulas and layouts); every step runs in the library's HIP kernels, there is no CPU path.  Arguments
are checked and outputs allocated in ``csrc/torch_history.cpp``.

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

from . import IKBO_OK, IkboError, lib

PAGE = 64                  # tokens per page of the 4-bit cache
MAX_USERS = 4096
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}

# The small calls are bound by the host: these are the cheap forms of current_device() and of
# current_stream(device).cuda_stream (0.1 us each against 0.2 and 2.8), with the public ones to fall back on.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _check(status: int, what: str) -> None:
    if status != IKBO_OK:
        raise IkboError(status, what)


@contextlib.contextmanager
def _on(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):   # a handle; 0 is the default stream
                stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
            s = stream
            with torch.cuda.stream(s):
                yield s.cuda_stream


def _run(device, stream, call, *args):
    """call(stream handle, *args) with ``device`` current and allocations on the stream."""
    if stream is None and _current_device() == device.index:
        return call(_current_stream(device.index), *args)
    with _on(device, stream) as handle:
        return call(handle, *args)


def _status_of(result, what: str):
    """A result of the binding, or the library's status raised."""
    if type(result) is int:
        raise IkboError(result, what)
    return result


_ext = None


def _binding():
    """The torch binding (``_ikbo_torch.so``) with the library's entry points; raises if either is not built."""
    global _ext
    if _ext is None:
        L = lib()
        try:
            from . import _ikbo_torch as ext
        except ImportError as e:
            raise ImportError("_ikbo_torch.so is not built; run `python -m broadcast_gemm_amd.build`") from e
        names = ("ikbo_kv_tables", "ikbo_rope", "ikbo_kv4_write", "ikbo_kv4_read", "ikbo_kv4_attention_workspace", "ikbo_kv4_attention")
        ext.bind([ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names])
        _ext = ext
    return _ext


def _device(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    return t.device


def kv_status(status, stream=None) -> int:
    """Wait for the stream, then return and clear the condition recorded in ``status`` (an IKBO_* code).

    Calls on other streams that share ``status`` must be over."""
    device = _device(status)
    if status.dtype != torch.int32 or status.numel() != 1:
        raise ValueError("status must be an int32 tensor of one element")
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
    res = _run(_device(lens), stream, _binding().kv_tables, counts, lens, block_table, ring, state, capacity, status, page_size, in_place,
               None if out is None else list(out))
    return StepTables._make(_status_of(res, "ikbo_kv_tables"))


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
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    q_out = k_out = None
    if out is not None:
        q_out, k_out = out
        _rope_out(q, k, q_out, k_out)
    return _status_of(_run(_device(x), stream, _binding().rope, q, k, positions, freq, ROPE_LAYOUTS[layout], factor, inverse, q_out, k_out),
                      "ikbo_rope")


def _rope_out(q, k, q_out, k_out) -> None:
    pairs = []
    for t, o in ((q, q_out), (k, k_out)):
        if (t is None) != (o is None):
            raise ValueError("out must hold the outputs of the tensors that are given")
        if t is not None:
            if t.dim() != 3 or o.dim() != 3:
                raise ValueError("q, k and out must be tensors [tokens, heads, head_dim]")
            _distinct("out", o)
            pairs.append((t, o))
    for own, o in pairs:
        for t, _ in pairs:
            same = t is own and o.data_ptr() == t.data_ptr() and o.stride() == t.stride() and o.shape == t.shape
            if not same and _meet(o, t):
                raise ValueError("an output overlaps an input that it is not")
    if len(pairs) == 2 and _meet(pairs[0][1], pairs[1][1]):
        raise ValueError("the outputs overlap")


def _meet(a, b) -> bool:
    """Whether two tensors may share memory (different heads, rows or columns of one tensor do not)."""
    x, y = _spans(a), _spans(b)
    return x[0] <= y[1] and y[0] <= x[1] and not _interleaved(a, b)


def _interleaved(a, b) -> bool:
    """Whether two tensors share no element although their spans may cross.

    Looks for places i in a and j in b with gap + sum_k j_k t_k - sum_k i_k s_k = 0, in bytes, the largest strides first
    and only where the rest can still get there: strides that nest, as those of tensors do, leave two choices each."""
    steps = {}
    for t, sign in ((a, -1), (b, 1)):
        for n, stride in zip(t.shape, t.stride()):
            if n > 1 and stride:
                lo, hi = steps.get(stride * t.element_size(), (0, 0))
                steps[stride * t.element_size()] = (lo - (n - 1), hi) if sign < 0 else (lo, hi + n - 1)
    steps = [(s, *steps[s]) for s in sorted(steps, reverse=True)]
    least, most = [0], [0]                                   # what the smaller strides can add
    for s, lo, hi in reversed(steps):
        least.append(least[-1] + lo * s)
        most.append(most[-1] + hi * s)
    below, above = -b.element_size(), a.element_size()       # elements meet if their distance lies between
    left = 10000                                             # strides that do not nest: give up, they may meet

    def reach(k, at):
        nonlocal left
        left -= 1
        if k == len(steps) or left < 0:
            return left < 0 or below < at < above
        s, lo, hi = steps[k]
        lo = max(lo, -((at + most[-2 - k] - below - 1) // s))
        hi = min(hi, (above - 1 - at - least[-2 - k]) // s)
        return any(reach(k + 1, at + d * s) for d in range(lo, hi + 1))

    return not reach(0, b.data_ptr() - a.data_ptr())


def kv4_write(k, v, slots, tiles, status, stream=None) -> None:
    """Put the rows k, v [T, H_kv, head_dim] (bf16 or float32) into the cache at their slots (``ikbo_kv4_write``)."""
    _check(_run(_device(k), stream, _binding().kv4_write, k, v, slots, tiles, status), "ikbo_kv4_write")


def kv4_read(slots, tiles, status, dtype=torch.bfloat16, out=None, stream=None):
    """The values of the cached rows at the slots: (k, v) [T, H_kv, head_dim] (``ikbo_kv4_read``).

    Rows of a slot of -1 are left as they were (unspecified without ``out``)."""
    k = v = None
    if out is not None:
        k, v = out
        for t in (k, v):
            if t.dim() != 3:
                raise ValueError("out must be tensors [tokens, heads, head_dim]")
            _distinct("out", t)
        if _meet(k, v):
            raise ValueError("the outputs overlap")
    return _status_of(_run(_device(tiles), stream, _binding().kv4_read, slots, tiles, status, dtype, k, v), "ikbo_kv4_read")


def kv4_attention(Q, tiles, block_table, lens, mp, status, positions=None, scale: float = 0.0, out=None, stream=None):
    """O = softmax(scale Q K[map]^T) V[map] over the cached histories (``ikbo_kv4_attention``).

    Q [B_c, H_q, L_q, head_dim] bf16 (or [B_c, H_q, head_dim]: one query each), any strides that are multiples of 8;
    ``mp`` [B_c] int32, or None where candidate b belongs to user b; -1 entries are padding.  ``positions`` [B_c, L_q]
    (or [B_c]) int32 limits each query to tokens up to its position.  O has Q's shape; the rows of padding are left as
    they were (unspecified without ``out``).  ``out`` may be Q, or else must not overlap it."""
    if out is not None:
        _distinct("out", out)
        same = out.data_ptr() == Q.data_ptr() and out.shape == Q.shape and all(x == y or n == 1 for x, y, n in zip(out.stride(), Q.stride(), Q.shape))
        if not same and _meet(out, Q):
            raise ValueError("out overlaps Q")
    return _status_of(_run(_device(Q), stream, _binding().kv4_attention, Q, tiles, block_table, lens, mp, status, positions, scale, out),
                      "ikbo_kv4_attention")


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
        # Everything that could refuse the write is checked before the tables move on.
        H, dim = self.tiles.shape[1], self.tiles.shape[2] // 68
        for name, x in (("k", k), ("v", v)):
            if x.device != self.tiles.device or x.dtype not in (torch.bfloat16, torch.float32) or x.dtype != k.dtype:
                raise ValueError(f"{name} must be bfloat16 or float32 on {self.tiles.device}, k and v alike")
            if x.dim() != 3 or x.shape != (k.shape[0], H, dim) or x.stride(2) != 1:
                raise ValueError(f"{name} must be [T, {H}, {dim}] with contiguous heads, k and v alike")
            whole = 8 if x.dtype == torch.bfloat16 else 4
            if x.data_ptr() % 16 or x.stride(0) % whole or x.stride(1) % whole:
                raise ValueError(f"{name}: rows must be 16-byte aligned")
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
        if stream is not None:   # the copies below are torch's, on its current stream: make that the call's
            with _on(self.tiles.device, stream):
                return self.attend(Q, mp, positions=positions, causal=causal, scale=scale, out=out)
        if self.freq is not None:
            q = Q.transpose(1, 2) if Q.dim() == 4 else Q          # [.., heads, head_dim], tokens first
            turned = rope(q.reshape(-1, *q.shape[-2:]), None, positions.reshape(-1), self.freq, layout=self.layout,
                          factor=self.factor)[0].view(q.shape)
            Q = turned.transpose(1, 2) if Q.dim() == 4 else turned
        return kv4_attention(Q, self.tiles, self.table, self.lens, mp, self.status, positions=positions if causal else None,
                             scale=scale, out=out)

    def check(self, stream=None) -> int:
        """Wait, then return and clear the condition that a step recorded."""
        return kv_status(self.status, stream)

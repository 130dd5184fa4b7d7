"""Training target attention: its forward with the statistics that the gradient needs, its gradient, and dropout.

The pages say the same kernels serve training once the ratio of candidates to users exceeds one (aibriefing article, the
paragraph on the three layers of the stack).  K and V stand at the user batch, and their gradients are formed there: nothing is replicated per candidate in
either direction.  The calls bind the C ABI (``ikbo_attention_*``, ``ikbo_dropout`` in ``include/ikbo.h``, which states
formulas, random numbers and layouts); every step runs in the library's HIP kernels, there is no CPU path.

    O, lse = attention(Q, K, V, map, status, lens=lens, dropout=0.1, rng=rng)
    dQ, dK, dV = attention_backward(dO, Q, K, V, O, lse, map, status, lens=lens, dropout=0.1, rng=rng)
    y = dropout(x, 0.1, rng, residual=r)                 # and dx = dropout(dy, 0.1, rng)

``autograd.IkboAttention`` and ``autograd.IkboDropout`` run these.

Random numbers come from a counter: ``rng`` is an int64 tensor (seed, offset) on the GPU, and equal ones give equal
numbers.  A step takes an offset of its own; nothing about the mask is stored, the backward forms it again.  Offsets
count modulo 2^32.

Nothing is kept between calls: outputs and workspaces come from torch's allocator on the stream the call runs on (the
current one, or ``stream``).  Conditions that only the device sees set bits of ``status`` (an int32 tensor of one
element, zeroed once); ``history.kv_status`` waits, returns and clears them.
"""
from __future__ import annotations

import ctypes

from . import lib
from .history import _binding, _device, _meet, _run, _status_of

_bound = None


def _training():
    """The torch binding with the library's training entry points."""
    global _bound
    if _bound is None:
        ext, L = _binding(), lib()
        names = ("ikbo_attention_workspace", "ikbo_attention_forward", "ikbo_attention_backward", "ikbo_dropout")
        ext.bind_training([ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names])
        _bound = ext
    return _bound


def attention(Q, K, V, mp, status, lens=None, positions=None, scale: float = 0.0, dropout: float = 0.0, rng=None, stream=None):
    """(O, lse): target attention and the logarithms of its rows' sums (``ikbo_attention_forward``).

    Q [B_c, H_q, L_q, head_dim], K and V [B_u, H_kv, L_kv, head_dim], bf16, any strides that are multiples of 8 with
    contiguous heads; H_q a multiple of H_kv.  ``mp`` [B_c] int32 names the candidates' users; -1 entries are padding, rows of
    zeros.  ``lens`` [B_u] int32 are the users' numbers of tokens, ``positions`` [B_c, L_q] int32 limits each query to tokens
    up to its position; a query that sees none gives O = 0, lse = -inf.  ``dropout`` is a probability in whole 256ths (the
    nearest), and needs ``rng``.  O [B_c, H_q, L_q, head_dim] bf16, lse [B_c, H_q, L_q] float32."""
    return _status_of(_run(_device(Q), stream, _training().attention_forward, Q, K, V, mp, status, lens, positions, scale, dropout, rng),
                      "ikbo_attention_forward")


def attention_backward(dO, Q, K, V, O, lse, mp, status, lens=None, positions=None, scale: float = 0.0, dropout: float = 0.0, rng=None,
                       stream=None):
    """(dQ, dK, dV) of the attention above for the upstream gradient dO (``ikbo_attention_backward``).

    The other arguments are those of the forward, O and lse its results.  dK and dV are summed over the user's candidates,
    their queries and the heads that share a head; users without candidates and tokens behind a history get zeros.  All three are computed, whichever are wanted."""
    return _status_of(_run(_device(Q), stream, _training().attention_backward, dO, Q, K, V, O, lse, mp, status, lens, positions, scale,
                           dropout, rng), "ikbo_attention_backward")


def dropout(x, p: float, rng, residual=None, out=None, stream=None):
    """residual + x / (1 - p) where an element stays, the residual (or 0) where it does not (``ikbo_dropout``).

    x, bf16 or float32, and ``residual`` are dense; ``p`` is a probability in whole 65536ths (the nearest).  The gradient of
    x is the same call on the gradient.  ``out`` may be x or ``residual``, or else must not overlap them."""
    if out is not None:
        for t in (x, residual):
            if t is not None and not (out.data_ptr() == t.data_ptr() and out.shape == t.shape and out.stride() == t.stride()) and _meet(out, t):
                raise ValueError("out overlaps an input that it is not")
    return _status_of(_run(_device(x), stream, _training().dropout, x, p, rng, residual, out), "ikbo_dropout")

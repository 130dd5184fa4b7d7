"""Training through the IKBO LCE: a torch.autograd.Function over the library's forward and
backward, and a module that owns the projections.

The pages say the same kernels serve training once the ratio of candidates to users exceeds one
(aibriefing article, the paragraph on the three layers of the stack).  Forward and backward both
run in ``libikbo`` (``ikbo_lce_forward`` / ``ikbo_lce_backward``); the gradients are those of

    Y[b] = W_u . U[map[b]] + W_c . C[b]

(dC[b] = W_c^T dY[b], dU[u] = W_u^T S[u], dW_c = sum_b dY[b] C[b]^T, dW_u = sum_u S[u] U[u]^T with
S[u] the sum of dY over the candidates of user u).  The library returns dW_u and dW_c in float32;
autograd wants a gradient in its parameter's dtype, so they are rounded to it once (the only
step outside the library, a dtype conversion).

    lce = IkboLce(K_u, K_c, M, D).cuda()           # W_u, W_c: bf16 parameters
    Y = lce(U, C, map)                               # U, C may require grad
    Y.backward(dY)                                   # lce.W_u.grad, lce.W_c.grad, U.grad, C.grad

Rotary positions train through ``IkboRope``: the gradient of a rotation is the rotation by the opposite
angle with the same factor, the same kernel.

    rope = IkboRope(head_dim).cuda()
    q, k = rope(q, k, positions)                     # [T, H, head_dim] each

Target attention trains through ``IkboAttention``, with dropout of its weights, and ``IkboDropout`` drops activations;
``IkboLce`` takes a ``dropout`` of its output.  Their masks are never stored: the backward forms them again from the
call's (seed, offset) (``training``), which is torch's to give, or the module's if it has a seed.

    attend = IkboAttention(dropout=0.1).cuda()
    O = attend(Q, K, V, map, lens=lens)              # Q, K, V may require grad; dK, dV at the user batch
"""
from __future__ import annotations

from typing import Dict, Tuple

import torch

from . import FLAG_BACKWARD, LcePlan
from . import history, training
from .rewrite import bucket_b_c, bucket_b_u


class _BackwardPlans:
    """Plans with the backward's workspace, keyed by (K_u, K_c, M, D), each sized to a batch range.

    A plan that a larger batch outgrows is dropped, not destroyed: autograd graphs recorded
    with it may still run their backward, and it is freed once none refers to it."""

    def __init__(self, make_plan=LcePlan):
        self._make = make_plan
        self._plans: Dict[Tuple[int, int, int, int], object] = {}

    def plan_for(self, B_u: int, B_c: int, K_u: int, K_c: int, M: int, D: int):
        key = (K_u, K_c, M, D)
        plan = self._plans.get(key)
        if plan is None or plan.max_B_u < B_u or plan.max_B_c < B_c:
            mu, mc = bucket_b_u(B_u), bucket_b_c(B_c)
            if plan is not None:
                mu, mc = max(mu, plan.max_B_u), max(mc, plan.max_B_c)
            plan = self._make(mu, mc, K_u, K_c, M, D, dtype="bf16", flags=FLAG_BACKWARD)
            self._plans[key] = plan
        return plan

    def close(self) -> None:
        for plan in self._plans.values():
            plan.close()
        self._plans.clear()


class LceFunction(torch.autograd.Function):
    """Y = W_u . U[map] + W_c . C with both directions in the library (bf16 tensors on the GPU)."""

    @staticmethod
    def forward(ctx, U, C, mp, W_u, W_c, plans: _BackwardPlans):
        B_u, K_u, D = U.shape
        B_c, K_c, _ = C.shape
        plan = plans.plan_for(B_u, B_c, K_u, K_c, W_u.shape[0], D)
        mp32 = mp.to(torch.int32).contiguous()
        U, C, W_u, W_c = (t.contiguous() for t in (U, C, W_u, W_c))
        Y = plan.forward(U, C, mp32, W_u, W_c)
        ctx.save_for_backward(U, C, mp32, W_u, W_c)
        ctx.plan = plan
        return Y

    @staticmethod
    def backward(ctx, dY):
        U, C, mp32, W_u, W_c = ctx.saved_tensors
        dU, dC, dW_u, dW_c = ctx.plan.backward(dY.contiguous(), U, C, mp32, W_u, W_c)
        need = ctx.needs_input_grad
        return (dU if need[0] else None, dC if need[1] else None, None,
                dW_u.to(W_u.dtype) if need[3] else None, dW_c.to(W_c.dtype) if need[4] else None, None)


class IkboLce(torch.nn.Module):
    """The LCE layer with trainable projections W_u [M, K_u] and W_c [M, K_c] (bf16).

    Initialised with standard deviation 1/sqrt(K_u + K_c), so that Y has about unit variance for
    unit-variance inputs.  While training, ``dropout`` of the output's elements are dropped (``IkboDropout``)."""

    def __init__(self, K_u: int, K_c: int, M: int, D: int, generator=None, dropout: float = 0.0):
        super().__init__()
        std = (K_u + K_c) ** -0.5
        self.W_u = torch.nn.Parameter((torch.randn(M, K_u, generator=generator) * std).to(torch.bfloat16))
        self.W_c = torch.nn.Parameter((torch.randn(M, K_c, generator=generator) * std).to(torch.bfloat16))
        self.D = D
        self.drop = IkboDropout(dropout) if dropout else None
        self._plans = _BackwardPlans()

    def forward(self, U, C, mp):
        Y = LceFunction.apply(U, C, mp, self.W_u, self.W_c, self._plans)
        return Y if self.drop is None else self.drop(Y)


class RopeFunction(torch.autograd.Function):
    """(q, k) turned by their positions (``inverse``: turned back), both directions in the library.

    The gradient is the same function the other way round, so it can be differentiated again."""

    @staticmethod
    def forward(ctx, q, k, positions, freq, layout, factor, inverse=False):
        q_out, k_out = history.rope(q, k, positions, freq, layout=layout, factor=factor, inverse=inverse)
        ctx.save_for_backward(positions, freq)
        ctx.how = (layout, factor, not inverse)
        return q_out, k_out

    @staticmethod
    def backward(ctx, dq, dk):
        positions, freq = ctx.saved_tensors
        dq, dk = (None if d is None or not need else d if d.stride(-1) == 1 else d.contiguous()
                  for d, need in zip((dq, dk), ctx.needs_input_grad))
        if dq is not None or dk is not None:
            dq, dk = RopeFunction.apply(dq, dk, positions, freq, *ctx.how)
        return dq, dk, None, None, None, None, None


class IkboRope(torch.nn.Module):
    """Rotary positions of q and k [T, H, head_dim] (k may be None), with gradients.

    ``rot_dim``, ``theta`` and ``scaling`` as in ``history.rope_frequencies``; the frequencies are a buffer that casts of
    the module (``bfloat16()``, ``to(dtype)``) leave in float64.  Forward and backward may be captured into a graph
    together, while no eager graph of the same leaves is alive (torch would accumulate their gradients on that one's
    stream)."""

    def __init__(self, head_dim: int, rot_dim: int = 0, theta: float = 10000.0, scaling=None, layout: str = "half"):
        super().__init__()
        self.layout = layout
        freq, self.factor = history.rope_frequencies(rot_dim or head_dim, theta, scaling, device="cpu")
        self.register_buffer("freq", freq, persistent=False)

    def _apply(self, fn, *args, **kwargs):
        freq = self.freq
        super()._apply(fn, *args, **kwargs)
        if self.freq.dtype != freq.dtype:   # moved and rounded: only the move is kept
            self.freq = freq.to(self.freq.device)
        return self

    def forward(self, q, k, positions):
        return RopeFunction.apply(q, k, positions, self.freq, self.layout, self.factor)


# Which run of autograd's engine this thread is in, -1 outside of backward passes.
_in_backward = getattr(torch._C, "_current_graph_task_id", None) or (lambda: -1)


class _Counter(torch.nn.Module):
    """A module with random numbers.

    Without a seed every call takes its (seed, offset) from torch's generator of the device, on the device.  They are then
    what torch's own dropout would have: set by ``torch.manual_seed``, new in every replay of a captured step, and the same
    when ``torch.utils.checkpoint`` runs a forward pass again, since it restores that generator.

    With a seed they are the module's own: ``rng`` (seed, offset), whose offset moves on with every call that uses them, on
    the device, so that replays of a captured step draw new ones; it is saved with the module's state (modules without a seed
    have it too, for states of either kind).  A copy of the module, and ranks whose buffers a wrapper keeps alike, draw the same
    ones.  Nothing moves it back for a forward pass that is run again, which would give gradients of another mask than the
    output's: within a backward pass such a module raises an error."""

    _counted = True

    def __init__(self, seed):
        super().__init__()
        self._counted = seed is not None
        if seed is None:   # from torch's generator: other modules have others
            seed = int(torch.randint(0, 1 << 62, ()))
        self.register_buffer("rng", torch.tensor([seed, 0], dtype=torch.int64))

    def _draw(self):
        rng = self.rng.clone()
        self.rng[1:].add_(1)
        return rng

    def _numbers(self, device):
        """(seed, offset) of one call."""
        if not self._counted:
            return torch.randint(0, 1 << 62, (2,), device=device)
        if _in_backward() != -1:
            raise RuntimeError("a module with a seed of its own cannot repeat its random numbers in a forward pass that is run again for the "
                               "backward (activation checkpointing); leave seed=None there")
        return self._draw()


def _probability(p: float, of: int) -> float:
    if not (p == 0.0 or (0.0 < p < 1.0 and 0 < round(p * of) < of)):
        raise ValueError(f"dropout must be 0, or a probability that is not 0 or 1 in whole {of}ths")
    return float(p)


class DropoutFunction(torch.autograd.Function):
    """residual + dropout(x) in the library; the gradient of x is the same dropout of the gradient."""

    @staticmethod
    def forward(ctx, x, residual, p, rng):
        ctx.save_for_backward(rng)
        ctx.p = p
        return training.dropout(x.contiguous(), p, rng, residual=None if residual is None else residual.contiguous())

    @staticmethod
    def backward(ctx, dy):
        dx = DropoutFunction.apply(dy, None, ctx.p, *ctx.saved_tensors) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None


class IkboDropout(_Counter):
    """x with ``p`` of its elements dropped and the others divided by 1 - p, added to ``residual`` if that is given.

    bf16 or float32 on the GPU; p in whole 65536ths (the nearest).  In evaluation nothing is dropped.  A residual of x's shape
    and type is added in the same kernel and the sum rounded once; any other that can be added to x is added to what the
    dropout rounded."""

    def __init__(self, p: float, seed=None):
        super().__init__(seed)
        self.p = _probability(p, 65536)

    def forward(self, x, residual=None):
        if not (self.training and self.p):
            return x if residual is None else residual + x
        rng = self._numbers(x.device)
        if residual is None or (torch.is_tensor(residual) and residual.shape == x.shape and residual.dtype == x.dtype):
            return DropoutFunction.apply(x, residual, self.p, rng)
        return residual + DropoutFunction.apply(x, None, self.p, rng)


class AttentionFunction(torch.autograd.Function):
    """O = softmax(scale Q K[map]^T) V[map] over the tokens that each query sees, both directions in the library."""

    @staticmethod
    def forward(ctx, Q, K, V, mp, lens, positions, scale, dropout, rng, status):
        Q, K, V = (_rows(t) for t in (Q, K, V))
        how = dict(lens=lens, positions=positions, scale=scale, dropout=dropout, rng=rng)
        O, lse = training.attention(Q, K, V, mp, status, **how)
        ctx.save_for_backward(Q, K, V, O, lse, mp, lens, positions, rng, status)
        ctx.how = scale, dropout
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, lse, mp, lens, positions, rng, status = ctx.saved_tensors
        scale, dropout = ctx.how
        grads = training.attention_backward(_rows(dO), Q, K, V, O, lse, mp, status, lens=lens, positions=positions, scale=scale,
                                            dropout=dropout, rng=rng)
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad)) + (None,) * 7


def _rows(t):
    """t, or a copy of it where its rows are not contiguous and 16-byte aligned."""
    whole = t.dim() == 4 and (t.shape[3] == 1 or t.stride(3) == 1) and t.data_ptr() % 16 == 0
    return t if whole and all(s % 8 == 0 for s, n in zip(t.stride()[:3], t.shape) if n > 1) else t.clone(memory_format=torch.contiguous_format)


def _int32(t):
    """t in 32 bits; what does not fit becomes the nearest that does, which is as far outside (a wrapped one might be a user)."""
    return (t.clamp(-1 << 31, (1 << 31) - 1) if t.dtype == torch.int64 else t).to(torch.int32).contiguous()


class IkboAttention(_Counter):
    """Target attention with gradients: Q [B_c, H_q, L_q, head_dim] over the K, V [B_u, H_kv, L_kv, head_dim] of the candidates'
    users, bf16.

    ``map`` [B_c] names the users, -1 is padding; ``lens`` [B_u] are the users' numbers of tokens, ``positions`` [B_c, L_q]
    limits each query to tokens up to its position (``training.attention``).  While training, ``dropout`` of the weights
    (in whole 256ths, the nearest) are dropped.  ``check`` waits, returns and clears what calls recorded about their
    device data.  Forward and backward may be captured into a graph together, while no eager graph of the same leaves is
    alive (torch would accumulate their gradients on that one's stream)."""

    def __init__(self, dropout: float = 0.0, scale: float = 0.0, seed=None):
        super().__init__(seed)
        self.dropout, self.scale = _probability(dropout, 256), float(scale)
        # Not a buffer: wrappers that give all ranks the first one's buffers would write over what was recorded.
        self.status = torch.zeros(1, dtype=torch.int32)

    def _apply(self, fn, *args, **kwargs):
        super()._apply(fn, *args, **kwargs)
        device, old = fn(torch.empty(0, dtype=torch.int32, device=self.status.device)).device, self.status
        if device != old.device:   # moved alone, and not cast
            self.status = torch.zeros(1, dtype=torch.int32, device=device) if old.is_meta else old.to(device)
        return self

    def forward(self, Q, K, V, mp, lens=None, positions=None):
        i32 = [None if t is None else _int32(t) for t in (mp, lens, positions)]
        drop = self.dropout if self.training else 0.0
        # A replica on another device (torch.nn.DataParallel) has the original's word, which only buffers would follow.
        status = self.status.to(Q.device) if getattr(self, "_is_replica", False) else self.status
        return AttentionFunction.apply(Q, K, V, *i32, self.scale, drop, self._numbers(Q.device) if drop else None, status)

    def check(self, stream=None) -> int:
        return history.kv_status(self.status, stream)

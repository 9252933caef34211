"""torch.autograd integration of the Lightning Attention forward and backward.

`lightning_attention(q, k, v, g, state_in=None, ...)` returns `(out, state_out)` like one
`lightning_attn_prefill` call (`lightning_attention_varlen` likewise for packed sequences,
`lightning_attention_sequence_parallel` for one rank's chunk of a sequence split across
ranks) and is differentiable in q, k, v, g, state_in and the norm weight: its backward is
one `lightning_attn_backward` call (the gradient reaching `state_out`, when the final state
feeds later computation, is passed to it as dstate_out).  When gradients are
needed in a norm mode, the forward runs the prefill in raw mode and then the output
transform, keeping the raw output y, which saves the backward its recompute of y.

`gated_recurrence`, `gated_recurrence_varlen` and `layer_norm` are the differentiable forms of
`lightning_attn_gated_recurrence[_varlen]` and `lightning_attn_layer_norm`, the backward of
each one call of the library's.  This module only orders the library calls and allocates their outputs; every computation runs
in the library's kernels.
"""
from __future__ import annotations

import torch

from . import lightning_attn as la
from . import sequence_parallel as sp


class _LightningAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, state_in, block_size, phi, mode, eps, norm_weight):
        B, T, H, D = q.shape
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        g = None if g is None else g.contiguous()
        out = torch.empty((B, T, H * D), dtype=q.dtype, device=q.device)
        state_out = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device)
        s_in = None if state_in is None else state_in.detach().contiguous()
        keep_y = mode != la.LA_OUT_RAW and (any(ctx.needs_input_grad[:5]) or ctx.needs_input_grad[9])
        y = None
        if keep_y:   # raw prefill, then the norm (and gate) from the kept y
            y = torch.empty_like(out)
            ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_PREFILL, B, T, 0, H, D, block_size,
                                                                   la._dtype(q), la.LA_OUT_RAW), q.device)
            la.lightning_attn_prefill(q, k, v, None, y, s_in, state_out, block_size=block_size, phi=phi,
                                      mode=la.LA_OUT_RAW, workspace=ws)
            la.lightning_attn_output_transform(y.view(B, T, H, D), g, out, mode=mode, eps=eps,
                                               norm_weight=norm_weight)
        else:        # the fused kernel
            ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_PREFILL, B, T, 0, H, D, block_size,
                                                                   la._dtype(q), mode), q.device)
            la.lightning_attn_prefill(q, k, v, g, out, s_in, state_out, block_size=block_size, phi=phi, mode=mode,
                                      eps=eps, norm_weight=norm_weight, workspace=ws)
        ctx.save_for_backward(q, k, v, g, s_in, None if norm_weight is None else norm_weight.detach(), y)
        ctx.cfg = (block_size, phi, mode, eps)
        ctx.has_state = state_in is not None
        return out, state_out

    @staticmethod
    def backward(ctx, dout, dstate_out):
        q, k, v, g, s_in, norm_weight, y = ctx.saved_tensors
        block_size, phi, mode, eps = ctx.cfg
        B, T, H, D = q.shape
        if dout is None:
            dout = torch.zeros((B, T, H * D), dtype=q.dtype, device=q.device)
        dout = dout.to(q.dtype).contiguous()
        dq, dk, dv = (torch.empty_like(q) for _ in range(3))
        dg = torch.empty_like(g) if mode == la.LA_OUT_RMSNORM_GATE else None
        ds_in = torch.empty((B, H, D, D), dtype=torch.float32, device=q.device) if ctx.has_state else None
        dw = torch.empty((H * D,), dtype=torch.float32, device=q.device) if ctx.needs_input_grad[9] else None
        ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_BACKWARD, B, T, 0, H, D, block_size,
                                                               la._dtype(q), mode), q.device)
        la.lightning_attn_backward(q, k, v, g if mode == la.LA_OUT_RMSNORM_GATE else None, dout, dq, dk, dv, dg=dg,
                                   state_in=s_in, dstate_in=ds_in, block_size=block_size, phi=phi, mode=mode,
                                   eps=eps, norm_weight=norm_weight, workspace=ws,
                                   dstate_out=None if dstate_out is None else dstate_out.float().contiguous(), y=y,
                                   dnorm_weight=dw)
        return dq, dk, dv, dg, ds_in, None, None, None, None, dw


def lightning_attention(q, k, v, g=None, state_in=None, block_size: int = 256, phi: int = la.LA_PHI_SILU,
                        mode: int = la.LA_OUT_RMSNORM_GATE, eps: float = 1e-6, norm_weight=None):
    """Differentiable prefill: q, k, v [B, T, H, D]; g [B, T, H*D] (gated mode); state_in fp32
    [B, H, D, D] or None; norm_weight [H*D] or None.  Returns (out [B, T, H*D], state_out
    fp32 [B, H, D, D])."""
    if norm_weight is not None:
        norm_weight = norm_weight.float().contiguous()
    return _LightningAttention.apply(q, k, v, g, state_in, block_size, phi, mode, eps, norm_weight)


class _LightningAttentionVarlen(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, state_in, cu_seqlens, max_seqlen, block_size, phi, mode, eps, norm_weight):
        total, H, D = q.shape
        N = cu_seqlens.numel() - 1
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        g = None if g is None else g.contiguous()
        out = torch.empty((total, H * D), dtype=q.dtype, device=q.device)
        state_out = torch.empty((N, H, D, D), dtype=torch.float32, device=q.device)
        s_in = None if state_in is None else state_in.detach().contiguous()
        keep_y = mode != la.LA_OUT_RAW and (any(ctx.needs_input_grad[:5]) or ctx.needs_input_grad[11])
        y = None
        if keep_y:   # raw prefill, then the norm (and gate) from the kept y
            y = torch.empty_like(out)
            ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_PREFILL_VARLEN, N, max_seqlen, total, H, D,
                                                                   block_size, la._dtype(q), la.LA_OUT_RAW), q.device)
            la.lightning_attn_prefill_varlen(q, k, v, None, y, cu_seqlens, max_seqlen, s_in, state_out,
                                             block_size=block_size, phi=phi, mode=la.LA_OUT_RAW, workspace=ws)
            la.lightning_attn_output_transform(y.view(total, H, D), g, out, mode=mode, eps=eps,
                                               norm_weight=norm_weight)
        else:        # the fused kernel
            ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_PREFILL_VARLEN, N, max_seqlen, total, H, D,
                                                                   block_size, la._dtype(q), mode), q.device)
            la.lightning_attn_prefill_varlen(q, k, v, g, out, cu_seqlens, max_seqlen, s_in, state_out,
                                             block_size=block_size, phi=phi, mode=mode, eps=eps,
                                             norm_weight=norm_weight, workspace=ws)
        ctx.save_for_backward(q, k, v, g, s_in, cu_seqlens, None if norm_weight is None else norm_weight.detach(), y)
        ctx.cfg = (max_seqlen, block_size, phi, mode, eps)
        ctx.has_state = state_in is not None
        return out, state_out

    @staticmethod
    def backward(ctx, dout, dstate_out):
        q, k, v, g, s_in, cu, norm_weight, y = ctx.saved_tensors
        max_seqlen, block_size, phi, mode, eps = ctx.cfg
        total, H, D = q.shape
        N = cu.numel() - 1
        if dout is None:
            dout = torch.zeros((total, H * D), dtype=q.dtype, device=q.device)
        dout = dout.to(q.dtype).contiguous()
        dq, dk, dv = (torch.empty_like(q) for _ in range(3))
        dg = torch.empty_like(g) if mode == la.LA_OUT_RMSNORM_GATE else None
        ds_in = torch.empty((N, H, D, D), dtype=torch.float32, device=q.device) if ctx.has_state else None
        dw = torch.empty((H * D,), dtype=torch.float32, device=q.device) if ctx.needs_input_grad[11] else None
        ws = la.new_workspace(la.lightning_attn_workspace_size(la.LA_OP_BACKWARD_VARLEN, N, max_seqlen, total, H, D,
                                                               block_size, la._dtype(q), mode), q.device)
        la.lightning_attn_backward_varlen(q, k, v, g if mode == la.LA_OUT_RMSNORM_GATE else None, dout, dq, dk, dv, cu,
                                          max_seqlen, dg=dg, state_in=s_in, dstate_in=ds_in, block_size=block_size,
                                          phi=phi, mode=mode, eps=eps, norm_weight=norm_weight, workspace=ws,
                                          dstate_out=None if dstate_out is None else dstate_out.float().contiguous(),
                                          y=y, dnorm_weight=dw)
        return dq, dk, dv, dg, ds_in, None, None, None, None, None, None, dw


def lightning_attention_varlen(q, k, v, cu_seqlens, max_seqlen: int, g=None, state_in=None, block_size: int = 256,
                               phi: int = la.LA_PHI_SILU, mode: int = la.LA_OUT_RMSNORM_GATE, eps: float = 1e-6,
                               norm_weight=None):
    """Differentiable packed prefill: q, k, v [total, H, D] of N sequences (cu_seqlens int32
    device [N + 1], max_seqlen its longest); g [total, H*D] (gated mode); state_in fp32
    [N, H, D, D] or None.  Returns (out [total, H*D], state_out fp32 [N, H, D, D])."""
    if norm_weight is not None:
        norm_weight = norm_weight.float().contiguous()
    return _LightningAttentionVarlen.apply(q, k, v, g, state_in, cu_seqlens, int(max_seqlen), block_size, phi, mode,
                                           eps, norm_weight)


class _SequenceParallelLightningAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, state0, norm_weight, rank, all_gather, block_size, phi, mode, eps):
        _, T, H, D = q.shape
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        g = None if g is None else g.contiguous()
        s0 = None if state0 is None else state0.detach().contiguous()
        w = None if norm_weight is None else norm_weight.detach().contiguous()
        out = torch.empty((1, T, H * D), dtype=q.dtype, device=q.device)
        state_end = torch.empty((H, D, D), dtype=torch.float32, device=q.device)
        ws = sp.workspace_for(T, H, D, block_size, mode, q.device, la._dtype(q))
        y = None
        if mode != la.LA_OUT_RAW and any(ctx.needs_input_grad[:6]):   # keep the raw output for the backward
            y = torch.empty_like(out)
            prefix = sp.prefill_sequence_parallel(q, k, v, None, y, rank, all_gather, state0=s0, state_out=state_end,
                                                  block_size=block_size, phi=phi, mode=la.LA_OUT_RAW, workspace=ws)
            la.lightning_attn_output_transform(y.view(1, T, H, D), g, out, mode=mode, eps=eps, norm_weight=w)
        else:
            prefix = sp.prefill_sequence_parallel(q, k, v, g, out, rank, all_gather, state0=s0, state_out=state_end,
                                                  block_size=block_size, phi=phi, mode=mode, eps=eps, norm_weight=w,
                                                  workspace=ws)
        ctx.save_for_backward(q, k, v, g, prefix, w, y)
        ctx.cfg = (rank, all_gather, block_size, phi, mode, eps, state0 is not None)
        return out, state_end

    @staticmethod
    def backward(ctx, dout, dstate_end):
        q, k, v, g, prefix, w, y = ctx.saved_tensors
        rank, all_gather, block_size, phi, mode, eps, has_s0 = ctx.cfg
        _, T, H, D = q.shape
        if dout is None:
            dout = torch.zeros((1, T, H * D), dtype=q.dtype, device=q.device)
        dout = dout.to(q.dtype).contiguous()
        dq, dk, dv = (torch.empty_like(q) for _ in range(3))
        dg = torch.empty_like(g) if mode == la.LA_OUT_RMSNORM_GATE else None
        dw = torch.empty((H * D,), dtype=torch.float32, device=q.device) if ctx.needs_input_grad[5] else None
        ds_in = torch.empty((H, D, D), dtype=torch.float32, device=q.device) if has_s0 else None
        sp.backward_sequence_parallel(q, k, v, g, dout, dq, dk, dv, rank, prefix, all_gather,
                                      dstate_end=None if dstate_end is None else dstate_end.float().contiguous(),
                                      y=y, dg=dg, dnorm_weight=dw, dstate_in=ds_in, block_size=block_size, phi=phi,
                                      mode=mode, eps=eps, norm_weight=w)
        # state0 is the same tensor on every rank: rank 0 returns its whole gradient and the
        # others zero, so that adding the ranks' gradients (as for the norm weight's per-chunk
        # parts) gives the total
        if ds_in is not None and rank != 0:
            ds_in.zero_()
        return dq, dk, dv, dg, ds_in, dw, None, None, None, None, None, None


def lightning_attention_sequence_parallel(q, k, v, g=None, state0=None, norm_weight=None, rank: int = 0,
                                          all_gather=sp.nccl_all_gather, block_size: int = 256,
                                          phi: int = la.LA_PHI_SILU, mode: int = la.LA_OUT_RMSNORM_GATE,
                                          eps: float = 1e-6):
    """Differentiable sequence-parallel prefill: this rank's contiguous chunk q, k, v
    [1, T, H, D] (g [1, T, H*D]) of one sequence split across the group's ranks in order.
    Returns (out [1, T, H*D], the state at the end of this chunk fp32 [H, D, D]: on the last
    rank the sequence's final state).  One all-gather in the forward and one in the backward,
    so every rank must call it in the same order and back-propagate through its output.
    Gradients of state0 and the norm weight (the same tensors on every rank) come as per-rank
    parts to be added over the ranks, as data-parallel gradients are."""
    if norm_weight is not None:
        norm_weight = norm_weight.float().contiguous()
    return _SequenceParallelLightningAttention.apply(q, k, v, g, state0, norm_weight, rank, all_gather, block_size,
                                                     phi, mode, eps)


def _aligned(t):
    """t as the library takes it: contiguous, from a 16-byte boundary (a slice may start anywhere, and so may
    the gradients that torch.cat and split hand back).  A copy only where it is not."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _GatedRecurrence(torch.autograd.Function):
    """x, f [B, T, W] (cu_seqlens None) or packed [total, W]."""

    @staticmethod
    def forward(ctx, x, f, state_in, cu_seqlens, input_mode, workspace):
        ctx.set_materialize_grads(False)
        x, f, cu_seqlens = _aligned(x), _aligned(f), _aligned(cu_seqlens)
        W = x.shape[-1]
        tokens = x.shape[0] if cu_seqlens is not None else x.shape[0] * x.shape[1]
        n = x.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        out = torch.empty_like(x)
        state_out = torch.empty((n, W), dtype=torch.float32, device=x.device)
        s_in = None if state_in is None else _aligned(state_in.detach())
        saved = la.new_recurrence_checkpoints(tokens, W, x.device) if any(ctx.needs_input_grad) else None
        ws = workspace
        if ws is None:
            ws = la.new_workspace(la.lightning_attn_gated_recurrence_workspace_size(n, tokens, W, la._dtype(x)), x.device)
        if cu_seqlens is None:
            la.lightning_attn_gated_recurrence(x, f, out, s_in, state_out, saved, input_mode, ws)
        else:
            la.lightning_attn_gated_recurrence_varlen(x, f, out, cu_seqlens, s_in, state_out, saved, input_mode, ws)
        ctx.save_for_backward(x, f, s_in, cu_seqlens, saved)
        ctx.cfg = (n, tokens, input_mode, workspace)
        return out, state_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dstate_out):
        x, f, s_in, cu, saved = ctx.saved_tensors
        n, tokens, input_mode, ws = ctx.cfg
        W = x.shape[-1]
        dout = torch.zeros_like(x) if dout is None else _aligned(dout.to(x.dtype))
        ds_out = None if dstate_out is None else _aligned(dstate_out.float())
        dx, df = torch.empty_like(x), torch.empty_like(f)
        ds_in = torch.empty((n, W), dtype=torch.float32, device=x.device) if ctx.needs_input_grad[2] else None
        if ws is None:
            ws = la.new_workspace(la.lightning_attn_gated_recurrence_workspace_size(n, tokens, W, la._dtype(x), True),
                                  x.device)
        if cu is None:
            la.lightning_attn_gated_recurrence_backward(x, f, dout, dx, df, s_in, ds_out, ds_in, saved, input_mode, ws)
        else:
            la.lightning_attn_gated_recurrence_backward_varlen(x, f, dout, dx, df, cu, s_in, ds_out, ds_in, saved,
                                                               input_mode, ws)
        return dx, df, ds_in, None, None, None


def gated_recurrence(x, f, state_in=None, input_mode: int = la.LA_INPUT_TIED, workspace=None):
    """Differentiable gated recurrence h_t = a_t h_{t-1} + b_t, a = sigmoid(f), b = x or (1 - a) x:
    x, f [B, T, W]; state_in fp32 [B, W] or None.  Returns (out [B, T, W], state_out fp32 [B, W]).
    Failures found on the device (malformed cu_seqlens, a wait that ran out) are recorded in
    `workspace`, the caller's, where lightning_attn_check finds them after the forward and after the
    backward: from new_workspace, lightning_attn_gated_recurrence_workspace_size(..., backward=True)
    bytes.  Without one, each call makes its own and the record is lost with it."""
    return _GatedRecurrence.apply(x, f, state_in, None, input_mode, workspace)


def gated_recurrence_varlen(x, f, cu_seqlens, state_in=None, input_mode: int = la.LA_INPUT_TIED, workspace=None):
    """Differentiable gated recurrence over packed sequences: x, f [total, W]; cu_seqlens int32
    device [N + 1] with cu_seqlens[N] == total; state_in fp32 [N, W] or None; workspace as for
    gated_recurrence.  Returns (out [total, W], state_out fp32 [N, W])."""
    return _GatedRecurrence.apply(x, f, state_in, cu_seqlens, input_mode, workspace)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        ctx.set_materialize_grads(False)
        x, residual = _aligned(x), _aligned(residual)
        weight, bias = (None if t is None else _aligned(t.detach()) for t in (weight, bias))
        out = torch.empty_like(x)
        s = None if residual is None else torch.empty_like(x)
        la.lightning_attn_layer_norm(x, out, residual=residual, sum_out=s, weight=weight, bias=bias, eps=eps)
        ctx.save_for_backward(x if s is None else s, weight)
        ctx.eps = eps
        return out if s is None else (out, s)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dsum=None):
        s, weight = ctx.saved_tensors
        W = s.shape[-1]
        need = ctx.needs_input_grad
        dout = torch.zeros_like(s) if dout is None else _aligned(dout.to(s.dtype))
        dsum = None if dsum is None else _aligned(dsum.to(s.dtype))
        dx = torch.empty_like(s)
        dw, db = (torch.empty(W, dtype=torch.float32, device=s.device) if n else None for n in need[1:3])
        ws = None
        if need[1] or need[2]:
            ws = la.new_workspace(la.lightning_attn_layer_norm_workspace_size(s.numel() // W, W), s.device)
        la.lightning_attn_layer_norm_backward(s, dout, dx, dsum=dsum, weight=weight, dweight=dw, dbias=db,
                                              eps=ctx.eps, workspace=ws)
        return dx if need[0] else None, dw, db, dx if need[3] else None, None


def layer_norm(x, weight=None, bias=None, residual=None, eps: float = 1e-5):
    """Differentiable layer norm of x (+ residual) over the last axis: x, residual [..., W]; weight,
    bias [W] or None.  Returns out, or (out, x + residual) where a residual is given."""
    weight, bias = (None if t is None else t.float().contiguous() for t in (weight, bias))
    return _LayerNorm.apply(x, weight, bias, residual, eps)

"""torch.autograd wrappers of the attention-boundary re-layouts.

A training step needs the re-layouts on both passes.  The gradient of a
permutation is its inverse, so each forward call's backward is the library's
call in the other direction (include/basp.h, "Backward pass of the same
boundary"):

* ``seq_to_head_qkv(plan, q, k, v)`` runs ``basp_seq_to_head`` (fused Q, K, V
  sequence-sharded -> head-sharded) and, on the backward pass,
  ``basp_head_to_seq_qkv`` (the fused gradient head-sharded -> dQ, dK, dV
  sequence-sharded);
* ``head_to_seq_o(plan, o)`` runs ``basp_head_to_seq`` (attention output
  head-sharded -> sequence-sharded) and, on the backward pass,
  ``basp_seq_to_head_o`` (dO sequence-sharded -> head-sharded).

The index-driven re-layouts (include/basp.h, "Index-driven re-layouts") have
their gradients in the same way:

* ``route_to_expert(expert_plan, x, ids)`` sorts the tokens by expert and
  returns their rows with the index; ``seq_to_expert(expert_plan, x, index)``
  moves by an index that is there; backward: ``basp_seq_to_expert_grad``;
* ``expert_to_seq(expert_plan, rows, weights, index)`` returns the weighted
  sums of the tokens' rows; backward: ``basp_expert_to_seq_grad``, one call that
  computes the gradients of rows and of weights, also where only one of them is
  asked for (rows and weights are kept until then);
* ``embed_to_seq(embed_plan, ids, table, scale)`` looks rows up into the
  sequence-sharded layout; backward, for the table (whose gradient has the
  plan's grad_dtype until autograd casts it to the table's):
  ``basp_embed_to_seq_grad``.

Tensors are contiguous and of the plan's dtype and element counts, as the
binding checks; outputs are allocated with torch on the inputs' device.  Only
buffers are marshalled here: every element is moved by the library's kernels.
The gradients are not themselves differentiable: a loss with one of them in it
is refused.  An index, rows or ids that a backward pass still needs must not be
written again through the binding's calls before it: torch does not see these
writes.

In HIP graphs, capture a backward pass together with its forward pass, on leaf
tensors that no live graph of eager calls holds: torch ties a leaf's gradient to
the stream of its first use.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding as b


class _Gradient(torch.autograd.Function):
    """compute(*tensors) of a backward pass.  With create_graph, autograd sees
    that the gradient depends on these tensors, and differentiating it again
    is an error wherever it stands in a loss."""

    @staticmethod
    def forward(ctx, compute, *tensors):
        return compute(*tensors)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients of the re-layouts are not themselves differentiable")


class _SeqToHeadQKV(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, q, k, v):
        i = plan.info
        out = torch.empty(i["qkv_elems"], dtype=q.dtype, device=q.device)
        b.basp_seq_to_head(plan, q, k, v, out)
        ctx.plan = plan
        return out

    @staticmethod
    def backward(ctx, grad):
        def compute(grad):
            i = ctx.plan.info
            dev, dt = grad.device, grad.dtype
            dq = torch.empty(i["q_elems"], dtype=dt, device=dev)
            dk = torch.empty(i["kv_elems"], dtype=dt, device=dev)
            dv = torch.empty(i["kv_elems"], dtype=dt, device=dev)
            b.basp_head_to_seq_qkv(ctx.plan, grad.contiguous(), dq, dk, dv)
            return dq, dk, dv

        return (None, *_Gradient.apply(compute, grad))


class _HeadToSeqO(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, o):
        out = torch.empty(plan.info["q_elems"], dtype=o.dtype, device=o.device)
        b.basp_head_to_seq(plan, o, out)
        ctx.plan = plan
        return out

    @staticmethod
    def backward(ctx, grad):
        def compute(grad):
            do = torch.empty(ctx.plan.info["q_elems"], dtype=grad.dtype, device=grad.device)
            b.basp_seq_to_head_o(ctx.plan, grad.contiguous(), do)
            return do

        return None, _Gradient.apply(compute, grad)


def seq_to_head_qkv(plan, q, k, v):
    """Fused Q/K/V seq -> head with its backward (see the module docstring).
    Returns the head-sharded HEAD(Q) || HEAD(K) || HEAD(V) buffer."""
    return _SeqToHeadQKV.apply(plan, q, k, v)


def head_to_seq_o(plan, o):
    """Attention output head -> seq with its backward (see the module
    docstring).  Returns the sequence-sharded output."""
    return _HeadToSeqO.apply(plan, o)


# ------------------------------------------------ index-driven re-layouts --

class ExpertIndex(NamedTuple):
    """What basp_expert_sort returns: int32 tensors on the device."""
    pos: torch.Tensor
    order: torch.Tensor
    offsets: torch.Tensor
    counts: torch.Tensor


def _index_buffers(plan, device):
    i = plan.info
    return ExpertIndex(*(torch.empty(n, dtype=torch.int32, device=device)
                         for n in (i["slots"], i["max_rows"], i["E"] + 1, i["E"])))


def _workspace(plan, device):
    return torch.empty(plan.info["workspace_bytes"], dtype=torch.uint8, device=device)


def _tokens_grad(plan, shape, pos):
    def compute(grad):
        dx = torch.empty(shape, dtype=grad.dtype, device=grad.device)
        b.basp_seq_to_expert_grad(plan, grad.contiguous(), pos, dx)
        return dx
    return compute


class _RouteToExpert(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, ids):
        i = plan.info
        index = _index_buffers(plan, x.device)
        rows = torch.empty(i["max_rows"], i["D"], dtype=x.dtype, device=x.device)
        b.basp_route_to_expert(plan, x, ids, *index, rows, _workspace(plan, x.device))
        ctx.plan, ctx.shape = plan, x.shape
        ctx.save_for_backward(index.pos)
        ctx.mark_non_differentiable(*index)
        return (rows, *index)

    @staticmethod
    def backward(ctx, grad, *_):
        (pos,) = ctx.saved_tensors
        return None, _Gradient.apply(_tokens_grad(ctx.plan, ctx.shape, pos), grad), None


class _SeqToExpert(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, x, pos, order):
        i = plan.info
        rows = torch.empty(i["max_rows"], i["D"], dtype=x.dtype, device=x.device)
        b.basp_seq_to_expert(plan, x, pos, order, rows)
        ctx.plan, ctx.shape = plan, x.shape
        ctx.save_for_backward(pos)
        return rows

    @staticmethod
    def backward(ctx, grad):
        (pos,) = ctx.saved_tensors
        return None, _Gradient.apply(_tokens_grad(ctx.plan, ctx.shape, pos), grad), None, None


class _ExpertToSeq(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, rows, weights, pos, order):
        i = plan.info
        out = torch.empty(i["T"], i["D"], dtype=rows.dtype, device=rows.device)
        b.basp_expert_to_seq(plan, rows, pos, weights, out)
        ctx.plan = plan
        ctx.save_for_backward(rows, weights, pos, order)
        return out

    @staticmethod
    def backward(ctx, grad):
        rows, weights, pos, order = ctx.saved_tensors

        def compute(grad, rows, weights):
            drows, dweights = torch.empty_like(rows), torch.empty_like(weights)
            b.basp_expert_to_seq_grad(ctx.plan, grad.contiguous(), rows, pos, order, weights, drows, dweights)
            return drows, dweights

        return (None, *_Gradient.apply(compute, grad, rows, weights), None, None)


class _EmbedToSeq(torch.autograd.Function):
    @staticmethod
    def forward(ctx, plan, ids, table, scale):
        i = plan.info
        out = torch.empty(i["T"], i["D"], dtype=table.dtype, device=table.device)
        b.basp_embed_to_seq(plan, ids, table, scale, out)
        ctx.plan, ctx.scale, ctx.shape = plan, scale, table.shape
        ctx.save_for_backward(ids)
        return out

    @staticmethod
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        plan = ctx.plan

        def compute(grad):
            dtable = torch.empty(ctx.shape, dtype=plan.grad[0], device=grad.device)
            b.basp_embed_to_seq_grad(plan, ids, grad.contiguous(), ctx.scale, False, dtable,
                                     _workspace(plan, grad.device))
            return dtable

        return None, None, _Gradient.apply(compute, grad), None


def sort_by_expert(plan, ids):
    """The ExpertIndex of ids [T][K] (basp_expert_sort)."""
    index = _index_buffers(plan, ids.device)
    b.basp_expert_sort(plan, ids, *index, _workspace(plan, ids.device))
    return index


def route_to_expert(plan, x, ids):
    """Tokens sorted by expert with their backward (see the module docstring).
    Returns (rows [max_rows][D], ExpertIndex)."""
    rows, *index = _RouteToExpert.apply(plan, x, ids)
    return rows, ExpertIndex(*index)


def seq_to_expert(plan, x, index):
    """The rows [max_rows][D] of tokens x by an ExpertIndex, with backward."""
    return _SeqToExpert.apply(plan, x, index.pos, index.order)


def expert_to_seq(plan, rows, weights, index):
    """Weighted sums [T][D] of the tokens' rows, with backward for both."""
    return _ExpertToSeq.apply(plan, rows, weights, index.pos, index.order)


def embed_to_seq(plan, ids, table, scale=1.0):
    """Scaled rows [T][D] of the table in the plan's order, with backward for
    the table."""
    return _EmbedToSeq.apply(plan, ids, table, scale)

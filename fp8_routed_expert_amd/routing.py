"""Tokens sorted by expert and back, differentiable: the autograd form of
moe_sort_tokens, moe_permute_rows and moe_combine_rows, for experts that are
trained in float32, bfloat16 or float16.

    table = sort_tokens(topk_idx, E, rows)
    a = permute_tokens(x, table)             # [rows_total, H], empty rows 0
    y = ...                                  # experts, segment by segment
    out = combine_tokens(y, topk_w, table)   # [T, H]

All calls run on the current stream of the tensors' device.  sort_tokens
allocates its table, so a table that a backward pass still needs is not
overwritten by the next one.  Nothing is read back: the calls can be captured
in a graph (table.status then tells, after a replay, of bad ids and dropped
rows).  As with every captured backward pass, free the eager passes over the
same leaves first: an accumulation that belongs to another stream's pass ends
the capture and the process.
"""

import torch

from . import ops


class SortedTokens:
    """The table that sort_tokens returns: counts [E], offsets [E + 1],
    slot_of [T, K], row_src and row_expert [rows_total], status [1] (all int32;
    the meaning and status bits of moe_dispatch_layout)."""

    __slots__ = ("T", "K", "E", "rows_total", "counts", "offsets", "slot_of", "row_src",
                 "row_expert", "status")


def sort_tokens(topk_idx, E, rows, layout=ops.LAYOUT_CONTIGUOUS, align_m=128):
    """Sorts the picks topk_idx (int32 [T, K]; -1: none) by expert.  rows: rows
    of the buffer (contiguous) or of each expert's segment (masked)."""
    T, K = topk_idx.shape
    d = topk_idx.device
    R = E * rows if layout == ops.LAYOUT_MASKED else rows
    s = SortedTokens()
    s.T, s.K, s.E, s.rows_total = T, K, E, R
    new = lambda *shape: torch.empty(shape, dtype=torch.int32, device=d)  # noqa: E731
    s.counts, s.offsets, s.slot_of, s.row_src, s.row_expert = (new(E), new(E + 1), new(T, K),
                                                               new(R), new(R))
    s.status = torch.zeros(1, dtype=torch.int32, device=d)
    ws = torch.empty(max(1, ops.moe_layout_workspace_bytes(T, K, E)), dtype=torch.uint8, device=d)
    ops.moe_sort_tokens(topk_idx, E, layout, align_m, rows, s.counts, s.offsets, s.slot_of,
                        s.row_src, s.row_expert, ws, s.status)
    return s


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table):
        ctx.table = table
        a = x.new_empty(table.rows_total, x.shape[1])
        ops.moe_permute_rows(x.contiguous(), table.slot_of, a, table.status, table.row_src)
        return a

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, da):
        t = ctx.table
        dx = da.new_empty(t.T, da.shape[1])
        ops.moe_permute_rows_grad(da.contiguous(), t.slot_of, dx, t.status)
        return dx, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, topk_w, table):
        y, topk_w = y.contiguous(), topk_w.contiguous()
        ctx.table = table
        # y's gradient reads the weights, the weights' y: nothing else is kept
        needs_y, needs_w = ctx.needs_input_grad[:2]
        ctx.save_for_backward(y if needs_w else None, topk_w if needs_y else None)
        out = y.new_empty(table.T, y.shape[1])
        ops.moe_combine_rows(y, table.slot_of, topk_w, out, table.status)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        t = ctx.table
        y, w = ctx.saved_tensors
        dy = dout.new_empty(t.rows_total, dout.shape[1]) if ctx.needs_input_grad[0] else None
        dw = dout.new_empty(t.T, t.K, dtype=torch.float32) if ctx.needs_input_grad[1] else None
        ops.moe_combine_rows_grad(dout.contiguous(), y, t.slot_of, w, dy, dw, t.status, t.row_src)
        return dy, dw, None


def permute_tokens(x, table):
    """a [rows_total, H] with a[slot_of[t, k]] = x[t] and zeros in the rows that
    no token goes to.  x [T, H] float32, bfloat16 or float16."""
    return _Permute.apply(x, table)


def combine_tokens(y, topk_w, table):
    """out [T, H] = sum_k topk_w[t, k] * y[slot_of[t, k]]; gradients for y
    (zero in the rows that no token has) and topk_w (float32 [T, K])."""
    if y.shape[0] != table.rows_total:
        raise ValueError(f"y: {y.shape[0]} rows, the table's buffer has {table.rows_total}")
    return _Combine.apply(y, topk_w, table)

"""A routed-expert block that is trained, or kept in float32, bfloat16 or
float16: the norm, the router and the experts' products under autograd, next to
the sorting of the tokens (routing.py).

    xn = layer_norm(x, weight, bias)                      # [T, H]
    topk_idx, topk_w, scores = route_tokens(logits, K)    # logits [T, E]
    table = sort_tokens(topk_idx, E, contiguous_rows(T * K, E))
    a = permute_tokens(xn, table)
    q = gated_act(grouped_linear(a, w13, table), table)   # w13 [E, 2I, H]
    y = grouped_linear(q, w2, table)                      # w2 [E, H, I]
    out = combine_tokens(y, topk_w, table)                # [T, H]

RoutedExperts is that block as a module.  All calls run on the current stream
of the tensors' device, read nothing back and can be captured in a graph (free
the eager passes over the same leaves first, as routing.py says).  Every call
allocates its own workspace.  Rows of a buffer that no expert has come out as
zeros.
"""

import torch

from . import ops
from .layer import contiguous_rows
from .routing import combine_tokens, permute_tokens, sort_tokens


def _workspace(nbytes, device):
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = x.contiguous().view(-1, x.shape[-1])
        y = torch.empty_like(rows)
        mean = rows.new_empty(rows.shape[0], dtype=torch.float32)
        rstd = torch.empty_like(mean)
        weight = None if weight is None else weight.contiguous()
        bias = None if bias is None else bias.contiguous()
        ops.moe_layer_norm(rows, weight, bias, eps, y, mean, rstd)
        ctx.save_for_backward(rows, weight, mean, rstd)
        ctx.param = next((p.dtype for p in (weight, bias) if p is not None), None)
        return y.view(x.shape)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        rows, weight, mean, rstd = ctx.saved_tensors
        T, H = rows.shape
        want = ctx.needs_input_grad
        dx = torch.empty_like(rows) if want[0] else None
        dw = rows.new_empty(H, dtype=ctx.param) if want[1] else None
        db = rows.new_empty(H, dtype=ctx.param) if want[2] else None
        ops.moe_layer_norm_grad(dy.contiguous().view(T, H), rows, weight, mean, rstd, dx, dw, db,
                                _workspace(ops.moe_layer_norm_workspace_bytes(T, H), rows.device))
        return None if dx is None else dx.view(dy.shape), dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension of x (float32, bfloat16 or float16);
    weight and bias [H] of x's type or float32, or None."""
    return _Norm.apply(x, weight, bias, eps)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, bias, kw, status):
        logits = logits.contiguous()
        T, E = logits.shape
        idx = logits.new_empty(T, K, dtype=torch.int32)
        w = logits.new_empty(T, K, dtype=torch.float32)
        scores = logits.new_empty(T, E, dtype=torch.float32)
        ops.moe_route_tokens(logits, idx, w, status, bias, scores=scores, **kw)
        ctx.save_for_backward(logits, idx)
        ctx.status = status
        ctx.kw = {k: kw[k] for k in ("score", "renorm", "scale")}
        ctx.mark_non_differentiable(idx)
        ctx.set_materialize_grads(False)
        return idx, w, scores

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, dw, dscores):
        logits, idx = ctx.saved_tensors
        if dw is None and dscores is None:
            return None, None, None, None, None
        dw = logits.new_zeros(idx.shape, dtype=torch.float32) if dw is None else dw.contiguous()
        dscores = None if dscores is None else dscores.contiguous()
        dlogits = torch.empty_like(logits)
        ops.moe_route_tokens_grad(logits, idx, dw, dlogits, ctx.status, dscores=dscores, **ctx.kw)
        return dlogits, None, None, None, None


def route_tokens(logits, K, bias=None, score=ops.SCORE_SOFTMAX, groups=1, top_groups=1,
                 group_best=1, renorm=True, scale=1.0, status=None):
    """Picks (int32 [T, K], -1: none), weights (float32 [T, K]) and scores
    (float32 [T, E]) of logits [T, E]; gradients from weights and scores to the
    logits.  bias [E] float32 moves the choice and gets none.  status (int32
    [1], zeroed by the caller) tells of NaN logits."""
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=logits.device)
    kw = dict(score=score, groups=groups, top_groups=top_groups, group_best=group_best,
              renorm=renorm, scale=scale)
    return _Route.apply(logits, K, bias, kw, status)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, w, table):
        a, w = a.contiguous(), w.contiguous()
        ctx.table = table
        # a's gradient reads the weights, the weights' a: nothing else is kept
        needs_a, needs_w = ctx.needs_input_grad[:2]
        ctx.save_for_backward(a if needs_w else None, w if needs_a else None)
        ctx.shapes = a.shape, w.shape
        c = a.new_empty(a.shape[0], w.shape[1])
        ops.moe_grouped_gemm_float(a, w, table.offsets, table.counts, c, table.status, True)
        return c

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dc):
        t = ctx.table
        a, w = ctx.saved_tensors
        (R, K), (E, N, _) = ctx.shapes
        dc = dc.contiguous()
        da = dw = None
        if ctx.needs_input_grad[0]:
            da = dc.new_empty(R, K)
            ops.moe_grouped_gemm_float_grad_rows(dc, w, t.offsets, t.counts, da, t.status, True)
        if ctx.needs_input_grad[1]:
            dw = dc.new_empty(E, N, K)
            ws = _workspace(ops.moe_grouped_gemm_float_workspace_bytes(E, R, N, K), dc.device)
            ops.moe_grouped_gemm_float_grad_weights(dc, a, t.offsets, t.counts, dw, ws, t.status)
        return da, dw, None


class _Act(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, table):
        h = h.contiguous()
        ctx.table = table
        ctx.save_for_backward(h)
        q = h.new_empty(h.shape[0], h.shape[1] // 2)
        ops.moe_gated_act(h, table.offsets, table.counts, q, table.status, True)
        return q

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq):
        t = ctx.table
        h, = ctx.saved_tensors
        dh = torch.empty_like(h)
        ops.moe_gated_act_grad(dq.contiguous(), h, t.offsets, t.counts, dh, t.status, True)
        return dh, None


def _rows_of(table, t, name):
    if t.shape[0] != table.rows_total:
        raise ValueError(f"{name}: {t.shape[0]} rows, the table's buffer has {table.rows_total}")


def grouped_linear(a, w, table):
    """c [rows_total, N]: row r of a [rows_total, K] with its expert's weights
    w[e] [N, K] (both float32, bfloat16 or float16)."""
    _rows_of(table, a, "a")
    if w.shape[0] != table.E:
        raise ValueError(f"w: {w.shape[0]} experts, the table has {table.E}")
    return _Linear.apply(a, w, table)


def gated_act(h, table):
    """silu(h[:, :I]) * h[:, I:] of h [rows_total, 2I]."""
    _rows_of(table, h, "h")
    return _Act.apply(h, table)


class RoutedExperts(torch.nn.Module):
    """x [T, H] -> [T, H]: norm, router, experts and the weighted sum of their
    outputs (the residual is the caller's).  The router's product is in float32.
    bias [E] float32 (a buffer, not a parameter) moves the choice of experts; a
    balancing scheme writes it.  After a call, `scores` holds the router's
    scores [T, E] and `table` the sorted tokens (its status tells of dropped
    rows, `route_status` of NaN logits).  with_scores=True returns (output,
    scores): what a balancing loss takes where the call is checkpointed, since a
    re-entrant checkpoint's first pass leaves `scores` without a graph."""

    def __init__(self, E, H, I, K, score=ops.SCORE_SOFTMAX, groups=1, top_groups=1, group_best=1,
                 renorm=True, scale=1.0, eps=1e-5, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        new = lambda *s, dt=dtype: torch.nn.Parameter(  # noqa: E731
            torch.empty(*s, dtype=dt, device=device))
        self.E, self.K, self.eps = E, K, eps
        self.route = dict(score=score, groups=groups, top_groups=top_groups, group_best=group_best,
                          renorm=renorm, scale=scale)
        self.norm_weight, self.norm_bias = new(H), new(H)
        self.router = new(E, H, dt=torch.float32)
        self.w13, self.w2 = new(E, 2 * I, H), new(E, H, I)
        self.register_buffer("bias", torch.zeros(E, dtype=torch.float32, device=device))
        torch.nn.init.ones_(self.norm_weight)
        torch.nn.init.zeros_(self.norm_bias)
        for w in (self.router, self.w13, self.w2):
            torch.nn.init.normal_(w, std=0.02)
        self.scores = self.table = self.route_status = None

    def __getstate__(self):
        # (a copy starts without what the last call left: a graph's tensors
        # cannot be copied)
        return {**self.__dict__, "scores": None, "table": None, "route_status": None}

    def forward(self, x, with_scores=False):
        # what the last call left holds its graph, whose accumulations belong
        # to that call's stream and would end a capture of this one
        self.scores = self.table = self.route_status = None
        xn = layer_norm(x, self.norm_weight, self.norm_bias, self.eps)
        # (router and bias are float32, unless the module was converted)
        with torch.autocast(x.device.type, enabled=False):
            logits = torch.nn.functional.linear(xn.float(), self.router.float())
        self.route_status = torch.zeros(1, dtype=torch.int32, device=x.device)
        idx, w, self.scores = route_tokens(logits, self.K, self.bias.float(),
                                           status=self.route_status, **self.route)
        t = self.table = sort_tokens(idx, self.E, contiguous_rows(idx.numel(), self.E))
        a = permute_tokens(xn, t)
        q = gated_act(grouped_linear(a, self.w13, t), t)
        out = combine_tokens(grouped_linear(q, self.w2, t), w, t)
        return (out, self.scores) if with_scores else out

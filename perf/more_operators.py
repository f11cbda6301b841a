"""What is measured of the operators around the experts that are trained: the
router (scores, groups, top-k, weights) and its gradient, the layer norm and its
gradient, the experts' products in 32- and 16-bit types with both gradients, and
the gated activation between them with its gradient.

`run` computes a case in its plain form (elementary torch operations) or, with
`own` set, through this package's calls; both take what `prepare` gives.
"""

import math

import torch

own = False

CONTIGUOUS, MASKED = 0, 1
SOFTMAX, SIGMOID = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
ALIGN = 128                  # rows that a contiguous segment is rounded up to
LEAST_SUM = 2.0 ** -64       # picked scores that sum to less are divided by this


# ---------------------------------------------------------------- the cases
def _route(op, T, E, K, dtype, score=SIGMOID, groups=1, top_groups=1, group_best=1, bias=True, renorm=True,
           scale=1.0, padded=False, aux=False):
    """T tokens' logits over E experts.  padded: some tokens are padding, all
    of whose logits are -infinity.  aux: a loss reads the scores as well."""
    return {"op": op, "T": T, "E": E, "K": K, "dtype": dtype, "score": score, "groups": groups,
            "top_groups": top_groups, "group_best": group_best, "bias": bias, "renorm": renorm, "scale": scale,
            "padded": padded, "aux": aux}


def _norm(op, T, H, dtype, w_dtype, bias=True):
    return {"op": op, "T": T, "H": H, "dtype": dtype, "w_dtype": w_dtype, "bias": bias}


def _experts(op, R, E, N, K, dtype, layout=CONTIGUOUS, capacity=0, w_dtype=""):
    """R routed rows on E experts.  Products: N outputs from K inputs, weights'
    gradients of w_dtype (the rows' type by default).  Activations: N = 2 K."""
    return {"op": op, "R": R, "E": E, "N": N, "K": K, "dtype": dtype, "layout": layout, "capacity": capacity,
            "w_dtype": w_dtype or dtype}


def listed():
    return [
        # one token of a decode step: all latency
        dict(_route("route", 1, 256, 8, "f32", SIGMOID, 8, 4, 2, scale=2.5), name="route one token"),
        # a prefill chunk, picks limited to 4 of 8 groups, a bias that balances the load
        dict(_route("route", 65536, 256, 8, "f32", SIGMOID, 8, 4, 2, scale=2.5, padded=True), name="route prefill"),
        # a training micro-batch's router, with a loss on the scores
        dict(_route("route_grad", 16384, 72, 6, "bf16", SOFTMAX, aux=True), name="route gradient"),
        # one token through the norm in front of the experts
        dict(_norm("norm", 1, 7168, "bf16", "bf16"), name="norm one token"),
        # a prefill chunk through it
        dict(_norm("norm", 65536, 7168, "bf16", "f32"), name="norm prefill"),
        # the norm's gradient in a training step
        dict(_norm("norm_grad", 32768, 7168, "bf16", "bf16"), name="norm gradient"),
        # gate and up of a decode step in the fixed-capacity layout: a few rows each
        dict(_experts("product", 256, 32, 4096, 7168, "bf16", MASKED, 16), name="product decode"),
        # gate and up of the prefill share: the largest product
        dict(_experts("product", 131040, 9, 4096, 7168, "bf16"), name="product prefill"),
        # a training micro-batch on 6 experts: gradients of the down product's rows and weights
        dict(_experts("product_grad", 6144, 6, 7168, 2048, "f16", w_dtype="f32"), name="product gradient"),
        # the same of a small model in 32 bits, with sizes that no tile divides
        dict(_experts("product_grad", 777, 5, 328, 520, "f32"), name="product gradient odd"),
        # the activation of a decode share
        dict(_experts("act", 1193, 32, 4096, 2048, "f16", MASKED, 128), name="act decode"),
        # its gradient at the prefill share
        dict(_experts("act_grad", 131040, 9, 4096, 2048, "bf16"), name="act gradient prefill"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "norm", "norm_grad", "product", "product", "product_grad",
                     "product_grad", "act", "act_grad"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 8, 512 // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        K = rng.randint(1, min(16, E * top_groups // groups))
        best = rng.choice([1, 2])
        return _route(op, _log(rng, 1, 65536), E, K, dtype, rng.choice([SOFTMAX, SIGMOID]), groups, top_groups, best,
                      rng.random() < 0.6, rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.random() < 0.4,
                      op == "route_grad" and rng.random() < 0.5)
    if op in ("norm", "norm_grad"):
        H = _log(rng, 64, 8192)
        T = min(_log(rng, 1, 65536), 32768 * 7168 // H)
        return _norm(op, T, H, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.7)
    E = _log(rng, 1, 64)
    R = _log(rng, 1, 131072)
    layout = rng.choice([CONTIGUOUS, MASKED])
    if op in ("act", "act_grad"):
        I = 8 * _log(rng, 16, 512)
        R = max(1, min(R, 131040 * 2048 // I // (2 if dtype == "f32" else 1)))
        N, K = 2 * I, I
    else:
        dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
        N, K = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 896)
        E = max(1, min(E, (1 << 30) // (N * K)))
        # no more multiplications than the largest listed case has, 1/32 of them in 32 bits
        most = 131040 * 4096 * 7168 // (32 if dtype == "f32" else 2)
        R = max(1, min(R, most // (N * K)))
    capacity = max(8, int(R / E * rng.choice([1.0, 1.5, 3.0]))) if layout == MASKED else 0
    return _experts(op, R, E, N, K, dtype, layout, capacity, rng.choice([dtype, "f32"]))


def _rows_total(c):
    """Rows of the buffer that a program sets aside for the case."""
    return c["E"] * c["capacity"] if c["layout"] == MASKED else c["R"] + (ALIGN - 1) * c["E"]


def work(c):
    op, b = c["op"], BYTES[c["dtype"]]
    if op in ("route", "route_grad"):
        T, E, K = c["T"], c["E"], c["K"]
        if op == "route":
            return {"bytes": T * (E * b + 8 * K), "flops": 10 * T * E}
        return {"bytes": T * (E * (2 * b + (4 if c["aux"] else 0)) + 8 * K), "flops": 12 * T * E}
    if op in ("norm", "norm_grad"):
        T, H, wb = c["T"], c["H"], BYTES[c["w_dtype"]]
        if op == "norm":
            return {"bytes": 2 * T * H * b + 2 * H * wb + 8 * T, "flops": 7 * T * H}
        return {"bytes": 3 * T * H * b + 3 * H * wb + 8 * T, "flops": 14 * T * H}
    R, E, N, K = c["R"], c["E"], c["N"], c["K"]
    if c["layout"] == MASKED:
        R = min(R, E * c["capacity"])
    if op == "act":
        return {"bytes": b * R * (N + K), "flops": 6 * R * K}
    if op == "act_grad":
        return {"bytes": b * R * (2 * N + K), "flops": 12 * R * K}
    used = E * (1 - math.exp(-R / E))
    if op == "product":
        return {"bytes": int(b * (R * K + used * N * K + R * N)), "flops": 2 * R * N * K}
    wb = BYTES[c["w_dtype"]]
    return {"bytes": int(b * (R * N + 2 * R * K + used * N * K) + wb * E * N * K), "flops": 4 * R * N * K}


# ---------------------------------------------------------------- inputs
def _normal(shape, dtype, g, scale=1.0):
    """Normal values, drawn in the type itself."""
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _segments(c, g):
    """Counts and segment starts of R rows on experts of uneven popularity."""
    R, E = c["R"], c["E"]
    p = torch.softmax(0.4 * torch.randn(E, generator=g, device="cuda"), 0)
    counts = torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E)
    size = torch.full_like(counts, c["capacity"]) if c["layout"] == MASKED else (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), size.cumsum(0)])
    return counts.to(torch.int32), offsets.to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = c["op"], TYPES[c["dtype"]]
    z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": dict(c), "status": z(1)}
    if op in ("route", "route_grad"):
        T, E, K = c["T"], c["E"], c["K"]
        # some experts are more popular than others
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") * 1.5 +
                       0.5 * torch.randn(E, generator=g, device="cuda")).to(dt)
        if c["padded"]:
            s["logits"][torch.rand(T, generator=g, device="cuda") < 0.1] = -math.inf
        s["bias"] = _normal((E,), torch.float32, g, 0.05) if c["bias"] else None
        if op == "route":
            s |= {"topk_idx": z(T, K), "topk_w": z(T, K, dtype=torch.float32)}
        else:
            s["topk_idx"] = _picks(c, s["logits"], s["bias"])[0]
            s["dtopk_w"] = _normal((T, K), torch.float32, g)
            s["dscores"] = _normal((T, E), torch.float32, g, 0.1) if c["aux"] else None
            s["dlogits"] = z(T, E, dtype=dt)
        return s
    if op in ("norm", "norm_grad"):
        T, H, wt = c["T"], c["H"], TYPES[c["w_dtype"]]
        # rows of different means and spreads
        s["x"] = _normal((T, H), dt, g).mul_((0.5 + torch.rand(T, 1, generator=g, device="cuda")).to(dt)).add_(
            _normal((T, 1), dt, g, 0.5))
        s["weight"] = (1 + _normal((H,), torch.float32, g, 0.1)).to(wt)
        s["bias"] = _normal((H,), wt, g, 0.1) if c["bias"] else None
        s["eps"] = 1e-5
        if op == "norm":
            s |= {"y": z(T, H, dtype=dt), "mean": z(T, dtype=torch.float32), "rstd": z(T, dtype=torch.float32)}
        else:
            # what the forward pass leaves
            s["mean"], s["rstd"] = _moments(s["x"], s["eps"])
            s["dy"] = _normal((T, H), dt, g)
            s |= {"dx": z(T, H, dtype=dt), "dweight": z(H, dtype=wt), "dbias": z(H, dtype=wt) if c["bias"] else None}
            # what the call may need beside its outputs: partial sums of the weight's and the bias's gradients
            s["workspace"] = z(8192 * H + 4096, dtype=torch.uint8)
        return s
    E, N, K, R = c["E"], c["N"], c["K"], _rows_total(c)
    s["counts"], s["offsets"] = _segments(c, g)
    if op in ("act", "act_grad"):
        s["h"] = _normal((R, N), dt, g, 2.0)
        if op == "act":
            s["q"] = z(R, K, dtype=dt)
        else:
            s["dq"], s["dh"] = _normal((R, K), dt, g), z(R, N, dtype=dt)
    else:
        s["a"] = _normal((R, K), dt, g)
        s["w"] = _normal((E, N, K), dt, g, 0.02)
        if op == "product":
            s["c"] = z(R, N, dtype=dt)
        else:
            s["dc"], s["da"] = _normal((R, N), dt, g), z(R, K, dtype=dt)
            s["dw"] = z(E, N, K, dtype=TYPES[c["w_dtype"]])
            # what the call may need beside its outputs: partial sums of the weights' gradients
            s["workspace"] = z(1 << 28, dtype=torch.uint8)
    # the plain form walks the segments on the host
    starts, counts = s["offsets"].tolist(), s["counts"].tolist()
    s["segments"] = [(b, min(b + n, e)) for b, n, e in zip(starts, counts, starts[1:])]
    return s


# ---------------------------------------------------------------- plain forms
def _scores(c, logits):
    """Scores in 64 bits (picks next to a border), 0 where the logit is -infinity."""
    l = logits.double()
    if c["score"] == SIGMOID:
        return 1 / (1 + torch.exp(-l))
    top = l.max(1, keepdim=True).values.clamp(min=-1e300)      # (a row of -infinity has no largest)
    e = torch.exp(l - top)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def _picks(c, logits, bias):
    """Picked experts (-1: none), their scores in 64 bits, and all scores."""
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    s = _scores(c, logits)
    key = s if bias is None else s + bias.double()
    key = key.masked_fill(logits == -math.inf, -math.inf)
    if G > 1:
        best = key.reshape(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_best"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    key, idx = key.sort(dim=1, descending=True, stable=True)
    key, idx = key[:, :K], idx[:, :K]
    none = key == -math.inf
    return torch.where(none, -1, idx).to(torch.int32), s.gather(1, idx).masked_fill(none, 0), s


def _moments(x, eps):
    """Mean and 1 / sqrt(variance + eps) of rows, in 32 bits."""
    f = x.float()
    mean = f.mean(1)
    return mean, torch.rsqrt((f - mean[:, None]).square().mean(1) + eps)


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op == "route":
        idx, w, _ = _picks(c, s["logits"], s["bias"])
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=LEAST_SUM)
        return {"idx": idx, "w": (w * c["scale"]).float()}
    if op == "route_grad":
        sc = _scores(c, s["logits"]).float()
        idx = s["topk_idx"].long()
        live = idx >= 0
        w = sc.gather(1, idx.clamp(min=0)).masked_fill_(~live, 0)
        d = s["dtopk_w"].masked_fill(~live, 0) * c["scale"]
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            by = total.clamp(min=LEAST_SUM)
            d = torch.where(total > LEAST_SUM, d - (d * w).sum(1, keepdim=True) / by, d) / by
        ds = torch.zeros_like(sc) if s["dscores"] is None else s["dscores"].clone()
        ds.scatter_add_(1, idx.clamp(min=0), d.masked_fill_(~live, 0))
        if c["score"] == SIGMOID:
            return (ds * sc * (1 - sc)).to(dt)
        return (sc * (ds - (sc * ds).sum(1, keepdim=True))).to(dt)
    if op == "norm":
        mean, rstd = _moments(s["x"], s["eps"])
        y = (s["x"].float() - mean[:, None]) * rstd[:, None] * s["weight"].float()
        if s["bias"] is not None:
            y += s["bias"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        wt = TYPES[c["w_dtype"]]
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        out = {"dweight": (dy * xh).sum(0, dtype=torch.float64).to(wt)}
        out["dbias"] = dy.sum(0, dtype=torch.float64).to(wt) if c["bias"] else 0
        dy *= s["weight"].float()
        out["dx"] = ((dy - dy.mean(1, keepdim=True) - xh * (dy * xh).mean(1, keepdim=True)) *
                     s["rstd"][:, None]).to(dt)
        return out
    if op == "act":
        I = c["K"]
        q = torch.zeros_like(s["q"])
        for b, n in s["segments"]:
            h = s["h"][b:n].float()
            q[b:n] = (h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]).to(dt)
        return q
    if op == "act_grad":
        I = c["K"]
        dh = torch.zeros_like(s["dh"])
        for b, n in s["segments"]:
            h, dq = s["h"][b:n].float(), s["dq"][b:n].float()
            gate, up = h[:, :I], h[:, I:]
            sig = 1 / (1 + torch.exp(-gate))
            dh[b:n, :I] = (dq * up * sig * (1 + gate * (1 - sig))).to(dt)
            dh[b:n, I:] = (dq * gate * sig).to(dt)
        return dh
    if op == "product":
        out = torch.zeros_like(s["c"])
        for e, (b, n) in enumerate(s["segments"]):
            if n > b:
                out[b:n] = (s["a"][b:n].float() @ s["w"][e].float().t()).to(dt)
        return out
    da, dw = torch.zeros_like(s["da"]), torch.zeros_like(s["dw"])
    for e, (b, n) in enumerate(s["segments"]):
        if n > b:
            dc = s["dc"][b:n].float()
            da[b:n] = (dc @ s["w"][e].float()).to(dt)
            dw[e] = (dc.t() @ s["a"][b:n].float()).to(dw.dtype)
    return {"da": da, "dw": dw}


# ---------------------------------------------------------------- the package's calls
def _own(s):
    import fp8_routed_expert_amd as fre
    c = s["case"]
    op = c["op"]
    if op == "route":
        fre.moe_route_tokens(s["logits"], s["topk_idx"], s["topk_w"], s["status"], s["bias"], c["score"], c["groups"],
                             c["top_groups"], c["group_best"], c["renorm"], c["scale"])
        return {"idx": s["topk_idx"], "w": s["topk_w"]}
    if op == "route_grad":
        fre.moe_route_tokens_grad(s["logits"], s["topk_idx"], s["dtopk_w"], s["dlogits"], s["status"], c["score"],
                                  c["renorm"], c["scale"], s["dscores"])
        return s["dlogits"]
    if op == "norm":
        fre.moe_layer_norm(s["x"], s["weight"], s["bias"], s["eps"], s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_grad":
        fre.moe_layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                s["workspace"])
        return {"dweight": s["dweight"], "dbias": s["dbias"] if c["bias"] else 0, "dx": s["dx"]}
    if op == "act":
        fre.moe_gated_act(s["h"], s["offsets"], s["counts"], s["q"], s["status"])
        return s["q"]
    if op == "act_grad":
        fre.moe_gated_act_grad(s["dq"], s["h"], s["offsets"], s["counts"], s["dh"], s["status"])
        return s["dh"]
    if op == "product":
        fre.moe_grouped_gemm_float(s["a"], s["w"], s["offsets"], s["counts"], s["c"], s["status"])
        return s["c"]
    fre.moe_grouped_gemm_float_grad_rows(s["dc"], s["w"], s["offsets"], s["counts"], s["da"], s["status"])
    fre.moe_grouped_gemm_float_grad_weights(s["dc"], s["a"], s["offsets"], s["counts"], s["dw"], s["workspace"],
                                            s["status"])
    return {"da": s["da"], "dw": s["dw"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    torch.set_default_device("cuda")
    try:
        return _exact(c, prepare(c, seed))
    finally:
        torch.set_default_device("cpu")


def _scores64(c, l):
    """Row by row from the definition; a row without a finite logit scores 0."""
    if c["score"] == SIGMOID:
        return torch.sigmoid(l)
    return torch.softmax(l, 1).nan_to_num(0.0)


def _exact_route(c, s):
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    l = s["logits"].double()
    score = _scores64(c, l)
    key = score.clone()
    if s["bias"] is not None:
        key += s["bias"].double()
    key[l == -math.inf] = -math.inf
    at = torch.arange(T)
    if G > 1:
        # the groups' scores, then the best group again and again
        part = key.view(T, G, E // G).clone()
        total = torch.zeros(T, G, dtype=torch.float64)
        for _ in range(min(c["group_best"], E // G)):
            top = part.max(2)
            total += top.values
            part.scatter_(2, top.indices[:, :, None], -math.inf)
        kept = torch.zeros(T, G, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            best = torch.where(kept, -math.inf, total).max(1, keepdim=True).values
            first = ((total >= best) & ~kept).to(torch.int8).argmax(1)
            kept[at, first] = True
        key[~kept[:, :, None].expand(T, G, E // G).reshape(T, E)] = -math.inf
    w = torch.zeros(T, K, dtype=torch.float64)
    for k in range(K):
        best = key.max(1, keepdim=True).values
        i = (key == best).to(torch.int8).argmax(1)
        w[:, k] = torch.where(best[:, 0] > -math.inf, score[at, i], 0.0)
        key[at, i] = -math.inf
    if c["renorm"]:
        w /= torch.clamp(w.sum(1, keepdim=True), min=LEAST_SUM)
    return {"idx": None, "w": c["scale"] * w}


def _exact(c, s):
    op = c["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "route_grad":
        l = s["logits"].double().requires_grad_()
        score = torch.sigmoid(l) if c["score"] == SIGMOID else torch.softmax(
            l.masked_fill((l == -math.inf).all(1, keepdim=True), 0.0), 1)
        live = s["topk_idx"] >= 0
        w = torch.where(live, score.gather(1, s["topk_idx"].clamp(min=0).long()), 0.0)
        if c["renorm"]:
            w = w / torch.clamp(w.sum(1, keepdim=True), min=LEAST_SUM)
        loss = (c["scale"] * w * s["dtopk_w"].double()).sum()
        if s["dscores"] is not None:
            loss = loss + torch.where(l == -math.inf, 0.0, score * s["dscores"].double()).sum()
        dl, = torch.autograd.grad(loss, l)
        return dl.masked_fill(l == -math.inf, 0.0)
    if op in ("norm", "norm_grad"):
        x, w = s["x"].double(), s["weight"].double()
        if op == "norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + s["eps"]) ** -0.5
            y = w * ((x - mean[:, None]) * rstd[:, None])
            return {"y": y if s["bias"] is None else y + s["bias"].double(), "mean": mean, "rstd": rstd}
        dy, r = s["dy"].double(), s["rstd"].double()[:, None]
        xh = r * (x - s["mean"].double()[:, None])
        dweight = torch.einsum("th,th->h", dy, xh)
        dbias = dy.sum(0) if c["bias"] else None
        g = w * dy
        H = c["H"]
        along = torch.einsum("th,th->t", g, xh)[:, None] / H
        return {"dweight": dweight, "dbias": dbias, "dx": r * (g - g.sum(1, keepdim=True) / H - along * xh)}
    R, E, N, K = _rows_total(c), c["E"], c["N"], c["K"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64)  # noqa: E731
    starts, ends = s["offsets"][:-1], torch.minimum(s["offsets"][:-1] + s["counts"], s["offsets"][1:])
    if op in ("act", "act_grad"):
        row = torch.arange(R)[:, None]
        valid = ((row >= starts) & (row < ends)).any(1)
        gate, up = s["h"].double().chunk(2, 1)
        sig = torch.sigmoid(gate)
        if op == "act":
            return torch.where(valid[:, None], gate * sig * up, 0.0)
        dq = torch.where(valid[:, None], s["dq"].double(), 0.0)
        return torch.cat([dq * up * (sig + gate * sig * torch.sigmoid(-gate)), dq * gate * sig], 1)
    a, w = s["a"], s["w"]
    out, da, dw = (new(R, N), None, None) if op == "product" else (None, new(R, K), new(E, N, K))
    for e in range(E):
        rows = slice(int(starts[e]), int(ends[e]))
        if rows.stop <= rows.start:
            continue
        if op == "product":
            torch.matmul(a[rows].double(), w[e].double().t(), out=out[rows])
        else:
            dc = s["dc"][rows].double()
            torch.matmul(dc, w[e].double(), out=da[rows])
            torch.matmul(dc.t(), a[rows].double(), out=dw[e])
    return out if op == "product" else {"da": da, "dw": dw}

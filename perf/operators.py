"""What is measured of the routed-expert operators: tokens sorted by expert and
back with their gradients, and the products in 8-bit integers with one scale
per token and one per output channel.

`run` computes a case in its plain form (elementary torch operations) or, with
`own` set, through this package's calls; both take what `prepare` gives.
"""

import math

import torch

own = False

CONTIGUOUS, MASKED = 0, 1
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases
def _routing(op, T, K, E, pool, H, dtype, layout=CONTIGUOUS, capacity=0):
    """T tokens pick K of `pool` experts, the first E of which are here."""
    return {"op": op, "T": T, "K": K, "E": E, "pool": pool, "H": H, "dtype": dtype,
            "layout": layout, "capacity": capacity}


def _linear(M, N, H, dtype):
    return {"op": "linear", "M": M, "N": N, "H": H, "dtype": dtype}


def _experts(op, T, K, E, pool, H, I, dtype, layout=CONTIGUOUS, capacity=0):
    return {"op": op, "T": T, "K": K, "E": E, "pool": pool, "H": H, "I": I, "dtype": dtype,
            "layout": layout, "capacity": capacity}


def listed():
    return [
        # the tiny workload: a few tokens, where a call is all latency
        dict(_routing("sort", 64, 2, 4, 8, 256, "bf16"), name="sort tiny"),
        # one prefill share of 9 experts: every row of the layer, moved once
        dict(_routing("sort", 65536, 8, 9, 36, 7168, "bf16"), name="sort prefill"),
        # a training micro-batch on 6 experts: the sort's gradient
        dict(_routing("sort_grad", 4096, 8, 6, 32, 7168, "f16"), name="sort gradient"),
        # a decode step in the fixed-capacity layout
        dict(_routing("combine", 1024, 8, 32, 220, 7168, "f16", MASKED, 128), name="back decode"),
        # a training step at the prefill share's size: gradients of rows and weights
        dict(_routing("combine_grad", 65536, 8, 9, 36, 7168, "bf16"), name="back gradient prefill"),
        # sizes that divide by nothing, in 32 bits: a small model's test run
        dict(_routing("combine_grad", 777, 3, 5, 7, 509, "f32"), name="back gradient odd"),
        # one token through a linear outside the experts: the weights are all there is to read
        dict(_linear(1, 4096, 7168, "bf16"), name="linear one token"),
        # a decode batch through one
        dict(_linear(96, 7168, 2048, "f16"), name="linear decode"),
        # a prefill chunk with a ragged end
        dict(_linear(8191, 7168, 2048, "bf16"), name="linear prefill"),
        # gate and up of 32 experts with a few dozen rows each: a decode step
        dict(_experts("gate_up", 1024, 8, 32, 220, 7168, 2048, "bf16", MASKED, 128), name="experts gate/up decode"),
        # the activation and the down product of a larger decode share
        dict(_experts("act_down", 4096, 8, 6, 32, 7168, 2048, "bf16"), name="experts act+down"),
        # gate and up of the prefill share: the largest product
        dict(_experts("gate_up", 65536, 8, 9, 36, 7168, 2048, "bf16"), name="experts gate/up prefill"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "sort_grad", "combine", "combine_grad", "linear", "linear", "gate_up", "act_down"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "linear":
        M, N, H = _log(rng, 1, 16384), 16 * _log(rng, 2, 512), 16 * _log(rng, 4, 512)
        return _linear(M, N, H, dtype)
    E = _log(rng, 1, 64)
    pool = E + _log(rng, 1, 256) - 1
    K = rng.randint(1, min(8, pool))
    layout = rng.choice([CONTIGUOUS, MASKED])
    if op in ("gate_up", "act_down"):
        H, I = 16 * _log(rng, 8, 448), 16 * _log(rng, 8, 128)
        T = _log(rng, 1, 32768)
    else:
        dtype = rng.choice(["bf16", "f16", "f32"])
        H, I = _log(rng, 64, 7168), 0
        T = _log(rng, 1, 65536)
    # no more routed rows than the largest listed case has
    most = 65536 if dtype == "f32" else 131072
    T = min(T, most // 2 if dtype == "f32" else T, max(1, most * pool // (K * E)))
    if T * K * E < 8 * pool:      # a few tokens alone: all of their experts are here
        pool, K = E, min(K, E)
    mean = T * K * E / pool / E
    capacity = max(8, int(mean * rng.choice([1.0, 1.5, 3.0]))) if layout == MASKED else 0
    if op in ("gate_up", "act_down"):
        return _experts(op, T, K, E, pool, H, I, dtype, layout, capacity)
    return _routing(op, T, K, E, pool, H, dtype, layout, capacity)


def _rows(c):
    """Rows of the sorted buffer that a program sets aside for the case: the
    mean number of routed rows and a tenth, each segment rounded up to 128."""
    if c["layout"] == MASKED:
        return c["capacity"]
    mean = c["T"] * c["K"] * c["E"] / c["pool"]
    return int(1.1 * mean) + 8 + 127 * c["E"]


def _rows_total(c):
    return c["E"] * _rows(c) if c["layout"] == MASKED else _rows(c)


def work(c):
    op = c["op"]
    b = BYTES[c["dtype"]]
    if op == "linear":
        M, N, H = c["M"], c["N"], c["H"]
        return {"bytes": b * M * H + N * H + 4 * N + b * M * N, "flops": 2 * M * N * H}
    T, K, E, H = c["T"], c["K"], c["E"], c["H"]
    R = T * K * E / c["pool"]           # on average
    if c["layout"] == MASKED:
        R = min(R, E * c["capacity"])
    rows = _rows_total(c)
    any_local = T * (1 - math.comb(c["pool"] - E, K) / math.comb(c["pool"], K)) if c["pool"] - E >= K else T
    if op == "sort":
        return {"bytes": int(4 * T * K + b * any_local * H + 4 * (T * K + 2 * rows) + b * R * H), "flops": 0}
    if op == "sort_grad":
        return {"bytes": int(b * R * H + 4 * T * K + b * T * H), "flops": int(R * H)}
    if op == "combine":
        return {"bytes": int(b * R * H + 8 * T * K + b * T * H), "flops": int(2 * R * H)}
    if op == "combine_grad":
        return {"bytes": int(b * any_local * H + 2 * b * R * H + 12 * T * K), "flops": int(3 * R * H)}
    I = c["I"]
    used = E * (1 - math.exp(-R / E))
    if op == "gate_up":
        return {"bytes": int(any_local * H + 2 * used * I * H + b * 2 * R * I), "flops": int(4 * R * I * H)}
    return {"bytes": int(2 * b * R * I + used * I * H + b * R * H), "flops": int(2 * R * I * H)}


# ---------------------------------------------------------------- inputs
def _topk(c, g):
    """Distinct picks of a skewed pool, -1 where the expert is elsewhere, and
    weights that sum to one over all K picks."""
    T, K, E, pool = c["T"], c["K"], c["E"], c["pool"]
    popularity = 0.4 * torch.randn(pool, generator=g, device="cuda")
    u = torch.rand(T, pool, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    picks = (popularity - torch.log(-torch.log(u))).topk(K, dim=1)
    idx = torch.where(picks.indices < E, picks.indices, -1).to(torch.int32)
    return idx.contiguous(), torch.softmax(picks.values, dim=1).contiguous()


def _normal(shape, dtype, g, scale=1.0):
    """Normal values, drawn in the type itself."""
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(scale)


def _codes(shape, g):
    """8-bit codes of normal rows and the rows' scales."""
    q = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).mul_(30).round_().clamp_(-127, 127)
    s = (0.5 + torch.rand(shape[:-1], generator=g, device="cuda")) / 40
    return q.to(torch.int8), s


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = c["op"], TYPES[c["dtype"]]
    z = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": dict(c)}
    if op == "linear":
        M, N, H = c["M"], c["N"], c["H"]
        s["x"] = _normal((M, H), dt, g)
        s["w"], s["w_scale"] = _codes((N, H), g)
        s["w_scale"] *= 0.05
        s["c"] = z(M, N, dtype=dt)
        # what the call may need beside its output: codes and scales of x
        s["workspace"] = z((M * (H + 4) + 1024), dtype=torch.uint8)
        return s
    T, K, E, H = c["T"], c["K"], c["E"], c["H"]
    R = _rows_total(c)
    s["topk_idx"], s["topk_w"] = _topk(c, g)
    s["status"] = z(1)
    if op == "sort":
        s["x"] = _normal((T, H), dt, g)
        s |= {"counts": z(E), "offsets": z(E + 1), "slot_of": z(T, K), "row_src": z(R), "row_expert": z(R)}
        s["a"] = z(R, H, dtype=dt)
        s["workspace"] = z(8 * E * (T * K // 1024 + 1), dtype=torch.uint8)
        return s
    # the others start from sorted tokens
    table = _sorted(c, s["topk_idx"])
    s |= dict(zip(("counts", "offsets", "slot_of", "row_src", "row_expert"), table))
    if op == "sort_grad":
        s["da"] = _normal((R, H), dt, g)
        s["dx"] = z(T, H, dtype=dt)
    elif op == "combine":
        s["y"] = _normal((R, H), dt, g)
        s["out"] = z(T, H, dtype=dt)
    elif op == "combine_grad":
        s["y"], s["dout"] = _normal((R, H), dt, g), _normal((T, H), dt, g)
        s["dy"], s["dw"] = z(R, H, dtype=dt), z(T, K, dtype=torch.float32)
    elif op == "gate_up":
        N = 2 * c["I"]
        s["x"], s["x_scale"] = _codes((T, H), g)
        s["w"], s["w_scale"] = _codes((E, N, H), g)
        s["w_scale"] *= 0.05
        s["c"] = z(R, N, dtype=dt)
    else:
        I = c["I"]
        s["h"] = _normal((R, 2 * I), dt, g, 2.0)
        s["w"], s["w_scale"] = _codes((E, H, I), g)
        s["w_scale"] *= 0.05
        s["q"], s["q_scale"] = z(R, I, dtype=torch.int8), z(R, dtype=torch.float32)
        s["y"] = z(R, H, dtype=dt)
    if op in ("gate_up", "act_down"):
        # the plain form walks the segments on the host
        starts, counts = s["offsets"].tolist(), s["counts"].tolist()
        s["segments"] = [(b, min(b + n, e, R)) for b, n, e in zip(starts, counts, starts[1:])]
    return s


# ---------------------------------------------------------------- plain forms
def _sorted(c, idx):
    """Counts, segment starts, slots, and each row's token and expert."""
    T, K, E = c["T"], c["K"], c["E"]
    masked, rows, R = c["layout"] == MASKED, _rows(c), _rows_total(c)
    e = idx.reshape(-1).long()
    local = e >= 0
    key = torch.where(local, e, E)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=e.device).scatter_add_(0, key, torch.ones_like(key))
    before = counts.cumsum(0) - counts
    rank = torch.empty_like(key)
    rank[order] = torch.arange(T * K, device=e.device) - before[key[order]]
    counts = counts[:E]
    size = torch.full_like(counts, rows) if masked else (counts + 127) // 128 * 128
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=e.device), size.cumsum(0)])
    slot = offsets[key] + rank
    keep = local & ((rank < rows) if masked else (slot < R))
    slot = torch.where(keep, slot, R)          # R: a row past the end, cut off below
    token = torch.arange(T * K, device=e.device) // K
    row_src = torch.full((R + 1,), -1, dtype=torch.int32, device=e.device)
    row_expert = row_src.clone()
    row_src[slot] = token.to(torch.int32)
    row_expert[slot] = key.to(torch.int32)
    slot_of = torch.where(keep, slot, -1).to(torch.int32).reshape(T, K)
    return (counts.to(torch.int32), offsets.to(torch.int32), slot_of, row_src[:R].contiguous(),
            row_expert[:R].contiguous())


def _gathered(y, slot_of):
    """y[slot_of] in 32 bits, zero where there is no slot."""
    rows = y[slot_of.clamp(min=0).long()].float()
    return rows.masked_fill_((slot_of < 0).unsqueeze(-1), 0)


def _quantized(x):
    """Codes and scales of rows: the scale in 32 bits, the quotient's rounding
    decided in 64 (values next to a border)."""
    amax = x.float().abs().amax(-1)
    s = (amax / 127).clamp(min=2.0 ** -126)
    s = torch.where(amax == 0, 1.0, s)
    return (x.double() / s.double().unsqueeze(-1)).round().float(), s


def _product(q, s, w, ws, dtype):
    return ((q @ w.float().t()) * (s.unsqueeze(-1) * ws)).to(dtype)


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op == "linear":
        q, sx = _quantized(s["x"])
        return _product(q, sx, s["w"], s["w_scale"], dt)
    if op == "sort":
        table = _sorted(c, s["topk_idx"])
        src = table[3]
        return {"a": s["x"][src.clamp(min=0).long()].masked_fill_((src < 0).unsqueeze(-1), 0), "table": table}
    if op == "sort_grad":
        return _gathered(s["da"], s["slot_of"]).sum(1).to(dt)
    if op == "combine":
        return (_gathered(s["y"], s["slot_of"]) * s["topk_w"].unsqueeze(-1)).sum(1).to(dt)
    if op == "combine_grad":
        # row by row: the row's token and its weight
        src, slot_of = s["row_src"], s["slot_of"]
        R = src.numel()
        w = torch.zeros(R + 1, device=src.device)
        w[torch.where(slot_of < 0, R, slot_of).long()] = s["topk_w"]
        g = s["dout"][src.clamp(min=0).long()].float()
        dy = (g * w[:R].unsqueeze(-1)).masked_fill_((src < 0).unsqueeze(-1), 0).to(dt)
        dots = g.mul_(s["y"].float()).sum(-1)
        return {"dy": dy, "dw": dots[slot_of.clamp(min=0).long()].masked_fill_(slot_of < 0, 0)}
    c_out = torch.zeros_like(s["c"] if op == "gate_up" else s["y"])
    if op == "act_down":
        I = c["I"]
        h = s["h"].float()
        q, sq = _quantized(h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:])
    for e, (b, n) in enumerate(s["segments"]):
        if n > b:
            if op == "gate_up":
                src = s["row_src"][b:n].long()
                c_out[b:n] = _product(s["x"][src].float(), s["x_scale"][src], s["w"][e], s["w_scale"][e], dt)
            else:
                c_out[b:n] = _product(q[b:n], sq[b:n], s["w"][e], s["w_scale"][e], dt)
    return c_out


# ---------------------------------------------------------------- the package's calls
def _own(s):
    import fp8_routed_expert_amd as fre
    c = s["case"]
    op = c["op"]
    if op == "linear":
        fre.moe_linear_int8(s["x"], s["w"], s["w_scale"], s["c"], s["workspace"])
        return s["c"]
    if op == "sort":
        fre.moe_sort_tokens(s["topk_idx"], c["E"], c["layout"], 128, _rows(c), s["counts"], s["offsets"],
                            s["slot_of"], s["row_src"], s["row_expert"], s["workspace"], s["status"])
        fre.moe_permute_rows(s["x"], s["slot_of"], s["a"], s["status"], s["row_src"])
        return {"a": s["a"], "table": (s["counts"], s["offsets"], s["slot_of"], s["row_src"], s["row_expert"])}
    if op == "sort_grad":
        fre.moe_permute_rows_grad(s["da"], s["slot_of"], s["dx"], s["status"])
        return s["dx"]
    if op == "combine":
        fre.moe_combine_rows(s["y"], s["slot_of"], s["topk_w"], s["out"], s["status"])
        return s["out"]
    if op == "combine_grad":
        fre.moe_combine_rows_grad(s["dout"], s["y"], s["slot_of"], s["topk_w"], s["dy"], s["dw"], s["status"],
                                  s["row_src"])
        return {"dy": s["dy"], "dw": s["dw"]}
    if op == "gate_up":
        fre.moe_grouped_gemm_int8_gather(s["x"], s["x_scale"], s["row_src"], s["w"], s["w_scale"], s["offsets"],
                                         s["counts"], s["c"], s["status"])
        return s["c"]
    fre.moe_act_requant_int8(s["h"], s["offsets"], s["counts"], s["q"], s["q_scale"], s["status"])
    fre.moe_grouped_gemm_int8(s["q"], s["q_scale"], s["w"], s["w_scale"], s["offsets"], s["counts"], s["y"],
                              s["status"])
    return s["y"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits
def _codes64(v):
    """Codes and scales of rows from the definition: the scale is held in 32
    bits, a code is the integer nearest the quotient, ties to even."""
    top = torch.maximum(v.max(-1).values, -v.min(-1).values)
    s = torch.where(top > 0, torch.clamp((top / 127).float(), min=2.0 ** -126), torch.ones(())).double()
    t = v / s[:, None]
    low = torch.floor(t)
    up = (t - low > 0.5) | ((t - low == 0.5) & (low.remainder(2) == 1))
    return low + up, s


def exact(c, seed):
    torch.set_default_device("cuda")
    try:
        return _exact(c, prepare(c, seed))
    finally:
        torch.set_default_device("cpu")


def _exact(c, s):
    op = c["op"]
    if op == "linear":
        q, sx = _codes64(s["x"].double())
        return sx[:, None] * (q @ s["w"].double().t()) * s["w_scale"].double()
    T, K, E, H = c["T"], c["K"], c["E"], c["H"]
    R = _rows_total(c)
    picks = s["topk_idx"].reshape(-1)
    # expert by expert: its picks in order, as many as fit
    rows, toks, ks = [], [], []
    start = 0
    for e in range(E):
        f = (picks == e).nonzero().flatten()
        b = e * c["capacity"] if c["layout"] == MASKED else start
        r = b + torch.arange(f.numel())
        fit = r < (b + c["capacity"] if c["layout"] == MASKED else R)
        rows.append(r[fit])
        toks.append(f[fit] // K)
        ks.append(f[fit] % K)
        start += -(-f.numel() // 128) * 128
    row, tok, k = torch.cat(rows), torch.cat(toks), torch.cat(ks)
    if op == "sort":
        a = torch.zeros(R, H, dtype=torch.float64)
        a[row] = s["x"].double()[tok]
        return {"a": a, "table": None}
    if op in ("sort_grad", "combine"):
        v = s["da" if op == "sort_grad" else "y"][row].double()
        if op == "combine":
            v *= s["topk_w"][tok, k].double()[:, None]
        return torch.zeros(T, H, dtype=torch.float64).index_add_(0, tok, v)
    if op == "combine_grad":
        v = s["dout"].double()[tok]
        dy, dw = torch.zeros(R, H, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
        dy[row] = v * s["topk_w"][tok, k].double()[:, None]
        dw[tok, k] = (v * s["y"][row].double()).sum(-1)
        return {"dy": dy, "dw": dw}
    out = torch.zeros(R, 2 * c["I"] if op == "gate_up" else H, dtype=torch.float64)
    for e in range(E):
        r, t = rows[e], toks[e]
        if not r.numel():
            continue
        if op == "gate_up":
            q, sq = s["x"][t].double(), s["x_scale"][t].double()
        else:
            gate, up = s["h"][r].double().split(c["I"], dim=-1)
            q, sq = _codes64(gate / (1 + torch.exp(-gate)) * up)
        out[r] = sq[:, None] * (q @ s["w"][e].double().t()) * s["w_scale"][e].double()
    return out

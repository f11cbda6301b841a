"""Helpers for the tests of the router, the layer norm and the experts'
products in 32 and 16 bits: inputs, guarded outputs and tolerances that count
roundings.  U is half a step of fp32 relative to the value; a value rounded to
a type t is off by at most finfo(t).eps / 2 of itself, or half the smallest
subnormal."""

import numpy as np
import torch

from tests.gpu_util import log

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24
GUARD = 64      # elements kept before and after a guarded output


def rounding(ref, dt):
    """What the last rounding to dt may move ref."""
    f = torch.finfo(dt)
    return f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2


def close(got, ref, tol, what):
    """got (any type) within tol of the 64-bit ref, elementwise, and no NaN."""
    got, ref = got.detach().double().cpu(), torch.as_tensor(ref).double().cpu()
    tol = torch.as_tensor(tol).double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs()
    log(f"{what}: {got.numel()} values, largest error over tolerance "
        f"{float((off / tol.clamp(min=1e-300)).max()) if got.numel() else 0:.3f}")
    assert not got.isnan().any(), what
    assert (off <= tol).all(), (what, float((off - tol).max()))


def values(seed, shape, dt, scale=1.0, shift=0.0, offset=0):
    """Device values of type dt and the same in 64 bits on the CPU; offset
    shifts the buffer by that many elements off its allocation."""
    g = np.random.default_rng(seed)
    n = int(np.prod(shape))
    v = torch.from_numpy(g.standard_normal(n + offset) * scale + shift).to(dt)
    return v.cuda()[offset:].view(shape), v[offset:].view(shape).double()


class Guarded:
    """Outputs in one allocation each, filled with a value that a right result
    does not have, with guard elements around them."""

    def __init__(self):
        self.all = []

    def new(self, *shape, dtype=torch.float32, fill=None, offset=0):
        fill = fill if fill is not None else (-7 if dtype in (torch.int32, torch.uint8) and
                                              dtype == torch.int32 else
                                              165 if dtype == torch.uint8 else float("nan"))
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * GUARD + offset,), fill, dtype=dtype, device="cuda")
        self.all.append((buf, GUARD + offset, n, buf.clone()))
        return buf[GUARD + offset:GUARD + offset + n].view(shape)

    def check(self):
        for buf, at, n, was in self.all:
            for part in (slice(0, at), slice(at + n, None)):
                a, b = buf[part].contiguous().view(torch.uint8), was[part].contiguous().view(torch.uint8)
                assert torch.equal(a, b), "written outside an output"


def table(counts, rows, layout=0, align=128, device="cuda"):
    """counts and offsets (int32, device), rows of the buffer, and the valid
    (start, end) of every expert."""
    counts = list(counts)
    if layout:
        offsets = [e * rows for e in range(len(counts) + 1)]
        total = rows * len(counts)
    else:
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + -(-c // align) * align)
        total = rows
    seg = []
    for e, c in enumerate(counts):
        b = min(offsets[e], total)
        seg.append((b, max(b, min(b + c, offsets[e + 1], total))))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
    return i32(counts), i32(offsets), total, seg


def valid_mask(seg, total):
    m = torch.zeros(total, dtype=torch.bool)
    for b, n in seg:
        m[b:n] = True
    return m

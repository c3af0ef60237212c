"""4-bit weights with group scales for the tests, and what they stand for in fp64.

What no element occupies -- fields past the columns, bytes between rows, rows of X that no slot names, the rest of
strided tensors -- holds noise or NaN: an access that should not matter shows.
"""
import numpy as np
import torch

import dense_packed_bit_gb300 as mm

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step, relative


def make_weights(seed, experts, rows, cols, group, dtype, zeros=True, spare=16, static=False, device="cuda"):
    """(the description for the kernels, the matrices [experts][rows][cols] float64); `spare`: bytes between rows of codes."""
    g = torch.Generator().manual_seed(seed)
    groups, held = -(-cols // group), 16 * -(-cols // 32)
    wide = torch.randint(0, 256, (experts, rows, held + spare), generator=g, dtype=torch.uint8)
    codes = wide[:, :, :held]
    # a NaN behind the last scale of each row
    s = torch.full((experts, rows, groups + 1), float("nan"), dtype=DT[dtype])
    s[:, :, :groups] = ((0.5 + torch.rand(experts, rows, groups, generator=g)) / np.sqrt(cols) / 5).to(DT[dtype])
    z = torch.randint(0, 256, (experts, rows, groups + 1), generator=g, dtype=torch.uint8) if zeros else None
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)[..., :cols].double()
    each = lambda a: a.double().repeat_interleave(group, -1)[..., :cols]  # noqa: E731
    dense = (code - (8.0 if z is None else each(z[:, :, :groups] & 15))) * each(s[:, :, :groups])
    wide, s = wide.to(device), s.to(device)
    z = None if z is None else z.to(device)[:, :, :groups]
    return mm.mm_packed4(wide[:, :, :held], s[:, :, :groups], z, cols, group, static), dense


def make_x(seed, n, cols, dtype, pad=8, device="cuda", bad=()):
    """Rows of X with NaN between them (and in rows `bad`); (tensor, float64)."""
    g = torch.Generator().manual_seed(seed)
    stride = -(-cols // 8) * 8 + pad
    x = torch.full((n, stride), float("nan"), dtype=DT[dtype])
    x[:, :cols] = torch.randn(n, cols, generator=g).to(DT[dtype])
    for r in bad:
        x[r] = float("nan")
    return x.to(device)[:, :cols], x[:, :cols].double()


def make_y(n, cols, dtype, pad=3, rows=2, device="cuda"):
    """Y [n][cols] inside a buffer of -7 with `pad` columns and `rows` rows more; (Y, buffer)."""
    buf = torch.full((n + rows, cols + pad), -7.0, dtype=DT[dtype], device=device)
    return buf[:n, :cols], buf


def untouched(y, buf):
    n, cols = y.shape
    assert bool((buf[:, cols:] == -7).all()) and bool((buf[n:] == -7).all()), "written outside Y"


def reference(x, w, swiglu):
    """Y of rows x [n][cols] and a matrix w [rows][cols], fp64, and how far each may be off: before the activation 1e-5 of
    the sum of the terms' magnitudes.

    silu has a slope of at most 1.1 (its largest is 1.0998), so silu(g) u is off by at most 1.1 |u| dg + |silu(g)| du + 1.1 dg
    du; computed in fp32 its own operations (an exponential of 2 ulp, a sum, a quotient, a product) add less than 8
    roundings of 2^-24, relative."""
    z, t = x @ w.T, 1e-5 * (x.abs() @ w.abs().T)
    if not swiglu:
        return z, t
    g, u, dg, du = z[:, ::2], z[:, 1::2], t[:, ::2], t[:, 1::2]
    s = g * torch.sigmoid(g)
    return s * u, 1.1 * u.abs() * dg + s.abs() * du + 1.1 * dg * du + 8 * 2.0 ** -24 * (s * u).abs()


def check(y, ref, tol, dtype, what=""):
    """|y - ref| within tol and one rounding to Y's type (2^-25: half the smallest subnormal number of fp16)."""
    got = y.double().cpu()
    off, may = (got - ref).abs(), tol + (ref.abs() + tol) * UNIT[dtype] + (2.0 ** -25 if dtype == "f16" else 0)
    bad = ~(off <= may)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / may).nan_to_num(9e9).max())} of the bound at {bad.nonzero()[0].tolist()}"

"""64-bit references of the many-adapter operators, written from their definitions, and the
error bounds their results have to keep.

Bounds. U = 2^-24 is half a step of fp32 (relative), h(dtype) that of the output type (bf16
2^-8). An fp32 sum of L terms in any order is off by at most (L - 1) U S to first order, S the
sum of the terms' magnitudes; the roundings' signs vary, so 4 sqrt(L) U S is used where each
addition rounds to nearest, and L / 16 steps of 2 U S for tensor-core sums, whose additions (16
terms each) may truncate. `mag` below is S.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def sum_bound(L, mag, dtype):
    if dtype == torch.bfloat16:
        return (2.0 * (L / 16 + 16) + 4.0 * np.sqrt(L)) * U * mag
    return (4.0 * np.sqrt(L) + 4.0) * U * mag


def make_ids(kind, T, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), n - 1, dtype=torch.int32)
    if kind == "wild":                       # every id from far below to far above [0, n)
        ids = torch.randint(-3, n + 3, (T,), generator=g).to(torch.int32)
        if T > 2:
            ids[0], ids[1] = 2 ** 31 - 1, -2 ** 31
        return ids
    if kind == "runs":                       # contiguous requests
        ids = torch.empty(T, dtype=torch.int32)
        at = 0
        while at < T:
            ln = int(torch.randint(1, 100, (1,), generator=g))
            ids[at:at + ln] = int(torch.randint(-1, n, (1,), generator=g))
            at += ln
        return ids
    return torch.randint(-1, n, (T,), generator=g).to(torch.int32)


def plan_ref(ids, n):
    key = [i if 0 <= i < n else n for i in ids.tolist()]
    order = sorted(range(len(key)), key=lambda t: (key[t], t))
    offsets = [0]
    for a in range(n + 1):
        offsets.append(offsets[-1] + key.count(a))
    return order, offsets


def groups(ids, n):
    for a in range(n):
        rows = (ids == a).nonzero().flatten()
        if rows.numel():
            yield a, rows


def lora_ref(x, a, b, ids, scale, base, g=None, u=None):
    """(y, |y| terms, u, |u| terms) and, with g, the gradients and their term magnitudes; all in
    float64 on the CPU. grad_b is that of the given u (the call's input) when u is not None."""
    x, a, b = x.double().cpu(), a.double().cpu(), b.double().cpu()
    n, r, K = a.shape
    N, T = b.shape[1], x.shape[0]
    out = {"y": torch.zeros(T, N, dtype=torch.float64) if base is None else base.double().cpu().clone(),
           "u": torch.zeros(T, r, dtype=torch.float64)}
    out["y_mag"], out["u_mag"] = out["y"].abs(), torch.zeros(T, r, dtype=torch.float64)
    if g is not None:
        g = g.double().cpu()
        for k, shape in (("grad_x", (T, K)), ("grad_a", a.shape), ("grad_b", b.shape)):
            out[k], out[k + "_mag"] = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for k, rows in groups(ids.cpu(), n):
        s = 1.0 if scale is None else float(scale[k])
        for sign, xs, as_, bs in (("", x[rows], a[k], b[k]), ("_mag", x[rows].abs(), a[k].abs(), b[k].abs())):
            s_ = abs(s) if sign else s
            uu = xs @ as_.t()
            out["u" + sign][rows] = uu
            out["y" + sign][rows] += s_ * uu @ bs.t()
            if g is not None:
                gs = g[rows].abs() if sign else g[rows]
                v = s_ * gs @ bs
                out["grad_x" + sign][rows] = v @ as_
                out["grad_a" + sign][k] = v.t() @ xs
                ug = uu if u is None else (u.double().cpu()[rows].abs() if sign else u.double().cpu()[rows])
                out["grad_b" + sign][k] = s_ * gs.t() @ ug
    return out


def assert_within(got, ref, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite"
    err = (got - ref).abs()
    over = err - bound
    worst = float((err / bound.clamp_min(1e-300)).max()) if err.numel() else 0.0
    assert bool((over <= 0).all()), f"{what}: {worst:.2f} times the bound"
    return worst

"""Adapters of many requests on the GPU: plan, low-rank and block-circulant adapters, forward and
backward, against 64-bit references (bounds: many_util.py and below)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import FP32_TOL, to_host_f64
from many_util import HALF, assert_within, groups, lora_ref, make_ids, plan_ref, sum_bound

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def rd():
    if not torch.cuda.is_available():
        pytest.fail("a CUDA GPU is required for the gpu tests")
    import block_circulant_layers_b200 as rd
    return rd


def randn(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


# ------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("T,n,kind", [(1, 1, "mixed"), (1, 1024, "none"), (31, 3, "wild"), (32, 1, "one"),
                                      (33, 5, "mixed"), (1000, 7, "runs"), (1024, 1024, "mixed"), (1025, 2, "wild"),
                                      (5000, 1000, "mixed"), (40000, 64, "runs"), (4096, 3, "none")])
def test_plan(rd, T, n, kind):
    ids = make_ids(kind, T, n, seed=T)
    order, offsets = plan_ref(ids, n)
    plan = rd.adapter_plan(ids.cuda(), n)
    for _ in range(2):                                   # made twice: the same, in place too
        assert plan.order.tolist() == order
        assert plan.offsets.tolist() == offsets
        plan = rd.adapter_plan(ids.cuda(), n, out=plan)
    # the tile lists: every position once, no tile across groups or above its size
    head = plan.buf[:16].tolist()
    assert head[:2] == [T, n]
    at = 16 + (n + 2 + 3) // 4 * 4 + 2 * ((T + 3) // 4 * 4)
    for l, size in enumerate((4, 16, 64)):
        cap = min(T, T // size + min(T, n + 1))
        tiles = plan.buf[at:at + 2 * head[2 + l]].view(-1, 2).tolist()
        at += (2 * cap + 3) // 4 * 4
        want = [[p, a] for a in range(n + 1) for p in range(offsets[a], offsets[a + 1], size)]
        assert len(want) <= cap and tiles == want


def test_plan_without_tokens(rd):
    plan = rd.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert plan.order.numel() == 0 and plan.offsets.tolist() == [0] * 5


# --------------------------------------------------------------------------- low rank
LORA = [  # T, K, N, r, n, ids
    (1, 4096, 4096, 16, 4, "one"), (1, 8, 8, 8, 1, "mixed"), (7, 40, 264, 8, 3, "none"), (16, 256, 4096, 64, 16, "mixed"),
    (33, 1032, 520, 24, 5, "wild"), (64, 4096, 1024, 128, 3, "mixed"), (100, 520, 72, 40, 200, "mixed"),
    (300, 2056, 1000, 16, 2, "runs"), (500, 1024, 2048, 128, 4, "runs"), (1000, 96, 8200, 32, 1, "one"),
    (257, 4104, 120, 64, 3, "runs"), (129, 72, 64, 112, 1, "wild"), (65, 64, 8, 48, 1, "one"),
    (150000, 64, 72, 8, 3, "runs"), (2000, 320, 4096, 64, 7, "mixed"), (3000, 1000, 264, 16, 700, "wild"),
    (1100, 136, 2056, 128, 30, "runs")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N,r,n,kind", LORA)
def test_lora(rd, T, K, N, r, n, kind, dtype):
    dt = DT[dtype]
    ids = make_ids(kind, T, n, seed=T + K)
    x, g = randn(1, T, K, dtype=dt), randn(2, T, N, dtype=dt)
    a, b = randn(3, n, r, K, std=K ** -0.5, dtype=dt), randn(4, n, N, r, std=r ** -0.5, dtype=dt)
    scale = 0.25 + torch.rand(n, generator=torch.Generator().manual_seed(5)).cuda()
    base = randn(6, T, N, dtype=dt)
    plan = rd.adapter_plan(ids.cuda(), n)
    u = torch.full((T, r), float("nan"), device="cuda")
    y = rd.lora_fwd(x, a, b, plan, scale=scale, base=base, u=u)
    gx, ga, gb = rd.lora_bwd(g, x, a, b, plan, u, scale=scale)
    ref = lora_ref(x, a, b, ids, scale, base, g, u)
    split = 2.0 ** -16 if dtype == "bf16" else 0.0       # mid as hi + lo
    assert_within(u, ref["u"], sum_bound(K, ref["u_mag"], dt), "u")
    assert_within(y, ref["y"], HALF[dt] * ref["y"].abs() + (sum_bound(K, 1, dt) + sum_bound(2 * r, 1, dt) + split)
                  * ref["y_mag"], "y")
    assert_within(gx, ref["grad_x"], HALF[dt] * ref["grad_x"].abs()
                  + (sum_bound(N, 1, dt) + sum_bound(2 * r, 1, dt) + split) * ref["grad_x_mag"], "grad_x")
    assert_within(ga, ref["grad_a"], (sum_bound(N, 1, dt) + sum_bound(3 * T, 1, dt)) * ref["grad_a_mag"], "grad_a")
    assert_within(gb, ref["grad_b"], sum_bound(3 * T, ref["grad_b_mag"], dt), "grad_b")
    # the same bits again; without base and scale; in place
    y2 = base.clone()
    rd.lora_fwd(x, a, b, plan, scale=scale, base=y2, y=y2)
    assert torch.equal(y, y2)
    again = rd.lora_bwd(g, x, a, b, plan, u, scale=scale)
    for p, q in zip((gx, ga, gb), again):
        assert torch.equal(p, q)
    y0 = rd.lora_fwd(x, a, b, plan)
    ref = lora_ref(x, a, b, ids, None, None)
    assert_within(y0, ref["y"], HALF[dt] * ref["y"].abs() + (sum_bound(K, 1, dt) + sum_bound(2 * r, 1, dt) + split)
                  * ref["y_mag"], "y without base")
    # each gradient alone is the same
    assert torch.equal(rd.lora_bwd(g, x, a, b, plan, None, scale=scale, need_grad_a=False, need_grad_b=False)[0], gx)
    assert torch.equal(rd.lora_bwd(g, x, a, b, plan, None, scale=scale, need_grad_x=False, need_grad_b=False)[1], ga)
    assert torch.equal(rd.lora_bwd(g, x, a, b, plan, u, scale=scale, need_grad_x=False, need_grad_a=False)[2], gb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lora_infinities_stay_in_their_token(rd, dtype):
    T, K, N, r, n = 40, 128, 192, 24, 3
    dt = DT[dtype]
    ids = make_ids("mixed", T, n, seed=9)
    x, base = randn(1, T, K, dtype=dt), randn(2, T, N, dtype=dt)
    a, b = randn(3, n, r, K, std=0.1, dtype=dt), randn(4, n, N, r, std=0.2, dtype=dt)
    bad = int((ids >= 0).nonzero()[0])
    none = int((ids < 0).nonzero()[0])
    plan = rd.adapter_plan(ids.cuda(), n)
    clean = rd.lora_fwd(x, a, b, plan, base=base)
    x[bad, 5] = float("inf")
    x[none, 7] = float("nan")                            # a token without an adapter: never read
    y = rd.lora_fwd(x, a, b, plan, base=base)
    rows = [t for t in range(T) if t != bad]
    assert torch.equal(y[rows], clean[rows])
    assert not bool(torch.isfinite(y[bad]).any())


def test_lora_without_tokens(rd):
    n, r, K, N = 2, 8, 64, 72
    plan = rd.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), n)
    a, b = randn(1, n, r, K), randn(2, n, N, r)
    x, g, u = (torch.empty(0, w, device="cuda") for w in (K, N, r))
    assert rd.lora_fwd(x, a, b, plan).shape == (0, N)
    gx, ga, gb = rd.lora_bwd(g, x, a, b, plan, u)
    assert gx.shape == (0, K) and not bool(ga.any()) and not bool(gb.any())


# -------------------------------------------------------------------- block circulant
# The arithmetic is fp32 for both dtypes (its bar: 1e-5 of the largest value) and a bf16 result is
# rounded once, by at most half a step, 2^-8 of the value. The bf16 bar of gpu_util (2e-2 of the
# rms) does not follow from that when rows without an adapter lower the rms: with rms 0.7 it is
# 1.4e-2, and the one rounding of a value of 3.9 already is 3.9 x 2^-8 = 1.52e-2.
def assert_rounded_once(got, ref, dtype, what):
    got = to_host_f64(got)
    assert np.all(np.isfinite(got)), what
    bound = FP32_TOL * np.abs(ref).max() + (HALF[DT[dtype]] * np.abs(ref) if dtype == "bf16" else 0.0)
    assert np.all(np.abs(got - ref) <= bound), f"{what}: {(np.abs(got - ref) / bound).max():.2f} times the bound"


CIRC = [  # T, D, p, n, ids
    (1, 4096, 128, 2, "one"), (5, 64, 64, 1, "mixed"), (9, 320, 64, 4, "wild"), (16, 4096, 128, 16, "mixed"),
    (37, 1024, 256, 3, "none"), (60, 1536, 512, 2, "runs"), (70, 4096, 512, 3, "runs"), (33, 2048, 1024, 2, "mixed"),
    (20, 1024, 1024, 4, "mixed"), (11, 4096, 2048, 3, "mixed"), (10, 2048, 2048, 2, "one"), (6, 8192, 4096, 2, "mixed"),
    (300, 4096, 128, 2, "runs"), (400, 1024, 128, 1, "one"), (700, 4096, 512, 5, "runs"), (333, 4096, 1024, 40, "mixed"), (280, 640, 128, 90, "mixed"), (5, 4096, 4096, 2, "one"),
    (9, 8192, 64, 2, "mixed")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,p,n,kind", CIRC)
def test_circ_many(rd, T, D, p, n, kind, dtype):
    dt, q = DT[dtype], D // p
    ids = make_ids(kind, T, n, seed=T + D + p)
    x, g, base = randn(1, T, D, dtype=dt), randn(2, T, D, dtype=dt), randn(3, T, D, dtype=dt)
    c = randn(4, n, q, q, p, std=D ** -0.5)
    c_hat = rd.rdfft_fwd(c.clone(), p)
    plan = rd.adapter_plan(ids.cuda(), n)
    y = rd.circ_fwd_many(x, c_hat, p, plan, base=base)
    gx, gc = rd.circ_bwd_many(g, x, c_hat, p, plan)
    xe, ge, be, ce = (to_host_f64(t) for t in (x, g, base, c))
    y_ref, gx_ref, gc_ref = be.copy(), np.zeros((T, D)), np.zeros((n, q, q, p))
    for k, rows in groups(ids, n):
        rows = rows.numpy()
        y_ref[rows] += oracle.circ_forward(xe[rows], ce[k])
        gx_ref[rows], gc_ref[k] = oracle.circ_backward(ge[rows], xe[rows], ce[k])
    assert_rounded_once(y, y_ref, dtype, "y")
    # tokens without an adapter: the base row and a zero gradient, bit for bit
    none = [t for t, k in enumerate(ids.tolist()) if not 0 <= k < n]
    assert torch.equal(y[none], base[none]) and not bool(gx[none].any())
    if gx_ref.any():
        assert_rounded_once(gx, gx_ref, dtype, "grad_x")
        assert_rounded_once(gc, gc_ref, "f32", "grad_c")
    idle = [k for k in range(n) if not (ids == k).any()]
    assert not bool(gc[idle].any())
    # in place and again: the same bits. One gradient alone may take other kernels than both.
    y2 = base.clone()
    rd.circ_fwd_many(x, c_hat, p, plan, base=y2, y=y2)
    assert torch.equal(y, y2)
    gx2, gc2 = rd.circ_bwd_many(g, x, c_hat, p, plan)
    assert torch.equal(gx, gx2) and torch.equal(gc, gc2)
    gx1 = rd.circ_bwd_many(g, x, c_hat, p, plan, need_grad_c=False)[0]
    gc1 = rd.circ_bwd_many(g, x, c_hat, p, plan, need_grad_x=False)[1]
    assert not bool(gx1[none].any()) and not bool(gc1[idle].any())
    if gx_ref.any():
        assert_rounded_once(gx1, gx_ref, dtype, "grad_x alone")
        assert_rounded_once(gc1, gc_ref, "f32", "grad_c alone")
    y0 = rd.circ_fwd_many(x, c_hat, p, plan)
    if gx_ref.any():
        assert_rounded_once(y0, y_ref - be, dtype, "y without base")


def test_circ_many_without_tokens(rd):
    plan = rd.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    c_hat = randn(1, 2, 2, 2, 64)
    x = torch.empty(0, 128, device="cuda")
    assert rd.circ_fwd_many(x, c_hat, 64, plan).shape == (0, 128)
    gx, gc = rd.circ_bwd_many(x, x, c_hat, 64, plan)
    assert gx.shape == (0, 128) and not bool(gc.any())


# ---------------------------------------------------------------- a plan of other sizes
def test_plan_of_other_sizes_is_reported(rd):
    """Through the C ABI (the binding refuses it earlier): nothing is written, and the device
    error says so."""
    T, n, K, N, r = 24, 2, 64, 64, 8
    assert rd.take_device_error() == 0
    plan = rd.adapter_plan(torch.zeros(40, dtype=torch.int32, device="cuda"), n)     # larger: reads stay inside
    x, a, b = randn(1, T, K), randn(2, n, r, K), randn(3, n, N, r)
    y = torch.full((T, N), 7.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert rd.lib.lora_fwd(x.data_ptr(), a.data_ptr(), b.data_ptr(), None, None, y.data_ptr(), None,
                           plan.buf.data_ptr(), T, K, N, r, n, 0, s) == 0
    assert rd.take_device_error() == rd.RDFFT_EPLAN
    assert bool((y == 7.0).all())
    c_hat = randn(4, n, 1, 1, 64)
    assert rd.lib.circ_fwd_many(x.data_ptr(), c_hat.data_ptr(), None, y.data_ptr(), plan.buf.data_ptr(), T, 64, 64, n,
                                0, s) == 0
    assert rd.take_device_error() == rd.RDFFT_EPLAN
    assert bool((y == 7.0).all()) and rd.take_device_error() == 0


# ------------------------------------------------------------------------- gradient norm
def flat64(ts):
    return torch.cat([t.detach().double().cpu().flatten() for t in ts])


@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [7, 8, 9, 1000, 65537], [32768] * 64, [13] * 600, [300, 0, 70000] * 500, [3_000_001]])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mixed"])
def test_grad_norm_and_clip(rd, sizes, dtype):
    kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[dtype]
    ts = [randn(i, m, dtype=kinds[i % len(kinds)]) if m else torch.empty(0, dtype=kinds[i % len(kinds)], device="cuda")
          for i, m in enumerate(sizes)]
    ref = float(flat64(ts).norm())
    # each 8-element sum is off by 8 U at most, the double sums by far less, then one root and rounding
    got = rd.grad_norm(ts)
    assert abs(float(got) - ref) <= 6 * 2.0 ** -24 * ref
    for max_norm in (0.25 * ref, 10.0 * ref, 0.0):
        out = [torch.full_like(t, float("nan")) for t in ts]
        before = [t.clone() for t in ts]
        norm = rd.clip_grad_norm(ts, max_norm, out=out)
        assert torch.equal(norm, got) and all(torch.equal(p, q) for p, q in zip(ts, before))
        coef = min(1.0, max_norm / (ref + 1e-6))
        for t, o in zip(ts, out):
            want = t.double().cpu() * coef
            half = HALF[t.dtype]
            assert_within(o, want, (half + 10 * 2.0 ** -24) * want.abs() + 1e-40, "clipped")
        if max_norm > ref:
            assert all(torch.equal(o, t) for o, t in zip(out, ts))
        inplace = [t.clone() for t in ts]
        rd.clip_grad_norm(inplace, max_norm)
        assert all(torch.equal(p, q) for p, q in zip(inplace, out))


def test_clip_of_unaligned_views(rd):
    """Views that start at any element, in and out with different remainders of 16 bytes."""
    for dt in (torch.bfloat16, torch.float32):
        buf, obuf = randn(1, 5000, dtype=dt), torch.full((5000,), 3.0, device="cuda", dtype=dt)
        ins = [buf[1:998], buf[1003:2000], buf[2000:2007], buf[3001:4999]]
        outs = [obuf[2:999], obuf[1004:2001], obuf[2005:2012], obuf[3001:4999]]
        norm = float(rd.clip_grad_norm(ins, 1.0, out=outs))
        ref = float(flat64(ins).norm())
        assert abs(norm - ref) <= 6 * 2.0 ** -24 * ref
        for t, o in zip(ins, outs):
            want = t.double().cpu() / (ref + 1e-6)
            assert_within(o, want, (HALF[dt] + 10 * 2.0 ** -24) * want.abs(), "clipped view")
        keep = torch.ones(5000, dtype=torch.bool)
        for lo, hi in ((2, 999), (1004, 2001), (2005, 2012), (3001, 4999)):
            keep[lo:hi] = False
        assert bool((obuf.cpu()[keep] == 3.0).all())


def test_grad_norm_of_extreme_values(rd):
    """Squares that overflow or underflow fp32, infinities and NaN."""
    for v in (1e25, 3e38, 1e-25, 2e-38, 1e19, 1e-15):
        t = torch.full((4097,), v, device="cuda")
        want = float(t.double().norm())
        if want < 3.4e38:
            assert abs(float(rd.grad_norm([t])) - want) <= 4 * 2.0 ** -24 * want
    assert float(rd.grad_norm([torch.zeros(100, device="cuda")])) == 0.0
    t = randn(1, 100)
    t[17] = float("inf")
    o = [torch.empty_like(t)]
    assert float(rd.clip_grad_norm([t], 1.0, out=o)) == float("inf")
    assert bool(o[0][17].isnan()) and not bool(o[0][:17].any())
    t[3] = float("nan")
    assert bool(rd.clip_grad_norm([t], 1.0, out=o).isnan()) and bool(o[0].isnan().all())

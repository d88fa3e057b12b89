"""The many-adapter operators as a program uses them: modules and their gradients, a chained
training step, other streams, captured and replayed steps, refusals of the binding, tensors
whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from many_util import HALF, assert_within, groups, lora_ref, make_ids, sum_bound

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


# ------------------------------------------------------------------------------ modules
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_low_rank_module(rd, dtype):
    n, K, N, r, T = 3, 128, 192, 16, 60
    bank = rd.LowRankAdapters(n, K, N, r, alpha=8.0, device="cuda")
    assert bank(randn(1, T, K), rd.adapter_plan(torch.zeros(T, dtype=torch.int32, device="cuda"), n)).eq(0).all()
    with torch.no_grad():
        bank.b.copy_(randn(2, n, N, r, std=r ** -0.5))
    ids = make_ids("mixed", T, n, seed=3)
    plan = rd.adapter_plan(ids.cuda(), n)
    x = randn(4, 5, T // 5, K, dtype=DT[dtype]).requires_grad_(True)        # leading dimensions
    base = randn(5, 5, T // 5, N, dtype=DT[dtype]).requires_grad_(True)
    g = randn(6, 5, T // 5, N, dtype=DT[dtype])
    y = bank(x, plan, base)
    y.backward(g)
    a2, b2 = bank.a.detach().to(DT[dtype]), bank.b.detach().to(DT[dtype])
    u = lora_ref(x.detach().reshape(T, K), a2, b2, ids, bank.scale, None)["u"]
    ref = lora_ref(x.detach().reshape(T, K), a2, b2, ids, bank.scale, base.detach().reshape(T, N), g.reshape(T, N), u)
    h, split = HALF[DT[dtype]], 2.0 ** -16 if dtype == "bf16" else 0.0
    s = lambda L: sum_bound(L, 1, DT[dtype])                                # noqa: E731
    assert_within(y.reshape(T, N), ref["y"], h * ref["y"].abs() + (s(K) + s(2 * r) + split) * ref["y_mag"], "y")
    assert_within(x.grad.reshape(T, K), ref["grad_x"],
                  h * ref["grad_x"].abs() + (s(N) + s(2 * r) + split) * ref["grad_x_mag"], "grad_x")
    assert_within(bank.a.grad, ref["grad_a"], (s(N) + s(3 * T)) * ref["grad_a_mag"], "grad_a")
    # grad_b's terms carry the kernel's own u, off by its sum's bound
    assert_within(bank.b.grad, ref["grad_b"], (s(3 * T) + s(K) * 40) * ref["grad_b_mag"], "grad_b")
    assert torch.equal(base.grad, g)


def test_low_rank_gradients_against_differences(rd):
    """Directional derivatives of a smooth loss in each input, central differences in fp32: the
    loss is 1/2 |y|^2, so the differences are exact up to rounding (y is linear in each input)."""
    n, K, N, r, T = 2, 64, 72, 8, 30
    ids = make_ids("mixed", T, n, seed=1)
    plan = rd.adapter_plan(ids.cuda(), n)
    scale = torch.tensor([0.5, 2.0], device="cuda")
    ins = [randn(k, *s, std=0.3) for k, s in ((2, (T, K)), (3, (n, r, K)), (4, (n, N, r)), (5, (T, N)))]
    leaves = [t.clone().requires_grad_(True) for t in ins]
    rd.low_rank_many(leaves[0], leaves[1], leaves[2], plan, scale, leaves[3]).square().sum().mul(0.5).backward()

    def loss(args):
        return float(rd.low_rank_many(args[0], args[1], args[2], plan, scale, args[3]).double().square().sum()) / 2

    for k in range(4):
        d = randn(10 + k, *ins[k].shape)
        eps = 2.0 ** -6
        up, dn = list(ins), list(ins)
        up[k], dn[k] = ins[k] + eps * d, ins[k] - eps * d
        # rounding: each y is off by about 2^-22 of its terms, so the difference by that of 2 x loss / (2 eps)
        num, ana = (loss(up) - loss(dn)) / (2 * eps), float((leaves[k].grad * d).double().sum())
        assert abs(num - ana) <= 2.0 ** -20 * (loss(up) + loss(dn)) / eps, (k, num, ana)


def test_circulant_gradients_against_differences(rd):
    n, p, q, T = 2, 64, 2, 26
    ids = make_ids("mixed", T, n, seed=7)
    plan = rd.adapter_plan(ids.cuda(), n)
    ins = [randn(2, T, q * p, std=0.3), randn(3, n, q, q, p, std=0.1), randn(4, T, q * p, std=0.3)]
    leaves = [t.clone().requires_grad_(True) for t in ins]
    rd.block_circulant_many(leaves[0], leaves[1], p, plan, leaves[2]).square().sum().mul(0.5).backward()

    def loss(args):
        return float(rd.block_circulant_many(args[0], args[1], p, plan, args[2]).double().square().sum()) / 2

    for k in range(3):
        d = randn(10 + k, *ins[k].shape)
        eps = 2.0 ** -6
        up, dn = list(ins), list(ins)
        up[k], dn[k] = ins[k] + eps * d, ins[k] - eps * d
        num, ana = (loss(up) - loss(dn)) / (2 * eps), float((leaves[k].grad * d).double().sum())
        assert abs(num - ana) <= 2.0 ** -20 * (loss(up) + loss(dn)) / eps, (k, num, ana)


def test_one_adapter_is_the_dense_layer(rd):
    """A bank of one adapter that every token uses gives BlockCirculantLinear's results (other
    kernel shapes may round differently in the last fp32 bits: compared at the fp32 bar)."""
    D, p, T = 1024, 256, 50
    layer = rd.BlockCirculantLinear(D, p, device="cuda", deterministic=True)
    bank = rd.BlockCirculantAdapters(1, D, p, device="cuda")
    with torch.no_grad():
        bank.c.copy_(layer.c[None])
    plan = rd.adapter_plan(torch.zeros(T, dtype=torch.int32, device="cuda"), 1)
    x, g = randn(1, T, D), randn(2, T, D)
    xs = [x.clone().requires_grad_(True) for _ in range(2)]
    ys = [layer(xs[0]), bank(xs[1], plan)]
    for y in ys:
        y.backward(g)
    for a, b in ((ys[0], ys[1]), (xs[0].grad, xs[1].grad), (layer.c.grad, bank.c.grad[0])):
        assert float((a - b).detach().abs().max()) <= 1e-5 * float(a.detach().abs().max())


def test_modules_skip_what_needs_no_gradient(rd):
    n, K, r, T = 2, 64, 8, 20
    plan = rd.adapter_plan(make_ids("mixed", T, n).cuda(), n)
    bank = rd.LowRankAdapters(n, K, K, r, device="cuda")
    bank.requires_grad_(False)
    x = randn(1, T, K).requires_grad_(True)
    bank(x, plan).sum().backward()
    assert x.grad is not None and bank.a.grad is None
    bank.a.requires_grad_(True)
    bank(x.detach(), plan).sum().backward()
    assert bank.a.grad is not None and bank.b.grad is None
    with torch.no_grad():
        assert not bank(x, plan).requires_grad


def test_modules_in_bf16_and_without_tokens(rd):
    n, K, r = 2, 64, 8
    bank = rd.LowRankAdapters(n, K, K, r, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        bank.b.copy_(randn(3, n, K, r))
    plan = rd.adapter_plan(make_ids("mixed", 20, n).cuda(), n)
    bank(randn(1, 20, K, dtype=torch.bfloat16), plan).float().square().sum().backward()
    assert bank.a.grad.dtype == bank.b.grad.dtype == torch.bfloat16 and bool(bank.b.grad.any())
    empty = rd.adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), n)
    x = torch.empty(0, K, device="cuda", requires_grad=True)
    for bank in (rd.LowRankAdapters(n, K, K, r, device="cuda"), rd.BlockCirculantAdapters(n, K, 64, device="cuda")):
        bank(x, empty).sum().backward()
        assert x.grad.shape == (0, K) and all(not bool(p.grad.any()) for p in bank.parameters())


def test_a_plan_made_again_fails_the_backward(rd):
    n, K, T = 2, 64, 16
    ids = make_ids("mixed", T, n).cuda()
    plan = rd.adapter_plan(ids, n)
    bank = rd.LowRankAdapters(n, K, K, 8, device="cuda")
    y = bank(randn(1, T, K), plan)
    rd.adapter_plan(ids.flip(0).contiguous(), n, out=plan)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# -------------------------------------------------------------------- the step together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step_of_both_kinds(rd, dtype):
    """Plan, shared projection, low-rank and block-circulant adapters beside it, backward, the
    gradients clipped together: against the same step in float64."""
    n, D, r, p, T = 3, 256, 8, 64, 90
    dt = DT[dtype]
    ids = make_ids("runs", T, n, seed=11)
    plan = rd.adapter_plan(ids.cuda(), n)
    w = randn(1, D, D, std=D ** -0.5, dtype=dt)
    low = rd.LowRankAdapters(n, D, D, r, device="cuda")
    circ = rd.BlockCirculantAdapters(n, D, p, device="cuda")
    with torch.no_grad():
        low.b.copy_(randn(2, n, D, r, std=r ** -0.5))
    x, target = randn(3, T, D, dtype=dt), randn(4, T, D, dtype=dt)
    y = circ(low(x, plan, x @ w.t()), plan, x)
    (y.float() - target.float()).square().mean().backward()
    grads = [low.a.grad, low.b.grad, circ.c.grad]
    before = [g.clone() for g in grads]
    norm = rd.clip_grad_norm(grads, 0.1)

    la, lb, cc = (t.detach().double().cpu().requires_grad_(True) for t in (low.a, low.b, circ.c))
    xd, wd, q = x.double().cpu(), w.double().cpu(), D // p
    m = torch.arange(p)
    h = xd @ wd.t()
    outs = []
    for t, k in enumerate(ids.tolist()):
        z = h[t]
        if 0 <= k < n:
            z = z + (lb[k] @ (la[k] @ xd[t])) * float(low.scale[k])
            dense = cc[k][:, :, (m[:, None] - m[None, :]) % p].permute(0, 2, 1, 3).reshape(D, D)
            outs.append(xd[t] + dense @ z)
        else:
            outs.append(xd[t])
    (torch.stack(outs) - target.double().cpu()).square().mean().backward()
    # bf16: the parameters, x @ w, the adapters' outputs and the loss gradient are rounded to half
    # a step (2^-8) each on the way; 8 such roundings, none amplified by more than the layer's gain
    # of about 2. fp32: the fp32 bar of the layer
    tol = 16 * 2.0 ** -8 if dtype == "bf16" else 1e-5
    for got, ref in zip(before, (la.grad, lb.grad, cc.grad)):
        assert float((got.double().cpu() - ref).abs().max()) <= tol * float(ref.abs().max())
    ref_norm = float(torch.cat([t.flatten() for t in before]).double().norm())
    assert abs(float(norm) - ref_norm) <= 1e-6 * ref_norm
    coef = min(1.0, 0.1 / (ref_norm + 1e-6))
    for g, b in zip(grads, before):
        assert float((g - b * coef).abs().max()) <= 1e-6 * float(b.abs().max())


def test_readme_example(rd):
    """The example runs, and its parameters get finite gradients, of the adapters in use only."""
    import os
    import re

    from conftest import ROOT
    with open(os.path.join(ROOT, "README.md")) as f:
        code = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    assert len(code) == 1
    scope = {}
    exec(code[0], scope)                                                     # noqa: S102
    low, circ, ids = scope["low"], scope["circ"], scope["ids"]
    assert set(ids.tolist()) == {-1, 0, 1} and bool(torch.isfinite(scope["norm"]))
    for t in (low.b.grad, circ.c.grad):
        assert bool(torch.isfinite(t).all()) and bool(t.flatten(1).any(1).all())
    assert not bool(low.a.grad.any())                                        # b starts at zero


def test_bucket_clip(rd):
    from block_circulant_layers_b200.dp import GradCBucket
    bucket = GradCBucket([torch.Size((2, 2, 64)), torch.Size((3,)), torch.Size((4, 4, 128))], "cuda")
    for k, v in enumerate(bucket.views):
        v.copy_(randn(k, *v.shape))
    before = bucket.flat.clone()
    norm = bucket.clip(1.0)
    ref = float(before.double().norm())
    assert abs(float(norm) - ref) <= 1e-6 * ref
    assert float((bucket.flat - before / (ref + 1e-6)).abs().max()) <= 1e-6
    assert all(v.data_ptr() >= bucket.flat.data_ptr() for v in bucket.views)


# ------------------------------------------------------------------- streams and graphs
def step_inputs(T, K, N, r, n, seed, dtype):
    return dict(x=randn(seed, T, K, dtype=dtype), a=randn(seed + 1, n, r, K, std=K ** -0.5, dtype=dtype),
                b=randn(seed + 2, n, N, r, std=r ** -0.5, dtype=dtype), g=randn(seed + 3, T, N, dtype=dtype))


def test_two_streams_at_once(rd):
    """Calls on two streams of their own, each behind work that fills the GPU."""
    T, K, N, r, n = 700, 1024, 768, 32, 3
    ids = [make_ids("mixed", T, n, seed=s).cuda() for s in (1, 2)]
    ins = [step_inputs(T, K, N, r, n, 100 * s, torch.bfloat16) for s in (1, 2)]
    c_hat = randn(9, n, 4, 4, 256)
    cx = randn(10, T, 1024, dtype=torch.bfloat16)

    def one(i):
        plan = rd.adapter_plan(ids[i], n)
        u = torch.empty(T, r, device="cuda")
        y = rd.lora_fwd(ins[i]["x"], ins[i]["a"], ins[i]["b"], plan, u=u)
        grads = rd.lora_bwd(ins[i]["g"], ins[i]["x"], ins[i]["a"], ins[i]["b"], plan, u)
        z = rd.circ_fwd_many(cx, c_hat, 256, plan)
        cg = rd.circ_bwd_many(z, cx, c_hat, 256, plan)
        norm = rd.grad_norm([*grads, *cg])
        return [y, *grads, z, *cg, norm]

    want = [one(0), one(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        got = [None, None]
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                busy @ busy
                got[i] = one(i)
        torch.cuda.synchronize()
        for i in range(2):
            for p, q in zip(got[i], want[i]):
                assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_step_with_new_ids(rd, dtype):
    """A step captured once, its plan made inside it, replayed on other ids and inputs."""
    T, K, N, r, n, p = 80, 512, 256, 8, 4, 128
    dt = DT[dtype]
    s = step_inputs(T, K, N, r, n, 1, dt)
    ids = make_ids("mixed", T, n, seed=1).cuda()
    c_hat, cx = randn(7, n, 2, 2, p), randn(8, T, 2 * p, dtype=dt)
    plan = rd.adapter_plan(ids, n)
    u = torch.empty(T, r, device="cuda")

    def step():
        rd.adapter_plan(ids, n, out=plan)
        y = rd.lora_fwd(s["x"], s["a"], s["b"], plan, u=u)
        grads = rd.lora_bwd(s["g"], s["x"], s["a"], s["b"], plan, u)
        z = rd.circ_fwd_many(cx, c_hat, p, plan, base=y)
        cg = rd.circ_bwd_many(y, cx, c_hat, p, plan)
        norm = rd.clip_grad_norm([*grads[1:], cg[1]], 1.0)
        return [y, *grads, z, *cg, norm]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        ids.copy_(make_ids(["mixed", "none", "one"][seed], T, n, seed=seed + 5))
        s["x"].copy_(randn(50 + seed, T, K, dtype=dt))
        cx.copy_(randn(60 + seed, T, 2 * p, dtype=dt))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_two_captured_graphs_in_turn(rd):
    """Two graphs of the same calls on other tensors, replayed in turn: neither disturbs the other."""
    T, K, N, r, n = 200, 256, 256, 16, 2
    ids = make_ids("runs", T, n, seed=3).cuda()
    plan = rd.adapter_plan(ids, n)
    ins = [step_inputs(T, K, N, r, n, 10 * k, torch.bfloat16) for k in (1, 2)]

    def step(s):
        u = torch.empty(T, r, device="cuda")
        y = rd.lora_fwd(s["x"], s["a"], s["b"], plan, u=u)
        grads = rd.lora_bwd(s["g"], s["x"], s["a"], s["b"], plan, u)
        return [y, *grads, rd.grad_norm(grads)]

    want = [[t.clone() for t in step(s)] for s in ins]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
    for k in (0, 1, 1, 0, 1, 0):
        graphs[k].replay()
        for p, q in zip(outs[k], want[k]):
            assert torch.equal(p, q)


def test_captured_backward_of_the_modules(rd):
    """Forward and backward of both modules captured (no eager graph of the leaves alive)."""
    n, D, p, T = 2, 256, 64, 40
    low = rd.LowRankAdapters(n, D, D, 8, device="cuda")
    with torch.no_grad():
        low.b.copy_(randn(2, n, D, 8))
    circ = rd.BlockCirculantAdapters(n, D, p, device="cuda")
    ids = make_ids("mixed", T, n, seed=4).cuda()
    x = randn(3, T, D)
    plan = rd.adapter_plan(ids, n)
    params = [low.a, low.b, circ.c]

    def step():
        return torch.autograd.grad(circ(low(x, plan, x), plan).square().sum(), params)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# --------------------------------------------------------------- refusals of the binding
def test_binding_refusals(rd):
    T, K, N, r, n = 12, 64, 72, 8, 2
    ids = make_ids("mixed", T, n).cuda()
    plan = rd.adapter_plan(ids, n)
    x, a, b, g = randn(1, T, K), randn(2, n, r, K), randn(3, n, N, r), randn(4, T, N)
    u = torch.zeros(T, r, device="cuda")
    for bad in (ids.cpu(), ids.long(), ids[None]):
        with pytest.raises(TypeError):
            rd.adapter_plan(bad, n)
    with pytest.raises(rd.RdfftError):
        rd.adapter_plan(ids, 0)
    with pytest.raises(ValueError):
        rd.adapter_plan(ids, n, out=rd.adapter_plan(ids[:4].contiguous(), n))
    with pytest.raises(TypeError):
        rd.lora_fwd(x.cpu(), a, b, plan)
    with pytest.raises(TypeError):
        rd.lora_fwd(x.half(), a.half(), b.half(), plan)
    for kw in (dict(x=x.t().contiguous().t()), dict(x=x[:, :32].contiguous()), dict(x=x[:5]), dict(a=a.bfloat16()),
               dict(b=b[:1]), dict(base=g.bfloat16()), dict(base=g[:3]), dict(scale=torch.ones(n)),
               dict(scale=torch.ones(n + 1, device="cuda")), dict(y=torch.empty(T, K, device="cuda")),
               dict(u=u.bfloat16())):
        args = dict(x=x, a=a, b=b, plan=plan)
        args.update(kw)
        with pytest.raises((ValueError, TypeError)):                         # TypeError: not on the GPU
            rd.lora_fwd(**args)
    with pytest.raises(rd.RdfftError):                                       # a rank of 4
        rd.lora_fwd(x, a[:, :4].contiguous(), b[..., :4].contiguous(), plan)
    with pytest.raises(rd.RdfftError):                                       # u in a's memory
        rd.lora_fwd(x, a, b, plan, u=a.view(-1)[:T * r].view(T, r))
    with pytest.raises(ValueError):
        rd.lora_bwd(g, x, a, b, plan, None)                                  # grad_b needs u
    with pytest.raises(ValueError):
        rd.lora_bwd(g[:, :64].contiguous(), x, a, b, plan, u)
    c_hat = randn(5, n, 1, 1, 64)
    for kw in (dict(x=x[:3]), dict(c_hat=c_hat[:1]), dict(p=32), dict(base=x.bfloat16())):
        args = dict(x=x, c_hat=c_hat, p=64, plan=plan)
        args.update(kw)
        with pytest.raises(ValueError):
            rd.circ_fwd_many(**args)
    with pytest.raises(TypeError):
        rd.circ_fwd_many(x, c_hat.bfloat16(), 64, plan)
    with pytest.raises(ValueError):
        rd.grad_norm([])
    for bad in ([x.half()], [x.cpu()], [x.t()], [3]):
        with pytest.raises(TypeError):
            rd.clip_grad_norm(bad, 1.0)
    with pytest.raises(ValueError):
        rd.clip_grad_norm([x, g], 1.0, out=[x])
    with pytest.raises(ValueError):
        rd.clip_grad_norm([x], 1.0, out=[x.bfloat16()])
    for bad in (-1.0, float("nan")):
        with pytest.raises(rd.RdfftError):
            rd.clip_grad_norm([x], bad)
    with pytest.raises(rd.RdfftError):
        rd.clip_grad_norm([x, x], 1.0)                                       # the same tensor twice
    assert float(rd.grad_norm([x, x])) > 0                                   # which a norm alone may take
    with pytest.raises(ValueError):
        rd.low_rank_many(x, a, b, plan, torch.ones(n, device="cuda", requires_grad=True))
    assert rd.take_device_error() == 0


# ---------------------------------------------------------------- offsets past 32 bits
def test_lora_offsets_past_32_bits(rd):
    """x of 2.16e9 elements; the last tokens and a few others against float64."""
    T, K, N, r, n = 66000, 32768, 8, 8, 2
    assert T * K > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    a, b, g = randn(2, n, r, K, std=K ** -0.5, dtype=x.dtype), randn(3, n, N, r, dtype=x.dtype), randn(4, T, N, dtype=x.dtype)
    ids = (torch.arange(T) % 3 - 1).int()
    plan = rd.adapter_plan(ids.cuda(), n)
    u = torch.empty(T, r, device="cuda")
    y = rd.lora_fwd(x, a, b, plan, u=u)
    gx, _, gb = rd.lora_bwd(g, x, a, b, plan, u, need_grad_a=False)
    rows = torch.tensor([0, 1, 2, 40000, 65534, 65535, 65536, T - 3, T - 2, T - 1])
    ref = lora_ref(x[rows.cuda()], a, b, ids[rows], None, None, g[rows.cuda()])
    s = lambda L: sum_bound(L, 1, x.dtype)                                   # noqa: E731
    h = HALF[x.dtype]
    assert_within(y[rows.cuda()], ref["y"], h * ref["y"].abs() + (s(K) + s(2 * r) + 2.0 ** -16) * ref["y_mag"], "y")
    assert_within(gx[rows.cuda()], ref["grad_x"],
                  h * ref["grad_x"].abs() + (s(N) + s(2 * r) + 2.0 ** -16) * ref["grad_x_mag"], "grad_x")
    assert not bool(y[ids.cuda() < 0].any())
    want = sum((g[ids.cuda() == k].double().t() @ u[ids.cuda() == k].double()).norm() for k in range(n))
    assert abs(float(gb.double().norm(dim=(1, 2)).sum() - want)) <= 1e-4 * float(want)


def test_circ_offsets_past_32_bits(rd):
    import oracle
    T, D, p, n = 530000, 4096, 512, 2
    assert T * D > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    c = randn(2, n, 8, 8, p, std=D ** -0.5)
    c_hat = rd.rdfft_fwd(c.clone(), p)
    ids = (torch.arange(T) % 3 - 1).int()
    plan = rd.adapter_plan(ids.cuda(), n)
    y = rd.circ_fwd_many(x, c_hat, p, plan, base=x)
    gx, _ = rd.circ_bwd_many(x, x, c_hat, p, plan)
    for t in (1, 2, 524287, 524288, 524289, T - 3, T - 2, T - 1):
        k = int(ids[t])
        xe = x[t].double().cpu().numpy()[None]
        ye, ge = xe.copy(), np.zeros_like(xe)
        if k >= 0:
            ce = c[k].double().cpu().numpy()
            ye += oracle.circ_forward(xe, ce)
            ge = oracle.circ_backward(xe, xe, ce)[0]
        for got, ref in ((y[t], ye), (gx[t], ge)):
            err = np.abs(got.double().cpu().numpy() - ref[0])
            assert np.all(err <= 2.0 ** -8 * np.abs(ref[0]) + 1e-5 * np.abs(xe).max() * 4), t

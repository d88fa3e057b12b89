"""Edges of the many-adapter operators: adapters that no token uses, values that are not finite,
long sums, plans that do not fit, and what a call leaves behind."""
import pytest
import torch

from many_util import make_ids

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


# ----------------------------------------------------------------- adapters without tokens
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,r", [(0, 16), (30, 8), (30, 64), (1200, 24), (1200, 128)])
def test_an_idle_adapters_scale_is_not_used(rd, T, r, dtype):
    """The gradients of an adapter without tokens are zeros even where its scale is not finite, and
    the others' gradients have the same bits as with a finite one."""
    n, K, N, dt = 6, 136, 200, DT[dtype]
    ids = make_ids("mixed", T, 3, seed=2) * 2                 # adapters 0, 2 and 4, or -2: none
    x, g = randn(1, T, K, dtype=dt), randn(2, T, N, dtype=dt)
    a, b = randn(3, n, r, K, std=0.1, dtype=dt), randn(4, n, N, r, std=0.2, dtype=dt)
    scale = 0.5 + torch.rand(n, generator=torch.Generator().manual_seed(5)).cuda()
    plan = rd.adapter_plan(ids.cuda(), n)
    u = torch.empty(T, r, device="cuda")
    rd.lora_fwd(x, a, b, plan, scale=scale, u=u)
    want = rd.lora_bwd(g, x, a, b, plan, u, scale=scale)
    for k, bad in ((1, float("nan")), (3, float("inf")), (5, -float("inf"))):
        scale[k] = bad
    got = rd.lora_bwd(g, x, a, b, plan, u, scale=scale)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    for t in got[1:]:
        assert not bool(t[1::2].any())


# ------------------------------------------------------------------------------ long sums
def shrink(got, ref):
    """Mean over all elements of how far the result falls short, relative (its terms all positive)."""
    return float(((ref - got.double()) / ref).mean())


@pytest.mark.parametrize("T,K,r", [(16, 65536, 16), (40, 65536, 128), (2048, 65536, 16), (1100, 65536, 128),
                                   (262144, 256, 16), (65536, 256, 64), (32768, 256, 128)])
def test_long_bf16_sums_do_not_shrink(rd, T, K, r):
    """u, grad_a and grad_b (fp32) of positive bf16 operands in 64 bits. Roundings to nearest have mean
    zero; truncating ones would make every sum smaller, in proportion to its length. A tensor-core
    accumulator takes at most 12 additions (three products of 64 tokens), 8 for u and v, each short by
    at most a step, 2 U; 4 U for what the roundings to nearest leave in the mean."""
    U, n, N = 2.0 ** -24, 1, 64 if K > 1024 else 256
    x, g = randn(1, T, K).abs().bfloat16(), randn(2, T, N).abs().bfloat16()
    a, b = (randn(3, n, r, K).abs() * K ** -0.5).bfloat16(), (randn(4, n, N, r).abs() * r ** -0.5).bfloat16()
    plan = rd.adapter_plan(torch.zeros(T, dtype=torch.int32, device="cuda"), n)
    u = torch.empty(T, r, device="cuda")
    rd.lora_fwd(x, a, b, plan, u=u)
    _, ga, gb = rd.lora_bwd(g, x, a, b, plan, u)
    v = g.double() @ b[0].double()
    ref_u = torch.cat([t.double() @ a[0].double().t() for t in x.split(1 << 13)])
    ref_ga = sum(p.t() @ t.double() for p, t in zip(v.split(1 << 13), x.split(1 << 13)))
    ref_gb = g.double().t() @ u.double()
    assert abs(shrink(u, ref_u)) <= (8 * 2 + 4) * U
    assert abs(shrink(gb[0], ref_gb)) <= (12 * 2 + 4) * U
    assert abs(shrink(ga[0], ref_ga)) <= (12 * 2 + 8 * 2 + 4) * U          # v is such a sum as well


# -------------------------------------------------------------------- a module's own dtype
def test_a_converted_bank_keeps_its_scale(rd):
    """alpha / r = 8 / 24 in a bank converted to bf16, with fp32 activations and weights that make
    y = scale x_0: two roundings of half a step (2^-24), of the scale and of the product."""
    n, K, r, T = 1, 64, 24, 40
    bank = rd.LowRankAdapters(n, K, 8, r, alpha=8.0, device="cuda").to(torch.bfloat16)
    with torch.no_grad():
        bank.a.zero_()
        bank.a[0, 0, 0] = 1.0                                 # u = (x_0, 0, ...)
        bank.b[0, :, 0] = 1.0                                 # y = scale x_0 in every column
    x = torch.arange(1, T + 1, device="cuda", dtype=torch.float32)[:, None].repeat(1, K)
    plan = rd.adapter_plan(torch.zeros(T, dtype=torch.int32, device="cuda"), n)
    y = bank(x, plan)                                         # fp32 activations, bf16 weights
    want = x[:, :8].double() * (8.0 / 24.0)
    assert float(((y.detach().double() - want) / want).abs().max()) <= 2 * 2.0 ** -24
    y.sum().backward()
    assert bank.b.grad.dtype == torch.bfloat16
    want_b = float(x[:, 0].double().sum()) * (8.0 / 24.0)     # each column's sum of scale u, rounded to bf16
    assert float((bank.b.grad[0, :, 0].double() - want_b).abs().max()) <= (2.0 ** -8 + 1e-6) * want_b


# ------------------------------------------------------------------- plans that do not fit
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("wants", [(1, 0, 1), (1, 1, 1), (0, 1, 0), (0, 0, 1)])
def test_backward_with_a_plan_of_other_sizes(rd, wants, dtype):
    """Through the C ABI (the binding refuses it earlier), the plan made again right behind it and
    used: nothing is written by the first call, the device error says so, the second is right."""
    T, n, K, N, r, dt = 90, 2, 64, 72, 8, (torch.float32, torch.bfloat16)[dtype]
    ids = make_ids("mixed", T, n, seed=1).cuda()
    x, g, a, b = (randn(k, *s, dtype=dt) for k, s in ((1, (T, K)), (2, (T, N)), (3, (n, r, K)), (4, (n, N, r))))
    good = rd.adapter_plan(ids, n)
    u = torch.empty(T, r, device="cuda")
    rd.lora_fwd(x, a, b, good, u=u)
    want = rd.lora_bwd(g, x, a, b, good, u)
    buf = rd.adapter_plan(torch.zeros(4 * T, dtype=torch.int32, device="cuda"), n).buf     # larger: reads stay inside
    outs = [torch.full_like(t, 7.0) if w else None for t, w in zip(want, wants)]
    v = torch.full((T, r), 7.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert rd.take_device_error() == 0

    def call():
        p = [None if t is None else t.data_ptr() for t in outs]
        assert rd.lib.lora_bwd(g.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), None, u.data_ptr(),
                               v.data_ptr(), *p, buf.data_ptr(), T, K, N, r, n, dtype, s) == 0

    call()
    kept = [None if t is None else t.clone() for t in [*outs, v]]
    assert rd.lib.adapter_plan(ids.data_ptr(), T, n, buf.data_ptr(), s) == 0
    call()
    assert rd.take_device_error() == rd.RDFFT_EPLAN and rd.take_device_error() == 0
    assert all(t is None or bool((t == 7.0).all()) for t in kept)
    assert all(t is None or torch.equal(t, w) for t, w in zip(outs, want))


def test_a_plan_whose_buffer_does_not_hold_it_is_refused(rd):
    T, n, K = 200, 3, 64
    ids = make_ids("mixed", T, n).cuda()
    plan = rd.adapter_plan(ids, n)
    x, a, b, c_hat = randn(1, T, K), randn(2, n, 8, K), randn(3, n, K, 8), randn(4, n, 1, 1, K)
    u = torch.zeros(T, 8, device="cuda")
    for buf in (plan.buf[:-4], plan.buf[:0], plan.buf.float(), plan.buf.cpu(), torch.stack([plan.buf] * 2, 1)[:, 0]):
        bad = rd.AdapterPlan(T, n, buf)
        for call in (lambda: rd.adapter_plan(ids, n, out=bad), lambda: rd.lora_fwd(x, a, b, bad),
                     lambda: rd.lora_bwd(x, x, a, b, bad, u), lambda: rd.circ_fwd_many(x, c_hat, K, bad),
                     lambda: rd.circ_bwd_many(x, x, c_hat, K, bad)):
            with pytest.raises(ValueError):
                call()
    rd.lora_fwd(x, a, b, plan)
    assert rd.take_device_error() == 0


# ------------------------------------------------------------------- what a call leaves behind
def test_a_graph_notices_what_a_call_overwrites(rd):
    """Tensors that a call writes into count as modified in place, and no others do; a backward pass that
    saved one fails instead of using the new values. Tensors made in inference mode are written too."""
    T, n, K, r = 30, 2, 64, 8
    plan = rd.adapter_plan(make_ids("mixed", T, n).cuda(), n)
    x, a, b, g = randn(1, T, K), randn(2, n, r, K), randn(3, n, K, r), randn(4, T, K)
    c_hat = randn(5, n, 1, 1, K)
    new = {k: torch.empty(s, device="cuda") for k, s in dict(
        y=(T, K), u=(T, r), gx=(T, K), ga=(n, r, K), gb=(n, K, r), ws=(T, r), gc=(n, 1, 1, K), out=(T, K)).items()}
    import ctypes
    need = ctypes.c_size_t()
    rd.lib.circ_bwd_many_workspace_size(T, K, K, n, 0, 1, ctypes.byref(need))
    new["cws"] = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    inputs = [x, a, b, g, c_hat]
    seen = {k: t._version for k, t in new.items()}

    def advanced():
        k = {k for k, t in new.items() if t._version != seen[k]}
        seen.update((k, t._version) for k, t in new.items())
        return k

    rd.lora_fwd(x, a, b, plan, y=new["y"], u=new["u"])
    assert advanced() == {"y", "u"}
    kw = dict(grad_x=new["gx"], grad_a=new["ga"], grad_b=new["gb"], workspace=new["ws"])
    rd.lora_bwd(g, x, a, b, plan, new["u"], **kw)
    assert advanced() == {"gx", "ga", "gb", "ws"}
    rd.lora_bwd(g, x, a, b, plan, new["u"], need_grad_x=False, need_grad_a=False, **kw)
    assert advanced() == {"gb"}
    rd.circ_fwd_many(x, c_hat, K, plan, y=new["y"])
    assert advanced() == {"y"}
    rd.circ_bwd_many(g, x, c_hat, K, plan, grad_x=new["gx"], grad_c=new["gc"], workspace=new["cws"])
    assert advanced() == {"gx", "gc", "cws"}
    rd.grad_norm([x, new["gx"]])
    rd.clip_grad_norm([x], 1.0, out=[new["out"]])
    assert advanced() == {"out"}
    rd.clip_grad_norm([new["gx"], new["ga"]], 1.0)
    assert advanced() == {"gx", "ga"}
    with pytest.raises(rd.RdfftError):
        rd.clip_grad_norm([new["gx"]], -1.0)                  # refused: nothing written
    assert advanced() == set() and all(t._version == 0 for t in inputs)

    leaf = x.clone().requires_grad_(True)
    h = leaf * 2.0
    loss = h.square().sum()                                   # saves h
    rd.circ_fwd_many(x, c_hat, K, plan, base=h.detach(), y=h.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        held = torch.zeros(T, K, device="cuda")
        kept = rd.adapter_plan(make_ids("one", T, n).cuda(), n)
    rd.circ_fwd_many(x, c_hat, K, plan, y=held)
    rd.clip_grad_norm([held], 1.0)
    assert bool(held.any())
    assert rd.adapter_plan(make_ids("none", T, n).cuda(), n, out=kept).offsets.tolist() == [0, 0, 0, T]


@pytest.mark.parametrize("count", [1, 100])
def test_a_kept_norm_keeps_no_workspace(rd, count):
    ts = [randn(k, 100) for k in range(count)]
    for norm in (rd.grad_norm(ts), rd.clip_grad_norm(ts, 1.0)):
        assert norm.shape == () and norm.dtype == torch.float32 and norm.untyped_storage().nbytes() == 4


def run_alone(code):
    """Runs a program of its own and returns the last line it prints."""
    import subprocess
    import sys

    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return r.stdout.strip().splitlines()[-1]


def test_reading_the_device_error_costs_one_copy_per_word(rd):
    """Every copy waits for the device: three words of the transforms' kernels, and one of all kernels
    that take a plan, read only once one of them has been launched."""
    code = """
import torch, block_circulant_layers_b200 as rd
from torch.profiler import profile, ProfilerActivity
def copies():
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
        assert rd.take_device_error() == 0
    return sum("Memcpy DtoH" in e.name for e in p.events())
x = torch.randn(4, 128, device="cuda")
rd.rdfft_fwd(x, 64)
copies()
before = copies()
plan = rd.adapter_plan(torch.zeros(4, dtype=torch.int32, device="cuda"), 1)
rd.circ_fwd_many(x, torch.randn(1, 2, 2, 64, device="cuda"), 64, plan)
rd.lora_fwd(x, torch.randn(1, 8, 128, device="cuda"), torch.randn(1, 64, 8, device="cuda"), plan)
print(before, copies())
"""
    assert run_alone(code) == "3 4"


def test_a_programs_first_calls_are_captured(rd):
    """Nothing of the library is loaded before the capture begins; the replay gives an eager call's bits."""
    code = """
import torch, block_circulant_layers_b200 as rd
torch.manual_seed(0)
T, n, K = 40, 2, 128
ids = torch.randint(-1, n, (T,), dtype=torch.int32, device="cuda")
x, a, b = torch.randn(T, K, device="cuda"), torch.randn(n, 8, K, device="cuda"), torch.randn(n, K, 8, device="cuda")
c, u = torch.randn(n, 2, 2, 64, device="cuda"), torch.empty(T, 8, device="cuda")
def step():
    plan = rd.adapter_plan(ids, n)
    y = rd.lora_fwd(x, a, b, plan, u=u)
    grads = [*rd.lora_bwd(y, x, a, b, plan, u), rd.circ_fwd_many(x, c, 64, plan), *rd.circ_bwd_many(y, x, c, 64, plan)]
    return [y, *grads, rd.grad_norm(grads)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
print(all(torch.equal(p, q) for p, q in zip(got, want)), rd.take_device_error())
"""
    assert run_alone(code) == "True 0"


# ----------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,r,kind", [(40, 24, "mixed"), (1500, 24, "runs"), (1500, 64, "runs"), (1030, 128, "mixed")])
def test_values_that_are_not_finite_stay_where_they_belong(rd, T, r, kind, dtype):
    """An infinity or NaN in one token's x, g or base reaches that token's rows and its adapter's weight
    gradients only, with the tiles of 16 and of 64 tokens and whatever shares a tile with it; in a
    token without an adapter it reaches nothing but a copied base row. All else has the same bits."""
    n, K, N, dt = 5, 136, 200, DT[dtype]
    ids = make_ids(kind, T, n, seed=3)
    x, g, base = randn(1, T, K, dtype=dt), randn(2, T, N, dtype=dt), randn(3, T, N, dtype=dt)
    a, b = randn(4, n, r, K, std=0.1, dtype=dt), randn(5, n, N, r, std=0.2, dtype=dt)
    plan = rd.adapter_plan(ids.cuda(), n)
    u = torch.empty(T, r, device="cuda")

    def calls():
        y = rd.lora_fwd(x, a, b, plan, base=base, u=u)
        return [y, u.clone(), *rd.lora_bwd(g, x, a, b, plan, u)]

    clean = calls()
    assert all(bool(torch.isfinite(t).all()) for t in clean)
    bad = int((ids == 2).nonzero()[1])
    none = int((ids < 0).nonzero()[0])
    others = torch.ones(T, dtype=torch.bool)
    others[bad] = False
    for value in (float("inf"), float("nan")):
        for t in (x, g):
            keep = t.clone()
            t[bad, 5] = value
            t[none, 7] = value                                # a token without an adapter: never read
            y, uu, gx, ga, gb = calls()
            t.copy_(keep)
            for got, want in ((y, clean[0]), (uu, clean[1]), (gx, clean[2])):
                assert torch.equal(got[others.cuda()], want[others.cuda()])
            for got, want in ((ga, clean[3]), (gb, clean[4])):
                rest = [k for k in range(n) if k != 2]
                assert torch.equal(got[rest], want[rest])
            if t is x:
                assert not bool(torch.isfinite(y[bad]).any()) and not bool(torch.isfinite(uu[bad]).any())
                assert not bool(torch.isfinite(gb[2]).any())                # through u
                assert not bool(torch.isfinite(ga[2, :, 5]).any())          # v x, column 5 alone
                assert torch.equal(ga[2, :, :5], clean[3][2, :, :5]) and torch.equal(gx, clean[2])
            else:
                assert not bool(torch.isfinite(gx[bad]).any())
                assert not bool(torch.isfinite(ga[2]).any())                # through v
                assert not bool(torch.isfinite(gb[2, 5]).any())             # g u, row 5 alone
                assert torch.equal(gb[2, :5], clean[4][2, :5]) and torch.equal(y, clean[0])
    keep = base.clone()
    base[none, 7] = base[bad, 9] = float("nan")
    y, uu, gx, ga, gb = calls()
    base.copy_(keep)
    wrong = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    wrong[none, 7] = wrong[bad, 9] = True
    assert bool(y[wrong].isnan().all()) and torch.equal(y[~wrong], clean[0][~wrong])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,p", [(40, 512, 64), (600, 4096, 512), (90, 1024, 1024), (300, 4096, 128), (50, 640, 128)])
def test_a_circulant_value_that_is_not_finite_stays_where_it_belongs(rd, T, D, p, dtype):
    """The same for the block-circulant adapters."""
    n, q, dt = 4, D // p, DT[dtype]
    ids = make_ids("runs", T, n, seed=3)
    ids[::7], ids[1], ids[2] = -1, 2, 1
    x, g, base = randn(1, T, D, dtype=dt), randn(2, T, D, dtype=dt), randn(3, T, D, dtype=dt)
    c_hat = rd.rdfft_fwd(randn(4, n, q, q, p, std=D ** -0.5), p)
    plan = rd.adapter_plan(ids.cuda(), n)

    def calls():
        return [rd.circ_fwd_many(x, c_hat, p, plan, base=base), *rd.circ_bwd_many(g, x, c_hat, p, plan)]

    clean = calls()
    others = torch.ones(T, dtype=torch.bool)
    others[1] = False
    others = others.cuda()
    for value in (float("inf"), float("nan")):
        for t in (x, g):
            keep = t.clone()
            t[1, 5] = t[0, 3] = value                         # token 0 has no adapter
            y, gx, gc = calls()
            t.copy_(keep)
            assert torch.equal(y[others], clean[0][others]) and torch.equal(gx[others], clean[1][others])
            rest = [k for k in range(n) if k != 2]
            assert torch.equal(gc[rest], clean[2][rest]) and bool((~torch.isfinite(gc[2])).any())
            assert bool((~torch.isfinite(y[1] if t is x else gx[1])).any())
            assert torch.equal(gx if t is x else y, clean[1] if t is x else clean[0])


# ------------------------------------------------------------------- offsets past 32 bits
# The tokens past element 2^31 are 16 times as large as the others, so that the sums are theirs.
@pytest.mark.parametrize("wide", ["x", "g"])
def test_lora_weight_gradients_past_32_bits(rd, wide):
    T, W, r, n = 66000, 32768, 8, 2
    first = 2 ** 31 // W
    assert first < T
    gen = torch.Generator(device="cuda").manual_seed(1)
    big = torch.empty(T, W, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    big[first:] *= 16
    small = randn(2, T, 8, dtype=torch.bfloat16)
    K, N = (W, 8) if wide == "x" else (8, W)
    x, g = (big, small) if wide == "x" else (small, big)
    a, b = randn(3, n, r, K, std=K ** -0.5, dtype=x.dtype), randn(4, n, N, r, std=0.3, dtype=x.dtype)
    ids = ((torch.arange(T) % 3 - 1).int()).cuda()
    plan = rd.adapter_plan(ids, n)
    u = torch.empty(T, r, device="cuda")
    rd.lora_fwd(x, a, b, plan, u=u)
    _, ga, gb = rd.lora_bwd(g, x, a, b, plan, u, need_grad_x=False)
    from many_util import assert_within, sum_bound
    for k in range(n):
        rows = (ids == k).nonzero().flatten()
        gd = torch.cat([t.double() @ b[k].double() for t in g[rows].split(2048)])        # v
        gm = torch.cat([t.double().abs() @ b[k].double().abs() for t in g[rows].split(2048)])
        ud = u[rows].double()
        for at in (0, W // 2 + 24, W - 64):
            cols = slice(at, at + 64)
            xs, gs = x[rows, cols if wide == "x" else slice(None)], g[rows, cols if wide == "g" else slice(None)]
            ref, mag = gd.t() @ xs.double(), gm.t() @ xs.double().abs()
            got = ga[k][:, cols] if wide == "x" else ga[k]
            bound = sum_bound(N, 1, x.dtype) + sum_bound(3 * rows.numel(), 1, x.dtype)
            assert_within(got, ref.cpu(), (bound * mag).cpu(), "grad_a")
            ref, mag = gs.double().t() @ ud, gs.double().abs().t() @ ud.abs()
            got = gb[k][cols] if wide == "g" else gb[k]
            assert_within(got, ref.cpu(), (sum_bound(3 * rows.numel(), 1, x.dtype) * mag).cpu(), "grad_b")


@pytest.mark.parametrize("alone", [False, True])
def test_circulant_weight_gradients_past_32_bits(rd, alone):
    T, D, p, n = 530000, 4096, 512, 2
    first = 2 ** 31 // D
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    x[first:] *= 16
    g[first:] *= 16
    ids = ((torch.arange(T) % 3 - 1).int()).cuda()
    plan = rd.adapter_plan(ids, n)
    c_hat = rd.rdfft_fwd(randn(2, n, 8, 8, p, std=D ** -0.5), p)
    gc = rd.circ_bwd_many(g, x, c_hat, p, plan, need_grad_x=not alone)[1]
    for k in range(n):
        rows = (ids == k).nonzero().flatten()
        for i, j in ((0, 0), (3, 6), (7, 7)):
            s = torch.zeros(p // 2 + 1, dtype=torch.complex128, device="cuda")
            mag = 0.0
            for part in rows.split(1 << 14):
                gi, xj = (t[part, c * p:(c + 1) * p].double() for t, c in ((g, i), (x, j)))
                s += (torch.fft.rfft(gi) * torch.fft.rfft(xj).conj()).sum(0)
                mag += float((gi.norm(dim=1) * xj.norm(dim=1)).sum())       # a term of a lag is at most this
            ref = torch.fft.irfft(s, n=p)
            # fp32 sums over a slice's tokens (148 slices), then over the slices, with the layer's own
            # error (1e-5 of the largest value) for the transforms
            bound = 4 * (T / 148 + 148) ** 0.5 * 2.0 ** -24 * mag + 1e-5 * float(ref.abs().max())
            assert float((gc[k, i, j].double() - ref).abs().max()) <= bound
            assert float(ref.norm()) / p ** 0.5 > 10 * bound                 # a lost part would show

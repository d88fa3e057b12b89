"""Adapters of many requests at once: the operators, their cases and their definitions.

A batch mixes tokens of requests that each use one of n adapters, or none, beside a shared
projection. The operators are
  plan      grouping the batch's tokens by adapter (once per step, kept for all its layers)
  lora_fwd  low-rank adapters:  y_t = base_t + s_a B_a (A_a x_t), a = the adapter of token t
  lora_bwd  its gradients: grad_x, grad_A, grad_B
  circ_fwd  block-circulant adapters: y_t = base_t + W(c_a) x_t, c_a given as its packed spectrum
  circ_bwd  its gradients: grad_x, grad_c
  clip      the global norm of many gradients, and the gradients clipped by it into a flat buffer

`run` computes them in plain torch operations, or, where `own` is true, through the calls of
block_circulant_layers_b200. `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ITEM = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's batch of one token per request: latency
        dict(name="plan_decode", op="plan", T=48, n=32, req=1),
        # a long mixed batch: prompts of many requests
        dict(name="plan_prompts", op="plan", T=32768, n=200, req=256),
        # decode: one token per request, 16 adapters loaded, rank 16, D = 4096
        dict(name="lora_fwd_decode", op="lora_fwd", T=32, K=4096, N=4096, r=16, n=16, req=1, dtype="bf16"),
        # a step of 4096 tokens (8 x 512) over 8 adapters beside the query projection
        dict(name="lora_fwd_step", op="lora_fwd", T=4096, K=4096, N=4096, r=16, n=8, req=512, dtype="bf16"),
        # a training step of the same adapters
        dict(name="lora_bwd_step", op="lora_bwd", T=4096, K=4096, N=4096, r=16, n=8, req=512, dtype="bf16"),
        # full-precision training of a narrow layer, ragged requests, odd feature sizes
        dict(name="lora_bwd_ragged_f32", op="lora_bwd", T=777, K=1032, N=2056, r=24, n=5, req=100, dtype="f32"),
        # decode with block-circulant adapters of the D = 4096, p = 128 layer
        dict(name="circ_fwd_decode", op="circ_fwd", T=16, D=4096, p=128, n=16, req=1, dtype="bf16"),
        # the 4096-token step with the D = 4096, p = 512 adapters
        dict(name="circ_fwd_step", op="circ_fwd", T=4096, D=4096, p=512, n=8, req=512, dtype="bf16"),
        dict(name="circ_bwd_step", op="circ_bwd", T=4096, D=4096, p=512, n=8, req=512, dtype="bf16"),
        # full-precision training of the D = p = 1024 layer on a ragged batch
        dict(name="circ_bwd_ragged_f32", op="circ_bwd", T=257, D=1024, p=1024, n=3, req=40, dtype="f32"),
        # the gradients of the 64 block-circulant adapters of a step (D = 4096, p = 512)
        dict(name="clip_adapters", op="clip", count=64, numel=32768, jitter=0, dtype="f32"),
        # the gradients of a whole model: many tensors of odd sizes
        dict(name="clip_model", op="clip", count=291, numel=1 << 20, jitter=1, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "lora_fwd", "lora_fwd", "lora_bwd", "circ_fwd", "circ_fwd", "circ_bwd", "clip"])
    if op == "plan":
        return dict(op=op, T=_log(rng, 1, 32768), n=_log(rng, 1, 512), req=_log(rng, 1, 512))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        return dict(op=op, count=_log(rng, 1, 291), numel=_log(rng, 100, 1 << 20), jitter=1, dtype=dtype)
    T = _log(rng, 1, 4096) if dtype == "bf16" else _log(rng, 1, 1500)
    req = 1 if T <= 64 else _log(rng, 8, 512)
    n = _log(rng, 1, 32)
    if op.startswith("lora"):
        return dict(op=op, T=T, K=8 * _log(rng, 16, 512), N=8 * _log(rng, 16, 512), r=rng.choice([8, 16, 24, 32, 64]),
                    n=n, req=req, dtype=dtype)
    p = rng.choice([64, 128, 256, 512, 1024, 2048])
    q = rng.choice([d for d in (1, 2, 4, 5, 8, 16, 32) if 256 <= d * p <= 4096])
    return dict(op=op, T=T, D=q * p, p=p, n=min(n, 12), req=req, dtype=dtype)


def _numels(case):
    """Elements of each gradient: `numel`, or with jitter anything from half of it to all of it."""
    if not case["jitter"]:
        return [case["numel"]] * case["count"]
    sizes = random.Random(case["count"] * 7919 + case["numel"])
    return [sizes.randint(max(1, case["numel"] // 2), case["numel"]) for _ in range(case["count"])]


def work(case):
    op = case["op"]
    if op == "plan":
        return {"bytes": 4 * (2 * case["T"] + case["n"] + 2), "flops": 0}
    if op == "clip":
        total = sum(_numels(case))
        return {"bytes": 2 * total * ITEM[case["dtype"]], "flops": 3 * total}
    es, T, n = ITEM[case["dtype"]], case["T"], case["n"]
    na = min(n, max(1, T // case["req"]))          # adapters that tokens can use
    if op.startswith("lora"):
        K, N, r = case["K"], case["N"], case["r"]
        w = r * (K + N)
        if op == "lora_fwd":                       # x, base, y; each adapter's A and B
            return {"bytes": es * (T * (K + 2 * N) + na * w) + 4 * T, "flops": 2 * T * w}
        return {"bytes": es * (T * (2 * K + N) + na * w) + 4 * (n * w + T * r + T), "flops": 4 * T * w}
    D, p = case["D"], case["p"]
    q = D // p
    fft = 2.5 * D * math.log2(p)
    c = 4 * D * q                                  # bytes of one c_hat
    if op == "circ_fwd":
        return {"bytes": es * 3 * T * D + na * c + 4 * T, "flops": int(T * (2 * fft + 4 * q * D))}
    return {"bytes": es * 3 * T * D + (na + n) * c + 4 * T, "flops": int(T * (3 * fft + 8 * q * D))}


# ------------------------------------------------------------------------------ inputs
def _ids(gen, T, n, req):
    """Adapter of each token: requests of random lengths (mean `req`), each with one adapter
    of n or, for one request in ten, none (-1)."""
    if req == 1:
        ids = torch.randint(0, n, (T,), generator=gen)
        return torch.where(torch.rand(T, generator=gen) < 0.1, torch.full_like(ids, -1), ids)
    ids = torch.empty(T, dtype=torch.int64)
    at = 0
    while at < T:
        ln = int(torch.randint(max(1, req // 2), req + req // 2 + 1, (1,), generator=gen))
        a = int(torch.randint(0, n, (1,), generator=gen))
        if float(torch.rand(1, generator=gen)) < 0.1:
            a = -1
        ids[at:at + ln] = a
        at += ln
    return ids


def _packed_dft(p, device):
    """F with (row @ F) = packed spectrum of a real row, 32 bits from 64-bit angles: slots 0 and
    p/2 real, Re Y_k at k, Im Y_k at p - k."""
    k = torch.arange(p, dtype=torch.int64, device=device)
    ang = (torch.outer(k, k) % p).double() * (2 * math.pi / p)
    f = torch.cos(ang)                             # [n, k], right for k <= p/2
    f[:, p // 2 + 1:] = -torch.sin(ang[:, 1:p // 2].flip(1))
    return f


def _tensors(case, gen, dev):
    return [(torch.randn(m, generator=gen, device=dev) * 0.02).to(DTYPES[case["dtype"]]) for m in _numels(case)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "clip":
        st["grads"] = _tensors(case, gen, dev)
        st["max_norm"] = 1.0
        # the step's flat gradient buffer, each tensor's part starting on 16 bytes
        step = 16 // ITEM[case["dtype"]]
        st["at"] = [0]
        for t in st["grads"]:
            st["at"].append(st["at"][-1] + (t.numel() + step - 1) // step * step)
        st["flat"] = torch.zeros(st["at"][-1], dtype=DTYPES[case["dtype"]], device=dev)
        st["out"] = [st["flat"][i:i + t.numel()] for i, t in zip(st["at"], st["grads"])]
        return st

    T, n = case["T"], case["n"]
    ids = _ids(torch.Generator().manual_seed(seed), T, n, case["req"])
    st["ids"] = ids.to(torch.int32).to(dev)
    if case["op"] == "plan":
        return st
    # the plan of the batch, kept for every layer of a step
    if own:
        import block_circulant_layers_b200 as rd
        st["plan"] = rd.adapter_plan(st["ids"], n)
    st["groups"] = [(a, torch.nonzero(ids == a).flatten().to(dev)) for a in sorted(set(ids.tolist())) if a >= 0]

    dt = DTYPES[case["dtype"]]

    def randn(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    if case["op"].startswith("lora"):
        K, N, r = case["K"], case["N"], case["r"]
        st["x"] = randn(T, K)
        st["a"] = randn(n, r, K, std=K ** -0.5)
        st["b"] = randn(n, N, r, std=r ** -0.5)
        st["scale"] = 0.25 + 0.5 * torch.rand(n, generator=gen, device=dev)
        if case["op"] == "lora_fwd":
            st["base"] = randn(T, N)
        else:
            st["g"] = randn(T, N)
            st["u"] = torch.zeros(T, r, device=dev)        # A_a x_t, kept by the forward pass
            for a, idx in st["groups"]:
                st["u"][idx] = st["x"][idx].float() @ st["a"][a].float().t()
        return st

    D, p = case["D"], case["p"]
    q = D // p
    st["x"] = randn(T, D)
    st["f"] = _packed_dft(p, dev)
    c = torch.randn(n, q, q, p, generator=gen, device=dev) * D ** -0.5
    st["c_hat"] = (c.double() @ st["f"]).float()            # kept while the adapters do not change
    # rows of the inverse: (spectrum @ fi) = the real row
    wgt = torch.full((p, 1), 2.0 / p, dtype=torch.float64, device=dev)
    wgt[0] = wgt[p // 2] = 1.0 / p
    st["fi"] = (st["f"].t() * wgt).float()
    st["f"] = st["f"].float()
    if case["op"] == "circ_fwd":
        st["base"] = randn(T, D)
    else:
        st["g"] = randn(T, D)
    return st


# ------------------------------------------------------------------------- plain forms
def _bins(z, p):
    """Complex bins 0..p/2 (re, im) of packed rows."""
    h = p // 2
    im = torch.zeros_like(z[..., :h + 1])
    im[..., 1:h] = z[..., h + 1:].flip(-1)
    return z[..., :h + 1], im


def _pack(re, im, p):
    return torch.cat([re, im[..., 1:p // 2].flip(-1)], dim=-1)


def _plain_plan(st):
    n = st["case"]["n"]
    ids = st["ids"].long()
    key = torch.where((ids < 0) | (ids >= n), torch.full_like(ids, n), ids)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(n + 1, device=key.device)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=key.device), counts.cumsum(0)])
    return order.int(), offsets.int()


def _plain_lora_fwd(st):
    y = st["base"].float().clone()
    for a, idx in st["groups"]:
        u = st["x"][idx].float() @ st["a"][a].float().t()
        y[idx] += st["scale"][a] * (u @ st["b"][a].float().t())
    return y.to(st["x"].dtype)


def _plain_lora_bwd(st):
    ga = torch.zeros(st["a"].shape, device=st["a"].device)
    gb = torch.zeros(st["b"].shape, device=st["b"].device)
    gx = torch.zeros_like(st["x"])
    for a, idx in st["groups"]:
        g, x = st["g"][idx].float(), st["x"][idx].float()
        v = st["scale"][a] * (g @ st["b"][a].float())
        gx[idx] = (v @ st["a"][a].float()).to(gx.dtype)
        ga[a] = v.t() @ x
        gb[a] = st["scale"][a] * (g.t() @ st["u"][idx])
    return gx, ga, gb


def _plain_circ_fwd(st):
    p, T = st["case"]["p"], st["case"]["T"]
    q = st["case"]["D"] // p
    y = st["base"].float().clone()
    for a, idx in st["groups"]:
        xr, xi = _bins(st["x"][idx].float().view(-1, q, p) @ st["f"], p)
        cr, ci = _bins(st["c_hat"][a], p)
        yr = torch.einsum("tjk,ijk->tik", xr, cr) - torch.einsum("tjk,ijk->tik", xi, ci)
        yi = torch.einsum("tjk,ijk->tik", xi, cr) + torch.einsum("tjk,ijk->tik", xr, ci)
        y[idx] += (_pack(yr, yi, p) @ st["fi"]).reshape(-1, q * p)
    return y.to(st["x"].dtype)


def _plain_circ_bwd(st):
    p = st["case"]["p"]
    q = st["case"]["D"] // p
    gx = torch.zeros_like(st["x"])
    gc = torch.zeros_like(st["c_hat"])
    for a, idx in st["groups"]:
        xr, xi = _bins(st["x"][idx].float().view(-1, q, p) @ st["f"], p)
        gr, gi = _bins(st["g"][idx].float().view(-1, q, p) @ st["f"], p)
        cr, ci = _bins(st["c_hat"][a], p)
        zr = torch.einsum("tik,ijk->tjk", gr, cr) + torch.einsum("tik,ijk->tjk", gi, ci)
        zi = torch.einsum("tik,ijk->tjk", gi, cr) - torch.einsum("tik,ijk->tjk", gr, ci)
        gx[idx] = (_pack(zr, zi, p) @ st["fi"]).reshape(-1, q * p).to(gx.dtype)
        sr = torch.einsum("tik,tjk->ijk", gr, xr) + torch.einsum("tik,tjk->ijk", gi, xi)
        si = torch.einsum("tik,tjk->ijk", gi, xr) - torch.einsum("tik,tjk->ijk", gr, xi)
        gc[a] = _pack(sr, si, p) @ st["fi"]
    return gx, gc


def _plain_clip(st):
    total = torch.zeros((), dtype=torch.float64, device=st["grads"][0].device)
    for t in st["grads"]:
        total += t.float().square().sum(dtype=torch.float64)
    norm = total.sqrt().float()
    coef = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
    for t, o in zip(st["grads"], st["out"]):
        o.copy_(t.float() * coef)
    return norm, st["flat"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "lora_fwd": _plain_lora_fwd, "lora_bwd": _plain_lora_bwd,
                "circ_fwd": _plain_circ_fwd, "circ_bwd": _plain_circ_bwd, "clip": _plain_clip}[op](state)
    import block_circulant_layers_b200 as rd
    if op == "plan":
        plan = rd.adapter_plan(state["ids"], state["case"]["n"])
        return plan.order, plan.offsets
    if op == "lora_fwd":
        return rd.lora_fwd(state["x"], state["a"], state["b"], state["plan"], scale=state["scale"],
                           base=state["base"])
    if op == "lora_bwd":
        return rd.lora_bwd(state["g"], state["x"], state["a"], state["b"], state["plan"], state["u"],
                           scale=state["scale"])
    if op == "circ_fwd":
        return rd.circ_fwd_many(state["x"], state["c_hat"], state["case"]["p"], state["plan"], base=state["base"])
    if op == "circ_bwd":
        return rd.circ_bwd_many(state["g"], state["x"], state["c_hat"], state["case"]["p"], state["plan"])
    norm = rd.clip_grad_norm(state["grads"], state["max_norm"], out=state["out"])
    return norm, state["flat"]


# ------------------------------------------------------------------- definition, 64 bits
def _dense_circulant(c_hat, p):
    """The D x D matrix of one adapter: block (i, j) has first column c_ij."""
    q = c_hat.shape[0]
    z = c_hat.double()
    re, h = z[..., :p // 2 + 1], p // 2
    im = torch.zeros_like(re)
    for k in range(1, h):
        im[..., k] = z[..., p - k]
    c = torch.fft.irfft(torch.complex(re, im), n=p)
    m = torch.arange(p, device=c.device)
    w = c[:, :, (m[:, None] - m[None, :]) % p]               # [i, j, row, column]
    return w.permute(0, 2, 1, 3).reshape(q * p, q * p)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        n = case["n"]
        ids = st["ids"].tolist()
        order, offsets = [], [0]
        buckets = [[] for _ in range(n + 1)]
        for t, a in enumerate(ids):
            buckets[a if 0 <= a < n else n].append(t)
        for bucket in buckets:
            order += bucket
            offsets.append(len(order))
        return torch.tensor(order, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32)
    if op == "clip":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in st["grads"]]))
        coef = min(1.0, st["max_norm"] / (float(norm) + 1e-6))
        flat = torch.zeros_like(st["flat"], dtype=torch.float64)
        for t, i in zip(st["grads"], st["at"]):
            flat[i:i + t.numel()] = t.double() * coef
        return norm, flat
    ids = st["ids"].long()
    x = st["x"].double()
    y = st["base"].double() if "base" in st else torch.zeros_like(x)
    gx = torch.zeros_like(x)
    ws = {"lora_fwd": ("a", "b"), "lora_bwd": ("a", "b"), "circ_fwd": (), "circ_bwd": ("c_hat",)}[op]
    gw = [torch.zeros_like(st[k], dtype=torch.float64) for k in ws]
    for a in range(case["n"]):
        rows = (ids == a).nonzero().flatten()
        if rows.numel() == 0:
            continue
        if op.startswith("lora"):
            s, wa, wb = float(st["scale"][a]), st["a"][a].double(), st["b"][a].double()
            if op == "lora_fwd":
                y[rows] += torch.einsum("tk,rk,nr->tn", x[rows], wa, s * wb)
                continue
            g = st["g"][rows].double()
            gx[rows] = (g @ wb) @ wa * s
            gw[0][a] = s * torch.einsum("nr,nk->rk", wb, g.t() @ x[rows])
            gw[1][a] = s * g.t() @ st["u"][rows].double()
            continue
        p = case["p"]
        q = case["D"] // p
        w = _dense_circulant(st["c_hat"][a], p)
        if op == "circ_fwd":
            y[rows] += x[rows] @ w.t()
            continue
        g = st["g"][rows].double()
        gx[rows] = g @ w
        dw = (g.t() @ x[rows]).view(q, p, q, p)
        col = torch.arange(p, device=dw.device)
        for m in range(p):                                   # the m-th wrapped diagonal of each block
            gw[0][a, :, :, m] = dw[:, (col + m) % p, :, col].sum(0)
    if op.endswith("fwd"):
        return y
    return (gx, *gw)

"""Adapters of many requests without a GPU: the launch rules and the plan's sizes (through the
host test library), and the C ABI's refusals, which come before any CUDA call."""
import ctypes
import os
import random

import pytest

from conftest import ROOT
from test_abi_host import A, BF16, EALIGN, EDTYPE, EINVAL, ENULL, EOVERLAP, ESPACE, F32, OK

PKG = os.path.join(ROOT, "block_circulant_layers_b200")
i64, i32, vp, f32, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
EPLAN = 9
NAN = float("nan")


@pytest.fixture(scope="module")
def emu():
    from block_circulant_layers_b200 import build
    build.build_emulator()
    L = ctypes.CDLL(os.path.join(PKG, "librdfft_hostemu.so"))
    L.rdfft_plan_tile_cap.argtypes, L.rdfft_plan_tile_cap.restype = [i64, i32, i32], i64
    L.rdfft_lora_list.argtypes = [i64, i32]
    L.rdfft_lora_cluster.argtypes = [i64, i32, i32, i32, i32]
    L.rdfft_lora_token_split.argtypes = [i64, i32, i32, i32, i32]
    L.rdfft_circ_many_tokens.argtypes = [i64, i32, i32, i32, i32, i32]
    L.rdfft_circ_many_slices.argtypes = [i64, i32, i32, i32, i32]
    return L


@pytest.fixture(scope="module")
def lib():
    from block_circulant_layers_b200 import build
    build.build_lib()
    L = ctypes.CDLL(os.path.join(PKG, "librdfft.so"))
    L.adapter_plan_size.argtypes = [i64, i32, ctypes.POINTER(i64)]
    L.adapter_plan.argtypes = [vp, i64, i32, vp, vp]
    L.lora_fwd.argtypes = [vp] * 8 + [i64] + [i32] * 5 + [vp]
    L.lora_bwd.argtypes = [vp] * 11 + [i64] + [i32] * 5 + [vp]
    L.circ_fwd_many.argtypes = [vp] * 5 + [i64] + [i32] * 4 + [vp]
    L.circ_bwd_many_workspace_size.argtypes = [i64] + [i32] * 5 + [ctypes.POINTER(sz)]
    L.circ_bwd_many.argtypes = [vp] * 6 + [i64] + [i32] * 4 + [vp, sz, vp]
    L.grad_norm_workspace_size.argtypes = [i32, ctypes.POINTER(sz)]
    L.grad_norm.argtypes = [vp, vp, vp, i32, vp, vp, sz, vp]
    L.clip_grad_norm.argtypes = [vp, vp, vp, vp, i32, f32, vp, vp, sz, vp]
    L.rdfft_strerror.argtypes, L.rdfft_strerror.restype = [i32], ctypes.c_char_p
    return L


# ------------------------------------------------------------------------------- rules
def test_tile_lists_hold_every_grouping(emu):
    rng = random.Random(0)
    for _ in range(2000):
        T, n = rng.randint(0, 300), rng.choice([1, 2, 5, 40, 1024])
        used = rng.sample(range(n + 1), min(n + 1, rng.randint(1, 6)))
        counts = [0] * len(used)
        for _ in range(T):
            counts[rng.randrange(len(used))] += 1
        for tile in (4, 16, 64):
            assert sum(-(-c // tile) for c in counts) <= emu.rdfft_plan_tile_cap(T, n, tile) <= T


def test_rules_stay_in_their_ranges(emu):
    rng = random.Random(1)
    for _ in range(3000):
        T, n = int(2 ** rng.uniform(0, 30)), rng.randint(1, 1024)
        K, N = 8 * rng.randint(1, 8192), 8 * rng.randint(1, 8192)
        lst = emu.rdfft_lora_list(T, n)
        assert lst in (1, 2)
        tiles = emu.rdfft_plan_tile_cap(T, n, 4 ** (lst + 1))
        for is_f32 in (0, 1):
            c = emu.rdfft_lora_cluster(tiles, lst, is_f32, K, N)
            assert c in (1, 2, 4, 8) and tiles * c < 2 ** 31
        for per_sm in (1, 2, 3):
            c = emu.rdfft_lora_token_split(T, n, (K + 63) // 64 + (N + 63) // 64, 64, per_sm)
            assert 1 <= c <= 8
        q = rng.choice([1, 2, 3, 8, 32, 128])
        assert emu.rdfft_circ_many_tokens(T, n, q, 8, 148, 4) in (1, 2, 4)
        s = emu.rdfft_circ_many_slices(T, n, rng.choice([1, 2, 4]), rng.choice([1, 2, 4]), 148)
        assert 1 <= s <= 148


def test_groups_of_one_token_take_one_per_cta(emu):
    assert emu.rdfft_circ_many_tokens(64, 64, 8, 8, 148, 4) == 1
    assert emu.rdfft_circ_many_tokens(4096, 8, 8, 8, 148, 4) == 4
    assert emu.rdfft_lora_list(4096, 8) == 2 and emu.rdfft_lora_list(4096, 1000) == 1 and emu.rdfft_lora_list(64, 1) == 1


# ---------------------------------------------------------------------------- refusals
# aligned fake device addresses far apart; a call here must fail before any of them is used
B, C, D, E, F, G, H = (A + k * (1 << 36) for k in range(1, 8))


def words(lib, T, n):
    w = i64(-1)
    return lib.adapter_plan_size(T, n, ctypes.byref(w)), w.value


def test_plan_arguments(lib):
    assert words(lib, 0, 1)[0] == OK and words(lib, 100, 1024)[0] == OK
    assert words(lib, -1, 1) == (EINVAL, 0) and words(lib, 10, 0) == (EINVAL, 0) and words(lib, 10, 1025) == (EINVAL, 0)
    assert words(lib, (1 << 30) + 1, 1)[0] == EINVAL
    assert lib.adapter_plan_size(1, 1, None) == ENULL
    rc, w = words(lib, 100, 7)
    assert rc == OK and w % 4 == 0 and w >= 16 + 9 + 200
    f = lib.adapter_plan
    assert f(A, -1, 4, B, None) == EINVAL and f(A, 8, 0, B, None) == EINVAL
    assert f(None, 8, 4, B, None) == ENULL and f(A, 8, 4, None, None) == ENULL
    assert f(A + 2, 8, 4, B, None) == EALIGN and f(A, 8, 4, B + 4, None) == EALIGN
    assert f(A, 8, 4, A, None) == EOVERLAP


def test_lora_fwd_arguments(lib):
    T, K, N, r, n = 32, 64, 128, 16, 4

    def f(x=A, a=B, b=C, scale=D, base=E, y=F, u=G, plan=H, T=T, K=K, N=N, r=r, n=n, dt=BF16):
        return lib.lora_fwd(x, a, b, scale, base, y, u, plan, T, K, N, r, n, dt, None)

    assert f(T=0) == OK and f(T=0, x=None, y=None) == OK
    assert f(dt=2) == EDTYPE
    for bad in (dict(K=60), dict(K=0), dict(K=65544), dict(N=4), dict(r=0), dict(r=12), dict(r=136), dict(n=0),
                dict(n=1025), dict(T=-1), dict(T=(1 << 30) + 1)):
        assert f(**bad) == EINVAL, bad
    for name in ("x", "a", "b", "y", "plan"):
        assert f(**{name: None}) == ENULL, name
    for name, at in (("x", A), ("a", B), ("b", C), ("base", E), ("y", F), ("u", G), ("plan", H)):
        assert f(**{name: at + 8}) == EALIGN, name
    assert f(scale=D + 2) == EALIGN
    size_y = T * N * 2
    for other in ("x", "a", "b", "scale", "u", "plan"):
        assert f(**{other: F + size_y - 16}) == EOVERLAP, other
    assert f(base=F + 16) == EOVERLAP                       # base may be y, not a part of it
    for other in ("x", "a", "b", "base", "scale", "plan"):
        assert f(**{other: G}) == EOVERLAP, other


def test_lora_bwd_arguments(lib):
    T, K, N, r, n = 32, 64, 128, 16, 4
    names = ("g", "x", "a", "b", "scale", "u", "v", "gx", "ga", "gb", "plan")
    at = dict(zip(names, (A + k * (1 << 36) for k in range(11))))

    def f(T=T, K=K, N=N, r=r, n=n, dt=F32, **over):
        v = [over.get(k, at[k]) for k in names]
        return lib.lora_bwd(*v, T, K, N, r, n, dt, None)

    assert f(gx=None, ga=None, gb=None) == OK
    assert f(dt=9) == EDTYPE and f(r=4) == EINVAL and f(K=12) == EINVAL and f(n=2000) == EINVAL
    for name in ("g", "b", "a", "x", "v", "u", "plan"):
        assert f(**{name: None}) == ENULL, name
    assert f(ga=None, gb=None, x=None, u=None, v=None, a=None) == ENULL     # grad_x needs a
    assert f(T=0, ga=at["ga"] + 4) == EALIGN and f(T=0, ga=at["gb"]) == EOVERLAP
    for name in names:
        if name != "scale":
            assert f(**{name: at[name] + 4}) == EALIGN, name
    for out in ("gx", "ga", "gb", "v"):
        for other in names:
            if other != out:
                assert f(**{other: at[out]}) == EOVERLAP, (out, other)


def test_circ_many_arguments(lib):
    T, Dm, p, n = 16, 1024, 128, 3

    def f(x=A, c=B, base=C, y=D, plan=E, T=T, Dm=Dm, p=p, n=n, dt=BF16):
        return lib.circ_fwd_many(x, c, base, y, plan, T, Dm, p, n, dt, None)

    assert f(T=0) == OK and f(dt=3) == EDTYPE
    for bad in (dict(Dm=1000), dict(p=32), dict(p=100), dict(Dm=16384), dict(n=0), dict(n=1025), dict(T=-1)):
        assert f(**bad) == EINVAL, bad
    for name in ("x", "c", "y", "plan"):
        assert f(**{name: None}) == ENULL
        assert f(**{name: A + 4}) == EALIGN
    assert f(x=D) == EOVERLAP and f(c=D + 16) == EOVERLAP and f(plan=D) == EOVERLAP and f(base=D + 16) == EOVERLAP

    size = sz(7)
    w = lib.circ_bwd_many_workspace_size
    assert w(T, Dm, p, n, BF16, 1, None) == ENULL
    assert w(T, 1000, p, n, BF16, 1, ctypes.byref(size)) == EINVAL and size.value == 0
    assert w(0, Dm, p, n, BF16, 1, ctypes.byref(size)) == OK and size.value == 0
    for gx in (0, 1):
        assert w(T, Dm, p, n, BF16, gx, ctypes.byref(size)) == OK
        one = 8 * 8 * 128 * 4
        assert size.value % one == 0 and n < size.value // one <= 148 + n
    need = size.value

    def b(g=A, x=B, c=C, gx=D, gc=E, plan=F, ws=G, ws_bytes=need, T=T, Dm=Dm, p=p, n=n, dt=BF16):
        return lib.circ_bwd_many(g, x, c, gx, gc, plan, T, Dm, p, n, dt, ws, ws_bytes, None)

    assert b(gx=None, gc=None) == OK and b(dt=4) == EDTYPE and b(Dm=1000) == EINVAL and b(n=0) == EINVAL
    for name in ("g", "plan", "c", "x", "ws"):
        assert b(**{name: None}) == ENULL, name
    assert b(ws_bytes=need - 16) == ESPACE and b(gc=E + 4) == EALIGN and b(ws=G + 8) == EALIGN
    assert b(T=0, gx=None, gc=E + 8) == EALIGN
    for out in (D, E, G):
        assert b(g=out) == EOVERLAP and b(x=out) == EOVERLAP and b(c=out) == EOVERLAP and b(plan=out) == EOVERLAP
    assert b(gx=E) == EOVERLAP and b(ws=E) == EOVERLAP and b(ws=D) == EOVERLAP


def test_norm_arguments(lib):
    n = sz(3)
    assert lib.grad_norm_workspace_size(4, None) == ENULL
    assert lib.grad_norm_workspace_size(-1, ctypes.byref(n)) == EINVAL and n.value == 0
    assert lib.grad_norm_workspace_size(4097, ctypes.byref(n)) == EINVAL
    assert lib.grad_norm_workspace_size(0, ctypes.byref(n)) == OK and n.value == 0
    assert lib.grad_norm_workspace_size(4096, ctypes.byref(n)) == OK and n.value % 8 == 0

    def lists(ptrs, numels, codes):
        m = len(ptrs)
        return (vp * m)(*ptrs), (i64 * m)(*numels), (i32 * m)(*codes), m

    def call(ptrs=(A, B), outs=None, numels=(100, 7), codes=(F32, BF16), norm=C, ws=D, ws_bytes=1 << 20, max_norm=1.0,
             clip=True):
        p, m, c, k = lists(ptrs, numels, codes)
        if not clip:
            return lib.grad_norm(p, m, c, k, norm, ws, ws_bytes, None)
        o = (vp * k)(*(ptrs if outs is None else outs))
        return lib.clip_grad_norm(p, o, m, c, k, max_norm, norm, ws, ws_bytes, None)

    for clip in (False, True):
        assert call(codes=(F32, 5), clip=clip) == EDTYPE and call(numels=(100, -1), clip=clip) == EINVAL
        assert call(ptrs=(A, None), clip=clip) == ENULL and call(norm=None, clip=clip) == ENULL
        assert call(ws=None, clip=clip) == ENULL and call(ws_bytes=64, clip=clip) == ESPACE
        assert call(ptrs=(A + 2, B), clip=clip) == EALIGN and call(ptrs=(A, B + 1), clip=clip) == EALIGN
        assert call(norm=C + 2, clip=clip) == EALIGN and call(ws=D + 4, clip=clip) == EALIGN
    assert lib.grad_norm(None, None, None, 2, C, D, 1 << 20, None) == ENULL
    assert call(max_norm=-1.0) == EINVAL and call(max_norm=NAN) == EINVAL
    assert call(outs=(E, None)) == ENULL and call(outs=(E + 2, F)) == EALIGN
    assert call(ptrs=(A, A), codes=(F32, F32), numels=(100, 100)) == EOVERLAP       # the same tensor twice
    assert call(outs=(E, E + 396)) == EOVERLAP                                        # outputs overlap
    assert call(outs=(A + 4, E)) == EOVERLAP                                          # shifted over its input
    assert call(outs=(E, A)) == EOVERLAP                                              # over another's input
    assert call(norm=A + 40) == EOVERLAP and call(ws=B - 64) == EOVERLAP


def test_new_code_has_a_message(lib):
    assert b"plan" in lib.rdfft_strerror(EPLAN)

"""Refusals of the residual norm, the rotary positions, the prefix attention and the cache's page operations (nothing is
launched), pins of their oracle, and the rotary frequencies."""
import math
import os

import numpy as np
import pytest

from oracle import kvcache as kc
from oracle import rollout as ro

P = 0x10000        # a 16-byte aligned fake address: validation rejects every call below before any use
BAD = 0x10008
NULL, SHAPE, ALIGN, MODE, VALUE = -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def lib():
    import fp8_precision_rl_amd as jf
    if not os.path.exists(jf.LIB_PATH):
        from fp8_precision_rl_amd import build
        build.build()
    return jf.load_library()


# ------------------------------------------------------------------------------------------------ refusals
def _norm(lib, x=P, res=P, w=P, rows=4, cols=256, eps=1e-5, h=P, q=P, s=P, r=P, y=P):
    return lib.jetfp8_rmsnorm_add_quantize(x, res, w, rows, cols, eps, h, q, s, r, y, None)


def test_norm_refusals(lib):
    for k in ("x", "res", "w", "h", "q", "s"):
        assert _norm(lib, **{k: None}) == NULL, k
    for k in ("x", "res", "w", "h", "q", "s", "r", "y"):
        assert _norm(lib, **{k: BAD}) == ALIGN, k
    for kw in (dict(rows=0), dict(rows=1 << 31), dict(cols=200), dict(cols=8320), dict(cols=0)):
        assert _norm(lib, **kw) == SHAPE, kw
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert _norm(lib, eps=eps) == VALUE


def _back(lib, dy=P, h=P, w=P, r=P, dres=P, rows=4, cols=256, dx=P, dw=P, ws=P, size=1 << 40):
    return lib.jetfp8_rmsnorm_backward(dy, h, w, r, dres, rows, cols, dx, dw, ws, size, None)


def test_norm_backward_refusals(lib):
    for k in ("dy", "h", "w", "r", "dx", "ws"):
        assert _back(lib, **{k: None}) == NULL, k
    for k in ("dy", "h", "w", "r", "dres", "dx", "dw", "ws"):
        assert _back(lib, **{k: BAD}) == ALIGN, k
    for kw in (dict(rows=0), dict(rows=1 << 31), dict(cols=200), dict(cols=8320), dict(size=2 * 256 * 4 - 1)):
        assert _back(lib, **kw) == SHAPE, kw
    f = lib.jetfp8_rmsnorm_backward_workspace
    assert f(4, 256) == 2 * 256 * 4 and f(1, 128) == 512 and f(1 << 20, 8192) == 512 * 8192 * 4
    assert f(0, 128) == SHAPE and f(4, 100) == SHAPE and f(4, 8320) == SHAPE


def _rotary(lib, x=P, ldx=1024, T=4, H=8, D=128, pos=P, f=P, pairs=64, layout=0, amp=1.0, inv=0, dst=2 * P, ldd=1024):
    return lib.jetfp8_rotary(x, ldx, T, H, D, pos, f, pairs, layout, amp, inv, dst, ldd, None)


def test_rotary_refusals(lib):
    for k in ("x", "pos", "f", "dst"):
        assert _rotary(lib, **{k: None}) == NULL, k
        assert _rotary(lib, **{k: BAD}) == ALIGN, k
    for kw in (dict(T=0), dict(T=1 << 24), dict(H=0), dict(H=1 << 20, ldx=1 << 30, ldd=1 << 30), dict(D=120), dict(D=8),
               dict(D=528), dict(pairs=0), dict(pairs=4), dict(pairs=72), dict(ldx=1016), dict(ldd=1020), dict(ldd=0),
               dict(dst=P, ldd=2048)):
        assert _rotary(lib, **kw) == SHAPE, kw
    for layout in (-1, 2):
        assert _rotary(lib, layout=layout) == MODE
    for kw in (dict(amp=0.0), dict(amp=-1.0), dict(amp=math.inf), dict(amp=math.nan), dict(inv=2), dict(inv=-1)):
        assert _rotary(lib, **kw) == VALUE, kw


def test_positions_and_prefix_refusals(lib):
    pos = lambda units=P, n=8, T=8, out=P: lib.jetfp8_kv_positions(units, n, T, out, None)
    pre = lambda units=P, n=8, table=P, R=4, W=8, groups=P, out=P: lib.jetfp8_kv_prefix(units, n, table, R, W, groups, out, None)
    for k in ("units", "out"):
        assert pos(**{k: None}) == NULL and pos(**{k: BAD}) == ALIGN
    for kw in (dict(n=0), dict(T=0), dict(T=(1 << 19) + 1), dict(n=1 << 31)):
        assert pos(**kw) == SHAPE, kw
    for k in ("units", "table", "groups", "out"):
        assert pre(**{k: None}) == NULL and pre(**{k: BAD}) == ALIGN
    for kw in (dict(n=0), dict(R=0), dict(R=4097), dict(W=0), dict(W=1 << 25), dict(R=4096, W=1 << 19)):
        assert pre(**kw) == SHAPE, kw


def _attend(lib, q=P, ldq=512, T=8, units=P, n=8, prefix=P, table=P, R=4, W=64, codes=P, scales=P, blocks=8, recent=P,
            recents=9, max_new=1, max_seq=4000, Hq=4, H=2, D=128, scale=0.1, o=P, oq=None, os=None, ws=P, size=1 << 40):
    return lib.jetfp8_attention_prefix(q, ldq, T, units, n, prefix, table, R, W, codes, scales, blocks, recent, recents,
                                       max_new, max_seq, Hq, H, D, scale, o, oq, os, ws, size, None)


def test_attention_prefix_refusals(lib):
    for k in ("q", "units", "prefix", "table", "codes", "scales", "recent", "o", "ws"):
        assert _attend(lib, **{k: None}) == NULL, k
    for k in ("q", "units", "prefix", "table", "codes", "scales", "recent", "o", "ws"):
        assert _attend(lib, **{k: BAD}) == ALIGN, k
    need = lib.jetfp8_attention_prefix_workspace(8, 1, 4000, 4, 2, 128)
    assert need > 0
    for kw in (dict(D=96), dict(Hq=3), dict(n=0), dict(max_new=0), dict(max_seq=0), dict(recents=7), dict(ldq=500),
               dict(size=need - 1)):
        assert _attend(lib, **kw) == SHAPE, kw
    assert _attend(lib, scale=0.0) == VALUE and _attend(lib, scale=math.inf) == VALUE
    # a workspace of its own: rows that fill waves by themselves are split where blocks may be shared, 256 MB on
    f, g = lib.jetfp8_attention_prefix_workspace, lib.jetfp8_attention_workspace
    assert f(256, 1, 64, 8, 8, 128) == g(256, 1, 64, 8, 8, 128) == 0
    assert f(128, 1, 4096, 32, 8, 128) == g(128, 1, 4096, 32, 8, 128) > 0
    assert f(512, 4, 4033, 64, 8, 128) > g(512, 4, 4033, 64, 8, 128) == 0
    assert f(32, 4, 64, 64, 8, 128) == g(32, 4, 64, 64, 8, 128)
    assert f(1, 1, 64, 3, 2, 128) == SHAPE


def test_fork_refusals(lib):
    fork = lambda state=P, table=P, W=8, R=4, parents=P, ns=2 * P, nt=2 * P: \
        lib.jetfp8_kv_fork(state, table, W, R, parents, ns, nt, None)
    rec = lambda parents=P, state=P, R=4, H=2, D=128, recent=P, n=8: \
        lib.jetfp8_kv_fork_recent(parents, state, R, H, D, recent, n, None)
    for k in ("state", "table", "parents", "ns", "nt"):
        assert fork(**{k: None}) == NULL and fork(**{k: BAD}) == ALIGN
    for kw in (dict(W=0), dict(R=0), dict(R=4097), dict(W=1 << 25), dict(R=4096, W=1 << 19)):
        assert fork(**kw) == SHAPE, kw
    for k in ("parents", "state", "recent"):
        assert rec(**{k: None}) == NULL and rec(**{k: BAD}) == ALIGN
    for kw in (dict(R=0), dict(R=4097, n=9000), dict(H=0), dict(D=32), dict(n=7), dict(n=1 << 31), dict(R=4096, H=4096, n=8192)):
        assert rec(**kw) == SHAPE, kw


def test_sweep_and_move_refusals(lib):
    sweep = lambda state=P, table=P, W=8, R=4, n=100, free=P, head=P, live=P, nt=2 * P, moves=P, ws=None, size=0: \
        lib.jetfp8_kv_sweep(state, table, W, R, n, free, head, live, nt, moves, ws, size, None)
    move = lambda moves=P, n=4, H=2, D=64, codes=P, scales=P, blocks=8: \
        lib.jetfp8_kv_move(moves, n, H, D, codes, scales, blocks, None)
    for k in ("state", "table", "free", "head", "live", "nt", "moves"):
        assert sweep(**{k: None}) == NULL and sweep(**{k: BAD}) == ALIGN
    for kw in (dict(W=0), dict(R=0), dict(R=4097), dict(n=0), dict(n=(1 << 18) + 1), dict(W=1 << 25), dict(R=4096, W=1 << 19)):
        assert sweep(**kw) == SHAPE, kw
    f = lib.jetfp8_kv_sweep_workspace
    assert f(64, 128, 100) == 0 and f(65, 128, 100) == 2 * 2 * 8 and f(4096, 4096, 1 << 18) == 64 * (1 << 15)
    assert f(0, 8, 8) == SHAPE and f(1, 1, (1 << 18) + 1) == SHAPE
    assert sweep(R=65, W=128) == NULL and sweep(R=65, W=128, ws=P, size=31) == SHAPE and sweep(R=65, W=128, ws=BAD, size=32) == ALIGN
    for k in ("moves", "codes", "scales"):
        assert move(**{k: None}) == NULL and move(**{k: BAD}) == ALIGN
    for kw in (dict(n=0), dict(H=0), dict(D=96), dict(blocks=0), dict(n=1 << 23, H=2), dict(n=1 << 40, H=1 << 30)):
        assert move(**kw) == SHAPE, kw


def test_fork_and_sweep_in_place_are_refused(lib):
    """Both read tables that other thread blocks would be overwriting."""
    Q = 4 * P                                                # far from the buffers at P: 4 requests of 8 blocks, 128 bytes
    fork = lambda ns, nt: lib.jetfp8_kv_fork(2 * P, P, 8, 4, 3 * P, ns, nt, None)
    for at in (-16, 0, 16):
        assert fork(2 * P + at, Q) == SHAPE
    for at in (-112, 0, 16, 112):
        assert fork(Q, P + at) == SHAPE
        assert lib.jetfp8_kv_sweep(2 * P, P, 8, 4, 100, Q, Q + 512, Q + 528, P + at, Q + 1024, None, 0, None) == SHAPE
    # tables of more than 2^31 bytes
    assert lib.jetfp8_kv_fork(P, 2 * P, 1 << 20, 1024, P, 1 << 40, 2 * P + (1 << 32) - 16, None) == SHAPE
    assert lib.jetfp8_kv_sweep(P, 2 * P, 1 << 20, 1024, 100, P, P, P, 2 * P + (1 << 32) - 16, P, P, 1 << 40, None) == SHAPE


def test_binding_refuses_host_tensors():
    import torch
    import fp8_precision_rl_amd as jf
    bf, i32 = lambda *s: torch.zeros(s, dtype=torch.bfloat16), lambda *s: torch.zeros(s, dtype=torch.int32)
    for f in (lambda: jf.rmsnorm_add_quantize(bf(2, 128), bf(2, 128), bf(128), 1e-5),
              lambda: jf.rmsnorm_backward(bf(2, 128), bf(2, 128), bf(128), torch.zeros(2)),
              lambda: jf.rotary(bf(2, 1, 64), i32(2), torch.zeros(32, dtype=torch.float64)),
              lambda: jf.kv_positions(i32(4, 8), 4), lambda: jf.kv_prefix(i32(4, 8), i32(2, 8), i32(2)),
              lambda: jf.kv_fork(i32(2, 2), i32(2, 8), i32(2)), lambda: jf.kv_sweep(i32(2, 2), i32(2, 8), 10),
              lambda: jf.kv_fork_recent(i32(2), i32(2, 2), bf(4, 1, 2, 64 * 64)),
              lambda: jf.kv_move(i32(4, 2), torch.zeros((4, 1, 2, 64 * 64), dtype=torch.uint8), torch.zeros(4, 1, 2))):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------------------------------------------------ oracle pins
def test_backward_is_the_derivative():
    """The formula against central differences of sum(dy y) in float64."""
    rng = np.random.default_rng(0)
    R, C, eps, step = 3, 24, 1e-2, 1e-5
    h, dy, w = rng.standard_normal((R, C)), rng.standard_normal((R, C)), 1 + 0.1 * rng.standard_normal(C)
    loss = lambda h, w: (dy * h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w).sum()
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    dx, _, dw, _ = ro.rmsnorm_backward(dy, h, w, r)
    for i in range(R):
        for k in range(C):
            e = np.zeros((R, C))
            e[i, k] = step
            assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * step) - dx[i, k]) < 1e-8
    for k in range(C):
        e = np.zeros(C)
        e[k] = step
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * step) - dw[k]) < 1e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_transposed_map(interleaved):
    """<rotary(x), dy> = <x, inverse(dy)>, so the inverse is the backward pass; and scores depend on distances alone."""
    rng = np.random.default_rng(1)
    x, dy, f = rng.standard_normal((4, 2, 32)), rng.standard_normal((4, 2, 32)), 10.0 ** -np.arange(8)
    pos = np.array([0, 3, 1000, 12345])
    y, _ = ro.rotary(x, pos, f, interleaved, 1.5, False)
    dx, _ = ro.rotary(dy, pos, f, interleaved, 1.5, True)
    assert abs((y * dy).sum() - (x * dx).sum()) < 1e-9
    assert np.array_equal(y[..., 16:], x[..., 16:])
    a, _ = ro.rotary(x, pos, f, interleaved, 1.0, False)
    b, _ = ro.rotary(x, pos + 77, f, interleaved, 1.0, False)
    assert abs((a[0] * a[1]).sum() - (b[0] * b[1]).sum()) < 1e-9


def test_oracle_prefix():
    state = np.array([[640, 0], [700, 0], [600, 1], [1000, 0], [64, 0], [1200, 0]], np.int32)
    table = np.full((6, 20), -1, np.int32)
    for r, n in enumerate(state[:, 0]):
        table[r, :n // 64] = np.arange(n // 64)
    table[3, 9] = 99
    plan = lambda lens: kc.plan(state, lens, np.arange(200, 260, dtype=np.int32), 0, table, int(sum(lens)), max(lens))
    p = plan([1, 1, 1, 1, 1, 1])
    rec = lambda groups, p=p: ro.prefix(p["units"], p["table"], np.array(groups)).tolist()
    assert rec([0, 0, 0, 1, 1, 1]) == [[0, 3, 8, 0]] * 3 + [[3, 1, 0, 0], [4, 1, 0, 0], [5, 1, 0, 0]]
    assert rec([2, 2, -1, 2, -1, 2])[3:] == [[3, 1, 0, 0], [4, 1, 0, 0], [5, 1, 0, 0]]      # the same id apart
    assert rec([0] * 6) == [[k, 1, 0, 0] for k in range(6)]                                  # request 4 has one block
    p = plan([1, 0, 1, 65, 0, 1])                                                            # idle ones do not count
    assert [u[0] for u in p["units"][:6]] == [0, 2, 3, 3, 5, -1]
    assert rec([0] * 6, p)[:6] == [[0, 5, 8, 0]] * 5 + [[-1, 0, 0, 0]]


def test_oracle_fork_and_sweep():
    state = np.array([[130, 0], [64, 1], [0, 0], [200, 1]], np.int32)
    table = np.array([[4, 7, -1, 9], [5, 3, 3, 3], [6, 6, 6, 6], [4, 7, 8, 2]], np.int32)
    s, t = ro.fork(state, table, [3, -1, 0, 1])
    assert s.tolist() == [[200, 1], [64, 1], [130, 1], [64, 0]]
    assert t.tolist() == [[4, 7, 8, -1], [5, -1, -1, -1], [4, 7, -1, -1], [5, -1, -1, -1]]
    w = ro.sweep(state, table, 9, False)
    assert w["free_blocks"].tolist() == [0, 1, 2, 3, 6, -1, -1, -1, -1] and w["live"][0] == 4
    w = ro.sweep(state, table, 9, True)
    assert w["free_blocks"].tolist() == [4, 5, 6, 7, 8, -1, -1, -1, -1]
    assert w["moves"].tolist() == [[4, 0], [5, 1], [7, 2], [8, 3]]
    assert w["next_table"].tolist() == [[0, 2, -1, -1], [1, -1, -1, -1], [-1] * 4, [0, 2, 3, -1]]
    recent = np.arange(8)[:, None].copy()
    ro.fork_recent([3, -1, 0, 1], state, recent)
    assert recent[:, 0].tolist() == [0, 7, 2, 3, 4, 0, 3, 7]


# ------------------------------------------------------------------------------------------------ frequencies
def test_rotary_frequencies():
    import fp8_precision_rl_amd as jf
    f = lambda *a, **k: jf.rotary_frequencies(*a, device="cpu", **k).numpy()
    base = 10000.0 ** (-2 * np.arange(32) / 64)
    assert np.allclose(f(64), base, rtol=1e-14)
    assert np.allclose(f(64, 500.0), 500.0 ** (-2 * np.arange(32) / 64), rtol=1e-14)
    assert np.allclose(f(64, scaling="linear", factor=8), base / 8, rtol=1e-14)
    g = f(64, scaling="base", factor=8)
    assert np.isclose(g[0], 1) and np.isclose(g[-1], base[-1] / 8) and (np.diff(g) < 0).all()
    g = f(64, scaling="bands", factor=8, original=4096, low=1, high=4)
    turns = 4096 * base / (2 * np.pi)
    assert np.allclose(g[turns >= 4], base[turns >= 4]) and np.allclose(g[turns <= 1], base[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (g[mid] < base[mid]).all() and (g[mid] > base[mid] / 8).all()
    for kw in (dict(scaling="other"), dict(scaling="bands", factor=2), dict(scaling="bands", original=100, low=4, high=4),
               dict(base=0.0), dict(factor=-1.0)):
        with pytest.raises(ValueError):
            f(64, **kw)
    for dim in (0, 7, -2):
        with pytest.raises(ValueError):
            f(dim)
    with pytest.raises(ValueError):
        f(2, scaling="base", factor=2)

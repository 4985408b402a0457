"""The expert operators' argument checks, before any launch: no GPU needed."""
import ctypes
import os
import random

import pytest
import torch

import sparse_moe_layer_correction_amd as M

BASE = dict(R=100, E=4, N=64, K=128)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.library_path()):
        from sparse_moe_layer_correction_amd.build import build
        build()
    return M.load_library()


def dims(**over):
    return ctypes.byref(M._GroupedDims(**dict(BASE, **over)))


REFUSED = [
    (dict(R=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(K=-8), -1),
    (dict(ldx=120), -1), (dict(ldy=56), -1), (dict(ldw=64), -1), (dict(lddx=64), -1), (dict(w_stride=64 * 128 - 8), -1),
    (dict(ldx=-128), -1),
    (dict(N=60), -2), (dict(K=100), -2), (dict(ldx=132), -2), (dict(w_stride=64 * 128 + 4), -2),
    (dict(E=1025), -2), (dict(R=(1 << 30) + 1), -2), (dict(ldx=1 << 21), -2),
    (dict(R=1 << 30, N=1 << 20), -2), (dict(E=1024, N=1 << 15, K=1 << 15), -2),
    (dict(R=47 * 1024, E=1024, N=425984, K=16), -2),           # too many 32-row tiles, of the 8-bit product alone
]


@pytest.mark.parametrize("bad,code", REFUSED)
def test_grouped_dims(lib, bad, code):
    d = dims(**bad)
    assert lib.moe_grouped_workspace_bytes(d) == 0
    big = 1 << 50
    assert lib.moe_grouped_matmul(d, 256, 256, 256, 256, 256, big, None) == code
    assert lib.moe_grouped_matmul_grad(d, 256, 256, 256, 256, 256, 256, 0, 0, 256, big, None) == code


def test_grouped_pointers(lib):
    d = dims()
    n = lib.moe_grouped_workspace_bytes(d)
    assert n > 0 and n % 256 == 0
    f, g, q = lib.moe_grouped_matmul, lib.moe_grouped_matmul_grad, lib.moe_grouped_matmul_fp8
    for i in range(4):
        a = [256] * 4
        a[i] = None
        assert f(d, *a, 256, n, None) == -1
        if i != 2:
            a[i] = 264
            assert f(d, *a, 256, n, None) == -1
    assert f(None, 256, 256, 256, 256, 256, n, None) == -1
    big = dims(E=200, R=10000, N=640)              # needs a tile table
    bn = lib.moe_grouped_workspace_bytes(big)
    for ws, have in ((None, bn), (128, bn), (256, 1024)):
        assert f(big, 256, 256, 256, 256, ws, have, None) == -3
        assert g(big, 256, 256, 256, 256, 256, 256, 0, 0, ws, have, None) == -3
        assert q(big, *[256] * 6, ws, have, None) == -3
    # bf16 rows are quantised into the workspace
    assert lib.moe_grouped_matmul_fp8_rows(d, 256, 256, 256, 256, 256, 256, 100 * 128 - 1, None) == -3
    assert lib.moe_grouped_matmul_fp8_rows(d, 256, 256, 256, 256, 256, None, 0, None) == -3
    # a long reduction over few tiles keeps its pieces there
    assert f(dims(K=4096), 256, 256, 256, 256, None, 0, None) == -3
    assert q(dims(K=4096), *[256] * 6, None, 0, None) == -3
    assert g(dims(N=4096), 256, 256, 256, 256, 256, None, 0, 0, None, 0, None) == -3
    # and so does a weight gradient split over the rows
    assert g(dims(R=4096, E=1), 256, 256, 256, 256, None, 256, 0, 0, None, 0, None) == -3
    assert g(d, None, 256, 256, 256, 256, 256, 0, 0, 256, n, None) == -1
    assert g(d, 256, None, 256, 256, 256, 256, 0, 0, 256, n, None) == -1      # dw needs x
    assert g(d, 256, 256, None, 256, 256, 256, 0, 0, 256, n, None) == -1      # dx needs w
    assert g(d, 256, 256, 256, None, 256, 256, 0, 0, 256, n, None) == -1
    assert g(d, 256, 256, 256, 256, None, None, 0, 0, 256, n, None) == -1     # nothing to compute
    assert g(d, 256, 256, 256, 256, 256, 256, 2, 0, 256, n, None) == -1       # unknown type
    assert g(d, 256, 256, 256, 256, 264, 256, 0, 0, 256, n, None) == -1
    for i in range(6):
        a = [256] * 6
        a[i] = None
        assert q(d, *a, 256, n, None) == -1
    assert q(dims(K=136), *[256] * 6, 256, 1 << 40, None) == -2               # K a multiple of 16
    r = lib.moe_grouped_matmul_fp8_rows
    for i in range(5):
        a = [256] * 5
        a[i] = None
        assert r(d, *a, 256, n, None) == -1
    assert r(dims(ldx=120), *[256] * 5, 256, n, None) == -1
    assert r(dims(R=1 << 30, K=4096), *[256] * 5, 256, 1 << 50, None) == -2


def test_quantisers(lib):
    r, b = lib.moe_quantize_fp8_rows, lib.moe_quantize_fp8_blocks
    assert r(256, -1, 64, 0, 256, 256, None) == -1
    assert r(256, 4, 0, 0, 256, 256, None) == -1
    assert r(256, 4, 64, 56, 256, 256, None) == -1
    assert r(None, 4, 64, 0, 256, 256, None) == -1
    assert r(256, 4, 64, 0, 264, 256, None) == -1
    assert r(256, 4, 60, 0, 256, 256, None) == -2
    assert r(256, 4, 64, 68, 256, 256, None) == -2
    for R, K in (((1 << 28) - 15, 64), ((1 << 27) - 7, 136)):    # one more than the grid's threads can be counted for
        assert r(1 << 40, R, K, 0, 1 << 44, 1 << 46, None) == -2
        assert r(1 << 40, R - 1, K, 0, 1 << 40, 1 << 46, None) == -1       # (refused for the shared memory alone)
    assert b(256, -1, 64, 64, 256, 256, None) == -1
    assert b(256, 1, 64, 0, 256, 256, None) == -1
    assert b(256, 1, 64, 64, None, 256, None) == -1
    assert b(264, 1, 64, 64, 256, 256, None) == -1
    assert b(256, 1, 64, 60, 256, 256, None) == -2
    assert b(256, 1, 1 << 16, 1 << 15, 256, 256, None) == -2
    assert b(256, 1 << 24, 8, 8, 256, 256, None) == -2


def test_outputs_share_no_memory(lib):
    R, N, K = 100, 64, 128
    d, f, g = dims(), lib.moe_grouped_matmul, lib.moe_grouped_matmul_grad
    x, w, o, y, dx, dw, ws = (i << 24 for i in range(1, 8))
    for out in (x, x + R * K * 2 - 16, x - R * N * 2 + 16, w, w + 4 * N * K * 2 - 16, o, o + 16):
        assert f(d, x, w, o, out, None, 0, None) == -1, hex(out)
    n = lib.moe_grouped_workspace_bytes(d)
    for a, b in ((y, dw), (x, dw), (w, dw), (dw, dw), (o, dw), (dx, x), (dx, y), (dx, dx + 16), (dx, o)):
        assert g(d, y, x, w, o, a, b, 1, 0, ws, n, None) == -1, (hex(a), hex(b))
    # columns of one matrix that overlap: x in [0, 128), y in [120, 184) of rows of 256
    side = dims(ldx=256, ldy=256)
    assert f(side, x, w, o, x + 120 * 2, None, 0, None) == -1
    assert f(side, x + 120 * 2, w, o, x + 64 * 2, None, 0, None) == -1
    assert f(side, x, w, o, x + 200 * 2, None, 0, None) == -1          # ends in the next row's x
    xq, xs, wq, sw = (i << 24 for i in range(10, 14))
    for out in (xq, xs, wq, sw, o, xq + R * K - 16):
        assert lib.moe_grouped_matmul_fp8(d, xq, xs, wq, sw, o, out, None, 0, None) == -1, hex(out)
    assert lib.moe_grouped_matmul_fp8_rows(d, x, wq, sw, o, x, ws, n, None) == -1
    assert lib.moe_quantize_fp8_rows(x, R, K, 0, x, xs, None) == -1
    assert lib.moe_quantize_fp8_rows(x, R, K, 0, xq, xq + 64, None) == -1
    assert lib.moe_quantize_fp8_blocks(w, 4, N, K, wq, w + 64, None) == -1


def test_workspace_is_enough_for_every_call(lib):
    """Given moe_grouped_workspace_bytes, no call asks for more: those below share memory between an input and an
    output, and are refused for that (-1), after the workspace (-3)."""
    rng = random.Random(7)
    x, w, o, y, ws = (i << 40 for i in range(1, 6))
    cases = [(1100, 50, 64, 2048)] + [
        (int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 10)), 16 * rng.randint(1, 200), 16 * rng.randint(1, 200))
        for _ in range(2000)]
    for R, E, N, K in cases:
        d = ctypes.byref(M._GroupedDims(R, E, N, K))
        n = lib.moe_grouped_workspace_bytes(d)
        got = (lib.moe_grouped_matmul(d, x, w, o, x, ws, n, None),
               lib.moe_grouped_matmul_grad(d, y, x, w, o, y, None, 1, 0, ws, n, None),
               lib.moe_grouped_matmul_grad(d, y, x, w, o, None, x, 1, 0, ws, n, None),
               lib.moe_grouped_matmul_grad(d, y, x, w, o, y, x, 0, 0, ws, n, None),
               lib.moe_grouped_matmul_fp8(d, x, y, w, w, o, x, ws, n, None),
               lib.moe_grouped_matmul_fp8_rows(d, x, w, w, o, x, ws, n, None))
        assert set(got) == {-1}, (R, E, N, K, got)


def tensors(*spec):
    t = (M._GradTensor * max(1, len(spec)))()
    for e, (g, o, n, dt) in zip(t, spec):
        e.grad, e.out, e.n, e.dtype = g, o, n, dt
    return t


def test_grad_norm(lib):
    ok = tensors((256, None, 1000, 0), (4096, 16384, 1000, 1), (None, None, 0, 1))
    n = lib.moe_grad_norm_workspace_bytes(ok, 3)
    assert n > 0 and n % 256 == 0
    f, c = lib.moe_grad_norm, lib.moe_clip_grad_norm
    assert f(ok, 3, None, 256, n, None) == -1
    assert f(None, 3, 256, 256, n, None) == -1
    assert f(ok, -1, 256, 256, n, None) == -1
    assert f(ok, 3, 256, None, n, None) == -3
    assert f(ok, 3, 256, 256, n - 1, None) == -3
    assert f(ok, 3, 256, 264, n, None) == -3
    for bad in ((None, None, 5, 0), (257, None, 5, 0), (258, None, 5, 1), (256, 258, 5, 1), (256, None, -1, 0), (256, None, 5, 2)):
        t = tensors(bad)
        assert lib.moe_grad_norm_workspace_bytes(t, 1) == 0
        assert f(t, 1, 256, 256, 1 << 20, None) == -1
        assert c(t, 1, 1.0, 256, 256, 1 << 20, None) == -1
    assert f(tensors((256, None, (1 << 40) + 1, 0)), 1, 256, 256, 1 << 40, None) == -2
    assert c(ok, 3, -1.0, 256, 256, n, None) == -1
    assert c(ok, 3, float("nan"), 256, 256, n, None) == -1
    assert c(ok, 3, 1.0, None, 256, n, None) == -1


def test_clip_refuses_overlaps(lib):
    c = lib.moe_clip_grad_norm
    for spec in (
        [(256, None, 100, 1), (256, None, 100, 1)],             # the same tensor twice
        [(256, None, 100, 1), (652, None, 100, 1)],             # one element shared
        [(256, 4096, 100, 1), (8192, 4096 + 396, 100, 1)],      # outputs share one
        [(256, 4096, 100, 1), (4096, 8192, 100, 1)],            # an output over another gradient
        [(256, 260, 100, 1)],                                   # an output over its own gradient, shifted
        [(256, 8192, 1000, 1), (512, 260, 10, 1)],              # inside a longer one
    ):
        t = tensors(*spec)
        assert c(t, len(spec), 1.0, 1 << 30, 256, 1 << 20, None) == -1, spec
    for norm in (256, 256 + 396, 4096 + 200):                   # the norm's own place inside a gradient or an output
        assert c(tensors((256, 4096, 100, 1)), 1, 1.0, norm, 256, 1 << 20, None) == -1, norm


def test_binding_refuses():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.grouped_matmul(x, w, o)                               # not on the GPU
    with pytest.raises(ValueError):
        M.grouped_matmul(x[0], w, o)
    with pytest.raises(TypeError):
        M.grouped_matmul(None, w, o)
    with pytest.raises((TypeError, ValueError)):
        M.grouped_matmul_grad(x, x, w, o)
    with pytest.raises((TypeError, ValueError)):
        M.quantize_fp8_rows(x)
    with pytest.raises((TypeError, ValueError)):
        M.grouped_matmul_fp8(x, w, w, o)
    with pytest.raises(ValueError):
        M.grad_norm([])
    with pytest.raises(ValueError):
        M.clip_grad_norm([x], 1.0)
    with pytest.raises(TypeError):
        M.clip_grad_norm([o], 1.0)

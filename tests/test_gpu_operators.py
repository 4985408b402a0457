"""The expert operators on the GPU against 64-bit definitions: the grouped product and
its gradients, the 8-bit product and its quantisers, gradient norm and clipping.

Tolerances. A bf16 output is one rounding of an fp32 sum: half a step, 2^-8 of the
value, plus the sum's own error, at most one unit of 2^-23 of sum |terms| for each of
its additions (round to nearest or toward zero). fp32 outputs lack the first part's
rounding (2^-24 of the value instead).
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_correction_amd as M
import workloads as W
from gpu_util import device_inputs, log

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def rnd(shape, seed, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def offs(counts, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(counts)]), dtype=torch.int32).cuda()


def check(got, ref, terms, n, dtype, more=0.0):
    """got against ref (64 bits) with sum |terms| and the number of additions n; more: a further allowance."""
    g = got.double().cpu()
    tol = HALF[dtype] * ref.abs() + n * 2.0 ** -23 * terms + more + 1e-300
    bad = (g - ref).abs() > tol
    assert torch.isfinite(g).all()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float(((g - ref).abs() / tol).max()):.3g}"


def ranges(offsets, R):
    """Rows of each expert: the offsets' running maximum, clamped to [0, R]."""
    o = np.maximum.accumulate(np.clip(offsets.cpu().numpy(), 0, R))
    return [(int(a), int(b)) for a, b in zip(o[:-1], o[1:])]


def ref_product(x, w, rg):
    x, w = x.double().cpu(), w.double().cpu()
    y = torch.zeros(x.shape[0], w.shape[1], dtype=F64)
    s = torch.zeros_like(y)
    for e, (a, b) in enumerate(rg):
        y[a:b] = x[a:b] @ w[e].t()
        s[a:b] = x[a:b].abs() @ w[e].abs().t()
    return y, s


SHAPES = [
    # R, E, N, K, rows of each expert
    (1, 1, 8, 8, [1]),
    (5, 3, 8, 16, [0, 5, 0]),
    (64, 4, 64, 64, [1, 0, 62, 1]),
    (300, 5, 136, 72, [129, 0, 128, 1, 42]),
    (257, 2, 264, 200, [1, 256]),
    (700, 3, 520, 328, [513, 63, 124]),
    (2, 40, 256, 128, [0] * 20 + [1] + [0] * 18 + [1]),
    (1100, 64, 320, 1096, [17] * 60 + [0, 70, 9, 1]),
    (900, 1, 1000, 64, [900]),
]


@pytest.mark.parametrize("R,E,N,K,counts", SHAPES)
def test_grouped_matmul(R, E, N, K, counts):
    x, w, o = rnd((R, K), 1), rnd((E, N, K), 2, K ** -0.5), offs(counts)
    y = M.grouped_matmul(x, w, o)
    ref, s = ref_product(x, w, ranges(o, R))
    check(y, ref, s, K, BF)
    assert torch.equal(y, M.grouped_matmul(x, w, o))


@pytest.mark.parametrize("R,E,N,K,counts", SHAPES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_grouped_matmul_grad(R, E, N, K, counts, dt):
    x, w, dy, o = rnd((R, K), 3), rnd((E, N, K), 4, K ** -0.5), rnd((R, N), 5), offs(counts)
    dx, dw = M.grouped_matmul_grad(dy, x, w, o, dw_dtype=dt)
    rg = ranges(o, R)
    rx, sx = ref_product(dy, w.transpose(1, 2), rg)
    check(dx, rx, sx, N, BF)
    X, G = x.double().cpu(), dy.double().cpu()
    for e, (a, b) in enumerate(rg):
        check(dw[e], G[a:b].t() @ X[a:b], G[a:b].abs().t() @ X[a:b].abs(), b - a, dt)
    again = M.grouped_matmul_grad(dy, x, w, o, dw_dtype=dt)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    only_x = M.grouped_matmul_grad(dy, x, w, o, need_dw=False)
    only_w = M.grouped_matmul_grad(dy, x, w, o, need_dx=False, dw_dtype=dt)
    assert only_x[1] is None and torch.equal(only_x[0], dx)
    assert only_w[0] is None and torch.equal(only_w[1], dw)


@pytest.mark.parametrize("dt", [BF, F32])
def test_gradient_accumulates(dt):
    R, E, N, K, counts = 300, 5, 136, 72, [129, 0, 128, 1, 42]
    x, w, dy, o = rnd((R, K), 3), rnd((E, N, K), 4), rnd((R, N), 5), offs(counts)
    dw = rnd((E, N, K), 6, 3.0, dt)
    before = dw.double().cpu()
    out = M.grouped_matmul_grad(dy, x, w, o, need_dx=False, dw=dw, accumulate=True)[1]
    assert out is dw
    X, G = x.double().cpu(), dy.double().cpu()
    for e, (a, b) in enumerate(ranges(o, R)):
        check(dw[e], before[e] + G[a:b].t() @ X[a:b], before[e].abs() + G[a:b].abs().t() @ X[a:b].abs(), b - a + 1, dt)
    assert torch.equal(dw[1].double().cpu(), before[1])      # no rows: left as it was


def test_gradients_are_the_differences_of_the_product():
    """The product is linear: y(x + h) - y(x) pairs with dy as h pairs with dx, and the same for w. x, h, w and
    dy are small whole numbers, so every sum below 2^24 is exact and bf16 rounding the only error."""
    R, E, N, K, counts = 200, 4, 72, 136, [64, 0, 101, 35]
    g = torch.Generator().manual_seed(8)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g).to(BF).cuda()
    x, h, w, v, dy, o = ints(R, K), ints(R, K), ints(E, N, K), ints(E, N, K), ints(R, N), offs(counts)
    dx, dw = M.grouped_matmul_grad(dy, x, w, o, dw_dtype=F32)
    y = M.grouped_matmul(x, w, o).double()      # |y| <= 136 < 256: exact in bf16
    yh = M.grouped_matmul(x + h, w, o).double() # |y| <= 272: even numbers above 256 may round by 1
    yw = M.grouped_matmul(x, w + v, o).double()
    slack = float((yh.abs() > 256).sum() + (yw.abs() > 256).sum())
    assert abs(float(((yh - y) * dy.double()).sum()) - float((dx.double() * h.double()).sum())) <= slack
    assert abs(float(((yw - y) * dy.double()).sum()) - float((dw.double() * v.double()).sum())) <= slack


@pytest.mark.parametrize("N,K", [(136, 72), (1800, 2064)])
@pytest.mark.parametrize("raw", [
    [40, 60, 90, 150],          # rows before the first and behind the last expert
    [0, 120, 80, 200],          # descending: the second expert is empty, the third starts at 120
    [-5, 50, 1 << 30, 100],     # outside the rows
    [200, 200, 200, 200],
    [0, 0, 0, 0],
])
def test_rows_of_no_expert_and_bad_offsets(raw, N, K):
    """Short sums, and long ones that are split."""
    R, E = 200, 3
    o = torch.tensor(raw, dtype=torch.int32).cuda()
    rg = ranges(o, R)
    own = torch.zeros(R, dtype=torch.bool)
    for a, b in rg:
        own[a:b] = True
    x, w, dy = rnd((R, K), 1), rnd((E, N, K), 2), rnd((R, N), 5)
    clean, cdy = x.clone(), dy.clone()
    x[~own.cuda()] = float("nan")               # never read
    dy[~own.cuda()] = float("inf")
    ref, s = ref_product(clean, w, rg)
    check(M.grouped_matmul(x, w, o), ref, s, K, BF)                          # zero where no expert is
    out = torch.full((R, N), 7.0, dtype=BF, device="cuda")
    M.grouped_matmul(x, w, o, out=out)
    assert (out.cpu()[~own] == 7).all()                                      # left as they were
    check(out[own.cuda()], ref[own], s[own], K, BF)
    dx, dw = M.grouped_matmul_grad(dy, x, w, o)
    rx, sx = ref_product(cdy, w.transpose(1, 2), rg)
    check(dx, rx, sx, N, BF)
    for e, (a, b) in enumerate(rg):
        G, X = cdy.double().cpu()[a:b], clean.double().cpu()[a:b]
        check(dw[e], G.t() @ X, G.abs().t() @ X.abs(), b - a, BF)


def test_infinities_stay_with_their_rows():
    R, E, N, K, counts = 260, 3, 136, 72, [100, 60, 100]
    x, w, dy, o = rnd((R, K), 1), rnd((E, N, K), 2), rnd((R, N), 5), offs(counts)
    ref, s = ref_product(x, w, ranges(o, R))
    x[100:160] = float("inf")                   # the middle expert's rows only
    w[1] = float("nan")
    y = M.grouped_matmul(x, w, o)
    keep = torch.ones(R, dtype=torch.bool)
    keep[100:160] = False
    check(y[keep.cuda()], ref[keep], s[keep], K, BF)
    assert not torch.isfinite(y[100:160]).any()
    dx, dw = M.grouped_matmul_grad(dy, x, w, o)
    assert torch.isfinite(dx[keep.cuda()]).all() and torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all()
    assert not torch.isfinite(dw[1]).any()


def test_strided_operands():
    R, E, N, K, counts = 300, 5, 136, 72, [129, 0, 128, 1, 42]
    o, rg = offs(counts), ranges(offs(counts), R)
    X, Y, Wb = rnd((R, K + 24), 1), rnd((R, N + 8), 2), rnd((E, N + 3, K + 40), 3)
    x, dy, w = X[:, 8:8 + K], Y[:, :N], Wb[:, 1:1 + N, 16:16 + K]
    out, dx = torch.zeros(R, N + 16, dtype=BF, device="cuda"), torch.zeros(R, K + 8, dtype=BF, device="cuda")
    ref, s = ref_product(x, w, rg)
    check(M.grouped_matmul(x, w, o, out=out[:, 8:8 + N])[:, :], ref, s, K, BF)
    assert (out[:, :8] == 0).all() and (out[:, 8 + N:] == 0).all()
    _, dw = M.grouped_matmul_grad(dy, x, w, o, dx=dx[:, :K])
    rx, sx = ref_product(dy, w.transpose(1, 2), rg)
    check(dx[:, :K], rx, sx, N, BF)
    assert (dx[:, K:] == 0).all()
    for e, (a, b) in enumerate(rg):
        G, Z = dy.double().cpu()[a:b], x.double().cpu()[a:b]
        check(dw[e], G.t() @ Z, G.abs().t() @ Z.abs(), b - a, BF)


def test_columns_of_one_matrix():
    """Operands side by side in one matrix share its rows and no memory."""
    R, E, N, K = 150, 3, 136, 72
    both, w, o = torch.zeros(R, K + N, dtype=BF, device="cuda"), rnd((E, N, K), 2, K ** -0.5), offs([60, 0, 90])
    both[:, :K] = rnd((R, K), 1)
    x = both[:, :K].clone()
    y = M.grouped_matmul(x, w, o)
    assert M.grouped_matmul(both[:, :K], w, o, out=both[:, K:]).data_ptr() == both.data_ptr() + 2 * K
    assert torch.equal(both[:, K:], y) and torch.equal(both[:, :K], x)


@pytest.mark.parametrize("R,E,N,K", [(1100, 50, 64, 2048), (1100, 50, 2048, 64)])
def test_each_gradient_alone(R, E, N, K):
    """Alone, each gradient may take other tiles, and another workspace, than both together."""
    x, w, dy, o = rnd((R, K), 1), rnd((E, N, K), 2, K ** -0.5), rnd((R, N), 3), offs(ragged(R, E, 4, 5))
    dx = M.grouped_matmul_grad(dy, x, w, o, need_dw=False)[0]
    dw = M.grouped_matmul_grad(dy, x, w, o, need_dx=False, dw_dtype=F32)[1]
    for e, (a, b) in enumerate(ranges(o, R)):
        G, X, Wt = dy[a:b].double(), x[a:b].double(), w[e].double()
        check(dw[e], (G.t() @ X).cpu(), (G.abs().t() @ X.abs()).cpu(), b - a, F32)
        if b > a:
            check(dx[a:b], (G @ Wt).cpu(), (G.abs() @ Wt.abs()).cpu(), N, BF)


@pytest.mark.parametrize("tail", [3, 300])
def test_rows_past_32_bit_offsets(tail):
    """Rows of 8 KB, 600000 of them: byte offsets past 2^32 in x, y and dy, and the last rows still right."""
    R, E, N, K = 600000 + tail, 3, 4096, 64
    o = offs([599990, 0, R - 599990])
    x, w, dy = rnd((R, K), 1), rnd((E, N, K), 2, K ** -0.5), rnd((R, 1), 3).expand(R, N).contiguous()
    y = M.grouped_matmul(x, w, o)
    dx, dw = M.grouped_matmul_grad(dy, x, w, o, dw_dtype=F32)
    G, X, Wt = dy[599990:].double(), x[599990:].double(), w[2].double()
    check(y[599990:], (X @ Wt.t().contiguous()).cpu(), (X.abs() @ Wt.abs().t().contiguous()).cpu(), K, BF)
    check(dx[599990:], (G @ Wt).cpu(), (G.abs() @ Wt.abs()).cpu(), N, BF)
    check(dw[2], (G.t() @ X).cpu(), (G.abs().t() @ X.abs()).cpu(), R - 599990, F32)
    xt = dy[-tail:].clone()                                                 # and as the operand read along its rows
    wt = rnd((E, 72, N), 4, N ** -0.5)
    z = M.grouped_matmul(dy, wt, o)
    check(z[-tail:], (xt.double() @ wt[2].double().t().contiguous()).cpu(),
          (xt.double().abs() @ wt[2].double().abs().t().contiguous()).cpu(), N, BF)
    q, s = M.quantize_fp8_rows(dy)
    q2, s2 = M.quantize_fp8_rows(xt)
    assert torch.equal(q[-tail:], q2) and torch.equal(s[:, -tail:], s2)


def test_refused_on_the_gpu():
    """Layouts the kernels cannot read, refused by the binding or the library before any launch."""
    x, w, o, dy = rnd((16, 64), 1), rnd((2, 72, 64), 2), offs([8, 8]), rnd((16, 72), 3)
    bad = [
        lambda: M.grouped_matmul(x[:1].expand(16, 64), w, o),               # rows that share memory
        lambda: M.grouped_matmul(x, w[:1].expand(2, 72, 64), o),            # experts that share theirs
        lambda: M.grouped_matmul(x.t().contiguous().t(), w, o),             # columns not contiguous
        lambda: M.grouped_matmul(x, w, o.long()),
        lambda: M.grouped_matmul(x, w, o[:-1]),
        lambda: M.grouped_matmul(x.float(), w, o),
        lambda: M.grouped_matmul(x[:, :56], w, o),
        lambda: M.grouped_matmul(x, w, o, out=torch.empty(16, 64, dtype=BF, device="cuda")),
        lambda: M.grouped_matmul(x, w, o.cpu()),
        lambda: M.grouped_matmul(rnd((16, 65), 1)[:, :64], w, o),           # a row stride that is no multiple of 8
        lambda: M.grouped_matmul(rnd((16, 72), 1)[:, 4:68], w, o),          # not 16-byte aligned
        lambda: M.grouped_matmul(x[:, :60], w[:, :, :60], o),               # K no multiple of 8
        lambda: M.grouped_matmul_grad(dy, x, w, o, need_dx=False, need_dw=False),
        lambda: M.grouped_matmul_grad(dy, x, w, o, accumulate=True),
        lambda: M.grouped_matmul_grad(dy, x, w, o, dw_dtype=torch.float16),
        lambda: M.grouped_matmul_grad(dy, x, w, o, dw=torch.empty(2, 72, 64, device="cuda"), dw_dtype=BF),
        lambda: M.grouped_matmul_grad(x, x, w, o),
        lambda: M.grouped_matmul_fp8(x, w, torch.ones(2, 1, 1, device="cuda"), o),
        lambda: M.grouped_matmul_fp8(x, w.view(torch.uint8)[..., :64].contiguous(), torch.ones(2, 1, 2, device="cuda"), o),
        lambda: M.quantize_fp8_rows(x.float()),
        lambda: M.quantize_fp8_blocks(w.transpose(1, 2)),
        lambda: M.clip_grad_norm([x, x], 1.0),                              # twice the same: scaled twice
        lambda: M.clip_grad_norm([x, x[8:]], 1.0),
        lambda: M.clip_grad_norm([x], 1.0, out=[]),
        lambda: M.clip_grad_norm([x], 1.0, out=[x.float()]),
        lambda: M.clip_grad_norm([x.t()], 1.0),
        lambda: M.clip_grad_norm([x], -1.0),
        lambda: M.grad_norm([x, o]),
        lambda: M.grad_norm([x, x.cpu()]),
    ]
    sq = rnd((2, 64, 64), 4)
    bad += [
        lambda: M.grouped_matmul(x, sq, o, out=x),                          # an output over an input
        lambda: M.grouped_matmul_grad(x, x, sq, o, dx=x),
        lambda: M.grouped_matmul_grad(x, x.clone(), sq, o, dw=sq),
    ]
    for f in bad:
        with pytest.raises((TypeError, ValueError, M.MoEError)):
            f()
    assert float(M.grad_norm([x, x])) > 0                                   # the norm alone may count a tensor twice


def test_no_rows():
    E, N, K = 4, 64, 72
    x, w, o = torch.empty(0, K, dtype=BF, device="cuda"), rnd((E, N, K), 1), offs([0] * E)
    assert M.grouped_matmul(x, w, o).shape == (0, N)
    dx, dw = M.grouped_matmul_grad(torch.empty(0, N, dtype=BF, device="cuda"), x, w, o)
    assert dx.shape == (0, K) and (dw == 0).all()
    q, s = M.quantize_fp8_rows(x)
    assert q.shape == (0, K) and s.shape == (1, 0)


# ----------------------------------------------------------------------------
# 8 bits
# ----------------------------------------------------------------------------

def ref_quantise(blocks):
    """Values of the last axis as (codes' values, scale): the definition, in 64 bits."""
    v = blocks.double()
    amax = v.abs().amax(-1, keepdim=True)
    e = torch.full_like(amax, -126.0)
    up = amax > 448.0 * torch.exp2(e)
    while up.any():
        e = torch.where(up, e + 1, e)
        up = amax > 448.0 * torch.exp2(e)
    scaled = (v / torch.exp2(e)).float()                      # exact: bf16 values and powers of two
    return scaled.to(torch.float8_e4m3fn), torch.exp2(e)[..., 0]


def blocks_of_rows(x):
    R, K = x.shape
    kb = (K + 127) // 128
    return torch.nn.functional.pad(x.float().cpu(), (0, kb * 128 - K)).view(R, kb, 128)


@pytest.mark.parametrize("R,K", [(1, 8), (3, 128), (37, 136), (130, 1360), (1, 2048)])
def test_quantise_rows(R, K):
    x = rnd((R, K), R, 1.0)
    x *= torch.exp2(torch.randint(-30, 30, (R, 1), generator=torch.Generator().manual_seed(K)).float()).to(BF).cuda()
    x[R // 2, : K // 2] = 0
    q, s = M.quantize_fp8_rows(x)
    rq, rs = ref_quantise(blocks_of_rows(x))
    assert torch.equal(s.double().cpu(), rs.t())
    assert torch.equal(q.cpu(), rq.reshape(R, -1)[:, :K].contiguous().view(torch.uint8))


def test_quantise_every_value():
    """Every bf16 value in a block with 448 and its negative: each rounding, ties and the smallest steps."""
    bits = torch.arange(0x0000, 0x7F80, dtype=torch.int32)
    vals = bits.to(torch.int16).view(BF)
    vals = vals[(vals.float() <= 448)]
    n = vals.numel() // 126 * 126
    x = torch.cat([vals[:n].view(-1, 126), torch.full((n // 126, 1), 448.0).to(BF), torch.full((n // 126, 1), -1.5).to(BF)], 1)
    x = torch.cat([x, -x]).cuda()
    q, s = M.quantize_fp8_rows(x)
    rq, rs = ref_quantise(blocks_of_rows(x))
    assert torch.equal(s.double().cpu(), rs.t()) and (s == 1).all()
    assert torch.equal(q.cpu(), rq.reshape(x.shape).view(torch.uint8))


def test_quantise_special_blocks():
    x = torch.zeros(6, 256, dtype=BF)
    x[1, 3] = float("nan")
    x[1, 4] = 2.0
    x[2, 130] = float("-inf")
    x[2, 131] = 3.0
    x[3, 0] = 3.3e38
    x[4, 0] = 1e-40                                        # subnormal: the scale stays at 2^-126
    x[5, :128] = float("inf")
    q, s = M.quantize_fp8_rows(x.cuda())
    v = q.cpu().view(torch.float8_e4m3fn).double() * s.double().cpu().t().repeat_interleave(128, 1)
    assert (q.cpu()[0] == 0).all() and (s[:, 0].cpu() == 2.0 ** -126).all()
    assert torch.isnan(v[1, 3]) and v[1, 4] == 2.0 and torch.isnan(v[2, 130]) and v[2, 131] == 3.0
    assert torch.isfinite(v[1, 5:]).all() and torch.isnan(v[5, :128]).all() and (v[5, 128:] == 0).all()
    assert abs(float(v[3, 0]) / float(x[3, 0].double()) - 1) <= 2.0 ** -4 and torch.isfinite(v[4]).all()


@pytest.mark.parametrize("shape", [(1, 1, 8), (3, 128, 128), (2, 200, 136), (1, 130, 520)])
def test_quantise_blocks(shape):
    w = rnd(shape, 9, 0.05)
    q, s = M.quantize_fp8_blocks(w)
    E, N, K = shape
    nb, kb = (N + 127) // 128, (K + 127) // 128
    p = torch.nn.functional.pad(w.float().cpu(), (0, kb * 128 - K, 0, nb * 128 - N))
    p = p.view(E, nb, 128, kb, 128).permute(0, 1, 3, 2, 4).reshape(E, nb, kb, -1)
    rq, rs = ref_quantise(p)
    assert torch.equal(s.double().cpu(), rs)
    back = rq.view(torch.uint8).view(E, nb, kb, 128, 128).permute(0, 1, 3, 2, 4).reshape(E, nb * 128, kb * 128)
    assert torch.equal(q.cpu(), back[:, :N, :K])


SHAPES8 = [(r, e, n, (k + 15) // 16 * 16, c) for r, e, n, k, c in SHAPES]


def ref_product8(xv, wq, sw, rg):
    """xv [R, K] the rows' values (64 bits); y and the sum of |terms|."""
    wv = wq.cpu().view(torch.float8_e4m3fn).double()
    E, N, K = wv.shape
    wv = wv * sw.double().cpu().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    y = torch.zeros(xv.shape[0], N, dtype=F64)
    s = torch.zeros_like(y)
    for e, (a, b) in enumerate(rg):
        y[a:b] = xv[a:b] @ wv[e].t()
        s[a:b] = xv[a:b].abs() @ wv[e].abs().t()
    return y, s


def aligned_loss(xv, wq, sw, rg):
    """What the 8-bit matrix instruction may drop. It adds the products of 8 consecutive k after aligning them to
    the largest one's exponent, with 13 bits below it, truncating (read off the device: 2^16 + 2^3 arrives, of 2^16 +
    28.125 the 4.125 below a multiple of 2^3 are lost, toward zero for either sign, and only inside such 8). So each
    of the 7 others loses less than 2^-13 of the largest |x w| of its 8, which the product of the two operands'
    largest magnitudes bounds."""
    wv = wq.cpu().view(torch.float8_e4m3fn).double().abs()
    E, N, K = wv.shape
    wv = wv * sw.double().cpu().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    xm, wm = xv.abs().view(-1, K // 8, 8).amax(2), wv.view(E, N, K // 8, 8).amax(3)
    out = torch.zeros(xv.shape[0], N, dtype=F64)
    for e, (a, b) in enumerate(rg):
        out[a:b] = 7 * 2.0 ** -13 * (xm[a:b] @ wm[e].t())
    return out


@pytest.mark.parametrize("R,E,N,K,counts", SHAPES8)
def test_grouped_matmul_fp8(R, E, N, K, counts):
    x, o = rnd((R, K), 1), offs(counts)
    wq, sw = M.quantize_fp8_blocks(rnd((E, N, K), 2, K ** -0.5))
    sw = sw * (0.5 + torch.rand(sw.shape, generator=torch.Generator().manual_seed(3)).cuda())   # any scale, not only 2^e
    y = M.grouped_matmul_fp8(x, wq, sw, o)
    q, sx = ref_quantise(blocks_of_rows(x))
    xv = (q.double() * sx[..., None]).reshape(R, -1)[:, :K]
    ref, s = ref_product8(xv, wq, sw, ranges(o, R))
    # the two scales' product and its fma add two roundings a block
    check(y, ref, s, K + 2 * ((K + 127) // 128), BF, aligned_loss(xv, wq, sw, ranges(o, R)))
    codes, scales = M.quantize_fp8_rows(x)
    assert torch.equal(y, M.grouped_matmul_fp8(codes, wq, sw, o, x_scale=scales))


@pytest.mark.parametrize("R,E,N,K,counts", [
    (16, 8, 2680, 96, [0, 0, 9, 0, 1, 0, 6, 0]),
    (1, 3, 136, 2064, [0, 1, 0]),
    (22, 300, 520, 1040, [1 if e % 14 == 3 else 0 for e in range(300)]),
    (200, 16, 520, 512, [70, 0, 33, 32, 31, 1, 0, 0, 20, 5, 5, 1, 1, 1, 0, 0]),
    (32, 1, 1000, 2048, [32]), (31, 4, 264, 5072, [3, 0, 27, 1]), (300, 20, 1000, 128, [15] * 20),
    (150, 5, 2000, 256, [33, 0, 64, 3, 50]), (7, 2, 136, 2064, [4, 3]),
])
def test_fp8_few_rows(R, E, N, K, counts):
    """Few rows are quantised by the product itself: the same bits as from codes made before, call after call in one
    workspace, with every column tile's workgroups at it at once."""
    o = offs(counts)
    wq, sw = M.quantize_fp8_blocks(rnd((E, N, K), 2, K ** -0.5))
    ws = torch.full((M.grouped_workspace_bytes(R, E, N, K),), 255, dtype=torch.uint8, device="cuda")
    for rep in range(4):
        x = rnd((R, K + 8), 10 + rep, 10.0 ** (rep - 2))[:, :K]
        if rep == 3:
            x[:, :16] = 0
            x[R // 2, K - 3] = float("inf")
        codes, scales = M.quantize_fp8_rows(x)
        want = M.grouped_matmul_fp8(codes, wq, sw, o, x_scale=scales)
        assert torch.isfinite(want).all() or rep == 3
        bits = lambda t: t.view(torch.int16)
        assert torch.equal(bits(M.grouped_matmul_fp8(x, wq, sw, o, ws=ws)), bits(want))
        assert torch.equal(bits(M.grouped_matmul_fp8(x, wq, sw, o)), bits(want))


@pytest.mark.parametrize("K", [272, 2064])
def test_fp8_rows_of_no_expert_and_special_values(K):
    R, E, N = 300, 3, 136
    o = torch.tensor([20, 150, 150, 280], dtype=torch.int32).cuda()
    x = rnd((R, K), 1)
    wq, sw = M.quantize_fp8_blocks(rnd((E, N, K), 2, K ** -0.5))
    good = M.grouped_matmul_fp8(x, wq, sw, o)
    assert (good[:20] == 0).all() and (good[280:] == 0).all() and torch.isfinite(good).all()
    x[:20] = float("nan")
    x[280:] = float("inf")
    x[30, 200] = float("inf")                              # its own row only
    out = torch.full((R, N + 8), 7.0, dtype=BF, device="cuda")
    M.grouped_matmul_fp8(x, wq, sw, o, out=out[:, :N])
    keep = [i for i in range(20, 280) if i != 30]
    assert torch.equal(out[keep, :N], good[keep]) and torch.isnan(out[30, :N]).all()
    assert (out[:20] == 7).all() and (out[280:] == 7).all() and (out[:, N:] == 7).all()


# ----------------------------------------------------------------------------
# gradient norm and clipping
# ----------------------------------------------------------------------------

def norm64(ts):
    return float(torch.sqrt(sum((t.double() ** 2).sum() for t in ts)))


SIZES = [[1], [7, 0, 33000, 5], [65536], [65537], [2048] * 32, [2048] * 33, [1, 2, 3] * 40, [500] * 121, [0, 30000, 0, 40001], [1 << 15, (1 << 15) + 1, 100003], [3] * 301, [2_000_003]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_clip_grad_norm(sizes, shift):
    """Tensors at any element alignment, both types mixed; in place and into other tensors."""
    g = []
    for i, n in enumerate(sizes):
        dt = (BF, F32)[i % 2]
        g.append(rnd((n + shift,), 50 + i, 10.0 ** (i % 4 - 2), dt)[shift:])
    ref = norm64([t.cpu() for t in g])
    n = M.grad_norm(g)
    assert n.shape == () and n.dtype == F32 and abs(float(n) - ref) <= 2.0 ** -23 * ref
    for ratio in (0.3, 2.0):
        out = [torch.full((t.numel() + 5,), 9.0, dtype=t.dtype, device="cuda")[(i % 3):][:t.numel()] for i, t in enumerate(g)]
        n = M.clip_grad_norm(g, ratio * ref, out=out)
        assert abs(float(n) - ref) <= 2.0 ** -23 * ref
        f = min(1.0, float(np.float32(ratio * ref)) / ref)
        for a, b in zip(g, out):
            # half a step of the type, and the factor's own error
            r = a.double().cpu() * f
            assert ((b.double().cpu() - r).abs() <= (HALF[a.dtype] + 2.0 ** -40) * r.abs() + 1e-44).all()
            if ratio > 1:
                assert torch.equal(a, b)
        inplace = [t.clone() for t in g]
        M.clip_grad_norm(inplace, ratio * ref)
        assert all(torch.equal(a, b) for a, b in zip(inplace, out))


def test_clip_large_and_not_finite():
    big = [torch.full((1000,), 3e38, device="cuda"), torch.full((9,), -3e38, dtype=BF, device="cuda")]
    ref = norm64([t.cpu() for t in big])
    c = [t.clone() for t in big]
    n = M.clip_grad_norm(c, 1.0)
    assert torch.isinf(n)                                   # past fp32, though the clip knows it
    for a, b in zip(big, c):
        r = a.double().cpu() / ref
        assert ((b.double().cpu() - r).abs() <= (HALF[a.dtype] + 2.0 ** -40) * r.abs()).all()
    for bad in (float("nan"), float("inf")):
        g = [rnd((100,), 1), rnd((50,), 2, 1.0, F32)]
        g[1][7] = bad
        c = [t.clone() for t in g]
        n = M.clip_grad_norm(c, 0.1)
        assert not torch.isfinite(n)
        assert torch.equal(c[0], g[0]) and torch.equal(c[1][:7], g[1][:7]) and torch.equal(c[1][8:], g[1][8:])
    z = [torch.zeros(100, device="cuda")]
    assert float(M.clip_grad_norm(z, 0.0)) == 0 and (z[0] == 0).all()
    one = [torch.ones(100, device="cuda")]
    M.clip_grad_norm(one, 0.0)
    assert (one[0] == 0).all()


# ----------------------------------------------------------------------------
# together, captured, on other streams
# ----------------------------------------------------------------------------

def training_step(x, w_up, w_down, o, dy):
    """relu^2 experts forward and backward with the operators, gradients clipped to norm 1."""
    a = M.grouped_matmul(x, w_up, o)
    h = torch.relu(a).square()
    y = M.grouped_matmul(h, w_down, o)
    dh, d_down = M.grouped_matmul_grad(dy, h, w_down, o, dw_dtype=F32)
    da = (dh.float() * 2 * torch.relu(a).float()).to(BF)
    dx, d_up = M.grouped_matmul_grad(da, x, w_up, o)
    norm = M.clip_grad_norm([d_up, d_down], 1.0)
    return y, dx, d_up, d_down, norm


def test_a_training_step_of_the_experts():
    """Routed and permuted by the framework, through both products and back, clipped: against autograd in 64 bits."""
    d = device_inputs("tiny")
    cfg = d["cfg"]
    idx, _, _ = M.route(d["x"], d["w_router"], d["corr_bias"], cfg.K, cfg.routed_scaling)
    z = rnd((cfg.T, cfg.L), 70)
    o, row_token, _, x = M.permute(idx, cfg.E, z)
    dy = rnd((x.shape[0], cfg.L), 71)
    y, dx, d_up, d_down, norm = training_step(x, d["w_up"], d["w_down"], o, dy)
    X = x.double().cpu().requires_grad_()
    U, D = d["w_up"].double().cpu().requires_grad_(), d["w_down"].double().cpu().requires_grad_()
    out = torch.cat([(torch.relu(X[a:b] @ U[e].t()) ** 2) @ D[e].t() for e, (a, b) in enumerate(ranges(o, x.shape[0]))])
    out.backward(dy.double().cpu())
    n = float(torch.sqrt((U.grad ** 2).sum() + (D.grad ** 2).sum()))
    # a, h, y or dh, da and the gradient are each rounded to bf16 (2^-8 of a value, relu^2 doubling a's):
    # at most 6 half steps of the largest value, whatever cancels inside the sums
    rel = lambda g, r: float((g.double().cpu() - r).abs().max() / r.abs().max())
    assert rel(y, out.detach()) <= 6 * 2.0 ** -8 and rel(dx, X.grad) <= 6 * 2.0 ** -8
    assert abs(float(norm) / n - 1) <= 6 * 2.0 ** -8
    assert rel(d_up, U.grad / n) <= 6 * 2.0 ** -8 and rel(d_down, D.grad / n) <= 6 * 2.0 ** -8


def test_the_products_repeat_the_forward():
    """grouped_matmul on the forward's own latent rows and offsets gives its stored y."""
    d = device_inputs("tiny", T=300)
    cfg = d["cfg"]
    w = {k: d[k] for k in ("w_router", "corr_bias", "w_fc1", "w_up", "w_down", "w_fc2", "w_sh_up", "w_sh_down")}
    dims = M.dims_from(d["x"], w, cfg.K, cfg.routed_scaling)
    ws = torch.zeros(M.workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    M.forward(d["x"], w, cfg.K, cfg.routed_scaling, ws=ws)
    lay = M.workspace_layout(dims)
    part = lambda k, n, dt: ws[lay[k]: lay[k] + n * torch.empty(0, dtype=dt).element_size()].view(dt)
    TK = cfg.T * cfg.K
    o = part("offsets", cfg.E + 1, torch.int32)
    h, y = part("h", TK * cfg.I, BF).view(TK, cfg.I), part("y", TK * cfg.L, BF).view(TK, cfg.L)
    got = M.grouped_matmul(h, w["w_down"], o)
    ref, s = ref_product(h, w["w_down"], ranges(o, TK))
    check(got, ref, s, cfg.I, BF)
    check(y, ref, s, cfg.I, BF)


@pytest.mark.parametrize("kind", ["train", "fp8"])
def test_captured_calls_replay(kind):
    R, E, N, K, counts = 700, 6, 264, 200, [300, 0, 17, 250, 63, 70]
    x, wu, wd, dy, o = rnd((R, K), 1), rnd((E, N, K), 2, 0.1), rnd((E, K, N), 3, 0.1), rnd((R, K), 4), offs(counts)
    x8, o8 = rnd((R, 272), 5), offs(counts)
    wq, sw = M.quantize_fp8_blocks(rnd((E, N, 272), 6, 0.1))
    run = (lambda: training_step(x, wu, wd, o, dy)) if kind == "train" else (lambda: (M.grouped_matmul_fp8(x8, wq, sw, o8),))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    with torch.cuda.graph(g2):
        out2 = run()
    log(f"[operators] captured {kind}")
    for rep in range(3):
        for t in (x, x8, dy):
            t.copy_(rnd(t.shape, 100 * rep + t.shape[1]))
        o.copy_(offs([[300, 0, 17, 250, 63, 70], [0, 0, 700, 0, 0, 0], [1, 2, 3, 4, 5, 6]][rep]))
        o8.copy_(o)
        eager = [t.clone() for t in run()]
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(eager, out, out2):
            assert torch.equal(a, b) and torch.equal(a, c), f"replay {rep}"


def test_other_streams():
    """Calls in flight on two streams at once, each given the stream, give the single call's bits."""
    R, E, N, K, counts = 900, 8, 520, 328, [113] * 7 + [109]
    x, w, dy, o = rnd((R, K), 1), rnd((E, N, K), 2, 0.1), rnd((R, N), 3), offs(counts)
    grads = [rnd((300_001,), 4), rnd((70_000,), 5, 1.0, F32)]
    want = (M.grouped_matmul(x, w, o), *M.grouped_matmul_grad(dy, x, w, o), M.grad_norm(grads))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for rep in range(5):
        for s in streams:
            outs.append((M.grouped_matmul(x, w, o, stream=s), *M.grouped_matmul_grad(dy, x, w, o, stream=s),
                         M.grad_norm(grads, stream=s)))
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("R,E,N,K", [(300, 5, 136, 80), (1000, 200, 520, 80), (5000, 3, 136, 80), (70, 3, 1600, 2064)])
def test_workspace_of_the_caller(R, E, N, K):
    """Calls without a table, with one, and with the pieces of a split gradient, in a workspace full of junk."""
    x, w, dy = rnd((R, K), 1), rnd((E, N, K), 2), rnd((R, N), 3)
    o = offs(np.random.default_rng(4).multinomial(R, np.ones(E) / E))
    wq, sw = M.quantize_fp8_blocks(w)
    calls = (lambda ws: (M.grouped_matmul(x, w, o, ws=ws),), lambda ws: M.grouped_matmul_grad(dy, x, w, o, ws=ws),
             lambda ws: (M.grouped_matmul_fp8(x, wq, sw, o, ws=ws),))
    for call in calls:
        ws = torch.full((M.grouped_workspace_bytes(R, E, N, K) + 256,), 255, dtype=torch.uint8, device="cuda")
        for a, b in zip(call(ws[:-256]), call(None)):
            assert torch.equal(a, b)
        assert (ws[-256:] == 255).all()
    with pytest.raises(M.MoEError):
        M.grouped_matmul_fp8(x, wq, sw, o, ws=ws[:256])
    with pytest.raises(M.MoEError):
        M.grouped_matmul_fp8(x, wq, sw, o, ws=ws[1:])


def ragged(R, E, seed, holes=0):
    rng = np.random.default_rng(seed)
    p = rng.random(E)
    p[rng.permutation(E)[:holes]] = 0
    return rng.multinomial(R, p / p.sum()).tolist()


# every kind of plan: with a tile table (E > 128), big tiles with short last ones, four stages, split gradients
PLANS = [
    (2000, 200, 136, 80, ragged(2000, 200, 1, 60)),
    (9000, 40, 1032, 272, ragged(9000, 40, 2, 4)),
    (13000, 12, 1032, 528, [64, 1, 128, 129, 192, 193, 256, 257, 0, 5000, 3000, 3780]),
    (6000, 3, 136, 272, [0, 5999, 1]),
    (5000, 128, 8, 16, ragged(5000, 128, 3, 50)),
    (1500, 1, 200, 336, [1500]),
    (40000, 2, 264, 144, [33000, 7000]),
    (30000, 7, 520, 2064, ragged(30000, 7, 4)),
    (3, 14, 72, 5072, [0] * 4 + [1] + [0] * 5 + [2] + [0] * 3),
    (538, 2, 1816, 3808, [500, 38]),
    (900, 300, 72, 1552, ragged(900, 300, 5, 100)),
    (400, 1024, 40, 80, ragged(400, 1024, 6, 700)),
    (2000, 200, 1032, 80, ragged(2000, 200, 7, 60)),
    (60000, 150, 1032, 64, ragged(60000, 150, 8, 20)),
    (30000, 2, 136, 64, [29999, 1]),
    (1000, 100, 520, 1040, ragged(1000, 100, 9, 40)),
    (8100, 4, 1832, 144, [4000, 100, 3000, 1000]),             # 264 tiles of 256 x 256: the last 8 in quarters
    (8700, 4, 1832, 144, [4000, 200, 3300, 1200]),             # 280: the last 24 in halves
    (8100, 4, 144, 1840, [4000, 100, 3000, 1000]),
    (8700, 8, 1800, 1840, [4000, 200, 0, 3200, 100, 0, 1200, 0]),   # both gradients in one launch, with parts
    (33000, 140, 512, 528, ragged(33000, 140, 10, 20)),        # the same with a tile table
    (1000, 8, 2048, 256, ragged(1000, 8, 11, 1)),              # one launch: a split dx beside dW
    (2008, 3, 3032, 304, [1500, 0, 508]),                      # and both split
    (230, 4, 1824, 2096, [60, 100, 0, 70]),                    # dW in small tiles for it
    (300, 100, 72, 2064, [33, 0, 64, 32, 31, 1] + [2] * 69 + [1] + [0] * 24),
]


@pytest.mark.parametrize("R,E,N,K,counts", PLANS)
def test_every_plan(R, E, N, K, counts):
    """The larger plans, against 64-bit sums on the GPU."""
    x, w, dy, o = rnd((R, K), 3), rnd((E, N, K), 4, K ** -0.5), rnd((R, N), 5), offs(counts)
    X, Wt, G = x.double(), w.double(), dy.double()
    y = M.grouped_matmul(x, w, o)
    dx, dw = M.grouped_matmul_grad(dy, x, w, o, dw_dtype=F32)
    dwb = M.grouped_matmul_grad(dy, x, w, o, need_dx=False)[1]
    wq, sw = M.quantize_fp8_blocks(w)
    y8 = M.grouped_matmul_fp8(x, wq, sw, o)
    q, sx = M.quantize_fp8_rows(x)                            # (pinned against the definition above)
    XV = q.view(torch.float8_e4m3fn).double() * sx.double().t().repeat_interleave(128, 1)[:, :K]
    for e, (a, b) in enumerate(ranges(o, R)):
        ops = lambda u, v: ((u @ v).cpu(), (u.abs() @ v.abs()).cpu())
        ref, s = ops(G[a:b].t().contiguous(), X[a:b])
        check(dw[e], ref, s, b - a, F32)
        check(dwb[e], ref, s, b - a, BF)
        if a == b:
            continue
        check(y[a:b], *ops(X[a:b], Wt[e].t().contiguous()), K, BF)
        check(dx[a:b], *ops(G[a:b], Wt[e]), N, BF)
        wv = wq[e].view(torch.float8_e4m3fn).double() * sw[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        ref, s = ops(XV[a:b], wv.t().contiguous())
        loss = 7 * 2.0 ** -13 * (XV[a:b].abs().view(b - a, K // 8, 8).amax(2) @ wv.abs().view(N, K // 8, 8).amax(2).t())
        check(y8[a:b], ref, s, K + 2 * ((K + 127) // 128), BF, loss.cpu())
    # added to itself: fp32 sums double exactly, bf16 ones too (the sum, once rounded, plus the same fp32 sum
    # is within a step of twice it)
    keep, keepb = dw.clone(), dwb.clone()
    M.grouped_matmul_grad(dy, x, w, o, need_dx=False, dw=dw, accumulate=True)
    M.grouped_matmul_grad(dy, x, w, o, need_dx=False, dw=dwb, accumulate=True)
    assert torch.equal(dw, 2 * keep)
    joint = keep.clone()                                       # and beside dx
    dx2, _ = M.grouped_matmul_grad(dy, x, w, o, dw=joint, accumulate=True)
    assert torch.equal(dx2, dx) and torch.equal(joint, 2 * keep)
    assert ((dwb.double() - 2 * keepb.double()).abs() <= 2.0 ** -7 * 2 * keepb.double().abs()).all()

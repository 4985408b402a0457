"""What is measured of the expert operators, and their plain forms.

Four operators over rows that are grouped by expert (``offsets`` [E+1] int32:
the rows of expert e are ``offsets[e] .. offsets[e+1]``):

* ``product``   y[r] = x[r] . W[e]^T, bf16;
* ``gradient``  dx[r] = dy[r] . W[e] (bf16) and dW[e] = dy_e^T . x_e (fp32 or bf16);
* ``product8``  the product on E4M3 weights with one fp32 scale per 128 x 128
  block, the rows quantised on the way (E4M3, a power-of-two scale per 128);
* ``clip``      the global norm of many gradient tensors, and the tensors scaled to it.

``own`` false: plain torch operations in 32 bits, rounded once at the end.
``own`` true: the calls of ``sparse_moe_layer_correction_amd``.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def _product(kind, R, E, N, K, spread, **more):
    return dict(op=kind, R=R, E=E, N=N, K=K, spread=spread, **more)


def listed():
    return [
        # the tiny layer's expert up product, 64 tokens of top-4: launch latency
        dict(name="product_tiny", **_product("product", 256, 16, 128, 64, "even")),
        # a 64-token decode step of the 512-expert layer (top-22): weights stream once, 2-3 rows an expert
        dict(name="product_decode", **_product("product", 1408, 512, 5120, 2048, "even")),
        # its 16384-token prefill: about 700 rows an expert
        dict(name="product_prefill", **_product("product", 360448, 512, 5120, 2048, "even")),
        # a micro-batch of a small layer, experts without rows among them, sizes off every tile
        dict(name="gradient_odd", **_product("gradient", 1237, 24, 712, 328, "holes", dw="bf16")),
        # few wide experts with many rows each (a short long-axis sum for dx, a long one for dW), skewed
        dict(name="gradient_skew", **_product("gradient", 16384, 8, 2048, 1024, "skew", dw="fp32")),
        # the expert down product of the 128-expert layer, 4096 tokens of top-8, gradients kept in fp32
        dict(name="gradient_nano", **_product("gradient", 32768, 128, 2048, 5120, "even", dw="fp32")),
        # one token through 512 experts (22 rows): the single-token form in 8 bits
        dict(name="product8_decode", **_product("product8", 22, 512, 5120, 2048, "even")),
        # a ragged batch with sizes that end inside scale blocks
        dict(name="product8_odd", **_product("product8", 3001, 20, 1000, 1360, "holes")),
        # 8192 tokens of top-8 over 128 experts with hot and cold experts
        dict(name="product8_super", **_product("product8", 65536, 128, 5120, 2048, "skew")),
        # the weight gradients of the tiny layer: eight small tensors
        dict(name="clip_tiny", op="clip", count=8, largest=1 << 17, smallest=16, mix="bf16", ratio=0.25),
        # a model's worth of tensors, norms' vectors among matrices, in two types
        dict(name="clip_many", op="clip", count=320, largest=20_000_003, smallest=255, mix="both", ratio=0.5),
        # few tensors of expert size, fp32 gradients
        dict(name="clip_experts", op="clip", count=6, largest=700_000_000, smallest=100_000_000, mix="fp32", ratio=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "gradient", "product8", "clip"])
    if op == "clip":
        largest = _log(rng, 1 << 12, 50_000_000)
        return dict(op=op, count=_log(rng, 1, 400), largest=largest, smallest=_log(rng, 1, largest),
                    mix=rng.choice(["bf16", "fp32", "both"]), ratio=rng.choice([0.1, 0.5, 2.0]))
    E = _log(rng, 1, 512)
    R = _log(rng, 1, 100_000)
    step = 16 if op == "product8" else 8
    N = max(1, _log(rng, 64, 6000) // 8) * 8
    K = max(1, _log(rng, 64, 6000) // step) * step
    while E * N * K > 2_000_000_000:                 # keeps a drawn case within the listed ones
        E = max(1, E // 2)
    while R * N * K > 1_000_000_000_000:
        R = max(1, R // 2)
    case = _product(op, R, E, N, K, rng.choice(["even", "skew", "holes"]))
    if op == "gradient":
        case["dw"] = rng.choice(["bf16", "fp32"])
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _counts(case, seed):
    """Rows of each expert: a multinomial draw, even, Zipf(1.1) or with a third of the experts empty."""
    E, R = case["E"], case["R"]
    rng = np.random.default_rng([seed, 7])
    p = np.ones(E)
    if case["spread"] == "skew":
        p = (rng.permutation(E) + 1.0) ** -1.1
    elif case["spread"] == "holes" and E > 2:
        p[rng.permutation(E)[: E // 3]] = 0.0
    return rng.multinomial(R, p / p.sum()).tolist()


def _sizes(case):
    """Elements of each gradient tensor: the largest one, the rest spread over the range's logarithm."""
    rng = np.random.default_rng([case["count"], case["largest"], case["smallest"]])
    lo, hi = math.log(case["smallest"]), math.log(max(case["largest"], case["smallest"]))
    sizes = [int(round(math.exp(v))) for v in rng.uniform(lo, hi, case["count"])]
    sizes[0] = case["largest"]
    return sizes


def _mix(case):
    """The type of each gradient tensor."""
    return [case["mix"] if case["mix"] != "both" else ("bf16", "fp32")[i % 2] for i in range(case["count"])]


def _bucketed(case):
    """Zeroed flat buckets, one for each type, and the gradient tensors as views of them, each at a multiple of 16
    elements: as a trainer that reduces its gradients in buckets holds them."""
    sizes, mix = _sizes(case), _mix(case)
    total = {k: sum((n + 15) // 16 * 16 for n, m in zip(sizes, mix) if m == k) for k in sorted(set(mix))}
    buckets = {k: torch.zeros(n, dtype=_DT[k], device="cuda") for k, n in total.items()}
    at, views = dict.fromkeys(buckets, 0), []
    for n, k in zip(sizes, mix):
        views.append(buckets[k][at[k]:at[k] + n])
        at[k] += (n + 15) // 16 * 16
    return list(buckets.values()), views


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    if case["op"] == "clip":
        buckets, grads = _bucketed(case)
        for i, t in enumerate(grads):
            t.normal_(0.0, 10.0 ** ((i % 5) - 4), generator=g)
        # the bound as a share of the norm these gradients have
        total = math.sqrt(sum(t.numel() * 10.0 ** (2 * ((i % 5) - 4)) for i, t in enumerate(grads)))
        return dict(buckets=buckets, grads=grads, max_norm=case["ratio"] * total)
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    counts = _counts(case, seed)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    s = dict(counts=counts, offsets=offsets, x=normal((R, K), 1.0, torch.bfloat16))
    if case["op"] == "product8":
        codes = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
        for e in range(E):                           # values of a block fill the type's range
            codes[e] = normal((N, K), 90.0, torch.float32).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        nb, kb = (N + 127) // 128, (K + 127) // 128
        scale = torch.empty((E, nb, kb), device="cuda").uniform_(0.5, 2.0, generator=g) / (90.0 * math.sqrt(K))
        s.update(codes=codes, scale=scale)
    else:
        s["w"] = normal((E, N, K), 1.0 / math.sqrt(K), torch.bfloat16)
        if case["op"] == "gradient":
            s["dy"] = normal((R, N), 1.0, torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "clip":
        s["out_buckets"], s["out"] = _bucketed(case)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _ranges(counts):
    r0 = 0
    for e, n in enumerate(counts):
        if n:
            yield e, slice(r0, r0 + n)
        r0 += n


def _plain_product(s):
    x, w = s["x"], s["w"]
    y = torch.empty(x.shape[0], w.shape[1], dtype=torch.bfloat16, device=x.device)
    for e, r in _ranges(s["counts"]):
        y[r] = (x[r].float() @ w[e].float().t()).to(torch.bfloat16)
    return y


def _plain_gradient(s):
    x, w, dy, dt = s["x"], s["w"], s["dy"], _DT[s["case"]["dw"]]
    dx = torch.empty_like(x)
    dw = torch.zeros(w.shape, dtype=dt, device=x.device)
    for e, r in _ranges(s["counts"]):
        g = dy[r].float()
        dx[r] = (g @ w[e].float()).to(torch.bfloat16)
        dw[e] = (g.t() @ x[r].float()).to(dt)
    return dx, dw


def _plain_product8(s):
    x, codes, scale = s["x"], s["codes"], s["scale"]
    R, K = x.shape
    E, N, _ = codes.shape
    kb = (K + 127) // 128
    xb = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(R, kb, 128)
    amax = xb.abs().amax(2, keepdim=True)
    mant, ex = torch.frexp(amax)                     # amax = mant * 2^ex, mant in [0.5, 1)
    ex = torch.where(mant > 0.875, ex - 8, ex - 9).clamp(min=-126)   # the least with amax <= 448 * 2^ex
    ex = torch.where(amax == 0, torch.full_like(ex, -126), ex)
    q = torch.ldexp(xb, -ex).to(torch.float8_e4m3fn).float()
    xq = torch.ldexp(q, ex).view(R, kb * 128)[:, :K]
    y = torch.empty(R, N, dtype=torch.bfloat16, device=x.device)
    for e, r in _ranges(s["counts"]):
        sw = scale[e].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        y[r] = (xq[r] @ (codes[e].view(torch.float8_e4m3fn).float() * sw).t()).to(torch.bfloat16)
    return y


def _plain_clip(s):
    total = torch.zeros((), device="cuda")
    for t in s["grads"]:
        v = t.float()
        total = total + (v * v).sum()
    norm = total.sqrt()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm))
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * coef)
    return [norm] + s["out_buckets"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"product": _plain_product, "gradient": _plain_gradient, "product8": _plain_product8,
                "clip": _plain_clip}[op](state)
    import sparse_moe_layer_correction_amd as M
    if op == "product":
        return M.grouped_matmul(state["x"], state["w"], state["offsets"])
    if op == "gradient":
        return M.grouped_matmul_grad(state["dy"], state["x"], state["w"], state["offsets"],
                                     dw_dtype=_DT[state["case"]["dw"]])
    if op == "product8":
        return M.grouped_matmul_fp8(state["x"], state["codes"], state["scale"], state["offsets"])
    norm = M.clip_grad_norm(state["grads"], state["max_norm"], out=state["out"])
    return [norm] + state["out_buckets"]


# ----------------------------------------------------------------------------
# work and exact values
# ----------------------------------------------------------------------------

def work(case):
    if case["op"] == "clip":
        sizes = _sizes(case)
        size = {"bf16": 2, "fp32": 4}
        return {"bytes": 2 * sum(n * size[m] for n, m in zip(sizes, _mix(case))), "flops": 3 * sum(sizes)}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    # experts that get rows: each of E boxes, R balls
    live = E - (E // 3 if case["spread"] == "holes" and E > 2 else 0)
    hit = live * (1.0 - (1.0 - 1.0 / live) ** R)
    if case["op"] == "product":
        return {"bytes": int(2 * (R * K + R * N + hit * N * K)), "flops": 2 * R * N * K}
    if case["op"] == "product8":
        return {"bytes": int(2 * (R * K + R * N) + hit * N * K), "flops": 2 * R * N * K}
    size = 2 if case["dw"] == "bf16" else 4
    return {"bytes": int(2 * (2 * R * K + R * N + hit * N * K) + size * E * N * K), "flops": 4 * R * N * K}


def _round_e4m3(v):
    """float64 values of magnitude at most 448 to the nearest E4M3 value, ties to even."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (ex - 4).clamp(min=-9))    # three fraction bits, 2^-9 below 2^-6
    return torch.round(v / step) * step


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "clip":
        sq = 0.0
        for t in s["grads"]:
            for part in t.split(1 << 26):
                sq += float(part.double().pow(2).sum())
        norm = math.sqrt(sq)
        f = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
        return [torch.tensor(norm, dtype=torch.float64)] + [t.double() * f for t in s["buckets"]]
    x, counts = s["x"], s["counts"]
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(int).tolist()
    E, N, K = case["E"], case["N"], case["K"]
    rows = [(e, starts[e], starts[e + 1]) for e in range(E) if counts[e]]
    f64 = dict(dtype=torch.float64, device=x.device)
    if case["op"] == "gradient":
        dx, dw = torch.zeros(x.shape, **f64), torch.zeros((E, N, K), **f64)
        for e, a, b in rows:
            dx[a:b] = torch.mm(s["dy"][a:b].double(), s["w"][e].double())
            dw[e] = torch.mm(s["dy"][a:b].double().t().contiguous(), x[a:b].double())
        return dx, dw
    y = torch.zeros((x.shape[0], N), **f64)
    for e, a, b in rows:
        xe = x[a:b].double()
        if case["op"] == "product":
            y[a:b] = torch.mm(xe, s["w"][e].double().t().contiguous())
            continue
        we = s["codes"][e].view(torch.float8_e4m3fn).double()
        for i in range(0, K, 128):
            blk = xe[:, i:i + 128]
            top = blk.abs().amax(1, keepdim=True)
            # the least power of two 2^p with top / 2^p <= 448, not below 2^-126
            p = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)
            p = torch.where(top > 448.0 * torch.exp2(p), p + 1, p)
            p = torch.where((top <= 448.0 * torch.exp2(p - 1)) & (p > -126), p - 1, p)
            unit = torch.exp2(p)
            part = torch.mm(_round_e4m3(blk / unit), we[:, i:i + 128].t().contiguous()) * unit
            y[a:b] += part * s["scale"][e, :, i // 128].double().repeat_interleave(128)[:N]
    return y

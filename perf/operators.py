"""The 8-bit linear-layer operators as measured cases: the residual's addition
with the root-mean-square norm and an 8-bit output (``rmsquant``), its gradient
(``rmsgrad``), quantising a matrix and reading it back (``quant``, ``dequant``)
and the product of 8-bit matrices with scales (``gemmq``).

Tensors here are row-major with one token (or one output channel) a row, which
is the library's column-major storage with one token a column: m is the length
of a row (or the number of output channels of a product), n the number of
tokens, k a product's depth.  ``pad`` is what the leading dimensions have above
the row's length.  Types: 's' float, 'h' half, 'b' bfloat16.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"s": torch.float32, "h": torch.float16, "b": torch.bfloat16}
BYTES = {"s": 4, "h": 2, "b": 2}


def listed():
    return [
        # one token of a serving step: nothing but latency
        dict(name="rmsquant one token", op="rmsquant", type="b", m=4096, n=1, pad=0),
        # a ragged batch whose odd row length leaves no row after the first aligned
        dict(name="rmsquant ragged", op="rmsquant", type="s", m=4099, n=509, pad=0),
        # the norm before a layer over a long prompt or a training batch
        dict(name="rmsquant prompt", op="rmsquant", type="b", m=8192, n=16384, pad=0),
        # a small training batch, odd sizes, padded rows
        dict(name="rmsgrad ragged", op="rmsgrad", type="h", m=1543, n=257, pad=5),
        # a training batch
        dict(name="rmsgrad batch", op="rmsgrad", type="b", m=4096, n=16384, pad=0),
        # one vector quantised on its own and read back
        dict(name="quant one vector", op="quant", type="b", m=8192, n=1, pad=0),
        # a weight matrix made 8-bit, and read back for training
        dict(name="quant weights", op="quant", type="b", m=8192, n=8192, pad=0),
        # a serving step for one token: a matrix-vector product over weights that fit L2
        dict(name="gemmq one token", op="gemmq", type="b", m=4096, n=1, k=4096, pad=0),
        # the same over a matrix far larger than L2 (an output layer): HBM alone
        dict(name="gemmq one token, large", op="gemmq", type="b", m=32768, n=1, k=8192, pad=0),
        # a serving step for a ragged batch of requests
        dict(name="gemmq batch", op="gemmq", type="h", m=8192, n=37, k=4096, pad=0),
        # a short prompt with odd sizes: no row but the first is aligned
        dict(name="gemmq ragged", op="gemmq", type="s", m=2111, n=509, k=1543, pad=0),
        # a long prompt: arithmetic alone
        dict(name="gemmq prompt", op="gemmq", type="b", m=8192, n=8192, k=8192, pad=0),
    ]


def _length(rng, lo, hi):
    """A length between lo and hi, even over its logarithm; half of them multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v > 64:
        v -= v % 64
    if v == 3072:
        v += 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["rmsquant", "rmsgrad", "quant", "gemmq", "gemmq"])
    kind = rng.choice("shb")
    pad = rng.choice([0, 0, 1, 16])
    while True:
        if op == "gemmq":
            m, n, k = _length(rng, 64, 32768), _length(rng, 1, 8192), _length(rng, 64, 16384)
            if m * n * k <= 8192 ** 3 and m * k <= 8192 * 32768 and m * n <= 8192 * 8192:
                return dict(op=op, type=kind, m=m, n=n, k=k, pad=pad)
        else:
            m, n = _length(rng, 64, 32768), _length(rng, 1, 16384)
            most = {"rmsquant": 8192 * 16384, "rmsgrad": 4096 * 16384, "quant": 8192 * 8192}[op]
            if m * n * BYTES[kind] <= 2 * most:
                return dict(op=op, type=kind, m=m, n=n, pad=pad)


def _rows(g, n, m, pad, dtype, scale=1.0, outliers=False):
    """n rows of m normal values, m + pad apart; outliers: a few columns are
    much larger than the others, as a model's residual stream has them."""
    t = torch.empty((n, m + pad), dtype=dtype, device="cuda")
    gain = torch.full((m,), scale, device="cuda")
    if outliers:
        gain[torch.rand((m,), generator=g, device="cuda") < 0.01] *= 12.0
    step = max(1, (1 << 26) // (m + pad))
    for i in range(0, n, step):
        r = min(step, n - i)
        t[i:i + r, :m] = torch.randn((r, m), generator=g, device="cuda") * gain
        t[i:i + r, m:] = 0
    return t


def _eight_bit(g, n, m, pad, scale):
    """n rows of m 8-bit values, m + pad apart, and a scale a row."""
    q = torch.zeros((n, m + pad), dtype=torch.int8, device="cuda")
    s = torch.empty((n,), device="cuda")
    step = max(1, (1 << 26) // m)
    for i in range(0, n, step):
        r = min(step, n - i)
        x = torch.randn((r, m), generator=g, device="cuda") * scale
        s[i:i + r] = x.abs().amax(1) / 127.0
        q[i:i + r, :m] = torch.round(x / s[i:i + r, None]).to(torch.int8)
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, kind, m, n, pad = case["op"], case["type"], case["m"], case["n"], case["pad"]
    dtype = DTYPES[kind]
    # what 8-bit values are read back as: of 16 bits, as training takes them
    back = "b" if kind == "b" else "h"
    st = dict(op=op, kind=kind, back=back, m=m, n=n, pad=pad)

    def new(rows, cols, dt):
        return torch.zeros((rows, cols), dtype=dt, device="cuda")

    if op == "gemmq":
        k = case["k"]
        st["k"] = k
        st["w"], st["sw"] = _eight_bit(g, m, k, pad, 0.02)
        st["x"], st["sx"] = _eight_bit(g, n, k, pad, 1.0)
        st["y"] = new(n, m + pad, dtype)
        return st
    if op == "quant":
        st["x"] = _rows(g, n, m, pad, dtype, 0.02)
    else:
        st["g"] = (1.0 + 0.1 * torch.randn((m,), generator=g, device="cuda")).to(dtype)
    if op == "rmsquant":
        st["x"] = _rows(g, n, m, pad, dtype, 0.5)
        st["r"] = _rows(g, n, m, pad, dtype, 1.0, outliers=True)
        st["h"] = new(n, m + pad, dtype)
    if op == "rmsgrad":
        st["h"] = _rows(g, n, m, pad, dtype, 1.0, outliers=True)
        st["rstd"] = torch.rsqrt(st["h"][:, :m].float().square().mean(1) + EPS)
        st["dy"] = _rows(g, n, m, pad, dtype, 0.1)
        st["dr"] = _rows(g, n, m, pad, dtype, 0.1)
        st["dx"] = new(n, m + pad, dtype)
        st["dg"] = torch.zeros((m,), device="cuda")
    else:
        st["q"] = new(n, m + pad, torch.int8)
        st["s"] = torch.zeros((n,), device="cuda")
        st["rstd"] = torch.zeros((n,), device="cuda")
        st["v"] = new(n, m + pad, DTYPES[back])
    return st


def _outputs(st):
    """The outputs of the library's calls: the state's buffers without their padding."""
    m, op = st["m"], st["op"]
    if op == "gemmq":
        return {"y": st["y"][:, :m]}
    if op == "rmsgrad":
        return {"dx": st["dx"][:, :m], "dg": st["dg"]}
    out = {"v": st["v"][:, :m], "s": st["s"]}
    if op == "rmsquant":
        out.update(h=st["h"][:, :m], rstd=st["rstd"])
    return out


def _run_own(st):
    import symmetric_matrix_vector_gb300 as xs

    op, kind, m, n = st["op"], st["kind"], st["m"], st["n"]
    ld = m + st["pad"]
    if op == "gemmq":
        k = st["k"]
        ldk = k + st["pad"]
        xs.check(xs.gemmq(kind, m, n, k, 1.0, st["w"], ldk, st["sw"], st["x"], ldk, st["sx"], 0.0,
                          st["y"], ld))
    elif op == "rmsgrad":
        xs.check(xs.rmsgrad(kind, m, n, st["dy"], ld, st["h"], ld, st["g"], st["rstd"], st["dr"],
                            ld, st["dx"], ld, st["dg"]))
    else:
        if op == "rmsquant":
            xs.check(xs.rmsquant(kind, m, n, st["x"], ld, st["r"], ld, st["g"], EPS, st["h"], ld,
                                 st["q"], ld, st["s"], st["rstd"]))
        else:
            xs.check(xs.quant(kind, m, n, st["x"], ld, st["q"], ld, st["s"]))
        # 8-bit values come back as the values they stand for
        xs.check(xs.dequant(st["back"], m, n, st["q"], ld, st["s"], st["v"], ld))
    return _outputs(st)


def _quantised(y, back):
    """Rows of 32-bit values as their 8-bit values' values, and the scales."""
    s = y.abs().amax(1) / 127.0
    q = torch.where(s[:, None] > 0, torch.round(y / s[:, None]), torch.zeros_like(y))
    return (q * s[:, None]).to(DTYPES[back]), s


def _run_plain(st):
    op, m = st["op"], st["m"]
    dtype = DTYPES[st["kind"]]
    if op == "gemmq":
        k = st["k"]
        y = st["x"][:, :k].float() @ st["w"][:, :k].float().T
        return {"y": (y * st["sx"][:, None] * st["sw"][None, :]).to(dtype)}
    if op == "quant":
        v, s = _quantised(st["x"][:, :m].float(), st["back"])
        return {"v": v, "s": s}
    if op == "rmsquant":
        h = (st["x"][:, :m].float() + st["r"][:, :m].float()).to(dtype)
        hf = h.float()
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        v, s = _quantised(hf * rstd[:, None] * st["g"].float(), st["back"])
        return {"v": v, "s": s, "h": h, "rstd": rstd}
    h, dy, rstd = st["h"][:, :m].float(), st["dy"][:, :m].float(), st["rstd"]
    dyg = dy * st["g"].float()
    c = rstd.square() * (dyg * h).mean(1)
    dx = st["dr"][:, :m].float() + rstd[:, None] * (dyg - h * c[:, None])
    return {"dx": dx.to(dtype), "dg": (dy * h * rstd[:, None]).sum(0)}


def run(st):
    return _run_own(st) if own else _run_plain(st)


def work(case):
    op, m, n, b = case["op"], case["m"], case["n"], BYTES[case["type"]]
    if op == "gemmq":
        k = case["k"]
        return {"bytes": k * (m + n) + m * n * b + 4 * (m + n), "flops": 2 * m * n * k}
    if op == "rmsgrad":  # dy, h, dr in, dx out; g in, dg out; rstd in
        return {"bytes": 4 * m * n * b + m * b + 4 * m + 4 * n, "flops": 11 * m * n}
    # the 8-bit values out and in again, and what they are read back as out
    bytes_ = m * n * (b + 1) + m * n * (1 + 2) + 8 * n
    if op == "rmsquant":  # r in and h out as well; g in; rstd out
        bytes_ += 2 * m * n * b + m * b + 4 * n
    return {"bytes": bytes_, "flops": (9 if op == "rmsquant" else 4) * m * n}


def exact(case, seed):
    st = prepare(case, seed)
    op, m = case["op"], case["m"]

    def wide(name, cols=m):
        return st[name][..., :cols].to(torch.float64)

    if op == "gemmq":
        k = case["k"]
        y = torch.matmul(wide("x", k), wide("w", k).t())
        y.mul_(st["sx"].double().unsqueeze(1)).mul_(st["sw"].double())
        return {"y": y}
    if op == "rmsgrad":
        # the gradient of sum(dy * norm(h)) + sum(dr * h), from the norm's quotient:
        # with u = h / |h|_eps, d(u_i)/d(h_j) = (delta_ij - u_i u_j / m) / |h|_eps
        size = 1.0 / st["rstd"].double().unsqueeze(1)
        u = wide("h") / size
        dy = wide("dy")
        a = dy * st["g"].double()
        dx = (a - u * torch.mean(a * u, dim=1, keepdim=True)) / size + wide("dr")
        return {"dx": dx, "dg": torch.sum(dy * u, dim=0)}
    out = {}
    if op == "rmsquant":
        total = wide("x") + wide("r")
        # the norm is that of the stored sum
        h = total.to(DTYPES[case["type"]]).double()
        size = torch.sqrt(torch.sum(h * h, dim=1) / m + EPS)
        out.update(h=total, rstd=1.0 / size)
        y = h / size.unsqueeze(1) * st["g"].double()
    else:
        y = wide("x")
    top = torch.amax(torch.abs(y), dim=1)
    steps = torch.round(y * (127.0 / top).unsqueeze(1))
    out.update(v=torch.nan_to_num(steps, nan=0.0) * (top / 127.0).unsqueeze(1), s=top / 127.0)
    return out

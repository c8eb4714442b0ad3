"""GPU parity of the 8-bit row operators (x<quant>, x<dequant>, x<rmsquant>,
x<rmsgrad>) against plain 64-bit implementations: lengths from one element to
beyond what a block holds in registers, odd lengths, padded and unaligned
columns, every type, columns of zeros, infinities, NaN and values whose squares
leave float's range, in-place forms, the gradient against differences."""
import pytest
import torch

import symmetric_matrix_vector_gb300 as xs
from tests import q8_reference as ref
from tests.q8_reference import DTYPES, U32, UNIT, Matrix

pytestmark = pytest.mark.gpu

SIZES = [(1, 1), (2, 3), (7, 5), (31, 2), (64, 1), (128, 130), (257, 3), (1000, 4), (1543, 7),
         (4096, 3), (4099, 3), (8192, 2), (16384, 2), (16400, 2), (20001, 2), (32768, 2),
         (40000, 2), (65537, 1)]
# padding of the leading dimension, elements before the first
LAYOUTS = [(0, 0), (16, 0), (1, 0), (3, 1), (16, 8), (0, 16)]
EPS = 1e-5


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, n, m, kind, scale=1.0):
    return (torch.randn((n, m), generator=g, device="cuda") * scale).to(DTYPES[kind])


def check_quantised(q, s, y64, rel):
    """q and s against the rows of y64 that they quantise, known to a relative
    error `rel`: the scale to that and two roundings, every integer to half a step and what
    the relative errors of value and scale make of 127 steps"""
    steps, s64 = ref.quantised(y64)
    assert bool(((s.double() - s64).abs() <= (rel + 4 * U32) * s64).all())
    assert bool(((q.double() - steps).abs() <= 0.5 + 127 * (2 * rel + 8 * U32)).all())
    assert int(q.abs().max()) == 127


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m,n", SIZES)
def test_quant_and_dequant(kind, m, n):
    g = gen(m + n)
    for pad, off in LAYOUTS:
        x = Matrix(n, m, DTYPES[kind], m + pad, off, normal(g, n, m, kind, 0.03))
        q = Matrix(n, m, torch.int8, m + pad, off)
        s = torch.full((n,), -1.0, device="cuda")
        assert xs.quant(kind, m, n, x.ptr, x.ld, q.ptr, q.ld, s) == 0
        torch.cuda.synchronize()
        check_quantised(q.rows, s, x.rows.double(), 0.0)
        assert q.outside_untouched()
        for back in ("s", "h", "b"):
            v = Matrix(n, m, DTYPES[back], m + pad, off)
            assert xs.dequant(back, m, n, q.ptr, q.ld, s, v.ptr, v.ld) == 0
            torch.cuda.synchronize()
            assert torch.equal(v.rows, (q.rows.float() * s[:, None]).to(DTYPES[back]))
            assert v.outside_untouched()


@pytest.mark.parametrize("kind", ["h", "b"])
def test_quant_rounds_16_bit_values_exactly(kind):
    """127 x / max|x| to the nearest integer, ties to even, in whole numbers: values on
    few bits, where ties are common, and every largest value a half or bfloat16 has"""
    m, n = 600, 256
    g = gen(77)
    x = torch.randint(-255, 256, (n, m), generator=g, device="cuda").to(DTYPES[kind])
    x[:, 0] = torch.arange(n, device="cuda").to(DTYPES[kind])      # some columns' largest
    x[::2] = (x[::2] % 32).to(DTYPES[kind])
    scale = torch.tensor([1.0, 2.0 ** -14, 2.0 ** 7], device="cuda")[torch.arange(n, device="cuda") % 3]
    x = (x.float() * scale[:, None]).to(DTYPES[kind])
    q = torch.empty((n, m), dtype=torch.int8, device="cuda")
    s = torch.empty((n,), device="cuda")
    assert xs.quant(kind, m, n, x, m, q, m, s) == 0
    torch.cuda.synchronize()
    num = torch.round(x.double() / scale.double()[:, None] * 256).long() * 127     # whole
    top = torch.round(x.double().abs().amax(1) / scale.double() * 256).long()[:, None]
    safe = torch.where(top > 0, top, torch.ones_like(top))
    low = torch.div(num, safe, rounding_mode="floor")
    twice = 2 * (num - low * safe)                                 # against one top
    up = (twice > safe) | ((twice == safe) & (low % 2 != 0))
    want = torch.where(top > 0, low + up.long(), torch.zeros_like(low))
    assert torch.equal(q.long(), want)


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_quant_special_columns(kind):
    """zeros, one value, an infinity, a NaN in any place, the type's largest and
    smallest magnitudes"""
    m = 300
    dt = DTYPES[kind]
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    x = torch.zeros((9, m), dtype=dt, device="cuda")
    x[1, 299] = 3.0
    x[2] = normal(gen(1), 1, m, kind)[0]
    x[2, 0] = float("inf")
    x[3] = normal(gen(2), 1, m, kind)[0]
    x[3, 298] = float("nan")
    x[4] = torch.linspace(-1, 1, m, device="cuda") * big
    x[5] = (torch.linspace(-1, 1, m, device="cuda", dtype=torch.float64) * tiny).to(dt)
    x[6] = -big
    x[7] = normal(gen(3), 1, m, kind)[0]
    x[7, 5] = float("-inf")
    x[7, 6] = float("nan")
    x[8] = -0.0
    q = torch.full((9, m), 5, dtype=torch.int8, device="cuda")
    s = torch.full((9,), -1.0, device="cuda")
    assert xs.quant(kind, m, 9, x, m, q, m, s) == 0
    torch.cuda.synchronize()
    for j in (0, 8):
        assert float(s[j]) == 0.0 and not bool(q[j].any())
    assert int(q[1].abs().sum()) == 127 and int(q[1, 299]) == 127
    for j in (2, 3, 7):
        assert bool(torch.isnan(s[j])) and not bool(q[j].any())
    assert bool((q[6] == -127).all())
    check_quantised(q[4:5], s[4:5], x[4:5].double(), 0.0)
    # a scale that is subnormal is itself rounded to a multiple of 2^-149
    steps, s64 = ref.quantised(x[5:6].double())
    assert abs(float(s[5]) - float(s64[0])) <= max(2.0 ** -150, 2 * U32 * float(s64[0]))
    assert bool(((q[5:6].double() - steps).abs() <= 0.5 + 127 * 8 * U32).all())


def test_quant_smallest_columns():
    """float columns whose scale rounds to zero read back as zeros"""
    m = 40
    x = torch.zeros((2, m), device="cuda")
    x[0, 3] = 2.0 ** -149
    x[1, 3] = 2.0 ** -126
    x[1, 4] = -2.0 ** -127
    q = torch.full((2, m), 5, dtype=torch.int8, device="cuda")
    s = torch.full((2,), -1.0, device="cuda")
    assert xs.quant("s", m, 2, x, m, q, m, s) == 0
    torch.cuda.synchronize()
    assert float(s[0]) == 0.0 and not bool(q[0].any())
    assert q[1, 3:5].tolist() == [127, -64] and not bool(q[1, 5:].any())


def run_rmsquant(kind, m, n, x, r, g, eps, h, q, s, rstd):
    p = lambda t: None if t is None else t.ptr      # noqa: E731
    ld = lambda t: 0 if t is None else t.ld         # noqa: E731
    return xs.rmsquant(kind, m, n, x.ptr, x.ld, p(r), ld(r), g, eps, p(h), ld(h), q.ptr, q.ld, s,
                       rstd)


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m,n", SIZES)
def test_rmsquant(kind, m, n):
    g = gen(3 * m + n)
    dt = DTYPES[kind]
    rel = ref.sum_depth(m) * U32
    for pad, off in LAYOUTS:
        x = Matrix(n, m, dt, m + pad, off, normal(g, n, m, kind))
        r = Matrix(n, m, dt, m + pad, off, normal(g, n, m, kind, 3.0))
        w = (1 + 0.2 * torch.randn((m,), generator=g, device="cuda")).to(dt)
        h, q = Matrix(n, m, dt, m + pad, off), Matrix(n, m, torch.int8, m + pad, off)
        s, rstd = torch.full((2, n), -1.0, device="cuda")
        assert run_rmsquant(kind, m, n, x, r, w, EPS, h, q, s, rstd) == 0
        torch.cuda.synchronize()
        assert torch.equal(h.rows, (x.rows.float() + r.rows.float()).to(dt))
        y64, rstd64 = ref.rmsnorm(h.rows.double(), w.double(), EPS)
        assert bool(((rstd.double() - rstd64).abs() <= rel * rstd64).all())
        check_quantised(q.rows, s, y64, rel)
        assert h.outside_untouched() and q.outside_untouched()


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m", [5, 1024, 4099, 40000])
def test_rmsquant_optional_arguments(kind, m):
    """no residual, no weight, nothing stored but the 8-bit output; in place over
    X and over R: all give the bytes of the full call"""
    n, dt = 3, DTYPES[kind]
    g = gen(m)
    x0, r0 = normal(g, n, m, kind), normal(g, n, m, kind)
    ones = torch.ones((m,), dtype=dt, device="cuda")

    def call(x, r, w, h, with_rstd=True):
        q = Matrix(n, m, torch.int8)
        s, rstd = torch.full((2, n), -1.0, device="cuda")
        assert run_rmsquant(kind, m, n, x, r, w, EPS, h, q, s, rstd if with_rstd else None) == 0
        torch.cuda.synchronize()
        assert with_rstd or bool((rstd == -1.0).all())
        return q.rows.clone(), s.clone(), rstd.clone()

    x, r, h = Matrix(n, m, dt, values=x0), Matrix(n, m, dt, values=r0), Matrix(n, m, dt)
    q1, s1, rstd1 = call(x, r, ones, h)
    for place in ("x", "r"):
        x, r = Matrix(n, m, dt, values=x0), Matrix(n, m, dt, values=r0)
        at = x if place == "x" else r
        q2, s2, rstd2 = call(x, r, None, at)
        assert torch.equal(q1, q2) and torch.equal(s1, s2) and torch.equal(rstd1, rstd2)
        assert torch.equal(at.rows, h.rows)
    x, r = Matrix(n, m, dt, values=x0), Matrix(n, m, dt, values=r0)
    q2, s2, _ = call(x, r, None, None, with_rstd=False)
    assert torch.equal(q1, q2) and torch.equal(s1, s2)
    assert torch.equal(x.rows, x0) and torch.equal(r.rows, r0)
    # without a residual the sum is X itself
    summed, h2 = Matrix(n, m, dt, values=h.rows), Matrix(n, m, dt)
    q2, s2, rstd2 = call(summed, None, ones, h2)
    assert torch.equal(q1, q2) and torch.equal(s1, s2) and torch.equal(rstd1, rstd2)
    assert torch.equal(h2.rows, h.rows)
    q2, s2, _ = call(summed, None, ones, None)
    assert torch.equal(q1, q2) and torch.equal(s1, s2)


@pytest.mark.parametrize("scale,eps", [(1e30, 1e-5), (3e-30, 0.0), (1e-42, 0.0), (1e-30, 1e-5),
                                       (1.5e38, 0.0)])
def test_rmsquant_squares_out_of_range(scale, eps):
    """finite values whose squares overflow or underflow float"""
    n, m = 3, 1000
    x = Matrix(n, m, torch.float32)
    x.rows.copy_((torch.rand((n, m), generator=gen(9), device="cuda", dtype=torch.float64) * 2 - 1)
                 * scale)
    q = Matrix(n, m, torch.int8)
    s, rstd = torch.full((2, n), -1.0, device="cuda")
    assert run_rmsquant("s", m, n, x, None, None, eps, None, q, s, rstd) == 0
    torch.cuda.synchronize()
    y64, rstd64 = ref.rmsnorm(x.rows.double(), 1.0, eps)
    if float(rstd64.max()) > 3e38:      # the reciprocal itself is beyond float
        assert bool(torch.isinf(rstd).all()) and bool(torch.isnan(s).all())
        return
    rel = ref.sum_depth(m) * U32
    # eps is passed as a float: its own rounding adds 2^-24
    assert bool(((rstd.double() - rstd64).abs() <= (rel + U32) * rstd64 + 2.0 ** -149).all())
    # a reciprocal below float's normal range keeps fewer bits
    rel += max(0.0, 2.0 ** -150 / float(rstd64.min()))
    check_quantised(q.rows, s, y64, rel)


@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_rmsquant_special_columns(kind):
    """a column of zeros stays zeros; an infinity or a NaN makes its column, and only
    that, NaN"""
    n, m = 5, 513
    x0 = normal(gen(4), n, m, kind)
    x0[1] = 0
    x0[2, 512] = float("inf")
    x0[3, 7] = float("nan")
    x = Matrix(n, m, DTYPES[kind], values=x0)
    q = Matrix(n, m, torch.int8)
    s, rstd = torch.full((2, n), -1.0, device="cuda")
    assert run_rmsquant(kind, m, n, x, None, None, EPS, None, q, s, rstd) == 0
    torch.cuda.synchronize()
    assert float(s[1]) == 0.0 and not bool(q.rows[1].any())
    assert abs(float(rstd[1]) * EPS ** 0.5 - 1) <= 4 * U32
    assert bool(torch.isnan(s[2:4]).all()) and not bool(q.rows[2:4].any())
    rel = ref.sum_depth(m) * U32
    keep = [0, 4]
    y64, _ = ref.rmsnorm(x0[keep].double(), 1.0, EPS)
    check_quantised(q.rows[keep], s[keep], y64, rel)


def run_rmsgrad(kind, m, n, dy, h, w, rstd, dr, dx, dg):
    return xs.rmsgrad(kind, m, n, dy.ptr, dy.ld, h.ptr, h.ld, w, rstd,
                      None if dr is None else dr.ptr, 0 if dr is None else dr.ld, dx.ptr, dx.ld, dg)


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m,n", SIZES + [(96, 1000), (1024, 700), (33, 5000), (8200, 333),
                                         (4096, 400), (2048, 350), (16384, 310), (12000, 400)])
def test_rmsgrad(kind, m, n):
    g = gen(5 * m + n)
    dt = DTYPES[kind]
    depth = ref.sum_depth(m) * U32
    for pad, off in (LAYOUTS if m * n < 1 << 18 else LAYOUTS[:3]):
        dy = Matrix(n, m, dt, m + pad, off, normal(g, n, m, kind, 0.1))
        dr = Matrix(n, m, dt, m + pad, off, normal(g, n, m, kind, 0.1))
        h = Matrix(n, m, dt, m + pad, off, normal(g, n, m, kind, 2.0))
        w = (1 + 0.2 * torch.randn((m,), generator=g, device="cuda")).to(dt)
        rstd = torch.rsqrt(h.rows.float().square().mean(1) + EPS)
        dx, dg = Matrix(n, m, dt, m + pad, off), torch.full((m,), -1.0, device="cuda")
        assert run_rmsgrad(kind, m, n, dy, h, w, rstd, dr, dx, dg) == 0
        torch.cuda.synchronize()
        dx64, dg64, dx_size, dg_size = ref.rmsgrad(dy.rows.double(), h.rows.double(), w.double(),
                                                   rstd.double(), dr.rows.double())
        bound = UNIT[kind] * dx64.abs() + (1 + UNIT[kind]) * depth * dx_size
        if kind == "h":
            bound = bound + 2.0 ** -25      # half a subnormal step
        assert bool(((dx.rows.double() - dx64).abs() <= bound).all())
        # any order of n additions
        assert bool(((dg.double() - dg64).abs() <= (n + 40) * U32 * dg_size).all())
        assert dx.outside_untouched()


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m,n", [(5, 4), (1024, 9), (4099, 300), (40000, 3)])
def test_rmsgrad_optional_arguments_and_in_place(kind, m, n):
    """no weight, no residual gradient, no weight gradient; in place over dY, dR
    and H: all give the bytes of the full call"""
    g = gen(m + 1)
    dt = DTYPES[kind]
    dy0, dr0, h0 = normal(g, n, m, kind), normal(g, n, m, kind), normal(g, n, m, kind)
    ones, zeros = torch.ones((m,), dtype=dt, device="cuda"), torch.zeros((n, m), dtype=dt,
                                                                         device="cuda")
    rstd = torch.rsqrt(h0.float().square().mean(1) + EPS)

    def call(w, dr, place=None, with_dg=True):
        a = {"dy": Matrix(n, m, dt, values=dy0), "h": Matrix(n, m, dt, values=h0),
             "dr": None if dr is None else Matrix(n, m, dt, values=dr), "dx": Matrix(n, m, dt)}
        dx, dg = a[place or "dx"], torch.full((m,), -1.0, device="cuda")
        assert run_rmsgrad(kind, m, n, a["dy"], a["h"], w, rstd, a["dr"], dx,
                           dg if with_dg else None) == 0
        torch.cuda.synchronize()
        assert with_dg or bool((dg == -1.0).all())
        return dx.rows.clone(), dg

    dx1, dg1 = call(ones, dr0)
    for place in ("dy", "dr", "h"):
        dx2, dg2 = call(None, dr0, place)
        assert torch.equal(dx1, dx2) and torch.equal(dg1, dg2), place
    assert torch.equal(call(None, dr0, with_dg=False)[0], dx1)
    dx2, dg2 = call(ones, zeros)
    dx3, dg3 = call(ones, None)
    assert bool((dx2 == dx3).all()) and torch.equal(dg2, dg3)


def test_rmsgrad_against_differences():
    """central differences of sum(dY * norm(h) * G) + sum(dR * h) in 64 bits along
    random directions of h and of G"""
    m, n = 257, 6
    g = gen(11)
    h0, dy0, dr0 = (torch.randn((n, m), generator=g, device="cuda") for _ in range(3))
    w0 = 1 + 0.2 * torch.randn((m,), generator=g, device="cuda")

    def loss(h, w):
        return float(((ref.rmsnorm(h, w, EPS)[0] * dy0.double()) + dr0.double() * h).sum())

    rstd = ref.rmsnorm(h0.double(), 1.0, EPS)[1].float()
    h, dy, dr, dx = (Matrix(n, m, torch.float32, values=v) for v in (h0, dy0, dr0, dr0))
    dg = torch.zeros((m,), device="cuda")
    assert run_rmsgrad("s", m, n, dy, h, w0, rstd, dr, dx, dg) == 0
    torch.cuda.synchronize()
    t = 1e-5
    for _ in range(4):
        v = torch.randn((n, m), generator=g, device="cuda").double()
        num = (loss(h0.double() + t * v, w0.double()) - loss(h0.double() - t * v, w0.double())) / (2 * t)
        # third derivatives (order 10 here) times t^2, and the losses' rounding over t
        size = float((dx.rows.double() * v).abs().sum())
        assert abs(num - float((dx.rows.double() * v).sum())) <= 1e-6 * size + 1e-6
        v = torch.randn((m,), generator=g, device="cuda").double()
        num = (loss(h0.double(), w0.double() + t * v) - loss(h0.double(), w0.double() - t * v)) / (2 * t)
        size = float((dg.double() * v).abs().sum())
        assert abs(num - float((dg.double() * v).sum())) <= 1e-6 * size + 1e-6


def test_rmsgrad_of_no_tokens():
    dg = torch.full((70,), -1.0, device="cuda")
    assert xs.rmsgrad("b", 70, 0, None, 70, None, 70, None, None, None, 70, None, 70, dg) == 0
    torch.cuda.synchronize()
    assert not bool(dg.any())


@pytest.mark.parametrize("kind", ["s", "b"])
def test_rows_repeat_bitwise_on_another_stream(kind):
    m, n = 4100, 700
    g = gen(21)
    dt = DTYPES[kind]
    x, dy = normal(g, n, m, kind), normal(g, n, m, kind)
    torch.cuda.synchronize()
    outs = []
    for stream in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        with torch.cuda.stream(stream):
            h, dx = torch.empty_like(x), torch.empty_like(x)
            q = torch.empty((n, m), dtype=torch.int8, device="cuda")
            s, rstd = torch.empty((2, n), device="cuda")
            dg = torch.empty((m,), device="cuda")
            v = torch.empty((n, m), dtype=dt, device="cuda")
            assert xs.rmsquant(kind, m, n, x, m, dy, m, None, EPS, h, m, q, m, s, rstd) == 0
            assert xs.dequant(kind, m, n, q, m, s, v, m) == 0
            assert xs.rmsgrad(kind, m, n, dy, m, h, m, None, rstd, v, m, dx, m, dg) == 0
        stream.synchronize()
        outs.append((h, q, s, rstd, v, dx, dg))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_rows_offsets_beyond_32_bits():
    """columns so far apart that their offsets pass 2^32 elements"""
    m, n, ld = 1000, 4, (1 << 31) - 8
    flat = torch.empty(((n - 1) * ld + m,), dtype=torch.bfloat16, device="cuda")   # 12.9 GB
    rows = flat.as_strided((n, m), (ld, 1))
    rows.copy_(normal(gen(31), n, m, "b"))
    qf = torch.empty(((n - 1) * ld + m,), dtype=torch.int8, device="cuda")
    q = qf.as_strided((n, m), (ld, 1))
    s, rstd = torch.empty((2, n), device="cuda")
    assert xs.rmsquant("b", m, n, flat, ld, None, 0, None, EPS, None, 0, qf, ld, s, rstd) == 0
    torch.cuda.synchronize()
    y64, _ = ref.rmsnorm(rows.double(), 1.0, EPS)
    check_quantised(q, s, y64, ref.sum_depth(m) * U32)
    dg = torch.empty((m,), device="cuda")
    dx = torch.empty((n, m), dtype=torch.bfloat16, device="cuda")
    assert xs.rmsgrad("b", m, n, flat, ld, flat, ld, None, rstd, None, 0, dx, m, dg) == 0
    torch.cuda.synchronize()
    dg64 = (rows.double() ** 2 * rstd.double()[:, None]).sum(0)
    assert bool(((dg.double() - dg64).abs() <= 44 * U32 * dg64).all())
    assert xs.dequant("b", m, n, qf, ld, s, flat, ld) == 0
    torch.cuda.synchronize()
    assert torch.equal(rows, (q.float() * s[:, None]).bfloat16())
    del flat, qf, rows, q
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("m,n", [(3, 6000), (61, 6000), (515, 3001), (1543, 1500), (4101, 700)])
def test_rmsgrad_of_many_columns_at_every_alignment(kind, m, n):
    """several columns a block; operands that lie alike and that do not; NaN all around"""
    g = gen(m * n)
    dt = DTYPES[kind]
    nan = float("nan")

    class Placed:
        def __init__(self, pad, off, values):
            self.flat = torch.full((off + n * (m + pad) + 9,), nan, dtype=dt, device="cuda")
            self.rows = self.flat.as_strided((n, m), (m + pad, 1), off)
            self.rows.copy_(values)
            self.ptr, self.ld = self.flat.data_ptr() + off * self.flat.element_size(), m + pad

    dy0, dr0 = normal(g, n, m, kind, 0.1), normal(g, n, m, kind, 0.1)
    h0 = normal(g, n, m, kind, 2.0)
    w = (1 + 0.2 * torch.randn((m,), generator=g, device="cuda")).to(dt)
    rstd = torch.rsqrt(h0.float().square().mean(1) + EPS)
    dx64, dg64, dx_size, dg_size = ref.rmsgrad(dy0.double(), h0.double(), w.double(), rstd.double(),
                                               dr0.double())
    bound = UNIT[kind] * dx64.abs() + (1 + UNIT[kind]) * ref.sum_depth(m) * U32 * dx_size
    if kind == "h":
        bound = bound + 2.0 ** -25
    for at in (((0, 0),) * 4, ((1, 3),) * 4, ((8, 5),) * 4, ((0, 1), (3, 0), (2, 7), (1, 0)),
               ((0, 2), (0, 2), (0, 2), (0, 0)), ((0, 0), (8, 8), (16, 0), (0, 16))):
        dy, h, dr, dx = (Placed(*p, v) for p, v in zip(at, (dy0, h0, dr0, torch.zeros_like(h0))))
        dg = torch.full((m,), -1.0, device="cuda")
        assert run_rmsgrad(kind, m, n, dy, h, w, rstd, dr, dx, dg) == 0
        torch.cuda.synchronize()
        assert bool(((dx.rows.double() - dx64).abs() <= bound).all()), at
        assert bool(((dg.double() - dg64).abs() <= (n + 40) * U32 * dg_size).all()), at
        dx.rows.fill_(nan)
        assert bool(torch.isnan(dx.flat).all()), at

"""GPU parity of the product of 8-bit matrices (x<gemmq>) against a 64-bit
product: from one token to prompts, odd sizes, depths of zero and one, padded
and unaligned columns, every type, alpha and beta, missing scales, the largest
integers, NaN scales, offsets beyond 32 bits."""
import pytest
import torch

import symmetric_matrix_vector_gb300 as xs
from tests import q8_reference as ref
from tests.q8_reference import DTYPES, UNIT, Matrix

pytestmark = pytest.mark.gpu

LAYOUTS = [(0, 0), (16, 0), (1, 0), (3, 1), (16, 16), (0, 5)]
TOKENS = [1, 2, 3, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 127, 129, 256, 257, 300, 513]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def integers(g, n, k, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, (n, k), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def check(kind, m, n, k, g, pad=0, off=0, alpha=1.0, beta=0.0, scales=True, w=None, x=None):
    dt = DTYPES[kind]
    W = Matrix(m, max(k, 1), torch.int8, max(k, 1) + pad, off,
               integers(g, m, max(k, 1)) if w is None else w)
    X = Matrix(n, max(k, 1), torch.int8, max(k, 1) + pad, off,
               integers(g, n, max(k, 1)) if x is None else x)
    sw = torch.rand((m,), generator=g, device="cuda") * 1e-3 + 1e-5
    sx = torch.rand((n,), generator=g, device="cuda") * 1e-2 + 1e-4
    y0 = torch.randn((n, m), generator=g, device="cuda").to(dt)
    # beta = 0 must not read Y
    Y = Matrix(n, m, dt, m + pad, off, y0 if beta != 0 else torch.full_like(y0, float("nan")))
    assert xs.gemmq(kind, m, n, k, alpha, W.ptr, W.ld, sw if scales else None, X.ptr, X.ld,
                    sx if scales else None, beta, Y.ptr, Y.ld) == 0
    torch.cuda.synchronize()
    if not scales:
        sw, sx = torch.ones_like(sw), torch.ones_like(sx)
    y64, size = ref.gemmq(W.rows[:, :k], X.rows[:, :k], alpha, sw, sx, beta, y0)
    bound = UNIT[kind] * y64.abs() + (1 + UNIT[kind]) * size + (2.0 ** -25 if kind == "h" else 0)
    bad = ~((Y.rows.double() - y64).abs() <= bound)
    if kind == "h":     # beyond half's range
        bad &= ~(torch.isinf(Y.rows) & (y64.abs() > 65000))
    assert not bool(bad.any()), (kind, m, n, k, pad, off, int(bad.sum()))
    assert Y.outside_untouched()


@pytest.mark.parametrize("n", TOKENS)
def test_token_counts(n):
    g = gen(n)
    for kind, m, k in (("b", 256, 512), ("s", 129, 1000), ("h", 100, 64), ("s", 384, 2048)):
        for pad, off in ((0, 0), (1, 0)):
            check(kind, m, n, k, g, pad, off)


@pytest.mark.parametrize("kind,m,n,k,pad,off", [
    ("b", 8192, 2048, 256, 0, 0), ("h", 4099, 3001, 333, 1, 3), ("s", 2560, 6000, 128, 16, 0),
    ("b", 300, 9000, 1, 0, 0), ("h", 10000, 1000, 200, 0, 1), ("s", 5000, 1537, 1000, 8, 0)])
def test_many_tiles(kind, m, n, k, pad, off):
    """more tiles than the GPU forms at once, odd edges, queued one behind another"""
    g = gen(m + n)
    for alpha, beta in ((1.0, 0.0), (0.5, -2.0), (1.0, 0.0)):
        check(kind, m, n, k, g, pad, off, alpha, beta)


@pytest.mark.parametrize("k", [1, 2, 15, 16, 31, 32, 33, 63, 64, 65, 100, 127, 128, 130, 255, 256,
                               1000, 1543, 4096, 5000, 16384])
def test_depths(k):
    g = gen(k)
    for n, m in ((1, 130), (4, 64), (20, 257), (70, 128), (300, 200)):
        check("s", m, n, k, g)
        check("b", m, n, k, g, pad=16)


@pytest.mark.parametrize("m", [1, 2, 7, 8, 15, 16, 63, 64, 100, 127, 128, 129, 255, 257, 500, 1000,
                               2111, 4096, 33000])
def test_channel_counts(m):
    g = gen(m)
    for n, k in ((1, 256), (3, 100), (16, 512), (50, 128), (260, 192)):
        check("s", m, n, k, g)
        check("h", m, n, k, g, pad=1)


@pytest.mark.parametrize("pad,off", LAYOUTS)
@pytest.mark.parametrize("kind", ["s", "h", "b"])
def test_layouts_and_scalars(kind, pad, off):
    g = gen(7 * pad + off)
    for n in (1, 6, 24, 90, 270):
        for alpha, beta in ((1.0, 0.0), (-0.75, 1.0), (0.5, -2.0)):
            check(kind, 200, n, 320, g, pad, off, alpha, beta)
        check(kind, 200, n, 320, g, pad, off, 1e-4, 0.0, scales=False)


@pytest.mark.parametrize("n", [1, 4, 20, 80, 300])
def test_raw_integers_are_exact(n):
    """no scales, float output: the integer sums themselves, equal to the last bit
    while they are below 2^24"""
    g = gen(n)
    for k in (64, 777, 1024):
        w, x = integers(g, 150, k, -128, 127), integers(g, n, k, -128, 127)
        y = torch.empty((n, 150), device="cuda")
        assert xs.gemmq("s", 150, n, k, 1.0, w, k, None, x, k, None, 0.0, y, 150) == 0
        torch.cuda.synchronize()
        assert torch.equal(y.double(), x.double() @ w.double().T)


@pytest.mark.parametrize("n", [1, 4, 20, 80, 300])
def test_largest_integers(n):
    """every product at its largest, of one sign: sums beyond 2^24"""
    m, k = 140, 8192
    for a, b in ((-128, -128), (-128, 127), (127, 127)):
        w = torch.full((m, k), a, dtype=torch.int8, device="cuda")
        x = torch.full((n, k), b, dtype=torch.int8, device="cuda")
        check("s", m, n, k, gen(n), w=w, x=x)


@pytest.mark.parametrize("n", [1, 4, 20, 80, 300])
def test_nan_scales_stay_in_their_row_and_column(n):
    m, k = 150, 256
    g = gen(n)
    w, x = integers(g, m, k), integers(g, n, k)
    sw, sx = torch.ones((m,), device="cuda"), torch.ones((n,), device="cuda")
    sw[149] = float("nan")
    sx[n - 1] = float("nan")
    y = torch.zeros((n, m), device="cuda")
    assert xs.gemmq("s", m, n, k, 1.0, w, k, sw, x, k, sx, 0.0, y, m) == 0
    torch.cuda.synchronize()
    want = torch.zeros((n, m), dtype=torch.bool, device="cuda")
    want[:, 149] = True
    want[n - 1, :] = True
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("kind", ["s", "h", "b"])
@pytest.mark.parametrize("n", [1, 20, 200])
def test_no_product(kind, n):
    """alpha = 0 or k = 0: Y := beta * Y, nothing else read"""
    m, dt = 130, DTYPES[kind]
    y0 = torch.randn((n, m), generator=gen(n), device="cuda").to(dt)
    for alpha, k in ((0.0, 64), (1.0, 0)):
        for beta in (0.0, 0.5, 1.0):
            y = y0.clone() if beta != 0 else torch.full_like(y0, float("nan"))
            assert xs.gemmq(kind, m, n, k, alpha, None, 64, None, None, 64, None, beta, y, m) == 0
            torch.cuda.synchronize()
            assert torch.equal(y, (y0.float() * beta).to(dt) if beta != 0 else torch.zeros_like(y0))


@pytest.mark.parametrize("n", [1, 20, 200])
def test_repeats_bitwise_on_another_stream(n):
    m, k = 1000, 2000
    g = gen(n)
    w, x = integers(g, m, k), integers(g, n, k)
    sw, sx = torch.rand((m,), generator=g, device="cuda"), torch.rand((n,), generator=g, device="cuda")
    torch.cuda.synchronize()
    outs = []
    for stream in (torch.cuda.Stream(), torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            for _ in range(3):
                y = torch.empty((n, m), device="cuda")
                assert xs.gemmq("s", m, n, k, 1.0, w, k, sw, x, k, sx, 0.0, y, m) == 0
                outs.append(y)
        stream.synchronize()
    assert all(torch.equal(outs[0], y) for y in outs[1:])


@pytest.mark.parametrize("n", [1, 3, 8, 13, 30, 37, 64, 100, 200, 500, 1500, 4000])
def test_many_calls_in_a_row(n):
    """calls queued behind one another, different operands in turn, give what each
    gives alone"""
    m, k = 2048, 4096
    g = gen(n)
    sets = []
    for _ in range(3):
        w, x = integers(g, m, k), integers(g, n, k)
        y = torch.empty((n, m), device="cuda")
        sets.append((w, x, y))
    alone = []
    for w, x, y in sets:
        assert xs.gemmq("s", m, n, k, 1.0, w, k, None, x, k, None, 0.0, y, m) == 0
        torch.cuda.synchronize()
        want = x.double() @ w.double().T
        assert torch.equal(y.double(), want)
        alone.append(y.clone())
    for _ in range(40):
        for w, x, y in sets:
            y.fill_(float("nan"))
        for _ in range(3):
            for w, x, y in sets:
                assert xs.gemmq("s", m, n, k, 1.0, w, k, None, x, k, None, 0.0, y, m) == 0
        for (w, x, y), a in zip(sets, alone):
            assert torch.equal(y, a)
    assert xs.xsymv_sync_status() == 0


@pytest.mark.parametrize("n", [2, 40])
def test_offsets_beyond_32_bits(n):
    """channels, tokens and outputs so far apart that offsets pass 2^32 bytes"""
    m, k, ld = 5, 96, (1 << 30) - 16
    g = gen(n)
    wf = torch.empty(((m - 1) * ld + k,), dtype=torch.int8, device="cuda")     # 4.3 GB
    w = wf.as_strided((m, k), (ld, 1))
    w.copy_(integers(g, m, k))
    ldx = (1 << 32) // n // 16 * 16 + 16 if n > 2 else (1 << 31) - 16
    xf = torch.empty(((n - 1) * ldx + k,), dtype=torch.int8, device="cuda")
    x = xf.as_strided((n, k), (ldx, 1))
    x.copy_(integers(g, n, k))
    yf = torch.empty(((n - 1) * ldx + m,), dtype=torch.bfloat16, device="cuda")
    assert xs.gemmq("b", m, n, k, 1.0, wf, ld, None, xf, ldx, None, 0.0, yf, ldx) == 0
    torch.cuda.synchronize()
    assert torch.equal(yf.as_strided((n, m), (ldx, 1)),
                       (x.double() @ w.double().T).float().bfloat16())
    del wf, w, xf, x, yf
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["h", "b"])
def test_norm_feeds_product(kind):
    """rmsquant's output is the product's input as it stands: the layer against
    the same layer in 64 bits on the 8-bit values"""
    dt = DTYPES[kind]
    m, k = 300, 520
    for n in (1, 33):
        g = gen(n)
        x, r = (torch.randn((n, k), generator=g, device="cuda").to(dt) for _ in range(2))
        wt = (torch.randn((m, k), generator=g, device="cuda") * 0.05).to(dt)
        w, q = (torch.empty((c, k), dtype=torch.int8, device="cuda") for c in (m, n))
        sw, sq = torch.empty((m,), device="cuda"), torch.empty((n,), device="cuda")
        h, y = torch.empty_like(x), torch.empty((n, m), dtype=dt, device="cuda")
        assert xs.quant(kind, k, m, wt, k, w, k, sw) == 0
        assert xs.rmsquant(kind, k, n, x, k, r, k, None, 1e-5, h, k, q, k, sq, None) == 0
        assert xs.gemmq(kind, m, n, k, 1.0, w, k, sw, q, k, sq, 0.0, y, m) == 0
        torch.cuda.synchronize()
        y64 = (q.double() * sq.double()[:, None]) @ (w.double() * sw.double()[:, None]).T
        assert bool(((y.double() - y64).abs() <= UNIT[kind] * y64.abs() + 1e-6 * k ** 0.5).all())
        # and near the layer of the unquantised values: two roundings of half a step
        # per product, at most 1/254 of the largest of a column each
        hn, _ = ref.rmsnorm(h.double(), 1.0, 1e-5)
        full = hn @ wt.double().T
        worst = (hn.abs().amax(1)[:, None] * wt.double().abs().sum(1)[None, :]
                 + hn.abs().sum(1)[:, None] * wt.double().abs().amax(1)[None, :]) / 254 * 1.01
        assert bool(((y.double() - full).abs() <= worst + UNIT[kind] * full.abs() + 1e-3).all())


@pytest.mark.parametrize("n", [1, 5, 8, 20, 33, 64, 90, 300])
def test_queued_layers_see_their_own_activations(n):
    """norms and products queued behind one another through the same 8-bit buffers:
    every product reads what the norm before it wrote, not what was there earlier"""
    m, k, layers = 512, 1024, 24
    g = gen(n)
    w = integers(g, m, k)
    xs_in = torch.randn((layers, n, k), generator=g, device="cuda").bfloat16()
    q = torch.empty((n, k), dtype=torch.int8, device="cuda")
    s = torch.empty((n,), device="cuda")
    y = torch.empty((layers, n, m), device="cuda")
    qs, ss = torch.empty((layers, n, k), dtype=torch.int8, device="cuda"), torch.empty((layers, n), device="cuda")
    for i in range(layers):        # each alone
        assert xs.rmsquant("b", k, n, xs_in[i], k, None, 0, None, 1e-5, None, 0, qs[i], k, ss[i], None) == 0
        torch.cuda.synchronize()
    want = torch.stack([(qs[i].double() @ w.double().T) * ss[i].double()[:, None] for i in range(layers)])
    for _ in range(20):
        y.fill_(float("nan"))
        for i in range(layers):    # queued
            assert xs.rmsquant("b", k, n, xs_in[i], k, None, 0, None, 1e-5, None, 0, q, k, s, None) == 0
            assert xs.gemmq("s", m, n, k, 1.0, w, k, None, q, k, s, 0.0, y[i], m) == 0
        torch.cuda.synchronize()
        assert bool(((y.double() - want).abs() <= 4 * ref.U32 * want.abs()).all())


@pytest.mark.parametrize("n", [1, 20, 100])
def test_queued_weights(n):
    """the weights written by the kernel just before the product: every product reads
    its own, equal to those that the same call gives alone"""
    m, k = 512, 1024
    g = gen(n)
    x = integers(g, n, k)
    ws = torch.randn((12, m, k), generator=g, device="cuda").half()
    w = torch.empty((m, k), dtype=torch.int8, device="cuda")
    sw = torch.empty((m,), device="cuda")
    y = torch.empty((12, n, m), device="cuda")
    want = []
    for i in range(12):
        assert xs.quant("h", k, m, ws[i], k, w, k, sw) == 0
        torch.cuda.synchronize()
        want.append((x.double() @ w.double().T) * sw.double())
    want = torch.stack(want)
    for _ in range(10):
        for i in range(12):
            assert xs.quant("h", k, m, ws[i], k, w, k, sw) == 0
            assert xs.gemmq("s", m, n, k, 1.0, w, k, sw, x, k, None, 0.0, y[i], m) == 0
        torch.cuda.synchronize()
        assert bool(((y.double() - want).abs() <= 4 * ref.U32 * want.abs()).all())


@pytest.mark.parametrize("m,n,k", [(700, 20, 640), (700, 64, 640), (700, 100, 640), (130, 50, 64),
                                   (2048, 2048, 256), (4096, 4096, 512)])
def test_waits_that_run_out(m, n, k):
    """copies whose barrier expects bytes that never arrive (nothing faults): the
    kernel returns after the limit, Y is NaN, the status says so, and the next
    call is right"""
    g = gen(n)
    w, x = integers(g, m, k), integers(g, n, k)
    y = torch.zeros((n, m), device="cuda")

    def run():
        st = xs.gemmq("s", m, n, k, 1.0, w, k, None, x, k, None, 0.0, y, m)
        assert st == 0
        return xs.xsymv_sync_status()

    want = x.double() @ w.double().T
    assert run() == 0 and torch.equal(y.double(), want)
    xs.xsymv_set_wait_limit(2_000_000)
    try:
        xs.xsymv_test_stall(True)
        assert run() == -6
        assert bool(torch.isnan(y).all())
        xs.xsymv_test_stall(False)
        assert run() == 0 and torch.equal(y.double(), want)
    finally:
        xs.xsymv_test_stall(False)
        xs.xsymv_set_wait_limit(0)
    # a call without such waits reports none
    s = torch.empty((1,), device="cuda")
    assert xs.quant("s", 4, 1, y, 4, w, 4, s) == 0 and xs.xsymv_sync_status() == 0


@pytest.mark.parametrize("n", [9, 20, 32, 33, 47, 64])
@pytest.mark.parametrize("m", [1, 15, 17, 300, 2047, 2049, 4100])
def test_rows_off_the_16_byte_boundaries(n, m):
    """W's rows at every distance from a boundary, X's at another one or on it, the largest
    integers all around both; exact sums"""
    g = gen(m + n)
    for k, pad, off, pad_x, off_x in ((1, 0, 3, 0, 0), (15, 2, 0, 1, 0), (113, 0, 0, 15, 16),
                                      (128, 1, 15, 0, 0), (129, 15, 1, 15, 0), (127, 1, 1, 2, 9),
                                      (1000, 4, 2, 8, 0), (640, 8, 8, 0, 7)):
        def placed(rows, pad, off):
            flat = torch.full((off + rows * (k + pad) + 300,), 127, dtype=torch.int8, device="cuda")
            at = flat[off:off + rows * (k + pad)].view(rows, k + pad)
            at[:, :k] = integers(g, rows, k, -128, 127)
            return flat, at
        (wf, w), (xf, x) = placed(m, pad, off), placed(n, pad_x, off_x)
        y = torch.full((n + 1, m + 3), 7.0, device="cuda")
        assert xs.gemmq("s", m, n, k, 1.0, wf.data_ptr() + off, k + pad, None, xf.data_ptr() + off_x,
                        k + pad_x, None, 0.0, y, m + 3) == 0
        torch.cuda.synchronize()
        assert torch.equal(y[:n, :m].double(), x[:, :k].double() @ w[:, :k].double().T), (k, pad, off)
        assert bool((y[n:] == 7.0).all()) and bool((y[:, m:] == 7.0).all())


@pytest.mark.parametrize("m,n,k", [(2500, 20, 641), (2500, 40, 641), (4100, 64, 333), (700, 40, 640),
                                   (300, 48, 4096)])
def test_waits_that_run_out_off_the_boundaries(m, n, k):
    """the same for W's rows off the 16-byte boundaries, and for tiles of 48 tokens"""
    test_waits_that_run_out(m, n, k)


@pytest.mark.parametrize("n", [33, 40, 47, 48])
def test_tiles_of_48_tokens(n):
    """their depth shared by 1, 2, 4 and 8 CTAs"""
    g = gen(n)
    for kind, m, k, pad in (("b", 40000, 64, 0), ("h", 20000, 256, 16), ("s", 6000, 512, 0),
                            ("h", 257, 2000, 3), ("b", 128, 1024, 0), ("s", 129, 4097, 0)):
        check(kind, m, n, k, g, pad)
        check(kind, m, n, k, g, pad, 1, -0.5, 2.0)

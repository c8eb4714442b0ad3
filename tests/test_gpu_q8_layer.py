"""The example layer in 8 bits (q8_layer): its serving step against the same
layer in 64 bits on the same 8-bit values, and its gradients against
torch's own, the rounding taken as the identity."""
import pytest
import torch

from symmetric_matrix_vector_gb300 import q8_layer
from tests import q8_reference as ref
from tests.q8_reference import U32, UNIT

pytestmark = pytest.mark.gpu


def make(dtype, channels, width, tokens, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    layer = q8_layer.Q8Linear(normal(channels, width, scale=0.05), 1 + normal(width, scale=0.1))
    return layer, normal, normal(tokens, width), normal(tokens, width)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [1, 17, 200])
def test_serving_step(dtype, tokens):
    layer, _, x, r = make(dtype, 300, 520, tokens)
    y, h = layer.forward(x, r)
    _, q, scale, rstd = layer.norm(x, r)
    assert torch.equal(h, (x.float() + r.float()).to(dtype))
    y64, size = ref.gemmq(layer.w, q, 1.0, layer.sw, scale, 0.0, None)
    unit = UNIT[layer.kind]
    assert bool(((y.double() - y64).abs() <= unit * y64.abs() + (1 + unit) * size + 2.0 ** -25).all())


def test_training_step():
    """float: against autograd of the norm in 64 bits, with the weight's 8-bit values"""
    layer, normal, x, r = make(torch.float32, 96, 257, 40)
    dy, dh = normal(40, 96), normal(40, 257)
    y, dx, dg, dw = layer.train_step(x, r, dy, dh)
    h, q, scale, _ = layer.norm(x, r)
    w64 = layer.w.double() * layer.sw.double()[:, None]
    a64 = q.double() * scale.double()[:, None]
    h64 = h.double().requires_grad_()
    g64 = layer.g.double().requires_grad_()
    a = ref.rmsnorm(h64, g64, layer.eps)[0]
    ((a * (dy.double() @ w64)).sum() + (h64 * dh.double()).sum()).backward()
    # the 16- or 32-bit products of torch come in with sums of 96 and of 257 products
    def near(got, want, terms):
        return float((got.double() - want).abs().max()) <= terms * 4 * U32 * float(want.abs().max()) * 8
    assert near(y, a64 @ w64.T, 257)
    assert near(dx, h64.grad, 96 + 257)
    assert near(dg, g64.grad, 96 + 40)
    assert near(dw, dy.double().T @ a64, 40)


def test_example_runs(capsys):
    q8_layer.main(256, 384, 33)
    out = capsys.readouterr().out
    assert "training step" in out and out.count("within") == 4
    for line in out.splitlines():
        if "within" in line:
            # two roundings of at most half a 254th of the largest value to every product
            assert float(line.split("within ")[1].split()[0]) < 0.03


@pytest.mark.parametrize("tokens", [1, 17, 200])
def test_serving_step_in_a_graph(tokens):
    """captured after a first run on the stream, replayed on other inputs"""
    layer, normal, x, r = make(torch.bfloat16, 300, 520, tokens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.forward(x, r)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, h = layer.forward(x, r)
        y, h = layer.forward(y[:, :1] + x, h)
    for _ in range(3):
        x.copy_(normal(tokens, 520))
        graph.replay()
        torch.cuda.synchronize()
        y1, h1 = layer.forward(x, r)
        y1, h1 = layer.forward(y1[:, :1] + x, h1)
        assert torch.equal(y, y1) and torch.equal(h, h1)

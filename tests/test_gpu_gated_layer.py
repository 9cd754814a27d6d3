"""The gated block, its backward pass and clipping together with the operators
around them, as a training step and as a served layer run them: the example's
layer, eagerly and captured.

Each call is bit for bit the same in every run (its tests), so a captured step
equals an eager one exactly.  Against 64 bits: the bound of the layer's own test, e4m3
rounding of two products in a row, 0.11.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "moe_layer_example", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


CASES = [(300, 4, 8, 512, 256, None), (1, 2, 8, 256, 144, None), (513, 3, 16, 272, 400, 5)]




@pytest.mark.parametrize("case", CASES)
def test_served_layer(example, case):
    """Quantized rows only, as served: the same bits as the training forward."""
    x, ids, weights, w13, w2, _ = example.make_inputs(*case[:5], seed=1, local=case[5])
    layer = example.Fp8MoELayer(w13, w2)
    out, _ = layer.forward(x, ids, weights)
    assert torch.equal(layer.infer(x, ids, weights), out)


@pytest.mark.parametrize("case", CASES)
def test_captured_training_step(example, case):
    x, ids, weights, w13, w2, g = example.make_inputs(*case[:5], seed=2, local=case[5])
    gq = example.gq

    def step(layer, w13, w2):
        out, saved = layer.forward(x, ids, weights)
        dx, dweights, dw13, dw2 = layer.backward(g, saved)
        norm = layer.step(w13, w2, dw13, dw2, 0.01, 1.0)
        return out, dx, dweights, dw13, dw2, norm

    a13, a2 = w13.clone(), w2.clone()
    layer = example.Fp8MoELayer(a13, a2)
    want = [[t.clone() for t in step(layer, a13, a2)] + [a13.clone(), a2.clone()] for _ in range(2)]
    b13, b2 = w13.clone(), w2.clone()
    layer = example.Fp8MoELayer(b13, b2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # quantizes the weights that it finds, then makes a step
        layer.update(b13, b2)
        got = step(layer, b13, b2)
    for w in want:
        graph.replay()
        gq.check_device_error()
        for name, a, b in zip(("out", "dx", "dweights", "dw13", "dw2", "norm", "w13", "w2"), w, [*got, b13, b2]):
            assert torch.equal(a, b), name
        # both gradients together have a norm of 1, up to bf16's rounding of each element
        norm = sum(float(t.double().square().sum()) for t in got[3:5]) ** 0.5
        assert abs(norm - min(1.0, float(got[5]))) <= 2.0 ** -8


def test_two_layers_at_once(example):
    """Two layers on streams of their own, call by call in turn: neither sees
    the other's buffers."""
    inputs = [example.make_inputs(300, 4, 8, 512, 256, seed=s) for s in (3, 4)]
    layers = [example.Fp8MoELayer(i[3], i[4]) for i in inputs]

    def run(layer, i):
        out, saved = layer.forward(*i[:3])
        return (out, *layer.backward(i[5], saved))

    want = [run(l, i) for l, i in zip(layers, inputs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(5):
        got = []
        for s, l, i in zip(streams, layers, inputs):
            with torch.cuda.stream(s):
                got.append(run(l, i))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))

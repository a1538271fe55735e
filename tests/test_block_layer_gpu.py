"""The layer with norms around it: what it keeps between calls, and each of its options against the calls
that it is made of."""
import weakref

import pytest
import torch

import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def rand(g, *shape, std=1.0, dt=f32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def weights(g, H, I, E, dt):
    return (rand(g, H, E, std=H ** -0.5, dt=dt), rand(g, E, I, H, std=H ** -0.5, dt=dt),
            rand(g, E, I, H, std=H ** -0.5, dt=dt), rand(g, E, H, I, std=I ** -0.5, dt=dt))


def test_a_captured_gate_gradient_outlives_a_gate_of_the_other_form():
    """A step captured with a gate a token, then an eager step with one an element: the captured step's
    buffer is still the layer's, so a replay writes memory of nobody else."""
    g = torch.Generator(device=DEV).manual_seed(0)
    T, H, I, E, k, eps = 40, 128, 64, 4, 2, 1e-6
    w, ow = weights(g, H, I, E, bf), 1 + rand(g, H, std=0.2)
    x, dy = rand(g, T, H, dt=bf), rand(g, T, H, dt=bf)
    token, full = torch.sigmoid(rand(g, T)), torch.sigmoid(rand(g, T, H)).to(bf)
    layer, other = (moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, post_norm=eps) for _ in range(2))

    def step(m, gate):
        m.forward(x, *w, post_weight=ow, gate=gate)
        return m.backward(dy, x, *w)["dgate"]

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(layer, token)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step(layer, token)
    torch.cuda.synchronize()
    for _ in range(3):
        x.copy_(rand(g, T, H, dt=bf))
        got = step(layer, full)
        assert torch.equal(got, step(other, full)) and got.shape == (T, H)
        keep = got.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert any(t is captured for t in layer.buf.values())
        assert torch.equal(captured, step(other, token)) and torch.equal(got, keep)
        assert step(layer, token).data_ptr() == captured.data_ptr()


@pytest.mark.parametrize("form", ["train", "serve", "serve norms", "train post", "train pre"])
def test_a_layer_holds_no_tensor_that_it_does_not_read_again(form):
    """The residual, and in a layer built for the forward alone every input, is its caller's alone once
    forward() is back.  Training with a norm holds what the norm's backward reads."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, H, I, E, k, eps = 24, 64, 64, 4, 2, 1e-6
    w = weights(g, H, I, E, bf)
    train, pre, post = form.startswith("train"), form in ("serve norms", "train pre"), form in ("serve norms", "train post")
    layer = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, train=train, pre_norm=eps if pre else None,
                         post_norm=eps if post else None)
    given = {"x": rand(g, T, H, dt=bf)}
    if pre:
        given["pre_weight"] = torch.ones(H, device=DEV)
    else:
        given["residual"] = rand(g, T, H, dt=bf)
    if post:
        given.update(post_weight=torch.ones(H, device=DEV), gate=torch.rand(T, device=DEV))
    refs = {n: weakref.ref(t) for n, t in given.items()}
    layer.forward(given.pop("x"), *w, **given)
    del given
    held = {n for n, r in refs.items() if r() is not None}
    assert held == ({"train post": {"post_weight", "gate"}, "train pre": {"x", "pre_weight"}}.get(form, set()))

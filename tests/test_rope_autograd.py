"""Rope.apply under autograd: recorded where the input requires grad, refused
where it cannot be."""
import math

import pytest
import torch

import varlen_gqa_split_b200 as vg
from varlen_gqa_split_b200 import Rope, rope_table


@pytest.fixture(scope="module", autouse=True)
def _built():
    from varlen_gqa_split_b200 import build
    build.build()


def test_out_with_gradients_is_refused():
    rope = Rope(8, *rope_table(4))
    x, pos = torch.ones(1, 1, 8, requires_grad=True), torch.zeros(1, 1, dtype=torch.int32)
    y = torch.ones(1, 1, 8)
    for args in ((x, pos, y), (x, pos, x), (y, pos, x)):
        with pytest.raises(ValueError, match="gradient"):
            rope.apply(*args)
    with torch.no_grad(), pytest.raises((ValueError, RuntimeError)) as e:   # (goes on to device and tensors)
        rope.apply(x, pos, y)
    assert "gradient" not in str(e.value)
    with pytest.raises(RuntimeError):                                   # no truth value
        rope.apply(y, pos, grad=torch.ones(2))


def _rotate64(x, pos, freqs, axes, layout, scale, sign):
    n = len(freqs)
    theta = pos.double()[torch.tensor(axes, device=x.device)].t() * torch.tensor(freqs, dtype=torch.float64, device=x.device)
    c, s = torch.cos(theta)[:, None] * scale, torch.sin(theta)[:, None] * scale * sign
    at = torch.arange(n, device=x.device)
    u, w = (at, at + n) if layout == "half" else (2 * at, 2 * at + 1)
    y = x.double().clone()
    y[..., u], y[..., w] = x[..., u].double() * c - x[..., w].double() * s, x[..., u].double() * s + x[..., w].double() * c
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,eps", [(torch.float32, 2.0 ** -24), (torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8)])
def test_backward_is_the_transpose(layout, dtype, eps):
    freqs, axes = rope_table(12, (4, 8), base=1e3)
    rope = Rope(26, freqs, axes, layout=layout, scale=0.5)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(37, 3, 26, generator=g, device="cuda").to(dtype).requires_grad_()
    up = torch.randn(37, 3, 26, generator=g, device="cuda").to(dtype)
    pos = torch.randint(-500, 500, (2, 37), generator=g, device="cuda", dtype=torch.int32)
    y = rope.apply(x, pos)
    assert y.requires_grad and torch.equal(y.detach(), rope.apply(x.detach(), pos))
    (gx,) = torch.autograd.grad(y, x, up)
    ref = _rotate64(up, pos, freqs, axes, layout, 0.5, -1)
    # one rounding to the type, after an angle off by pi 2^-25, cosine and sine
    # by 2^-22, two products and a sum, relative to |u| + |w| <= 2 max
    tol = ref.abs() * eps * (1 + 2.0 ** -7) + up.abs().max() * 2 * (math.pi * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24) + 2.0 ** -25
    assert ((gx.double() - ref).abs() <= tol).all()
    assert torch.equal(gx, rope.apply(up, pos, grad=True))
    # the recorded transpose has the rotation for its gradient
    (gg,) = torch.autograd.grad(rope.apply(x, pos, grad=True), x, up)
    assert torch.equal(gg, rope.apply(up, pos))


@pytest.mark.gpu
def test_gradients_of_any_layout_and_twice():
    rope = Rope(64, *rope_table(32))
    base = torch.randn(20, 6, 64, device="cuda", requires_grad=True)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    x = base[:, 1:5]                                                # heads of a wider projection
    for make in (lambda y: y.sum(), lambda y: y[:, 2].sum(), lambda y: (y.transpose(0, 1).contiguous() * 2).sum(),
                 lambda y: y.permute(2, 0, 1).reshape(-1).square().sum()):
        (g,) = torch.autograd.grad(make(rope.apply(x, pos)), base)
        y = rope.apply(x.detach(), pos).requires_grad_()
        (gy,) = torch.autograd.grad(make(y), y)
        want = torch.zeros_like(base)
        want[:, 1:5] = rope.apply(gy.contiguous(), pos, grad=True)
        assert torch.equal(g, want)
    y = rope.apply(x, pos)
    (g,) = torch.autograd.grad((y ** 3).sum(), base, create_graph=True)
    (gg,) = torch.autograd.grad(g.sum(), base)                      # through the backward, once more
    v = torch.ones(20, 4, 64, device="cuda")
    t = rope.apply(x.detach(), pos)
    want = torch.zeros_like(base)
    want[:, 1:5] = rope.apply(6 * t * rope.apply(v, pos), pos, grad=True)
    torch.testing.assert_close(gg, want, rtol=2.0 ** -18, atol=2.0 ** -16)


@pytest.mark.gpu
def test_autograd_notices_what_is_written_in_place():
    rope = Rope(64, *rope_table(32))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    a = torch.randn(5, 2, 64, device="cuda", requires_grad=True)
    b = torch.randn(5, 2, 64, device="cuda")
    y = (a * b).sum()                                               # saves b
    rope.apply(b, pos, b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    z = rope.apply(a, pos).sum()
    pos.add_(1)                                                     # saved by the rotation
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.no_grad():                                           # nothing recorded, a written in place
        was = a._version
        assert rope.apply(a, pos, a) is a and a._version > was
    with torch.inference_mode():
        c = torch.randn(5, 2, 64, device="cuda")
        assert rope.apply(c, pos, c) is c


@pytest.mark.gpu
def test_backward_on_another_stream_and_captured():
    rope = Rope(64, *rope_table(32))
    pos = torch.arange(300, dtype=torch.int32, device="cuda")[None]
    x = torch.randn(300, 4, 64, device="cuda", requires_grad=True)
    up = torch.randn(300, 4, 64, device="cuda")
    want = rope.apply(up, pos, grad=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = rope.apply(x, pos, stream=side)
    side.synchronize()
    y.backward(up)
    torch.cuda.synchronize()
    assert torch.equal(x.grad, want)
    leaf = torch.randn(300, 4, 64, device="cuda", requires_grad=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.autograd.grad(rope.apply(leaf, pos), leaf, up)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        (g,) = torch.autograd.grad(rope.apply(leaf, pos), leaf, up)
    g.detach().zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, want)


@pytest.mark.gpu
def test_closed_table_in_backward():
    rope = Rope(64, *rope_table(32))
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    x = torch.ones(3, 1, 64, device="cuda", requires_grad=True)
    y = rope.apply(x, pos).sum()
    rope.close()
    with pytest.raises(vg.AttnError):
        y.backward()


@pytest.mark.gpu
def test_cosines_and_sines_of_far_positions():
    """Pairs (1, 0) turn into (cos, sin) themselves, in fp32 within 1.6 * 2^-24
    (a unit of the library's functions, half a one of a sum, 2 pi 2^-34 rad of
    the angle) and what 2^-60 |pos| rad of the angle and its 64-bit reference
    (pos freq off by 2^-53 of itself) are off by."""
    n = 32
    freqs = [1e4 ** (-i / n) for i in range(n)]
    rope = Rope(2 * n, freqs)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    pos = torch.randint(-(1 << 20), 1 << 20, (1, 20000), generator=g, device="cuda", dtype=torch.int32)
    x = torch.zeros(20000, 1, 2 * n, device="cuda")
    x[..., :n] = 1.0
    out = rope.apply(x, pos)[:, 0].double()
    theta = pos.double().t() * torch.tensor(freqs, dtype=torch.float64, device="cuda")
    bound = 1.6 * 2.0 ** -24 + 2.0 ** 20 * (2.0 ** -60 + 2.0 ** -52)
    assert (out[:, :n] - torch.cos(theta)).abs().max() <= bound
    assert (out[:, n:] - torch.sin(theta)).abs().max() <= bound
    back = rope.apply(x, pos, grad=True)[:, 0]
    assert torch.equal(back[:, :n].double(), out[:, :n]) and torch.equal(back[:, n:].double(), -out[:, n:])
    # quarter turns are exact
    quarter = Rope(2, [math.pi / 2])
    y = quarter.apply(torch.tensor([[[1.0, 0.0]]] * 4, device="cuda"), torch.arange(4, dtype=torch.int32, device="cuda")[None])
    want = torch.tensor([[1.0, 0.0], [0.0, 1.0], [-1.0, 0.0], [0.0, -1.0]], device="cuda")
    assert (y[:, 0] - want).abs().max() <= 2.0 ** -52

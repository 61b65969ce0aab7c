"""The layer operators and the codec together: a tensor-parallel feed-forward layer, forward and backward, against
64-bit arithmetic without the codec.

Bounds on the 2-norm.  A value that passes the codec once is within half a step of its format: E4M3 within 2^-4 of
itself in the transformed domain (an isometry); INT8 within 1/254 of its block's largest value, at most 5 times the
root mean square of 64 normal values: 0.012 of the norm; INT4 within 1/30 of a group's range, at most 7 such: 0.14
(half of it, 0.07, as a uniform error's root mean square is 1/sqrt 3 of its largest).  The all-reduce has two such
steps.  16-bit roundings along the way add 2^-8 for each of at most ten operations."""
import pytest
import torch

import quantized_tensor_activation_gb300 as qta
from quantized_tensor_activation_gb300 import tp_ffn
from gpu_util import device

pytestmark = pytest.mark.gpu

CODEC = {"taco_fp8": 2 * 2.0 ** -4, "int8_sym": 2 * 0.012, "int4_asym": 0.14 + 0.012}


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def reference(x, r, do, ds, p, kind):
    leaf = lambda t: None if t is None else t.double().requires_grad_(True)
    q = {k: [leaf(w) for w in v] if isinstance(v, list) else leaf(v) for k, v in p.items()}
    x64, r64 = leaf(x), leaf(r)
    s = x64 if r is None else x64 + r64
    c = s - s.mean(1, keepdim=True) if kind == "layer" else s
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * q["gamma"]
    if q["beta"] is not None:
        y = y + q["beta"]
    o = sum((torch.nn.functional.silu(y @ g.T) * (y @ u.T)) @ d.T for g, u, d in zip(q["wg"], q["wu"], q["wd"]))
    if q["bias"] is not None:
        o = o + q["bias"]
    torch.autograd.backward([o, s], [do.double(), ds.double()])
    return s.detach(), o.detach(), x64.grad, q


@pytest.mark.parametrize("codec", sorted(CODEC))
@pytest.mark.parametrize("rows,hidden,widths,kind,bias", [
    (256, 512, [264, 256, 200, 128], "rms", False), (333, 256, [344, 136], "layer", True), (1, 512, [128] * 4, "rms", False),
    (6, 1024, [344] * 2, "layer", True)])
def test_step(rows, hidden, widths, kind, bias, codec):
    device()
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + hidden)
    x, r, do, ds = (torch.randn(rows, hidden, generator=g, device="cuda").bfloat16() for _ in range(4))
    p = tp_ffn.random_params(hidden, widths, kind=kind, bias=bias, seed=7)
    layer = tp_ffn.TPFeedForward(rows, hidden, widths, kind=kind, codec=codec)
    s, o = layer.forward(x, p, residual=r)
    dx, grads = layer.backward(do, p, ds=ds)
    torch.cuda.synchronize()
    assert qta.qta_device_error() == 0
    s64, o64, dx64, q = reference(x, r, do, ds, p, kind)
    few, codec_err = 10 * 2.0 ** -8, CODEC[codec]
    assert rel(s, s64) < 2.0 ** -8
    assert rel(o, o64) < codec_err + few
    # the weights' gradients do not pass the codec, those behind the backward all-reduce do
    for k in ("wg", "wu", "wd"):
        for a, b in zip(grads[k], q[k]):
            assert rel(a, b.grad) < few, k
    if bias:
        assert rel(grads["bias"], q["bias"].grad) < few
    assert rel(dx, dx64) < codec_err + few
    assert rel(grads["gamma"], q["gamma"].grad) < codec_err + few
    if kind == "layer":
        assert rel(grads["beta"], q["beta"].grad) < codec_err + few


def test_second_step_and_stream():
    """Buffers are reused: a second step, on another stream, gives the same bits."""
    device()
    rows, hidden, widths = 200, 512, [136, 128]
    p = tp_ffn.random_params(hidden, widths)
    x, r, do = (torch.randn(rows, hidden, device="cuda").bfloat16() for _ in range(3))
    layer = tp_ffn.TPFeedForward(rows, hidden, widths)

    def step(stream=None):
        _, o = layer.forward(x, p, residual=r, stream=stream)
        dx, g = layer.backward(do, p, stream=stream)
        return [o.clone(), dx.clone(), g["wg"][1].clone(), g["gamma"].clone()]

    a = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_refusals():
    device()
    with pytest.raises(ValueError):
        tp_ffn.TPFeedForward(8, 512, [64], codec="fp4")
    with pytest.raises(ValueError):
        tp_ffn.AllReduce(2, 8, 200, "bf16", "taco_fp8")

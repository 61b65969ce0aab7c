"""Argument checks of the layer operators' C ABI, on the host (no GPU; no call here enqueues anything) and the
binding's C layouts."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_tensor_activation_gb300 as qta  # noqa: E402
from quantized_tensor_activation_gb300 import layer  # noqa: E402

OK, INV, ALN, UNS = qta.QTA_OK, qta.QTA_ERR_INVALID_ARG, qta.QTA_ERR_ALIGNMENT, qta.QTA_ERR_UNSUPPORTED
A, B, C, D, E, F, G, W = (0x10000000 * i for i in range(1, 9))   # addresses that nothing dereferences


@pytest.fixture(scope="module")
def L():
    qta.build()
    return layer._lib()


def M(p, ld=0):
    return layer.Mat(p, ld)


def test_layouts(L):
    assert ctypes.sizeof(layer.Mat) == 16
    assert ctypes.sizeof(layer.NormDesc) == 32 and layer.NormDesc.eps.offset == 28
    assert ctypes.sizeof(layer.LinearDesc) == 48 and layer.LinearDesc.act.offset == 40
    assert ctypes.sizeof(layer.FfnDesc) == 40 and layer.FfnDesc.act.offset == 32


def test_linear_refusals(L):
    f = L.qta_linear
    d = qta.linear_desc(4, 64, 128, "bf16")
    assert f(None, M(A), M(B), None, None, M(C), None) == INV
    for bad, want in (((-1, 64, 128, "bf16"), INV), ((4, 0, 128, "bf16"), INV), ((4, 64, 0, "bf16"), INV),
                      ((4, 64, 128, "fp32"), UNS), ((4, 64, 128, 7), UNS), ((1 << 31, 64, 128, "bf16"), UNS),
                      ((4, 1 << 31, 128, "bf16"), UNS), ((4, 64, 128, "bf16", 9), UNS),
                      ((4, 64, 128, "bf16", "none", "fp16"), UNS), ((4, 64, 128, "bf16", "none", None, "fp16"), UNS),
                      ((4, 64, 128, "bf16", "none", None, None, "fp16"), UNS)):
        assert f(qta.linear_desc(*bad), M(A), M(B), None, None, M(C), None) == want, bad
    assert f(d, None, M(B), None, None, M(C), None) == INV
    assert f(d, M(None), M(B), None, None, M(C), None) == INV
    assert f(d, M(A), None, None, None, M(C), None) == INV
    assert f(d, M(A), M(B), None, None, None, None) == INV
    assert f(d, M(A), M(B), None, M(None), M(C), None) == INV
    assert f(d, M(A, 64), M(B), None, None, M(C), None) == INV      # rows overlap
    assert f(d, M(A, -128), M(B), None, None, M(C), None) == INV
    assert f(d, M(A, 132), M(B), None, None, M(C), None) == ALN     # rows off 16 bytes
    assert f(d, M(A + 8), M(B), None, None, M(C), None) == ALN
    assert f(d, M(A), M(B + 2), None, None, M(C), None) == ALN
    assert f(d, M(A), M(B), C + 1, None, M(D), None) == ALN
    assert f(d, M(A), M(B), None, None, M(C + 1), None) == ALN
    assert f(d, M(A), M(B), None, None, M(A + 512), None) == INV    # y over x
    assert f(d, M(A), M(B), None, None, M(B + 128 * 2), None) == INV
    assert f(d, M(A), M(B), None, M(C + 2), M(C), None) == INV      # y over the residual, not in place
    assert f(d, M(A), M(B), None, M(C, 70), M(C, 80), None) == INV
    assert f(d, M(A), M(B), C + 16, None, M(C), None) == INV        # y over the bias
    odd = qta.linear_desc(4, 64, 127, "bf16")
    assert f(odd, M(A), M(B), None, None, M(C), None) == ALN        # contiguous rows of 127 elements
    # nothing to do: no pointer is looked at
    assert f(qta.linear_desc(0, 64, 128, "bf16"), None, None, None, None, None, None) == OK


def test_linear_bwd_refusals(L):
    f = L.qta_linear_bwd
    d = qta.linear_desc(4, 64, 128, "bf16", "silu")
    assert f(None, M(A), M(B), M(C), None, M(D), M(E), F, W, None) == INV
    assert f(d, None, M(B), M(C), None, M(D), M(E), F, W, None) == INV
    assert f(d, M(A), M(B), M(C), None, M(D), M(E), F, None, None) == INV     # no workspace
    assert f(d, M(A), M(B), M(C), None, M(D), M(E), F, W + 8, None) == ALN
    assert f(d, M(A + 2), M(B), M(C), None, M(D), M(E), F, W, None) == ALN
    assert f(d, M(A), M(B), M(C), None, M(D), M(E), F + 2, W, None) == ALN
    assert f(d, M(A), M(B), M(C), None, M(B + 2), M(E), F, W, None) == INV    # dx over x
    assert f(d, M(A), M(B), M(C), None, M(D), M(D + 64), F, W, None) == INV   # dw over dx
    assert f(d, M(A), M(B), M(C), None, M(D), M(E), W + 64, W, None) == INV   # dbias in the workspace
    assert f(d, M(A), M(B), M(C), None, M(W + 16), M(E), F, W, None) == INV   # dx in the workspace
    n = qta.linear_bwd_workspace_bytes(d)
    assert n >= 4 * 64 * 2 + 64 * 4
    assert qta.linear_bwd_workspace_bytes(qta.linear_desc(4, 0, 128, "bf16")) == 0


def test_ffn_refusals(L):
    f, b = L.qta_gated_ffn, L.qta_gated_ffn_bwd
    d = qta.ffn_desc(4, 64, 128, "fp16")
    assert f(None, M(A), M(B), M(C), M(D), None) == INV
    assert f(qta.ffn_desc(4, 64, 128, "fp32"), M(A), M(B), M(C), M(D), None) == UNS
    assert f(qta.ffn_desc(4, 64, 128, "fp16", 5), M(A), M(B), M(C), M(D), None) == UNS
    assert f(qta.ffn_desc(4, 0, 128, "fp16"), M(A), M(B), M(C), M(D), None) == INV
    assert f(d, M(A), M(B), None, M(D), None) == INV
    assert f(d, M(A), M(B), M(C + 2), M(D), None) == ALN
    assert f(d, M(A), M(B), M(C), M(C + 64), None) == INV
    assert f(qta.ffn_desc(0, 64, 128, "fp16"), None, None, None, None, None) == OK
    assert b(d, M(A), M(B), M(C), M(D), M(E), M(F), None, W, None) == INV       # dwg without dwu
    assert b(d, M(A), M(B), M(C), M(D), M(E), M(F), M(F + 2), W, None) == INV   # on top of each other
    assert b(d, M(A), M(B), M(C), M(D), M(E), M(F), M(G), None, None) == INV
    assert b(d, M(A), M(B), M(C), M(D), M(E), M(F), M(G), W + 4, None) == ALN
    assert b(d, M(A), M(B), M(C), M(D), M(W + 32), M(F), M(G), W, None) == INV
    assert qta.gated_ffn_bwd_workspace_bytes(d) >= 2 * 4 * 128 * 2


def test_norm_refusals(L):
    f, b = L.qta_norm, L.qta_norm_bwd
    d, rms = qta.norm_desc(4, 100, "bf16"), qta.norm_desc(4, 100, "bf16", "rms")
    assert f(None, M(A), None, B, None, M(C), None, None, None, None) == INV
    for bad, want in (((-1, 8, "bf16"), INV), ((4, 0, "bf16"), INV), ((4, 8, 5), UNS), ((4, 8, "bf16", 2), UNS),
                      ((4, 8, "bf16", "layer", -1.0), INV), ((4, 8, "bf16", "layer", float("nan")), INV),
                      ((4, 8, "bf16", "layer", float("inf")), INV), ((4, 8, "bf16", "layer", 1e-5, "fp16"), UNS),
                      ((1 << 31, 8, "bf16"), UNS)):
        assert f(qta.norm_desc(*bad), M(A), None, B, None, M(C), None, None, None, None) == want, bad
    assert f(d, M(A), None, None, None, M(C), None, None, None, None) == INV
    assert f(d, M(A + 1), None, B, None, M(C), None, None, None, None) == ALN
    assert f(d, M(A), None, B, None, M(C), None, D + 2, None, None) == ALN
    assert f(d, M(A), None, B, None, M(A), None, None, None, None) == INV            # y over x
    assert f(d, M(A), M(B), C, None, M(D), M(B), None, None, None) == INV            # sum over the residual
    assert f(d, M(A), None, B, None, M(C), M(C + 200), None, None, None) == INV      # y over sum
    assert f(rms, M(A), None, B, C, M(D), None, None, None, None) == INV             # RMS has no beta
    assert f(rms, M(A), None, B, None, M(D), None, C, None, None) == INV             # and no mean
    assert f(qta.norm_desc(0, 8, "bf16"), None, None, None, None, None, None, None, None, None) == OK
    assert b(d, M(A), M(B), C, None, D, None, M(E), F, G, W, None) == INV            # the layer norm's mean
    assert b(rms, M(A), M(B), C, None, D, None, M(E), F, G, W, None) == INV          # RMS has no dbeta
    assert b(d, M(A), M(B), C, D, D + 64, None, M(E), None, G, W, None) == INV       # no dgamma
    assert b(d, M(A), M(B), C, D, D + 64, None, M(E), F, F + 200, W, None) == INV    # dbeta over dgamma
    assert b(d, M(A), M(B), C, D, D + 64, None, M(A), F, G, W, None) == INV          # dx over dy
    assert b(d, M(A), M(B), C, D, D + 64, None, M(E), F, G, None, None) == INV
    assert b(d, M(A), M(B), C, D, D + 64, None, M(E), F, G, W + 4, None) == ALN
    assert qta.norm_bwd_workspace_bytes(d) >= 4 * 100 * 8


def test_names_are_checked():
    with pytest.raises(ValueError):
        qta.linear_desc(1, 8, 8, "int8")
    with pytest.raises(ValueError):
        qta.norm_desc(1, 8, "bf16", "batch")
    with pytest.raises(AttributeError):
        qta.no_such_call


def test_cpu_tensors_are_refused():
    d = qta.linear_desc(4, 32, 64, "bf16")
    x, w, y = (torch.zeros(a, b, dtype=torch.bfloat16) for a, b in ((4, 64), (32, 64), (4, 32)))
    with pytest.raises(ValueError):
        qta.qta_linear(d, x, w, y, stream=0)

"""The example layer (norm to 8 bits -> 8-bit product -> 4-bit product and their
gradients): each stage against the oracle on what the stage before it put out, so
that the bounds are those of the single operators."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from oracle import qmm_oracle as O
from _helpers import half_ulp
from test_gpu_fp4 import check_product
from test_gpu_rms_norm import check_backward, check_forward, f32

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantised_layer.py")
_spec = importlib.util.spec_from_file_location("quantised_layer", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def inputs(M, H, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, res, dh = (torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    return x, res, torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16), dh


def check_y(layer, qv, scale, y):
    want = O.a8w8(qv.cpu().numpy(), layer.W1.cpu().numpy(), scale.cpu().numpy(), layer.scale1.cpu().numpy(), "bf16")
    assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,H,F,N", [(1, 256, 512, 128), (70, 200, 300, 130), (300, 512, 384, 256)])
def test_serve(M, H, F, N, block):
    layer, _ = example.make(H, F, N, block)
    x, res, _, _ = inputs(M, H, N, M)
    z, h = layer.serve(x, res)
    q.check_device_error()
    n = q.qmm_rms_norm_s8(x, layer.norm, residual=res, eps=layer.eps, save_rstd=True)
    check_forward(x, res, layer.norm, n, layer.eps)
    assert torch.equal(h, n.h)
    y = q.qmm_a8w8(n.q, layer.W1, n.scale, layer.scale1)
    check_y(layer, n.q, n.scale, y)
    check_product(y, layer.W2, block, torch.bfloat16, z)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,H,F,N", [(70, 200, 300, 130), (300, 512, 384, 256)])
def test_train_step(M, H, F, N, block):
    layer, _ = example.make(H, F, N, block)
    x, res, dz, dh = inputs(M, H, N, 3 * M)
    s = layer.train_step(x, res, dz, dh)
    q.check_device_error()
    check_forward(x, res, layer.norm, q.RmsNormS8(s["q"], s["scale"], s["h"], s["rstd"]), layer.eps)
    check_y(layer, s["q"], s["scale"], s["y"])
    check_product(s["y"], layer.W2, block, torch.bfloat16, s["z"])
    check_product(dz, layer.W2.T.contiguous(), block, torch.bfloat16, s["dy"])
    check_product(dz.T.contiguous(), s["y"].T.contiguous(), block, torch.float32, s["dW2"])
    # bf16 times int8 with a float32 sum of F terms (F additions of half an ulp at most), then bf16
    A, B = f32(s["dys"]).astype(np.float64), layer.W1.cpu().numpy().astype(np.float64).T
    want = A @ B
    err = np.abs(f32(s["dn"]).astype(np.float64) - want)
    assert (err <= F * 2.0 ** -24 * (np.abs(A) @ np.abs(B)) + 1.01 * half_ulp(want, 7)).all()
    check_backward(s["dn"], s["h"], layer.norm, s["rstd"], dh, s["dx"], s["dnorm"])


def test_near_the_unquantised_layer():
    """8 bits are off by about 0.3 % of a product's size (a step of max / 127 against values of about
    max / 4, evened out over both operands) and 4-bit blocks of 32 by about 0.11 an operand, so two of them
    by 0.16; twice that is the bound for the forward product and the gradient that goes through two more."""
    M, H, F, N = 512, 512, 768, 512
    layer, W1 = example.make(H, F, N, 32)
    x, res, dz, dh = inputs(M, H, N, 5)
    s = layer.train_step(x, res, dz, dh)
    want = example.plain(layer, W1, x, res, dz, dh)
    for k in ("z", "dx", "dnorm", "dW2"):
        rel = float((s[k].double() - want[k]).norm() / want[k].norm())
        assert rel < 0.32, (k, rel)

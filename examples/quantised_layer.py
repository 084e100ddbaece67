"""A residual layer on the library's quantised operators, run for one token, for a
prompt and through a training step:

    h = x + residual            n = h / rms(h) * norm          (8 bits, a scale a row)
    y = n @ W1                  frozen, 8 bits, a scale a column
    z = y @ W2^T                trained, 4-bit blocks

serve() reads W1 at one byte a weight and W2 at 0.53 (0.56 in blocks of 16);
train_step() returns the gradients of x (and, equally, of the residual), of the
norm's weight and of W2.

    python examples/quantised_layer.py [--hidden 4096] [--inner 11008] [--tokens 2048] [--block 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_int8_matmul_gb300 as q  # noqa: E402


class QuantisedLayer:
    """norm [H]; W1 float [H, F], kept as int8 with a scale a column; W2 bf16 [N, F]."""

    def __init__(self, norm, W1, W2, block=32, eps=1e-6):
        self.norm, self.W2, self.block, self.eps = norm, W2, block, eps
        amax = W1.float().abs().amax(dim=0).clamp_min(1e-30)
        self.scale1 = amax / 127
        self.W1 = (W1.float() / self.scale1).round().clamp(-127, 127).to(torch.int8)
        self.W1t = self.W1.T.contiguous()   # for the gradient of n
        self.ones = torch.ones(W1.shape[0], device=W1.device)
        self.W2q = q.qmm_fp4_quantize(W2, block=block)

    def serve(self, x, residual):
        """(z, h) for any number of tokens; h is the next layer's residual."""
        n = q.qmm_rms_norm_s8(x, self.norm, residual=residual, eps=self.eps)
        y = q.qmm_a8w8(n.q, self.W1, n.scale, self.scale1)
        return q.qmm_fp4_matmul(q.qmm_fp4_quantize(y, block=self.block), self.W2q), n.h

    def train_step(self, x, residual, dz, dh):
        """The step's values by name, from the gradients of z and of h (what the layers above send down)."""
        b = self.block
        n = q.qmm_rms_norm_s8(x, self.norm, residual=residual, eps=self.eps, save_rstd=True)
        y = q.qmm_a8w8(n.q, self.W1, n.scale, self.scale1)
        # each product sums over another axis of its operands, so each is packed along both
        yq, yt = q.qmm_fp4_quantize_both(y, block=b)
        wq, wt = q.qmm_fp4_quantize_both(self.W2, block=b)
        z = q.qmm_fp4_matmul(yq, wq)
        dzq, dzt = q.qmm_fp4_quantize_both(dz, block=b)
        dy = q.qmm_fp4_matmul(dzq, wt)
        dW2 = q.qmm_fp4_matmul(dzt, yt, out_dtype=torch.float32)
        # the columns' scales of W1 are on the axis that the gradient sums over
        dys = (dy * self.scale1).to(torch.bfloat16)
        dn = q.qmm_w8_dequant(dys, self.W1t, self.ones, out_dtype=torch.bfloat16)
        dx, dnorm = q.qmm_rms_norm_backward(dn, n.h, self.norm, n.rstd, dh=dh)
        return {"z": z, "h": n.h, "rstd": n.rstd, "y": y, "dy": dy, "dys": dys, "dn": dn, "dx": dx, "dnorm": dnorm,
                "dW2": dW2, "q": n.q, "scale": n.scale}


def make(H, F, N, block=32, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    norm = (1 + 0.1 * torch.randn(H, generator=g, device=device)).to(torch.bfloat16)
    W1 = torch.randn(H, F, generator=g, device=device) / H ** 0.5
    W2 = (torch.randn(N, F, generator=g, device=device) / F ** 0.5).to(torch.bfloat16)
    return QuantisedLayer(norm, W1, W2, block), W1


def plain(layer, W1, x, residual, dz, dh):
    """z and the gradients in float64, with nothing quantised."""
    h = (x + residual).double().requires_grad_()
    w, W2 = layer.norm.double().requires_grad_(), layer.W2.double().requires_grad_()
    n = h * torch.rsqrt(h.pow(2).mean(dim=1, keepdim=True) + layer.eps) * w
    z = n @ W1.double() @ W2.T
    torch.autograd.backward([z, h], [dz.double(), dh.double()])
    return {"z": z.detach(), "dx": h.grad, "dnorm": w.grad, "dW2": W2.grad}


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=11008)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--block", type=int, default=32, choices=(16, 32))
    a = p.parse_args()
    layer, W1 = make(a.hidden, a.inner, a.hidden, a.block)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res, dz, dh = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    step = layer.train_step(x, res, dz, dh)
    z1, _ = layer.serve(x[:1], res[:1])
    zs, _ = layer.serve(x, res)
    q.check_device_error()
    want = plain(layer, W1, x, res, dz, dh)
    print(f"{a.tokens} tokens, {a.hidden} -> {a.inner} -> {a.hidden}, blocks of {a.block}")
    print("relative distance from the same layer in float64 without quantisation:")
    for name, got, ref in (("one token", z1, want["z"][:1]), ("prompt", zs, want["z"]),
                           *((k, step[k], want[k]) for k in ("z", "dx", "dnorm", "dW2"))):
        print(f"  {name:10s} {float((got.double() - ref).norm() / ref.norm()):.4f}")


if __name__ == "__main__":
    main()

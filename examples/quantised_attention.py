"""An attention block on the library's quantised operators, for prompts and for single
tokens of several sequences at once:

    h = x + residual            n = h / rms(h) * norm                (8 bits, a scale a row)
    qkv = n @ Wqkv              8 bits, a scale a column
    keys and queries rotated to their positions, keys and values into the cache (8 bits)
    a = softmax(q k^T) v        over the cache
    z = a @ Wo^T                4-bit blocks

    python examples/quantised_attention.py [--heads 32] [--kv-heads 8] [--prompt 1000] [--tokens 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_int8_matmul_gb300 as q  # noqa: E402


class AttentionBlock:
    """norm [H]; Wqkv float [H, (heads + 2 kv_heads) * dim]; Wo bf16 [H, heads * dim]."""

    def __init__(self, norm, Wqkv, Wo, heads, kv_heads, positions, base=500000.0, eps=1e-6):
        self.norm, self.eps, self.heads, self.kv_heads = norm, eps, heads, kv_heads
        self.dim = Wo.shape[1] // heads
        self.scale = Wqkv.float().abs().amax(dim=0).clamp_min(1e-30) / 127
        self.Wqkv = (Wqkv.float() / self.scale).round().clamp(-127, 127).to(torch.int8)
        self.Wo = q.qmm_fp4_quantize(Wo, block=16)
        half = self.dim // 2
        # angles of far positions need more than float32
        angle = (torch.arange(positions, dtype=torch.float64, device=norm.device)[:, None]
                 * base ** (-torch.arange(half, dtype=torch.float64, device=norm.device) / half))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def __call__(self, x, residual, cache, table, lengths, starts=None, max_tokens=None):
        """The step's values by name: x, residual [tokens, H], the sequences' tokens behind each other
        (starts; None: one each), lengths with the new tokens."""
        n = q.qmm_rms_norm_s8(x, self.norm, residual=residual, eps=self.eps)
        qkv = q.qmm_a8w8(n.q, self.Wqkv, n.scale, self.scale).view(x.shape[0], -1, self.dim)
        k, v = qkv[:, self.heads:-self.kv_heads], qkv[:, -self.kv_heads:]
        turned = q.qmm_kv_append(cache, k, v, table, lengths, starts=starts, q=qkv[:, :self.heads], cos=self.cos,
                                 sin=self.sin)
        a = q.qmm_kv_attention(turned, cache, table, lengths, starts=starts, max_tokens=max_tokens)
        z = q.qmm_fp4_matmul(q.qmm_fp4_quantize(a.view(x.shape[0], -1), block=16), self.Wo)
        return {"z": z, "h": n.h, "qkv": qkv, "q": turned, "a": a}


def make(heads, kv_heads, dim, positions, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    H = heads * dim
    norm = (1 + 0.1 * torch.randn(H, generator=g, device=device)).to(torch.bfloat16)
    Wqkv = torch.randn(H, (heads + 2 * kv_heads) * dim, generator=g, device=device) / H ** 0.5
    Wo = (torch.randn(H, H, generator=g, device=device) / H ** 0.5).to(torch.bfloat16)
    return AttentionBlock(norm, Wqkv, Wo, heads, kv_heads, positions), Wqkv, Wo


def plain(block, Wqkv, Wo, x, residual):
    """z of one sequence from its beginning, in float64 with nothing quantised."""
    h = (x + residual).double()
    n = h * torch.rsqrt(h.pow(2).mean(dim=1, keepdim=True) + block.eps) * block.norm.double()
    qkv = (n @ Wqkv.double()).view(len(x), -1, block.dim)
    c, s = (t[:len(x), None].double() for t in (block.cos, block.sin))

    def turn(t):
        a, b = t.chunk(2, dim=2)
        return torch.cat([a * c - b * s, b * c + a * s], dim=2)

    k, v = turn(qkv[:, block.heads:-block.kv_heads]), qkv[:, -block.kv_heads:]
    k, v = (t.repeat_interleave(block.heads // block.kv_heads, dim=1) for t in (k, v))
    score = torch.einsum("thd,shd->hts", turn(qkv[:, :block.heads]), k) / block.dim ** 0.5
    score.masked_fill_(torch.ones_like(score[0], dtype=torch.bool).triu(1), -torch.inf)
    return torch.einsum("hts,shd->thd", score.softmax(dim=2), v).reshape(len(x), -1) @ Wo.double().T


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--dim", type=int, default=128, choices=(64, 128))
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--tokens", type=int, default=20)
    a = p.parse_args()
    total = a.prompt + a.tokens
    block, Wqkv, Wo = make(a.heads, a.kv_heads, a.dim, total)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randn(total, a.heads * a.dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pages = -(-total // 64)
    cache = q.qmm_kv_cache(pages, a.kv_heads, a.dim)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).view(1, -1)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    z = [block(x[:a.prompt], res[:a.prompt], cache, table, ints(a.prompt), starts=ints(0, a.prompt))["z"]]
    for i in range(a.prompt, total):
        z.append(block(x[i:i + 1], res[i:i + 1], cache, table, ints(i + 1), max_tokens=1)["z"])
    q.check_device_error()
    want = plain(block, Wqkv, Wo, x, res)
    print(f"{a.heads} query heads on {a.kv_heads} of {a.dim}: relative distance from float64 without quantisation")
    for name, part, ref in (("prompt", z[0], want[:a.prompt]), ("tokens", torch.cat(z[1:]), want[a.prompt:])):
        if len(ref):
            print(f"  {name:7s} {float((part.double() - ref).norm() / ref.norm()):.4f}")


if __name__ == "__main__":
    main()

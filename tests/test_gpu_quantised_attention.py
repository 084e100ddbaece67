"""The example attention block (norm to 8 bits -> 8-bit product -> cache -> attention ->
4-bit product): prompts, then token by token, of several sequences; each stage against
the oracle on what the stage before it put out."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from _kv import assert_attention, attention_bound, rounded
from test_gpu_fp4 import check_product

pytestmark = pytest.mark.gpu
q = pytest.importorskip("quantized_int8_matmul_gb300")

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantised_attention.py")
_spec = importlib.util.spec_from_file_location("quantised_attention", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 2, 64, 16), (8, 1, 128, 48)])
def test_prompts_and_tokens(heads, kv_heads, dim, page):
    prompts, steps = [37, 5, 130], 6
    block, _, Wo = example.make(heads, kv_heads, dim, max(prompts) + steps)
    width = -(-(max(prompts) + steps) // page)
    cache = q.qmm_kv_cache(3 * width + 1, kv_heads, dim, page=page)
    rng = np.random.default_rng(0)
    table = rng.permutation(3 * width).astype(np.int32).reshape(3, width)
    arrays = [t.cpu().numpy() for t in cache]
    dt = torch.from_numpy(table).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    cos, sin = block.cos.cpu().numpy(), block.sin.cpu().numpy()
    for step in range(steps + 1):
        new = prompts if step == 0 else [1, 1, 1]
        lengths = np.array([n + step for n in prompts], np.int32)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x, res = (torch.randn(sum(new), heads * dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        r = block(x, res, cache, dt, torch.from_numpy(lengths).cuda(),
                  starts=torch.from_numpy(starts).cuda() if step == 0 else None, max_tokens=max(new))
        q.check_device_error()
        qkv = r["qkv"].float().cpu().numpy()
        want_q = ko.append(*arrays, qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], table, lengths, starts, cos,
                           sin, False, qkv[:, :heads])
        for got, want in zip(cache, arrays):
            assert np.array_equal(got.cpu().numpy(), want)
        turned = r["q"].float().cpu().numpy()
        assert np.array_equal(turned, rounded(want_q, "bf16"))
        exact, mag, top, seen = ko.attention(turned.astype(np.float64), *arrays, table, lengths, starts, dim ** -0.5, True,
                                             detail=True)
        assert_attention(r["a"].double().cpu().numpy(), exact, attention_bound(exact, mag, top, seen, "bf16", dim))
        check_product(r["a"].view(len(x), -1), Wo, 16, torch.bfloat16, r["z"])


def test_a_token_at_a_time_is_the_prompt():
    """The last row of a prompt and the same token appended alone see the same cache but for the blocks' scales:
    here each block's largest numbers come first, so that not even those differ."""
    block, _, _ = example.make(4, 2, 64, 64)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v, x = (torch.randn(40, h, 64, generator=g, device="cuda") for h in (2, 2, 4))
    decay = torch.where(torch.arange(40, device="cuda") % 16 == 0, 1.0, 0.05)[:, None, None]
    k, v, x = (k * decay).bfloat16(), (v * decay).bfloat16(), x.bfloat16()
    ints = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda")
    whole, single = q.qmm_kv_cache(3, 2, 64, page=16), q.qmm_kv_cache(3, 2, 64, page=16)
    qw = q.qmm_kv_append(whole, k, v, table, ints(40), starts=ints(0, 40), q=x, cos=block.cos, sin=block.sin)
    qs = torch.cat([q.qmm_kv_append(single, k[i:i + 1], v[i:i + 1], table, ints(i + 1), q=x[i:i + 1], cos=block.cos,
                                    sin=block.sin) for i in range(40)])
    assert torch.equal(qw, qs)
    for a, b in zip(whole, single):
        assert torch.equal(a, b)
    rows = q.qmm_kv_attention(qw, whole, table, ints(40), starts=ints(0, 40))
    one = q.qmm_kv_attention(qs[39:], single, table, ints(40))
    assert torch.allclose(rows[39:].float(), one.float(), rtol=2 ** -7, atol=1e-5)


def test_the_example_runs():
    import sys
    argv, sys.argv = sys.argv, ["quantised_attention.py", "--heads", "4", "--kv-heads", "2", "--dim", "64", "--prompt", "50",
                                "--tokens", "3"]
    try:
        example.main()
    finally:
        sys.argv = argv

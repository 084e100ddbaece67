"""Attention over values near the largest float32: parts of a long sequence are joined without leaving its range."""
import numpy as np
import pytest
import torch

from _kv import Batch
from test_gpu_kv_attention import q, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,group", [([(1, 9000)], 2), ([(2, 5000), (1, 40)], 2), ([(40, 6000)], 4), ([(150, 150)], 2)])
def test_values_near_the_largest_number(q, kind, seqs, group):  # noqa: F811
    for dim in (64, 128):
        b = Batch(seqs, 1, dim, 64, seed=15)
        b.ke[:] = 118
        b.ve[:] = 249                                  # a step of 2^122: 63 of them are below 2^128
        b.vc[:] = b.rng.integers(40, 64, b.vc.shape) * b.rng.choice([-1, 1], dim).astype(np.int8)
        y = run(q, b, kind, group, max_tokens=max(n for n, _ in seqs))
        assert torch.isfinite(y).all()

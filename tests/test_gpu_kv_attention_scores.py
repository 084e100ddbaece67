"""Attention over the 8-bit cache for scores of any finite size. Keys are zeros but for one element each, so that
a row's scores are whole multiples of one large number: its softmax picks the largest ones, shared evenly."""
import numpy as np
import pytest
import torch

from _kv import TYPES, Batch
from test_gpu_kv_attention import q  # noqa: F401

pytestmark = pytest.mark.gpu

FEW = [(1, 1), (8, 69), (3, 130), (1, 1700)]
MANY = [(128, 128), (100, 260), (20, 2500)]


def picked(b, sign, group, causal):
    """The mean of the visible values whose key is the largest (sign +1) or the smallest."""
    out, mag = (np.zeros((b.rows, b.heads * group, b.dim)) for _ in range(2))
    for s, (n, length) in enumerate(b.seqs):
        at = b.table[s, np.arange(length) // b.page], np.arange(length) % b.page
        step = 2.0 ** (b.ve[at[0], :, at[1] // 16].astype(int) - 127)
        v = b.vc[at[0], :, at[1]] * step[..., None]                     # [tokens, heads, dim]
        k = b.kc[at[0], :, at[1], 0].astype(int) * sign
        for i in range(n):
            lim = length - n + i + 1 if causal else length
            for h in range(b.heads):
                best = k[:lim, h] == k[:lim, h].max()
                out[b.starts[s] + i, h * group:(h + 1) * group] = v[:lim, h][best].mean(axis=0)
                mag[b.starts[s] + i, h * group:(h + 1) * group] = np.abs(v[:lim, h][best]).mean(axis=0)
    return out, mag


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("seqs,group", [(FEW, 2), (MANY, 4)])
@pytest.mark.parametrize("magnitude", [2.0 ** e for e in (14, 20, 27, 30, 40, 70, 100, 112)])
def test_scores_of_any_size(q, kind, seqs, group, magnitude):  # noqa: F811
    """All below zero, all above it, and of either sign. The softmax is the mean of one or a few tokens: P is the same for
    each of them, off by its own rounding (2^-11, in two parts 2^-21); O is summed 16 tokens at a time, at most 2500 in
    all, and a handful of operations follow, each off by 2^-23 or less, doubled for the numerator and the sum."""
    for low, high in ((-127, -1), (1, 127), (-127, 127)):
        for sign in (1, -1):
            for causal in (True, False):
                b = Batch(seqs, 2, 64, 32, seed=14)
                b.kc[..., 1:] = 0
                b.kc[..., 0] = b.rng.integers(low, high + 1, b.kc.shape[:-1])
                b.ke[:] = 150
                b.ve[:] = 120
                x = np.zeros((b.rows, 2 * group, 64), np.float32)
                x[..., 0] = sign * magnitude * 2.0 ** -23 * 1.25       # a score: 1.25 * magnitude / 8 * an integer
                y = q.qmm_kv_attention(torch.from_numpy(x).to(TYPES[kind]).cuda(), *b.device(q), causal=causal,
                                       max_tokens=max(n for n, _ in seqs))
                want, mag = picked(b, sign, group, causal)
                got = y.double().cpu().numpy()
                half, p = (2.0 ** -8, 2.0 ** -11) if kind == "bf16" else (2.0 ** -24, 2.0 ** -21)
                bound = np.abs(want) * half + mag * (p + (2500 / 16 + 8) * 2.0 ** -22)
                assert (np.abs(got - want) <= bound).all(), (low, high, sign, causal, np.abs(got - want).max())
    q.check_device_error()

"""Attention over the 8-bit cache where its values' scales lie far apart: what a row sees with little
weight, or not at all, must cost the rest of it no digits."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as ko
from _kv import TYPES, Batch, assert_attention, attention_bound, rounded
from test_gpu_kv_attention import q, run  # noqa: F401

pytestmark = pytest.mark.gpu

GAPS = [12, 24, 29, 31, 40, 60, 100, 120]
FEW = [(8, 69), (3, 130), (1, 70)]   # the kernel for single tokens
MANY = [(128, 128), (100, 260)]      # the tensor cores'


def set_bytes(b, exps, rule):
    """exps of block i of sequence s: rule(s, i)."""
    per = b.page // 16
    for s in range(len(b.seqs)):
        for i in range(b.width * per):
            if b.table[s, i // per] >= 0:
                exps[b.table[s, i // per], :, i % per] = rule(s, i)


def check(q, seqs, kind, rule, group=2, causal=True, dim=64, kernel=None, x=None, seed=11, zero=None):  # noqa: F811
    b = Batch(seqs, 2, dim, 32, seed=seed)
    b.ke[:] = 118
    set_bytes(b, b.ve, rule)
    if zero is not None:
        b.vc[np.repeat(b.ve == zero, 16, axis=2)] = 0
    run(q, b, kind, group, causal=causal, kernel=kernel, x=x, max_tokens=max(n for n, _ in seqs))


def each(f):
    for name, params in (("kind", ["bf16", "f32"]), ("seqs,group,kernel", [(FEW, 2, "kv_attention_rows"),
                                                                          (MANY, 4, None)])):
        f = pytest.mark.parametrize(name, params)(f)
    return f


@each
@pytest.mark.parametrize("gap", GAPS)
def test_values_that_grow(q, kind, seqs, group, kernel, gap):  # noqa: F811
    """From token 64 on values are 2^gap larger: rows before it do not see them, the first rows behind it see few."""
    check(q, seqs, kind, lambda s, i: 118 + gap * (i >= 4), group, kernel=kernel)
    check(q, seqs, kind, lambda s, i: 118 + gap * (i >= 4), group, kernel=kernel, dim=128)
    check(q, seqs, kind, lambda s, i: 118 + gap * (i >= 4), group, causal=False)


@each
@pytest.mark.parametrize("gap", GAPS)
def test_values_that_shrink_and_come_and_go(q, kind, seqs, group, kernel, gap):  # noqa: F811
    check(q, seqs, kind, lambda s, i: 118 + gap * (i < 4), group, kernel=kernel)
    check(q, seqs, kind, lambda s, i: 118 + gap * (i == 4), group, kernel=kernel)
    check(q, seqs, kind, lambda s, i: 118 + gap * (i % 2), group, kernel=kernel)
    check(q, seqs, kind, lambda s, i: max(118 - gap * (i % 3), 0), group, kernel=kernel)


@each
def test_every_block_at_a_scale_of_its_own(q, kind, seqs, group, kernel):  # noqa: F811
    for order in (1, -1):
        check(q, seqs, kind, lambda s, i: 10 + 29 * (order * i % 8), group,
              kernel=kernel)
    check(q, seqs, kind, lambda s, i: 40 + (53 * i) % 181, group, kernel=kernel)


@each
def test_blocks_of_zeros(q, kind, seqs, group, kernel):  # noqa: F811
    """A block of zeros has the smallest byte; so does one of numbers around 2^-121."""
    for rule in (lambda s, i: 0 if i % 2 else 120, lambda s, i: 120 if i == 2 else 0, lambda s, i: 0):
        check(q, seqs, kind, rule, group, kernel=kernel, zero=0)
        check(q, seqs, kind, rule, group, kernel=kernel)


@each
@pytest.mark.parametrize("gap", [12, 24, 30, 40, 60])
@pytest.mark.parametrize("where", ["first", "last", "middle"])
def test_large_values_of_next_to_no_weight(q, kind, seqs, group, kernel, gap, where):  # noqa: F811
    """One block's scores lie about 50 below the others', its values 2^gap above."""
    for dim in (64, 128):
        b = Batch(seqs, 2, dim, 32, seed=12)
        b.ke[:] = 120
        b.kc[..., 0] = 0
        per = b.page // 16
        at = lambda s: {"first": 0, "middle": 2, "last": (b.seqs[s][1] - 1) // 16}[where]  # noqa: E731
        set_bytes(b, b.ve, lambda s, i: 118 + gap * (i == at(s)))
        for s in range(len(seqs)):
            o = at(s) % per * 16
            b.kc[b.table[s, at(s) // per], :, o:o + 16, 0] = -127
        x = b.rng.standard_normal((b.rows, 2 * group, dim)) * 0.2
        x[..., 0] = 50 * dim ** 0.5
        run(q, b, kind, group, kernel=kernel, x=rounded(x, kind), max_tokens=max(n for n, _ in seqs))


@each
@pytest.mark.parametrize("dim", [64, 128])
def test_an_infinity_among_the_values(q, kind, seqs, group, kernel, dim):  # noqa: F811
    """It is stored as the largest number, and is nothing to the rows that do not see it, nor to the other elements."""
    t = TYPES[kind]
    for n, length in seqs:
        b = Batch([(length, length)], 2, dim, 32, seed=13)
        cache, table, lengths, starts = b.device(q)
        k, v = (rounded(b.rng.standard_normal((length, 2, dim)), kind) for _ in range(2))
        v[66, 0, 3], v[67, 1, dim - 1] = np.inf, -np.inf
        q.qmm_kv_append(cache, *(torch.from_numpy(a).to(t).cuda() for a in (k, v)), table, lengths, starts=starts)
        arrays = [c.cpu().numpy() for c in cache]
        starts = np.array([0, n], np.int32)
        x = rounded(b.rng.standard_normal((n, 2 * group, dim)), kind)
        y = q.qmm_kv_attention(torch.from_numpy(x).to(t).cuda(), cache, table, lengths,
                               starts=torch.from_numpy(starts).cuda())
        exact, mag, top, seen = ko.attention(x.astype(np.float64), *arrays, b.table, b.lengths, starts, dim ** -0.5, True,
                                             detail=True)
        assert_attention(y.double().cpu().numpy(), exact, attention_bound(exact, mag, top, seen, kind, dim))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("second", [4.0, 7.0, 8.0, 9.0])
def test_windows_that_come_back(q, kind, few, second):  # noqa: F811
    """Values, then blocks of zeros with scores 28 below, then values with scores above the first ones': what the first
    ones leave has to come through both changes."""
    size = 16 if few else 128                         # tokens of each of the three
    seqs = [(1, 3 * size)] * 300 if few else [(96, 3 * size), (100, 3 * size)]
    b = Batch(seqs, 8 if few else 2, 64, 16, seed=18)
    b.ke[:], b.ve[:] = 120, 118
    b.kc[..., 0] = 0
    for s in range(len(seqs)):
        for i in range(3 * size // 16):
            part = i * 16 // size
            b.kc[b.table[s, i], :, :, 0] = (0, -127, round(127 * second / 28))[part]
            v = b.vc[b.table[s, i]]
            v[:] = (np.abs(v) // 4 + 95, 0 * v, v // 16)[part]
            if part == 1:
                b.ve[b.table[s, i]] = 0
    group = 1 if few else 4
    x = b.rng.standard_normal((b.rows, b.heads * group, 64)) * 0.1
    x[..., 0] = 28 * 8 * 128 / 127
    run(q, b, kind, group, causal=False, x=rounded(x, kind), max_tokens=max(n for n, _ in seqs))

@each
@pytest.mark.parametrize("sharp", [3, 10])
def test_blocks_of_zeros_among_sharp_scores(q, kind, seqs, group, kernel, sharp):  # noqa: F811
    """Scores tens apart: what is left of a row where the zeros have most of its weight, and window after window of
    values with next to none. (No other value is 0: an element has something of every block.)"""
    for dim in (64, 128):
        for often in (0.1, 0.5):
            b = Batch(seqs, 2, dim, 32, seed=17)
            b.ke[:] = 121
            b.vc[b.vc == 0] = 1
            b.ve[:] = b.rng.integers(117, 121, b.ve.shape)
            zero = b.rng.random(b.ve.shape) < often
            b.ve[zero] = 0
            b.vc[np.repeat(zero, 16, axis=2)] = 0
            x = rounded(b.rng.standard_normal((b.rows, 2 * group, dim)) * sharp, kind)
            run(q, b, kind, group, kernel=kernel, x=x, max_tokens=max(n for n, _ in seqs))


@each
@pytest.mark.parametrize("drop", [4, 9, 14, 18, 22])
def test_values_as_large_as_their_weights_are_small(q, kind, seqs, group, kernel, drop):  # noqa: F811
    """One block's scores lie `drop` below the others', and its values above them by as much, by less and by more: what
    weighs most in the row is held by digits of its own."""
    for gap in sorted({round(drop * 1.4427) + d for d in (-8, -2, 0, 3, 7)}):
        b = Batch(seqs, 2, 64, 32, seed=19)
        b.ke[:] = 120
        b.kc[..., 0] = 0
        b.vc[b.vc == 0] = 1
        per = b.page // 16
        set_bytes(b, b.ve, lambda s, i: 118 + gap * (i == 2))
        for s in range(len(seqs)):
            o = 2 % per * 16
            b.kc[b.table[s, 2 // per], :, o:o + 16, 0] = -round(127 * drop / 25)
        x = b.rng.standard_normal((b.rows, 2 * group, 64)) * 0.2
        x[..., 0] = 25 * 8 * 128 / 127
        run(q, b, kind, group, kernel=kernel, x=rounded(x, kind), max_tokens=max(n for n, _ in seqs))

"""The key-value cache's plain forms against brute force in exact arithmetic and hand-worked values."""
import math
from fractions import Fraction

import numpy as np

from oracle import kv_oracle as ko

F = np.float32


def test_powers_and_bytes():
    assert float(ko.power(0)) == 2.0 ** -127 and float(ko.power(127)) == 1.0 and float(ko.power(255)) == 2.0 ** 128
    for k in (-100, -3, 0, 60):
        edge = 127.5 * 2.0 ** k
        assert ko.block_byte(F(edge)) == 128 + k                              # 127.5 steps round to 128: one more
        assert ko.block_byte(np.nextafter(F(edge), F(0))) == 127 + k
        assert ko.block_byte(F(64 * 2.0 ** k)) == 127 + k
        assert ko.block_byte(np.nextafter(F(63.75 * 2.0 ** k), F(0))) == 126 + k
    assert ko.block_byte(F(0)) == 0 and ko.block_byte(np.finfo(F).tiny) == 0
    assert ko.block_byte(np.finfo(F).max) == 249
    for amax in np.random.default_rng(0).standard_normal(200).astype(F) ** 9:
        b = ko.block_byte(abs(amax))
        assert abs(Fraction(float(amax))) < Fraction(255, 2) * Fraction(2) ** (b - 127)
        assert b == 0 or abs(Fraction(float(amax))) >= Fraction(255, 2) * Fraction(2) ** (b - 128)


def test_rotation_step_by_step():
    rng = np.random.default_rng(1)
    x, cos, sin = rng.standard_normal((3, 8)).astype(F), *rng.standard_normal((2, 5, 3)).astype(F)

    for inter in (False, True):
        y = ko.rotate(x, 4, cos, sin, inter)
        for h in range(3):
            for i in range(3):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 3)
                f = lambda p, q: F(float(Fraction(float(p)) * Fraction(float(q))))   # noqa: E731  (48 bits: exact in float64)
                assert y[h, a] == F(float(f(x[h, a], cos[4, i])) - float(f(x[h, b], sin[4, i])))
                assert y[h, b] == F(float(f(x[h, b], cos[4, i])) + float(f(x[h, a], sin[4, i])))
            assert (y[h, 6:] == x[h, 6:]).all()
    assert np.isnan(ko.rotate(x, 5, cos, sin, False)[:, :6]).all() and (ko.rotate(x, 0, None, None, False) == x).all()


def arrays(pages, heads, page, dim):
    return ([np.zeros((pages, heads, page, dim), np.int8) for _ in range(2)]
            + [np.zeros((pages, heads, page // 16), np.uint8) for _ in range(2)])


def test_append_by_hand():
    """One head of two numbers, a page of 16: 3.0 and -1.5, then a token that doubles the step twice."""
    kc, vc, ke, ve = arrays(2, 1, 16, 2)
    table, one = np.array([[1]], np.int32), np.ones((1, 1, 2), F)
    ko.append(kc, vc, ke, ve, one * np.array([3.0, -1.5], F), one, table, np.array([1], np.int32), None)
    assert ke[1, 0, 0] == 127 - 5 and kc[1, 0, 0].tolist() == [96, -48]         # step 2^-5: 3 / 127.5 < 2^-5
    ko.append(kc, vc, ke, ve, one * np.array([12.4, 0.0625], F), one, table, np.array([2], np.int32), None)
    assert ke[1, 0, 0] == 127 - 3 and kc[1, 0, :2].tolist() == [[24, -12], [99, 0]]   # 0.0625 is half a step: to even
    assert not kc[0].any() and ve[1, 0, 0] == 127 - 6 and vc[1, 0, :2].tolist() == [[64, 64], [64, 64]]


def test_append_against_rationals():
    rng = np.random.default_rng(2)
    kc, vc, ke, ve = arrays(3, 2, 32, 4)
    table = np.array([[2, 0]], np.int32)
    held = {}                                                                   # (kind, head, block) -> byte, ints
    length = 0
    for n in (3, 20, 1, 1, 9):
        k, v = (rng.standard_normal((n, 2, 4)) * 3.0 ** rng.integers(-2, 3) for _ in range(2))
        k, v = k.astype(F), v.astype(F)
        length += n
        ko.append(kc, vc, ke, ve, k, v, table, np.array([length], np.int32), np.array([0, n], np.int32))
        for kind, x in enumerate((k, v)):
            for h in range(2):
                for blk in range((length - n) // 16, (length - 1) // 16 + 1):
                    byte, ints = held.get((kind, h, blk), (0, {}))
                    fresh = {p: x[p - (length - n), h] for p in range(max(blk * 16, length - n), min(blk * 16 + 16, length))}
                    need = max(ko.block_byte(np.abs(t).max()) for t in fresh.values())
                    new = max(byte, need) if ints else need
                    ints = {p: [int(round(Fraction(q) / 2 ** (new - byte))) for q in t] for p, t in ints.items()}
                    for p, t in fresh.items():
                        ints[p] = [int(round(Fraction(float(q)) / Fraction(2) ** (new - 127))) for q in t]
                    held[kind, h, blk] = (new, ints)
    for (kind, h, blk), (byte, ints) in held.items():
        cache, exp = ((kc, ke), (vc, ve))[kind]
        page, off = table[0, blk // 2], blk % 2
        assert exp[page, h, off] == byte
        for p, t in ints.items():
            assert cache[page, h, p % 32].tolist() == t


def test_read_and_attention_by_brute_force():
    rng = np.random.default_rng(3)
    kc, vc, ke, ve = arrays(5, 2, 16, 4)
    for c in (kc, vc):
        c[:] = rng.integers(-127, 128, c.shape)
    for e in (ke, ve):
        e[:] = rng.integers(118, 124, e.shape)
    table = np.array([[3, 1], [0, 9], [4, -1]], np.int32)
    lengths, starts = np.array([20, 25, 2], np.int32), np.array([0, 3, 4, 8], np.int32)
    q = rng.standard_normal((9, 4, 4))
    back = ko.read(kc, ke, table, lengths, starts, 9)
    for causal in (True, False):
        got, mag, top, seen = ko.attention(q, kc, vc, ke, ve, table, lengths, starts, 0.5, causal, detail=True)
        assert np.isnan(got[8]).all()
        for b in range(3):
            n = starts[b + 1] - starts[b]
            for i in range(n):
                pos = lengths[b] - n + i
                for h in range(4):
                    kh, num, den, absn = h // 2, [[] for _ in range(4)], [], [[] for _ in range(4)]
                    for j in range(min(pos + 1 if causal else lengths[b], 32)):
                        page = table[b, j // 16]
                        if j < 0 or not 0 <= page < 5:
                            continue
                        k = [int(z) * 2.0 ** (int(ke[page, kh, 0]) - 127) for z in kc[page, kh, j % 16]]
                        v = [int(z) * 2.0 ** (int(ve[page, kh, 0]) - 127) for z in vc[page, kh, j % 16]]
                        p = math.exp(0.5 * math.fsum(x * y for x, y in zip(q[starts[b] + i, h], k)))
                        den.append(p)
                        for d in range(4):
                            num[d].append(p * v[d])
                            absn[d].append(p * abs(v[d]))
                        if j == pos and h % 2 == 0:
                            assert back[starts[b] + i, kh].tolist() == k
                    assert seen[starts[b] + i] == len(den)
                    for d in range(4):
                        want = math.fsum(num[d]) / math.fsum(den) if den else 0.0
                        wmag = math.fsum(absn[d]) / math.fsum(den) if den else 0.0
                        assert abs(got[starts[b] + i, h, d] - want) <= 1e-12 * (wmag + 1e-300)
                        assert abs(mag[starts[b] + i, h, d] - wmag) <= 1e-12 * (wmag + 1e-300)

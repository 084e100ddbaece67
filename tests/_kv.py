"""Inputs for the tests of the key-value cache: packed sequences over scattered pages."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rounded(x, kind):
    """float32 values that the type holds."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    return t.to(TYPES[kind]).float().numpy()


class Batch:
    """Sequences of (rows, tokens) over a cache of scattered pages; `bad`: (sequence,
    page index, page number) entries of the table that name no page."""

    def __init__(self, seqs, heads, dim, page, seed=0, spare=2, width=None, bad=(), starts=True):
        rng = np.random.default_rng(seed)
        self.rng, self.seqs, self.heads, self.dim, self.page = rng, seqs, heads, dim, page
        used = [-(-max(length, 0) // page) for _, length in seqs]
        self.width = max(used, default=0) if width is None else width
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(seqs), self.width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u][:self.width]
            at += u
        for b, p, number in bad:
            self.table[b, p] = number
        self.lengths = np.array([length for _, length in seqs], np.int32)
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32) if starts else None
        self.rows = int(sum(n for n, _ in seqs))
        self.kc = rng.integers(-127, 128, (self.pages, heads, page, dim)).astype(np.int8)
        self.vc = rng.integers(-127, 128, (self.pages, heads, page, dim)).astype(np.int8)
        self.ke = rng.integers(118, 123, (self.pages, heads, page // 16)).astype(np.uint8)
        self.ve = rng.integers(116, 124, (self.pages, heads, page // 16)).astype(np.uint8)

    def device(self, q):
        """(cache, table, lengths, starts) on the GPU; the arrays here stay the start's."""
        d = [torch.from_numpy(a.copy()).cuda() for a in (self.kc, self.vc, self.ke, self.ve)]
        return (q.KvCache(*d), torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lengths).cuda(),
                None if self.starts is None else torch.from_numpy(self.starts).cuda())

    def cache_arrays(self):
        return [a.copy() for a in (self.kc, self.vc, self.ke, self.ve)]


def turns(positions, half, base=10000.0):
    a = np.arange(positions)[:, None] * base ** (-np.arange(half) / max(half, 1))
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def attention_bound(exact, mag, top, seen, kind, dim):
    """How far an output may be off. A score is an fp32 sum of dim products and a few
    more roundings, at most (dim + 16) 2^-23 of sum |q k| * scale; exp2 and the
    subtraction of the maximum add 2^-20 for scores up to 2^3 above the maximum's
    magnitude; twice that, numerator and sum, weighted by p |v|. P is held in fp16 (2^-11)
    or in two fp16 parts (2^-21); O is summed over the tokens in fp32."""
    score = (dim + 16) * 2.0 ** -23 * (top[..., None] + 1) + 2.0 ** -20 + 2.0 ** -22 * top[..., None]
    p = 2.0 ** -11 if kind == "bf16" else 2.0 ** -21
    total = (seen[:, None, None] / 16 + 64) * 2.0 ** -23
    half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
    return mag * (2 * score + p + total) + np.abs(exact) * half + 1e-30


def assert_attention(got, exact, bound, what=""):
    err = np.abs(got - exact)
    bad = ~(err <= bound) & ~np.isnan(exact)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; first {i}: got {got[i]}, exact {exact[i]}, "
                             f"allowed {bound[i]}, worst ratio {np.nanmax(err / bound)}")

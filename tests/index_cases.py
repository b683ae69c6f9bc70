"""Plain forms of the index-driven re-layouts in 64 bits, inputs for them, and
the error bounds their tests use (no library code).

Bounds.  A sum of n products accumulated in fp32 in any order is off by at
most (n + 1) * 2^-24 times the sum of the absolute products, to first order;
twice that covers the higher orders at the sizes used here.  The result is
then rounded once to its type: half a step, eps/2 of its size, or half the
smallest subnormal."""
import numpy as np
import torch

FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def bound(dtype, exact, terms, n):
    """Largest error of one rounded fp32 sum of n products (arrays in fp64)."""
    fi = torch.finfo(dtype)
    err = 2 * (n + 1) * 2.0 ** -24 * terms
    return err + fi.eps / 2 * (np.abs(exact) + err) + fi.smallest_normal * fi.eps / 2


def check(got, exact, terms, n, what):
    dtype = got.dtype
    got = got.double().cpu().numpy().reshape(exact.shape)
    assert np.isfinite(got).all(), "%s: not finite, or not written" % what
    over = np.abs(got - exact) > bound(dtype, exact, terms, n)
    assert not over.any(), "%s: %d of %d over the bound, worst %g" % (
        what, over.sum(), over.size, np.abs(got - exact)[over].max())


def max_rows(T, K, E, align):
    M = T * K
    return (M + min(E, M) * (align - 1)) // align * align


def index(ids, E, align):
    """pos, order, offsets, counts of ids [T][K] by a walk over the slots."""
    T, K = ids.shape
    flat = ids.reshape(-1)
    counts = np.zeros(E, dtype=np.int64)
    rank = np.full(flat.size, -1, dtype=np.int64)
    for s, e in enumerate(flat.tolist()):
        if 0 <= e < E:
            rank[s] = counts[e]
            counts[e] += 1
    offsets = np.zeros(E + 1, dtype=np.int64)
    offsets[1:] = np.cumsum((counts + align - 1) // align * align)
    kept = rank >= 0
    pos = np.where(kept, offsets[np.where(kept, flat, 0)] + rank, -1)
    order = np.full(max_rows(T, K, E, align), -1, dtype=np.int64)
    order[pos[kept]] = np.nonzero(kept)[0]
    return pos, order, offsets, counts


def choices(rng, T, K, E, drop=0.0, id_bytes=8):
    """ids [T][K] of a skewed router, some outside [0, E): negative, E itself,
    and values that only look valid when cut to 32 bits."""
    p = np.exp(rng.normal(size=E))
    ids = rng.choice(E, size=(T, K), p=p / p.sum()).astype(np.int64)
    gone = rng.random((T, K)) < drop
    outside = [-1, E, -2**31, 2**31 - 1] + ([2**32, -2**32, 2**40 + 1] if id_bytes == 8 else [])
    ids[gone] = rng.choice(np.array(outside, dtype=np.int64), size=int(gone.sum()))
    return ids


def seq_place(N, B, S, G):
    """Place of every token of the order [B][S] in the sequence-sharded layout."""
    P, Bl = N // G, B // G
    St = S // P
    place = np.empty(B * S, dtype=np.int64)
    at = 0
    for rank in range(N):
        g, j = divmod(rank, P)
        for b in range(g * Bl, (g + 1) * Bl):
            place[b * S + j * St:b * S + (j + 1) * St] = np.arange(at, at + St)
            at += St
    return place


class Guarded:
    """A device buffer of n elements between two guards, all set to `fill`,
    starting `shift` elements past a 16-byte boundary."""

    PAD = 64

    def __init__(self, n, dtype, fill, shift=0, device="cuda"):
        self.whole = torch.full((n + 2 * self.PAD + shift,), fill, dtype=dtype, device=device)
        self.at, self.n, self.fill = self.PAD + shift, n, fill
        self.t = self.whole[self.at:self.at + n]

    def check(self, what):
        rest = torch.cat([self.whole[:self.at], self.whole[self.at + self.n:]])
        same = torch.isnan(rest) if self.fill != self.fill else rest == self.fill
        assert bool(same.all()), "%s: written outside the buffer" % what


def shifted(t, shift):
    """The same values at an address `shift` elements past a 16-byte boundary."""
    flat = t.reshape(-1)
    room = torch.empty(flat.numel() + shift, dtype=t.dtype, device=t.device)
    room[shift:] = flat
    return room[shift:]

"""Attention cases that tell the parts of the arithmetic apart, with their results in 64 bits and bounds of a few
roundings: every query has one value that is not zero, so a score is one product, and few slots are visible, so
that a lost part of a query or of a weight stands out.  `slip` plants such a mistake in the 64-bit form (numpy)."""
from __future__ import annotations

import numpy as np
import torch

import step_ref as ref

U = ref.U
LN2 = float(np.log(2.0))
SHIFT = {"f16": 9.0, "bf16": 0.0, "q8": 0.0}       # weights are held as 2^SHIFT times their value, at most


def cut(x, bits):
    """The leading `bits` bits of x, the rest cut off."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(np.ldexp(m, bits)), e - bits)


def high_part(x, kind, scale=1.0):
    """x without what a second (third) 16-bit part holds of scale * x."""
    if kind == "bf16":
        return cut(x, 16)                          # the third part lost
    return np.float16(x * scale).astype(np.float64) / scale


def two_slots(rng, kind, dim, n_seq, group):
    """n_seq sequences of two slots: a score of 0 and one between -2 and 0; values of either sign."""
    cache = ref.Cache(rng, kind, n_seq, 1, 16, dim)
    table = np.arange(n_seq, dtype=np.int32)[:, None]
    at = rng.integers(0, dim, n_seq)               # the dimension that the sequence's queries look at
    for s in range(n_seq):
        if kind == "q8":
            cache.kv[0][s, 0, 0, at[s]] = 0
            cache.kv[0][s, 0, 1, at[s]] = int(rng.integers(64, 128))
            cache.scale[0][s, 0, 1, at[s] // 32] = float(np.float16(rng.uniform(0.5, 1) / 127))
        else:
            cache.kv[0][s, 0, 0, at[s]] = 0
            cache.kv[0][s, 0, 1, at[s]] = float(rng.uniform(0.5, 1))
    q = np.zeros((n_seq, 1, group, dim), np.float32)
    q[np.arange(n_seq), 0, :, at] = -rng.uniform(0.3, 2.0, (n_seq, group))
    return cache, table, [2] * n_seq, q.reshape(n_seq, 1, -1)


def attn(cache, q, table, lens, scale, slip=None, seen=None, depth=0):
    """(out, bound) of one-hot queries over one kv head.  slip: a part that is lost, "q" or "weights".  seen[s, t]:
    the visible slots (default: the causal ones); depth: roundings of sums beyond those of a few slots."""
    kind, dim = cache.kind, cache.dim
    n_seq, n_tok, _ = q.shape
    x = q.reshape(n_seq, n_tok, -1, dim).astype(np.float64)
    out, tol = np.zeros(x.shape), np.zeros(x.shape)
    for s, n in enumerate(lens):
        k, v = cache.rows(0, table[s], n, 0), cache.rows(1, table[s], n, 0)
        for t in range(n_tok):
            j = np.arange(n - n_tok + t + 1) if seen is None else np.asarray(seen[s][t])
            for g in range(x.shape[2]):
                row = x[s, t, g]
                if slip == "q":
                    top = 2.0 ** (12 - np.floor(np.log2(np.abs(row).max())))
                    row = high_part(row, kind, top)
                z = scale * (k[j] @ row)
                sc = z / LN2                                             # the score in powers of two
                w = np.exp(z - z.max())
                total = w.sum()
                p = w * 2.0 ** SHIFT[kind]
                if slip == "weights":
                    p = high_part(p, kind)
                p = p / 2.0 ** SHIFT[kind]
                vv = v[j]
                out[s, t, g] = (p @ vv) / total
                # a score: two parts of q leave 2 U (three: nothing) and are added (f16, Q8_0: once, bf16: twice), a
                # Q8_0 scale is one rounding more, the factor and the product with it three
                r = {"f16": 6, "q8": 7, "bf16": 5}[kind] * U * np.abs(sc)
                # a weight: the reference and the difference are rounded, 2^x is good to 2^-22, and one factor 2^x
                # where parts of warps and CTAs are joined
                r = LN2 * (r + U * (np.abs(sc.max()) + SHIFT[kind]) + U * (np.abs(sc - sc.max()) + SHIFT[kind])) + 4 * U
                r = r + 5 * U
                # two parts leave 2 U, three nothing; a product with a scale is rounded once more
                parts = {"f16": 2, "bf16": 0, "q8": 3}[kind] * U
                # the products of 16 slots and what was there are added with a cut of 2 U each at most, in three (two)
                # instructions, of which those of the small parts weigh 2^-7 (2^-11); one rounded add
                few = min(len(j), 32)
                sums = (2 * (few + 1) * (1 + 2.0 ** -6) + 1 + depth) * U
                mass = (w @ np.abs(vv)) / total
                err = (w * (r + parts)) @ np.abs(vv) / total + sums * mass
                # the quotient: the sum of the weights, its reciprocal and the product
                of_sum = ((w * r).sum() / total + (few + depth + 2) * U)
                tol[s, t, g] = err + of_sum * np.abs(out[s, t, g])
    return out.reshape(q.shape), tol.reshape(q.shape)


def long_tail(kind, dim, n):
    """Twelve slots of weight 1 with values 0 (one in every tile that a warp begins with), and n - 12 of equal weights
    near 2^-22 with values 1, whose two f16 parts of 2^9 times the weight would leave more than 2^-13 of it."""
    page = 16
    n_pages = -(-n // page)
    cache = ref.Cache(np.random.default_rng(0), kind, n_pages, 1, page, dim)
    one = 64 if kind == "q8" else 1.0
    for i in range(2):
        cache.kv[i][:] = one
        if kind == "q8":
            cache.scale[i][:] = 2.0 ** -6
        cache.kv[i][:12, 0, 0] = 0
    q = np.zeros((1, 1, dim), np.float32)
    for x in np.linspace(-22.3 * LN2, -21.7 * LN2, 400).astype(np.float32):
        p = np.exp(np.float64(x)) * 2.0 ** 9
        if abs(p - high_part(p, "f16") - high_part(p - high_part(p, "f16"), "f16")) > 0.9 * 2.0 ** -12 * p:
            break
    q[0, 0, 3] = x
    return cache, np.arange(n_pages, dtype=np.int32)[None], [n], q

"""Plain 64-bit forms of the cache and logits operators (numpy, loops over rows), for the tests, with the
bounds that the kernels' f32 arithmetic has to keep.  Nothing of the library is used."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24          # half a step of f32


class Cache:
    """Pages on the CPU with the values they stand for; `device()` gives the pools."""

    def __init__(self, rng, kind, n_pages, n_kv, page, dim, layout="head", gap=0, fill=None):
        self.kind, self.n_pages, self.n_kv, self.page, self.dim = kind, n_pages, n_kv, page, dim
        self.layout, self.gap = layout, gap
        self.kv = []                                   # stored values, [n_pages, n_kv, page, dim]
        self.scale = []
        for _ in range(2):
            x = torch.from_numpy(rng.standard_normal((n_pages, n_kv, page, dim))).float()
            if kind == "q8":
                b = x.reshape(n_pages, n_kv, page, dim // 32, 32)
                d = (b.abs().amax(-1) / 127).half()
                self.kv.append((b / d.float()[..., None]).round().clamp(-127, 127).to(torch.int8).reshape(x.shape))
                self.scale.append(d)
            else:
                self.kv.append(x.to(torch.float16 if kind == "f16" else torch.bfloat16))
        if fill is not None:                           # [n_pages, n_kv or 1, page] bool: slots to spoil
            for i in range(2):
                where = torch.as_tensor(np.broadcast_to(fill, (n_pages, n_kv, page)).copy())
                (self.scale if kind == "q8" else self.kv)[i][where] = float("nan")

    def values(self, which):
        x = self.kv[which].double()
        if self.kind == "q8":
            x = (x.reshape(*x.shape[:3], -1, 32) * self.scale[which].double()[..., None]).reshape(x.shape)
        return x.numpy()

    def rows(self, which, table, n, h):
        """Slots 0..n-1 of a sequence, kv head h."""
        x = self.values(which) if not hasattr(self, "_v%d" % which) else getattr(self, "_v%d" % which)
        setattr(self, "_v%d" % which, x)
        j = np.arange(n)
        return x[np.asarray(table)[j // self.page], h, j % self.page]

    def _lay(self, x, device, gap):
        if self.layout == "token":
            x = x.transpose(1, 2).contiguous()
        if gap:                                        # unused elements after every row
            wide = torch.full((*x.shape[:-1], x.shape[-1] + gap), 7, dtype=x.dtype)
            wide[..., :x.shape[-1]] = x
            x = wide
        n = self.kv[0].shape[-1] if x.dtype != torch.float16 or self.kind != "q8" else self.dim // 32
        x = x.to(device)[..., :n]
        return x.transpose(1, 2) if self.layout == "token" else x

    def device(self, device="cuda"):
        k, v = (self._lay(x, device, self.gap) for x in self.kv)
        if self.kind != "q8":
            return k, v, None, None
        return k, v, *(self._lay(x, device, self.gap // 32) for x in self.scale)


def attn(cache, q, n_head, tables, lens, scale, window=0, n_sink=0, score=None):
    """(out, bound of its error, score, bound of its error) of q [n_seq, n_tok, n_head * dim]."""
    n_seq, n_tok, _ = q.shape
    d, group = cache.dim, n_head // cache.n_kv
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    score = None if score is None else score.astype(np.float64).copy()
    stol = None if score is None else np.zeros(score.shape)
    for s in range(n_seq):
        n = lens[s]
        for h in range(cache.n_kv):
            k, v = cache.rows(0, tables[s], n, h), cache.rows(1, tables[s], n, h)
            given, given_tol, seen_any = np.zeros(n), np.zeros(n), np.zeros(n, bool)
            for t in range(n_tok):
                p = n - n_tok + t
                j = np.arange(n)
                seen = (j <= p) & ((window == 0) | (j > p - window) | (j < n_sink)) if p >= 0 else np.zeros(n, bool)
                ok = np.asarray(tables[s])[j // cache.page] >= 0 if n else np.zeros(0, bool)
                seen &= ok
                if not seen.any():
                    continue
                seen_any |= seen
                kk, vv = k[seen], v[seen]
                for g in range(group):
                    cols = slice((h * group + g) * d, (h * group + g + 1) * d)
                    x = q[s, t, cols].astype(np.float64)
                    z = scale * (kk @ x)
                    w = np.exp(z - z.max())
                    total = w.sum()
                    w /= total
                    out[s, t, cols] = w @ vv
                    # a score: 2 d + 32 roundings of partial sums of at most sum |q k| each (truncating adds count
                    # twice), what the parts leave of q (2^-23 of its largest value), two of the score itself
                    absum = np.abs(kk) @ np.abs(x)
                    e = scale * ((2 * d + 32) * U * absum + 2 * U * np.abs(x).max() * np.abs(kk).sum(1)) + 4 * U * np.abs(z)
                    # a weight moves by twice the largest score error; sums over the slots round once a slot
                    rel = 2 * e.max() + 2 * U * (len(z) + 64)
                    tol[s, t, cols] = rel * (w @ np.abs(vv)) + 2 * U * rel
                    given[seen] += w
                    given_tol[seen] += w * rel
            if score is not None and n:
                new = np.arange(n) >= n - n_tok
                touched = seen_any | np.zeros(n, bool)
                old = np.where(new, 0.0, score[s, h, :n])
                res = np.where(touched, old + given, score[s, h, :n])
                stol[s, h, :n] = given_tol + 4 * U * np.abs(res)
                score[s, h, :n] = res
    return out, tol, score, stol


def rope(x, pos, inv_freq, rope_dim, pairs):
    """x [.., heads, dim] at position pos, in 64 bits."""
    x = x.astype(np.float64).copy()
    if rope_dim:
        a = pos * inv_freq.astype(np.float64)
        half = rope_dim // 2
        i = np.arange(half)
        first, second = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        u, w = x[..., first].copy(), x[..., second].copy()
        x[..., first] = u * np.cos(a) - w * np.sin(a)
        x[..., second] = u * np.sin(a) + w * np.cos(a)
    return x


def evict(score, lens, first, last, budget):
    """kept slots per sequence and head, in order."""
    kept = []
    for s, n in enumerate(lens):
        row = []
        for h in range(score.shape[1]):
            if n <= budget:
                row.append(list(range(n)))
                continue
            mid = list(range(first, n - last))
            z = score[s, h]
            mid.sort(key=lambda j: (-np.inf if np.isnan(z[j]) else z[j], 0 if np.isnan(z[j]) else 1, -j), reverse=True)
            row.append(sorted(list(range(first)) + mid[:budget - first - last] + list(range(n - last, n))))
        kept.append(row)
    return kept


def logits(z, hist=None, hist_len=None, params=None, bias_ids=None, bias_vals=None, bias_len=None, mask=None):
    """(adjusted logits in f32 steps, choice) -- every step rounds, as documented."""
    z = z.astype(np.float32).copy()
    n, v = z.shape
    idx = np.full(n, -1, np.int64)
    f = np.float32
    for r in range(n):
        if hist is not None:
            used = hist[r, :max(0, min(hist_len[r], hist.shape[1]))]
            ids, count = np.unique(used[(used >= 0) & (used < v)], return_counts=True)
            rep, freq, pres = (f(x) for x in params[r])
            for i, c in zip(ids, count):
                x = z[r, i]
                x = f(x / rep) if x > 0 else f(x * rep)
                z[r, i] = f(x - f(f(freq * f(c)) + pres))
        if bias_ids is not None:
            last = {}
            for i in range(max(0, min(bias_len[r], bias_ids.shape[1]))):
                if 0 <= bias_ids[r, i] < v:
                    last[int(bias_ids[r, i])] = bias_vals[r, i]
            for i, b in last.items():
                z[r, i] = f(z[r, i] + f(b))
        if mask is not None:
            i = np.arange(v)
            z[r, (mask[r, i // 32].astype(np.uint32) >> (i % 32).astype(np.uint32)) & 1 == 0] = -np.inf
        ok = z[r] > -np.inf
        if ok.any():
            idx[r] = np.argmax(np.where(ok, z[r], -np.inf))
    return z, idx

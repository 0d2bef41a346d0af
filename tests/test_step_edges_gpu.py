"""The cache and logits operators where a call's inputs leave the ordinary range: rows of wider tensors, lengths beyond
the table, values that the caches cannot hold; plain 64-bit forms in step_ref.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_decode_superblocks_b200 as q
import step_ref as ref
import step_tight as tight
import test_step_gpu as base
from test_step_gpu import dev, make_tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    q.build()
    q.qmv_check()
    yield
    assert q.qmv_check() == 0


# -------------------------------------------------------------------------------------- scores in a wider tensor --
def test_scores_in_a_slice_of_a_wider_tensor():
    """Lengths beyond the slice are clamped to it; nothing beside it changes."""
    rng = np.random.default_rng(1)
    lens, page, n_kv, dim, lo, hi = [90, 30], 16, 2, 64, 10, 60
    table, n_pages = make_tables(rng, lens, page)
    cache = ref.Cache(rng, "f16", 2 * n_pages + 8, n_kv, page, dim)
    x = rng.standard_normal((2, 1, 4 * dim)).astype(np.float32)
    k, v, _, _ = cache.device()
    c = q.KvCache(q.KV_F16, k, v)
    wide = dev(rng.random((2, n_kv, 100)).astype(np.float32))
    before = wide.cpu().numpy()
    out = torch.zeros(2, 1, 4 * dim, device="cuda")
    ws = torch.zeros(q.attn_ws_bytes(c, 4, 2, 1, table.shape[1], True), dtype=torch.uint8, device="cuda")
    tab, n = dev(table), dev(np.array(lens, np.int32))
    q.attn_decode(q.AttnArgs(c, dev(x), out, tab, n, ws, 0.125, score=wide[:, :, lo:hi]))
    assert q.qmv_check() == q.DEVERR_SEQ_LEN
    used = [hi - lo, 30]
    want, tol, want_score, stol = ref.attn(cache, x, 4, table, used, 0.125, score=before[:, :, lo:hi])
    got = wide.cpu().numpy()
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert (np.abs(got[:, :, lo:hi] - want_score) <= stol).all()
    assert np.array_equal(got[:, :, :lo], before[:, :, :lo]) and np.array_equal(got[:, :, hi:], before[:, :, hi:])
    # eviction by the same slice, to pages that the sequences do not use
    budget = 20
    dst = np.array([[n_pages, n_pages + 1], [n_pages + 2, n_pages + 3]], np.int32)
    kept, so = torch.full((2, n_kv, budget), -7, dtype=torch.int32, device="cuda"), torch.zeros(2, n_kv, budget, device="cuda")
    n_out = torch.zeros(2, dtype=torch.int32, device="cuda")
    q.kv_evict(q.EvictArgs(c, wide[:, :, lo:hi], tab, n, dev(dst), kept, so, n_out, 2, 3, budget))
    assert q.qmv_check() == q.DEVERR_SEQ_LEN
    z = got[:, :, lo:hi]
    rows = ref.evict(z, used, 2, 3, budget)
    for s in range(2):
        for h in range(n_kv):
            assert kept[s, h].tolist() == rows[s][h] and np.array_equal(so[s, h].cpu().numpy(), z[s, h, rows[s][h]])
    assert n_out.tolist() == [budget, budget]


# ------------------------------------------------------------------------------------------ append: what is stored --
def pools(cache, k, v, ks, vs):
    """What the pools hold now, bit by bit: the quants (16-bit values as integers), and the scales."""
    return [x.contiguous().view(torch.int16 if x.dtype != torch.int8 else torch.int8).cpu().numpy() for x in (k, v, ks, vs) if x is not None]


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("own_positions", [False, True])
def test_append_tokens_beyond_the_table_are_not_stored(kind, own_positions):
    """Every token goes to its own slot or nowhere: nothing is moved back over slots that are in use."""
    rng = np.random.default_rng(3)
    page, n_kv, n_head, dim, n_tok = 16, 2, 4, 64, 3
    lens = [32, 33, 34, 35, 36, 1000, 2 ** 31 - 1, 2, 0, -1, -2 ** 31]
    table = np.arange(2 * len(lens), dtype=np.int32).reshape(-1, 2)
    cache = ref.Cache(rng, kind, table.size, n_kv, page, dim)
    k, v, ks, vs = cache.device()
    before = pools(cache, k, v, ks, vs)
    x = rng.standard_normal((len(lens), n_tok, (n_head + 2 * n_kv) * dim)).astype(np.float32)
    inv = (10000.0 ** (-2.0 * np.arange(dim // 2) / dim)).astype(np.float32)
    qd, kd, vd = dev(x).split([n_head * dim, n_kv * dim, n_kv * dim], -1)
    out = torch.zeros(len(lens), n_tok, n_head * dim, device="cuda")
    pos = rng.integers(0, 5000, (len(lens), n_tok)).astype(np.int32)
    q.kv_append(q.AppendArgs(q.KvCache(base.KINDS[kind], k, v, ks, vs), qd, kd, vd, out, dev(table), dev(np.array(lens, np.int32)),
                             pos=dev(pos) if own_positions else None, inv_freq=dev(inv), rope_dim=dim))
    assert q.qmv_check() == q.DEVERR_SEQ_LEN
    after = pools(cache, k, v, ks, vs)
    got = out.double().cpu().numpy().reshape(len(lens), n_tok, n_head, dim)
    stored = {(s, n - n_tok + t) for s, n in enumerate(lens) for t in range(n_tok) if 0 <= n - n_tok + t < 32}
    for s, n in enumerate(lens):
        for t in range(n_tok):
            at = int(pos[s, t]) if own_positions else n - n_tok + t
            want = ref.rope(x[s, t, :n_head * dim].reshape(n_head, dim), float(at), inv, dim, False)
            assert (np.abs(got[s, t] - want) <= 2 * ref.U * np.abs(want) + 1e-12 * np.abs(x[s, t]).max()).all(), (n, t)
        for j in range(32):
            same = all(np.array_equal(a[2 * s + j // 16, :, j % 16], b[2 * s + j // 16, :, j % 16]) for a, b in zip(after, before))
            assert same == ((s, j) not in stored), (n, j)
    new = [(s, t) for s, n in enumerate(lens) for t in range(n_tok) if (s, n - n_tok + t) in stored]
    for s, t in new:                                    # the values are those of the token itself
        j = lens[s] - n_tok + t
        y = v[2 * s + j // 16, :, j % 16].double()
        if kind == "q8":
            y = (y.reshape(n_kv, -1, 32) * vs[2 * s + j // 16, :, j % 16].double()[..., None]).reshape(n_kv, dim)
        want = x[s, t, -n_kv * dim:].reshape(n_kv, dim).astype(np.float64)
        half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}.get(kind)
        # Q8_0: half a step of a block of 32, whose scale is rounded to f16
        lim = np.abs(want) * half + 2.0 ** -25 if half else np.repeat(np.abs(want.reshape(n_kv, -1, 32)).max(-1) / 127 * (0.5 + 127 * 2.0 ** -11 + 1e-3), 32, -1)
        assert (np.abs(y.cpu().numpy() - want) <= lim).all()


@pytest.mark.parametrize("what", [float("nan"), -float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dim", [64, 192, 256])
def test_append_keeps_nan_in_a_q8_cache(what, dim):
    """A block of 32 with a NaN reads as NaN throughout, one with an infinity at its largest scale; other blocks as ever."""
    rng = np.random.default_rng(dim)
    n_kv, page = 2, 16
    cache = ref.Cache(rng, "q8", 1, n_kv, page, dim)
    k, v, ks, vs = cache.device()
    x = rng.standard_normal((1, 1, 2 * n_kv * dim)).astype(np.float32)
    spots = [3, dim + 40, n_kv * dim + 63, 2 * n_kv * dim - 1]              # of k and of v, in either head
    x[0, 0, spots] = what
    kd, vd = dev(x).split([n_kv * dim, n_kv * dim], -1)
    q.kv_append(q.AppendArgs(q.KvCache(q.KV_Q8_0, k, v, ks, vs), None, kd, vd, None, dev(np.zeros((1, 1), np.int32)), dev(np.array([7], np.int32))))
    b = x.reshape(2, n_kv, dim // 32, 32)
    f = np.float32
    with np.errstate(invalid="ignore"):
        d = np.minimum(np.abs(b).max(-1) / f(127), f(65504)).astype(np.float16)
        df = d.astype(np.float32)[..., None]
        quant = np.clip(np.rint(b / df), -127, 127)
    quant = np.where(np.isnan(df), 0, quant).astype(np.int8)
    spoiled = 0
    for i, (pool, scale) in enumerate(((k, ks), (v, vs))):
        got_q = pool[0, :, 6].cpu().numpy().reshape(n_kv, -1, 32)
        got_d = scale[0, :, 6].cpu().numpy()
        assert np.array_equal(got_d, d[i], equal_nan=True) and np.array_equal(got_q, quant[i])
        spoiled += np.isnan(got_d).sum()
    assert spoiled == (4 if np.isnan(what) else 0)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("style", [q.ROPE_HALVES, q.ROPE_PAIRS])
def test_append_infinities_turn_as_the_formula_says(kind, style):
    """a cos - b sin with an infinity, with two, with a NaN, and with values whose sum passes f32's range."""
    dim, page, pos = 64, 16, [0, 1, 700, 31]
    inf, big = np.inf, np.float32(3e38)
    x = np.ones((len(pos), 1, 3 * dim), np.float32)
    for s in range(len(pos)):
        for i, (a, b) in enumerate([(inf, 1), (1, inf), (-inf, 2), (inf, inf), (inf, -inf), (np.nan, 1), (1, np.nan), (big, big), (big, -big), (-big, -big), (0, inf)]):
            at = (2 * i, 2 * i + 1) if style == q.ROPE_PAIRS else (i, i + dim // 2)
            for h in range(2):                          # q and k
                x[s, 0, h * dim + at[0]], x[s, 0, h * dim + at[1]] = a, b
    inv = np.full(dim // 2, 0.7, np.float32)
    cache = ref.Cache(np.random.default_rng(0), kind, len(pos), 1, page, dim)
    k, v, _, _ = cache.device()
    qd, kd, vd = dev(x).split([dim, dim, dim], -1)
    out = torch.zeros(len(pos), 1, dim, device="cuda")
    q.kv_append(q.AppendArgs(q.KvCache(base.KINDS[kind], k, v), qd, kd, vd, out, dev(np.arange(len(pos), dtype=np.int32)[:, None]),
                             dev(np.ones(len(pos), np.int32)), pos=dev(np.array(pos, np.int32)[:, None]), inv_freq=dev(inv), rope_dim=dim, rope_style=style))
    half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    with np.errstate(invalid="ignore", over="ignore"):
        for s, at in enumerate(pos):
            want = ref.rope(x[s, 0, :dim], at, inv, dim, style == q.ROPE_PAIRS).astype(np.float32).astype(np.float64)
            got = out[s, 0].double().cpu().numpy()
            ok = np.isfinite(want)
            assert np.array_equal(got[~ok], want[~ok], equal_nan=True), (at, got, want)
            assert (np.abs(got[ok] - want[ok]) <= 2 * ref.U * np.abs(want[ok]) + 1e-12).all()
            kept = k[s, 0, 0].double().cpu().numpy()
            if kind == "f16":                           # what is beyond 65504 is an infinity there
                want = want.astype(np.float16).astype(np.float64)
                ok = np.isfinite(want)
            else:
                ok = np.abs(want) < 3.38e38
            assert np.array_equal(np.isnan(kept), np.isnan(want)) and np.array_equal(np.sign(kept[~np.isnan(kept)]), np.sign(want[~np.isnan(want)]))
            assert np.isinf(kept[np.isinf(want)]).all() and (np.abs(kept[ok] - want[ok]) <= 2 * half * np.abs(want[ok]) + 2.0 ** -24).all()


# ----------------------------------------------------------------------- attention: what single roundings leave --
def run_one_head(cache, qx, table, lens, scale, window=0):
    """qx [n_seq, n_tok, heads * dim] over one kv head, and the workspace it leaves."""
    k, v, ks, vs = cache.device()
    c = q.KvCache(base.KINDS[cache.kind], k, v, ks, vs)
    n_seq, n_tok, width = qx.shape
    ws = torch.zeros(q.attn_ws_bytes(c, width // cache.dim, n_seq, n_tok, table.shape[1]), dtype=torch.uint8, device="cuda")
    out = torch.full(qx.shape, float("nan"), device="cuda")
    q.attn_decode(q.AttnArgs(c, dev(qx), out, dev(table), dev(np.array(lens, np.int32)), ws, scale, window))
    return out.double().cpu().numpy()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("typical", [0.01, 1e-5])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 65504.0, -65504.0])
@pytest.mark.parametrize("group", [1, 3])
def test_attn_scales_a_query_does_not_see_change_nothing(dim, typical, bad, group):
    """Q8_0, eight tokens, a window: slots that only some of the queries see have scales far from all others'."""
    rng = np.random.default_rng(dim)
    n, n_tok, page, window = 44, 8, 16, 30
    cache = ref.Cache(rng, "q8", 3, 1, page, dim)
    table = np.array([[2, 0, 1]], np.int32)
    for i in range(2):
        cache.scale[i][:] = torch.from_numpy(typical * rng.uniform(0.5, 1, cache.scale[i].shape)).half()
    seen = [[np.arange(p - window + 1, p + 1) for p in range(n - n_tok, n)]]
    x = np.zeros((1, n_tok, group, dim), np.float32)
    at = rng.integers(0, dim, (n_tok, group))
    for t in range(n_tok):
        for g in range(group):
            x[0, t, g, at[t, g]] = rng.uniform(0.5, 1) / (127 * typical)
    x = x.reshape(1, n_tok, -1)
    want, tol = tight.attn(cache, x, table, [n], 1.0, seen=seen, depth=8)
    first = seen[0][0][0]                               # the first slots of the first queries, the last ones of the last
    for j in (first, first + 1, n - 2, n - 1):
        for i in range(2):
            cache.scale[i][table[0, j // page], 0, j % page] = bad
    got = run_one_head(cache, x, table, [n], 1.0, window)
    clear = slice(2, n_tok - 2)                         # queries that see none of these
    assert (np.abs(got[:, clear] - want[:, clear]) <= tol[:, clear]).all(), np.max(np.abs(got - want)[:, clear] / tol[:, clear])


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("n_tok,group", [(1, 1), (1, 8), (4, 3)])
def test_attn_a_large_scale_of_little_weight_leaves_the_others_exact(dim, n_tok, group):
    """Q8_0: the first slot's values are up to 65504 times 127, its weight is about 2^-40."""
    rng = np.random.default_rng(dim + n_tok)
    n, page = 30, 16
    cache = ref.Cache(rng, "q8", 2, 1, page, dim)
    table = np.array([[1, 0]], np.int32)
    cache.scale[1][:] = torch.from_numpy(1e-4 * rng.uniform(0.5, 1, cache.scale[1].shape)).half()
    cache.scale[1][1, 0, 0] = 65504.0
    x = np.zeros((1, n_tok, group, dim), np.float32)
    x[..., 5] = 1.0
    x = x.reshape(1, n_tok, -1)
    cache.kv[0][:, :, :, 5] = torch.from_numpy(rng.integers(-20, 20, (2, 1, page))).to(torch.int8)
    cache.scale[0][:, :, :, 0] = 2.0 ** -5
    cache.kv[0][1, 0, 0, 5] = -127
    cache.scale[0][1, 0, 0, 0] = 0.2185                 # a score of -27.75, 40 halvings
    want, tol = tight.attn(cache, x, table, [n], 1.0, depth=8)
    got = run_one_head(cache, x, table, [n], 1.0)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("kind,dim", [(k, d) for k in ("f16", "bf16", "q8") for d in (32, 64, 128, 256) if (k, d) != ("q8", 32)])
@pytest.mark.parametrize("group,n_seq", [(1, 1), (1, 900), (16, 900)])
def test_attn_a_long_tail_of_small_weights_keeps_its_sum(kind, dim, group, n_seq):
    """700 slots of about 2^-22 of the first ones' weight: their errors are alike and add up.  Many sequences share the
    pages, so that a CTA runs over whole ones."""
    n = 700
    cache, table, lens, x = tight.long_tail(kind, dim, n)
    x = np.tile(x, (1, 1, group))
    want, tol = tight.attn(cache, x, table, lens, 1.0, depth=100)
    got = run_one_head(cache, np.tile(x, (n_seq, 1, 1)), np.tile(table, (n_seq, 1)), lens * n_seq, 1.0)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("kind,dim", [("f16", 16), ("f16", 64), ("f16", 128), ("f16", 256), ("bf16", 64), ("bf16", 128), ("bf16", 256), ("q8", 64), ("q8", 128), ("q8", 256)])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_attn_two_slots_keep_every_part(kind, dim, group):
    """Bounds of a few roundings, which a lost part of a query or a weight passes many times over."""
    rng = np.random.default_rng(dim + group)
    cache, table, lens, x = tight.two_slots(rng, kind, dim, 50, group)
    want, tol = tight.attn(cache, x, table, lens, 1.0)
    got = run_one_head(cache, x, table, lens, 1.0)
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / np.maximum(tol, 1e-30))


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("n_kv,n_seq", [(8, 20), (1, 1)])
def test_attn_every_counter_is_zero_again(kind, n_kv, n_seq):
    """64 wide with one query: as many CTAs as an instance can have, nearly all of them with a segment that they share."""
    rng = np.random.default_rng(n_kv)
    lens = [int(x) for x in rng.integers(2500, 3500, n_seq)] if n_seq > 1 else [60000]
    table, n_pages = make_tables(rng, lens, 64)
    cache = ref.Cache(rng, kind, n_pages, n_kv, 64, 64)
    k, v, ks, vs = cache.device()
    c = q.KvCache(base.KINDS[kind], k, v, ks, vs)
    x = dev(rng.standard_normal((n_seq, 1, n_kv * 64)).astype(np.float32))
    ws = torch.zeros(q.attn_ws_bytes(c, n_kv, n_seq, 1, table.shape[1]), dtype=torch.uint8, device="cuda")
    tab, n, first = dev(table), dev(np.array(lens, np.int32)), None
    for _ in range(4):
        out = torch.full(x.shape, float("nan"), device="cuda")
        q.attn_decode(q.AttnArgs(c, x, out, tab, n, ws, 0.125))
        torch.cuda.synchronize()
        assert int(ws[:480 * 4].sum()) == 0             # the counters of the most CTAs that a call has
        first = out if first is None else first
        assert torch.equal(first, out) and bool(torch.isfinite(out).all())


# --------------------------------------------------------------------------------------------------------- eviction --
def test_evict_long_caches_beyond_the_keys_of_a_cluster():
    """Eight CTAs hold the keys of 327680 slots; the others are made anew in every round."""
    n = 330000
    rng = np.random.default_rng(5)
    z = rng.standard_normal((1, 1, n)).astype(np.float32)
    z[rng.random(z.shape) < 0.01] = np.nan
    z[rng.random(z.shape) < 0.01] = -np.inf
    base.run_evict("f16", 16, 1, 256, [n], 4, 100, 2000, z)
    base.run_evict("f16", 16, 1, 256, [n], 0, 0, 1500, rng.integers(0, 4, (1, 1, n)).astype(np.float32))      # ties

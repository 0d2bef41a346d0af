"""The cache and logits operators on a B200 against plain 64-bit forms (step_ref.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_decode_superblocks_b200 as q
import step_ref as ref

pytestmark = pytest.mark.gpu

KINDS = {"f16": q.KV_F16, "bf16": q.KV_BF16, "q8": q.KV_Q8_0}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    q.build()
    q.qmv_check()
    yield
    assert q.qmv_check() == 0


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def make_tables(rng, lens, page, spare=3, n_pages=None):
    """Scattered pages for every sequence; entries behind its length are -1."""
    need = [-(-n // page) for n in lens]
    most = max(1, max(need)) + 1
    total = n_pages or sum(need) + spare
    order = rng.permutation(total)
    table = np.full((len(lens), most), -1, np.int32)
    i = 0
    for s, k in enumerate(need):
        table[s, :k] = order[i:i + k]
        i += k
    return table, total


def unused(table, lens, page, n_pages):
    """[n_pages, 1, page]: slots that belong to no sequence."""
    free = np.ones((n_pages, 1, page), bool)
    for s, n in enumerate(lens):
        for j in range(n):
            if table[s, j // page] >= 0:
                free[table[s, j // page], 0, j % page] = False
    return free


def run_attn(cache, qx, n_head, table, lens, scale, window=0, n_sink=0, score=None, ws=None, max_lens=None, out_pad=0, n_kv=None):
    k, v, ks, vs = cache.device()
    c = q.KvCache(KINDS[cache.kind], k, v, ks, vs)
    n_seq, n_tok, width = qx.shape
    tab = dev(table)
    if ws is None:
        ws = torch.zeros(q.attn_ws_bytes(c, n_head, n_seq, n_tok, tab.shape[1], score is not None), dtype=torch.uint8, device="cuda")
    out = torch.full((n_seq, n_tok, width + out_pad), float("nan"), device="cuda")
    sc = None if score is None else dev(score)
    args = q.AttnArgs(c, dev(qx), out[..., :width], tab, dev(np.asarray(lens, np.int32)), ws, scale, window, n_sink, sc)
    q.attn_decode(args)
    torch.cuda.synchronize()
    assert int(ws[:1280].sum()) == 0                   # the counters are back to zero
    if out_pad:
        assert bool(torch.isnan(out[..., width:]).all())
    return out[..., :width].double().cpu().numpy(), None if sc is None else sc.double().cpu().numpy()


def check_attn(kind, dim, n_kv, group, n_tok, page, lens, layout="head", window=0, n_sink=0, score=False, gap=0, seed=0, out_pad=0, spoil=True):
    rng = np.random.default_rng(seed)
    table, n_pages = make_tables(rng, lens, page)
    fill = unused(table, lens, page, n_pages) if spoil else None
    cache = ref.Cache(rng, kind, n_pages, n_kv, page, dim, layout, gap, fill)
    n_head = n_kv * group
    qx = (1.5 * rng.standard_normal((len(lens), n_tok, n_head * dim))).astype(np.float32)
    sc = rng.random((len(lens), n_kv, table.shape[1] * page)).astype(np.float32) if score else None
    scale = dim ** -0.5
    out, got_score = run_attn(cache, qx, n_head, table, lens, scale, window, n_sink, sc, out_pad=out_pad)
    want, tol, want_score, stol = ref.attn(cache, qx, n_head, table, lens, scale, window, n_sink, sc)
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= tol).all(), np.max(np.abs(out - want) - tol)
    if score:
        assert (np.abs(got_score - want_score) <= stol + 0.0).all(), np.max(np.abs(got_score - want_score) - stol)
    return out


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 127, 129, 500])
def test_attn_one_token_lengths(kind, n):
    check_attn(kind, 64, 2, 4, 1, 16, [n], seed=n)


@pytest.mark.parametrize("kind,dim", [("f16", d) for d in (16, 32, 64, 80, 96, 112, 128, 160, 192, 256)] +
                         [("bf16", d) for d in (16, 48, 64, 80, 128, 144, 256)] + [("q8", d) for d in (64, 128, 192, 256)])
def test_attn_head_dims(kind, dim):
    check_attn(kind, dim, 2, 3, 1, 16, [37, 200], seed=dim)
    check_attn(kind, dim, 1, 5, 4, 8, [3, 141], seed=dim + 1, layout="token")


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 33, 64, 256])
def test_attn_page_sizes_and_layouts(kind, page):
    for layout in ("head", "token"):
        check_attn(kind, 64, 3, 2, 2, page, [70, 1, 130], layout, gap=64 if kind == "q8" else 8, seed=page)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("group,n_tok", [(1, 1), (1, 8), (2, 3), (4, 2), (4, 8), (7, 5), (8, 8), (16, 1), (9, 1), (33, 2), (128, 8)])
def test_attn_groups_and_tokens(kind, group, n_tok):
    check_attn(kind, 64, 1 if group > 30 else 2, group, n_tok, 16, [90, n_tok, 33], seed=group * 10 + n_tok)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (5, 0), (16, 4), (17, 20), (40, 3), (100, 100), (64, 0), (1000, 4)])
@pytest.mark.parametrize("n_tok", [1, 4, 8])
def test_attn_window_and_first_tokens(kind, window, n_sink, n_tok):
    check_attn(kind, 64, 2, 4, n_tok, 16, [200, 3, 64, 16, 33], window=window, n_sink=n_sink, score=True, seed=window + n_sink)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_pages_behind_the_window_are_not_read(kind):
    rng = np.random.default_rng(5)
    lens, page, window, n_sink = [300, 290], 16, 50, 20
    table, n_pages = make_tables(rng, lens, page)
    table[:, 2:13] = 2 ** 30                            # freed: slots 32..207 are seen by no query
    cache = ref.Cache(rng, kind, n_pages, 2, page, 64)
    qx = rng.standard_normal((2, 3, 8 * 64)).astype(np.float32)
    full = table.copy()
    full[:, 2:13] = 0
    out, _ = run_attn(cache, qx, 8, table, lens, 0.125, window, n_sink)
    want, tol, _, _ = ref.attn(cache, qx, 8, full, lens, 0.125, window, n_sink)
    assert (np.abs(out - want) <= tol).all()
    assert q.qmv_check() == 0


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_nothing_to_see_gives_zeros(kind):
    out = check_attn(kind, 64, 2, 4, 3, 16, [0, 1, 2, 3, 50], seed=3)
    assert (out[0] == 0).all() and (out[1, :2] == 0).all() and (out[1, 2] != 0).any()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_long_ragged_batch(kind):
    """Sequences shared by several CTAs, several sequences in one CTA, both at once."""
    check_attn(kind, 64, 4, 2, 1, 16, [5000, 1, 17, 2300, 900, 0, 40], seed=1)
    check_attn(kind, 128, 2, 4, 8, 32, [3001, 12, 600], "token", seed=2, out_pad=4)


def test_attn_many_sequences():
    rng = np.random.default_rng(7)
    check_attn("f16", 64, 1, 2, 1, 16, [int(x) for x in rng.integers(0, 40, 300)], seed=8)
    check_attn("q8", 64, 1, 1, 1, 16, [int(x) for x in rng.integers(0, 10, 1024)], seed=9)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_scores_accumulate(kind):
    check_attn(kind, 64, 2, 4, 1, 16, [100, 1, 1500], score=True, seed=4)
    check_attn(kind, 128, 2, 5, 3, 16, [100, 2, 700], score=True, seed=6)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
def test_attn_values_a_query_does_not_see_never_reach_it(kind, bad):
    """Every query of the newest eight but the last one misses the last slot; a window hides the first ones
    from the later queries only."""
    rng = np.random.default_rng(11)
    lens, page, n_tok, window = [77], 16, 8, 40
    table, n_pages = make_tables(rng, lens, page)
    cache = ref.Cache(rng, kind, n_pages, 1, page, 64)
    clean = ref.Cache(np.random.default_rng(0), kind, n_pages, 1, page, 64)
    clean.kv = [x.clone() for x in cache.kv]
    value = torch.finfo(cache.kv[0].dtype).min if bad == "lowest" else bad
    last, early = 76, 76 - 7 - window + 1               # seen by the last query only / by the first query only
    for j in (last, early):
        for i in range(2):
            cache.kv[i][table[0, j // page], :, j % page] = value
    qx = rng.standard_normal((1, n_tok, 2 * 64)).astype(np.float32)
    out, _ = run_attn(cache, qx, 2, table, lens, 0.125, window)
    want, tol, _, _ = ref.attn(clean, qx, 2, table, lens, 0.125, window)
    inner = slice(1, 7)                                 # these see neither
    assert (np.abs(out[:, inner] - want[:, inner]) <= tol[:, inner]).all()


def test_attn_large_and_tiny_queries():
    """q's parts keep their bits at any magnitude: the scores stay exact to f32."""
    for kind in ("f16", "bf16", "q8"):
        for mag in (1e-30, 1e-6, 1e4, 1e15):
            rng = np.random.default_rng(2)
            table, n_pages = make_tables(rng, [50], 16)
            cache = ref.Cache(rng, kind, n_pages, 1, 16, 64)
            qx = (mag * rng.standard_normal((1, 1, 64))).astype(np.float32)
            scale = float(np.float32(0.125 / mag))
            out, _ = run_attn(cache, qx, 1, table, [50], scale)
            want, tol, _, _ = ref.attn(cache, qx, 1, table, [50], scale)
            assert (np.abs(out - want) <= tol).all(), (kind, mag)


def test_attn_steep_scores():
    """Scores far apart: all weights but a few vanish, and the maximum moves along the cache."""
    for kind in ("f16", "bf16", "q8"):
        for sign in (1, -1):
            rng = np.random.default_rng(3)
            n = 400
            table, n_pages = make_tables(rng, [n], 16)
            cache = ref.Cache(rng, kind, n_pages, 1, 16, 64)
            for j in range(n):                          # keys grow (or shrink) along the sequence
                cache_k = cache.scale[0] if kind == "q8" else cache.kv[0]
                cache_k[table[0, j // 16], :, j % 16] *= 1 + sign * 0.9 * (2 * j / n - 1)
            qx = (20 * rng.standard_normal((1, 1, 64))).astype(np.float32)
            out, _ = run_attn(cache, qx, 1, table, [n], 0.125)
            want, tol, _, _ = ref.attn(cache, qx, 1, table, [n], 0.125)
            assert (np.abs(out - want) <= tol).all()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_bad_pages_and_lengths_are_left_out_and_reported(kind):
    rng = np.random.default_rng(4)
    lens, page = [100, 60], 16
    table, n_pages = make_tables(rng, lens, page)
    cache = ref.Cache(rng, kind, n_pages, 2, page, 64)
    qx = rng.standard_normal((2, 1, 8 * 64)).astype(np.float32)
    for bad in (-1, n_pages, -2 ** 31, 2 ** 31 - 1):
        t = table.copy()
        t[0, 2] = bad
        out, _ = run_attn(cache, qx, 8, t, lens, 0.125)
        hide = t.copy()
        hide[0, 2] = -1
        want, tol, _, _ = ref.attn(cache, qx, 8, hide, lens, 0.125)
        assert (np.abs(out - want) <= tol).all()
        assert q.qmv_check() == q.DEVERR_PAGE_ID
    # one entry more than the sequences need, filled here: a length beyond the table is clamped to it
    full = table.copy()
    full[full < 0] = 0
    out, _ = run_attn(cache, qx, 8, full, [2 ** 31 - 1, -5], 0.125)
    want, tol, _, _ = ref.attn(cache, qx, 8, full, [full.shape[1] * page, 0], 0.125)
    assert (np.abs(out - want) <= tol).all()
    assert q.qmv_check() == q.DEVERR_SEQ_LEN


def test_attn_results_do_not_vary_and_workspaces_serve_other_shapes():
    rng = np.random.default_rng(6)
    lens = [2000, 31, 700]
    table, n_pages = make_tables(rng, lens, 16)
    cache = ref.Cache(rng, "bf16", n_pages, 2, 16, 128)
    qx = rng.standard_normal((3, 8, 8 * 128)).astype(np.float32)
    k, v, _, _ = cache.device()
    c = q.KvCache(q.KV_BF16, k, v)
    ws = torch.zeros(q.attn_ws_bytes(c, 8, 3, 8, table.shape[1]), dtype=torch.uint8, device="cuda")
    first, _ = run_attn(cache, qx, 8, table, lens, 0.09, ws=ws)
    run_attn(cache, qx[:1, :1], 8, table[:1], lens[:1], 0.09, ws=ws)
    for _ in range(3):
        again, _ = run_attn(cache, qx, 8, table, lens, 0.09, ws=ws)
        assert np.array_equal(first, again)


def test_attn_captured_and_replayed_with_growing_lengths_and_on_two_streams():
    rng = np.random.default_rng(8)
    lens = [40, 130]
    table, n_pages = make_tables(rng, [200, 200], 16)
    cache = ref.Cache(rng, "f16", n_pages, 2, 16, 64)
    qx = rng.standard_normal((2, 1, 8 * 64)).astype(np.float32)
    k, v, _, _ = cache.device()
    c = q.KvCache(q.KV_F16, k, v)
    tab, qd = dev(table), dev(qx)
    sets = []
    for _ in range(2):
        n = dev(np.asarray(lens, np.int32))
        out = torch.zeros(2, 1, 8 * 64, device="cuda")
        ws = torch.zeros(q.attn_ws_bytes(c, 8, 2, 1, table.shape[1]), dtype=torch.uint8, device="cuda")
        sets.append((n, out, q.AttnArgs(c, qd, out, tab, n, ws, 0.125)))
    q.attn_decode(sets[0][2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.attn_decode(sets[0][2])
    other = torch.cuda.Stream()
    for step in range(0, 61, 20):
        now = [x + step for x in lens]
        for n, _, _ in sets:
            n.copy_(torch.tensor(now, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        q.attn_decode(sets[1][2], other)
        torch.cuda.synchronize()
        want, tol, _, _ = ref.attn(cache, qx, 8, table, now, 0.125)
        for _, out, _ in sets:
            assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def test_attn_a_pool_beyond_32_bits():
    """A slot whose element lies past 2^32: page 70000 of a pool of 65536-element pages, most of it never touched."""
    page, dim, n_kv = 256, 128, 2
    n_pages = 70001
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * page * dim * n_kv * 2:
        pytest.skip("needs 28 GB")
    pool = torch.empty(2, n_pages, n_kv, page, dim, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(1)
    small = ref.Cache(rng, "bf16", 2, n_kv, page, dim)
    ids = [n_pages - 1, 65537]
    for i in range(2):
        for s, t in enumerate(ids):
            pool[i, t] = small.kv[i][s].cuda()
    qx = rng.standard_normal((1, 1, 8 * dim)).astype(np.float32)
    c = q.KvCache(q.KV_BF16, pool[0], pool[1])
    out = torch.zeros(1, 1, 8 * dim, device="cuda")
    ws = torch.zeros(q.attn_ws_bytes(c, 8, 1, 1, 2), dtype=torch.uint8, device="cuda")
    q.attn_decode(q.AttnArgs(c, dev(qx), out, dev(np.array([ids], np.int32)), dev(np.array([500], np.int32)), ws, 0.1))
    want, tol, _, _ = ref.attn(small, qx, 8, [[0, 1]], [500], 0.1)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


# ------------------------------------------------------------------------------------------------------ append --
@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 16), ("f16", 80), ("bf16", 128), ("bf16", 256), ("q8", 64), ("q8", 192), ("q8", 256)])
@pytest.mark.parametrize("style", [q.ROPE_HALVES, q.ROPE_PAIRS])
@pytest.mark.parametrize("n_tok,layout", [(1, "head"), (5, "token"), (8, "head")])
def test_append(kind, dim, style, n_tok, layout):
    rng = np.random.default_rng(dim + n_tok)
    n_kv, n_head, page, lens = 3, 6, 7, [n_tok + 3, n_tok, 2, 40, 0]
    rope_dim = {16: 16, 80: 40}.get(dim, dim if n_tok == 1 else dim // 2)
    table, n_pages = make_tables(rng, lens, page)
    cache = ref.Cache(rng, kind, n_pages, n_kv, page, dim, layout, 64 if kind == "q8" else 8)
    before = [cache.values(i).copy() for i in range(2)]
    x = (3 * rng.standard_normal((len(lens), n_tok, (n_head + 2 * n_kv) * dim))).astype(np.float32)
    x[0, 0, n_head * dim:(n_head + 1) * dim] = 0       # a head of zeros
    pos = rng.integers(0, 2_000_000, (len(lens), n_tok)).astype(np.int32)
    inv = (10000.0 ** (-2.0 * np.arange(rope_dim // 2) / max(rope_dim, 1))).astype(np.float32)
    k, v, ks, vs = cache.device()
    c = q.KvCache(KINDS[kind], k, v, ks, vs)
    xd = dev(x)
    qd, kd, vd = xd.split([n_head * dim, n_kv * dim, n_kv * dim], -1)
    q_out = torch.zeros(len(lens), n_tok, n_head * dim, device="cuda")
    q.kv_append(q.AppendArgs(c, qd, kd, vd, q_out, dev(table), dev(np.asarray(lens, np.int32)), pos=dev(pos), inv_freq=dev(inv), rope_dim=rope_dim,
                             rope_style=style))
    got = []
    for pool, sc in ((k, ks), (v, vs)):
        y = pool.double().cpu()
        if kind == "q8":
            y = (y.reshape(*y.shape[:3], -1, 32) * sc.double().cpu()[..., None]).reshape(y.shape)
        got.append(y.numpy())
    want = [b.copy() for b in before]
    tol = [np.zeros_like(b) for b in before]
    heads = x.reshape(len(lens), n_tok, n_head + 2 * n_kv, dim)
    half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "q8": 0.0}[kind]
    q_want = np.zeros((len(lens), n_tok, n_head, dim))
    for s, n in enumerate(lens):
        for t in range(n_tok):
            turned = rope(heads[s, t, :n_head + n_kv], pos[s, t], inv, rope_dim, style == q.ROPE_PAIRS)
            q_want[s, t] = turned[:n_head]
            j = n - n_tok + t
            if j < 0:
                continue
            p, o = table[s, j // page], j % page
            for i, y in enumerate((turned[n_head:], heads[s, t, n_head + n_kv:].astype(np.float64))):
                if kind == "q8":
                    b = y.astype(np.float32).reshape(n_kv, -1, 32)
                    d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float16).astype(np.float32)
                    quant = np.clip(np.rint(b / np.where(d > 0, d, 1)[..., None]), -127, 127) * (d > 0)[..., None]
                    y = (quant.astype(np.float64) * d[..., None]).reshape(n_kv, dim)
                    want[i][p, :, o] = y
                else:
                    want[i][p, :, o] = y
                    # one rounding to f32 and one to the cache's type (f16: half a step of the subnormals at least)
                    tol[i][p, :, o] = np.abs(y) * (half + 2 * ref.U) + (2.0 ** -25 if kind == "f16" else 0)
    for i in range(2):
        assert (np.abs(got[i] - want[i]) <= tol[i]).all(), i
    q_got = q_out.double().cpu().numpy().reshape(q_want.shape)
    assert (np.abs(q_got - q_want) <= 2 * ref.U * np.abs(q_want) + 1e-12 * 3).all()


rope = ref.rope


def test_append_in_place_without_rope_and_without_q():
    rng = np.random.default_rng(1)
    dim, page, lens = 64, 16, [20]
    table, n_pages = make_tables(rng, lens, page)
    inv = np.array([1.0 / (i + 1) for i in range(32)], np.float32)
    for q_mode in ("in place", "none", "copy"):
        cache = ref.Cache(rng, "bf16", n_pages, 2, page, dim)
        k, v, _, _ = cache.device()
        c = q.KvCache(q.KV_BF16, k, v)
        x = rng.standard_normal((1, 2, 8 * dim)).astype(np.float32)
        xd = dev(x)
        qd, kd, vd = xd.split([4 * dim, 2 * dim, 2 * dim], -1)
        rd = 64 if q_mode == "in place" else 0
        out = {"in place": qd, "none": None, "copy": torch.zeros(1, 2, 4 * dim, device="cuda")}[q_mode]
        q.kv_append(q.AppendArgs(c, None if q_mode == "none" else qd, kd, vd, out, dev(table), dev(np.array(lens, np.int32)),
                                 inv_freq=dev(inv) if rd else None, rope_dim=rd))
        for t in range(2):                              # positions are the slots 18 and 19
            y = ref.rope(x[0, t, :6 * dim].reshape(6, dim), 18 + t, inv, rd, False)
            if out is not None:
                assert np.abs(out[0, t].double().cpu().numpy() - y[:4].reshape(-1)).max() <= 1e-6
            got = k[int(table[0, 1]), :, 2 + t].double().cpu().numpy()
            assert (np.abs(got - y[4:]) <= 2.0 ** -8 * np.abs(y[4:]) * 1.01).all()
    # a bad page: nothing stored, the query still rotated
    before = k.clone()
    t = table.copy()
    t[0, 1] = n_pages
    out.zero_()
    q.kv_append(q.AppendArgs(c, qd, kd, vd, out, dev(t), dev(np.array(lens, np.int32))))
    assert torch.equal(before, k) and torch.equal(out, qd)
    assert q.qmv_check() == q.DEVERR_PAGE_ID


# ------------------------------------------------------------------------------------------------------- evict --
def run_evict(kind, dim, n_kv, page, lens, first, last, budget, score, layout="head", seed=0, gap=0):
    rng = np.random.default_rng(seed)
    table, n_src = make_tables(rng, lens, page)
    new = [min(n, budget) for n in lens]
    dst, n_dst = make_tables(rng, new, page)
    dst[dst >= 0] += n_src
    dst[dst < 0] = -1
    # the budget has to fit the table
    wide = max(dst.shape[1], -(-budget // page))
    dst = np.concatenate([dst, np.full((len(lens), wide - dst.shape[1]), -1, np.int32)], 1)
    cache = ref.Cache(rng, kind, n_src + n_dst, n_kv, page, dim, layout, gap)
    k, v, ks, vs = cache.device()
    c = q.KvCache(KINDS[kind], k, v, ks, vs)
    sc = dev(score)
    kept = torch.full((len(lens), n_kv, budget), -7, dtype=torch.int32, device="cuda")
    score_out = torch.full((len(lens), n_kv, budget + 3), -7.0, device="cuda")
    len_out = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    q.kv_evict(q.EvictArgs(c, sc, dev(table), dev(np.asarray(lens, np.int32)), dev(dst), kept, score_out, len_out, first, last, budget))
    torch.cuda.synchronize()
    want = ref.evict(score, lens, first, last, budget)
    assert len_out.tolist() == new
    expect = [[x.clone() for x in cache.kv], [x.clone() for x in cache.scale]]
    kept, score_out = kept.cpu().numpy(), score_out.cpu().numpy()
    for s in range(len(lens)):
        for h in range(n_kv):
            w = want[s][h]
            assert kept[s, h, :len(w)].tolist() == w and (kept[s, h, len(w):] == -7).all(), (s, h)
            assert np.array_equal(score_out[s, h, :len(w)], score[s, h, w], equal_nan=True) and (score_out[s, h, len(w):] == -7).all()
            for part in expect:
                for x in part:
                    for i, j in enumerate(w):
                        x[dst[s, i // page], h, i % page] = x[table[s, j // page], h, j % page]
    for got, x in zip((k, v, ks, vs), expect[0] + expect[1]):
        assert torch.equal(got.cpu(), x)                # everything else as it was


@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 16), ("bf16", 112), ("bf16", 256), ("q8", 64), ("q8", 192), ("q8", 256)])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_evict(kind, dim, layout):
    rng = np.random.default_rng(dim)
    lens = [100, 0, 1, 41, 40, 333]
    score = rng.random((len(lens), 3, 340)).astype(np.float32)
    for first, last, budget in ((4, 10, 40), (0, 0, 1), (0, 0, 40), (20, 20, 40), (0, 40, 40), (3, 0, 17)):
        run_evict(kind, dim, 3, 16, lens, first, last, budget, score, layout, gap=64 if kind == "q8" else 0)


def test_evict_ties_nan_and_signs():
    rng = np.random.default_rng(2)
    lens = [700, 5000]
    score = rng.integers(0, 3, (2, 2, 5000)).astype(np.float32)     # many ties
    run_evict("f16", 32, 2, 7, lens, 1, 2, 300, score)
    score = rng.standard_normal((2, 2, 5000)).astype(np.float32)
    score[rng.random(score.shape) < 0.3] = np.nan
    score[rng.random(score.shape) < 0.05] = -np.inf
    score[rng.random(score.shape) < 0.05] = np.inf
    score[rng.random(score.shape) < 0.1] = -0.0
    score[rng.random(score.shape) < 0.1] = 0.0
    for budget in (10, 400, 4990):
        run_evict("f16", 32, 2, 16, lens, 2, 3, budget, score)
    run_evict("f16", 32, 1, 16, [5000], 0, 0, 4000, np.zeros((1, 1, 5000), np.float32))


@pytest.mark.parametrize("n", [4095, 4096, 4097, 40000])
def test_evict_long(n):
    rng = np.random.default_rng(n)
    run_evict("f16", 16, 1, 64, [n], 4, 100, 2000, rng.random((1, 1, n)).astype(np.float32))


def test_evict_bad_pages_are_reported_and_not_written():
    rng = np.random.default_rng(2)
    table = np.array([[0, 99, 1]], np.int32)
    cache = ref.Cache(rng, "f16", 4, 1, 16, 16)
    k, v, _, _ = cache.device()
    before = k.clone()
    c = q.KvCache(q.KV_F16, k, v)
    score = dev(np.arange(48, dtype=np.float32)[None, None])
    kept, so = torch.zeros(1, 1, 48, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, 48, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.kv_evict(q.EvictArgs(c, score, dev(table), dev(np.array([48], np.int32)), dev(np.array([[2, 3, -1]], np.int32)), kept, so, n, 0, 0, 48))
    assert kept[0, 0].tolist() == list(range(48)) and n.item() == 48
    assert torch.equal(k[2], before[0]) and torch.equal(k[3], before[3]) and torch.equal(k[:2], before[:2])
    assert q.qmv_check() == q.DEVERR_PAGE_ID


# ------------------------------------------------------------------------------------------------------ logits --
def run_logits(z, hist=None, hist_len=None, params=None, bias_ids=None, bias_vals=None, bias_len=None, mask=None, out_mode="own", stride_pad=0):
    n, v = z.shape
    zd = torch.full((n, v + stride_pad), 1e30, device="cuda")
    zd[:, :v] = dev(z)
    zd = zd[:, :v]
    out = {"own": torch.zeros(n, v, device="cuda"), "in place": zd, "none": None}[out_mode]
    idx = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    ws = torch.zeros(q.logits_ws_bytes(n), dtype=torch.uint8, device="cuda")
    g = lambda x: None if x is None else dev(x)  # noqa: E731
    args = q.LogitsArgs(zd, g(hist), g(hist_len), g(params), out, idx, ws, g(bias_ids), g(bias_vals), g(bias_len), g(mask))
    q.logits_argmax(args)
    torch.cuda.synchronize()
    assert int(ws.sum()) == 0
    want, want_idx = ref.logits(z, hist, hist_len, params, bias_ids, bias_vals, bias_len, mask)
    if out is not None:
        assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)
    assert idx.tolist() == want_idx.tolist()
    return args, out, idx


@pytest.mark.parametrize("v", [1, 31, 32, 33, 2047, 2048, 2049, 50257, 128000])
@pytest.mark.parametrize("n", [1, 5])
def test_logits(v, n):
    rng = np.random.default_rng(v + n)
    z = rng.standard_normal((n, v)).astype(np.float32)
    hist = rng.integers(-2, v + 2, (n, 300)).astype(np.int32)       # ids outside the vocabulary are skipped
    hist[:, :50] = hist[:, 50:100]                                  # repeats
    hist_len = np.array([300, 0, -3, 1000, 17][:n], np.int32)
    params = np.stack([1 + rng.random(n), rng.random(n), rng.random(n)], 1).astype(np.float32)
    ids = rng.integers(-1, v + 1, (n, 40)).astype(np.int32)
    ids[:, 20:] = ids[:, :20]                                       # the same token twice: the later entry counts
    vals = rng.standard_normal((n, 40)).astype(np.float32)
    blen = np.array([40, 30, 0, 99, -1][:n], np.int32)
    mask = rng.integers(-2**31, 2**31, (n, -(-v // 32) + 2)).astype(np.int32)
    run_logits(z)
    run_logits(z, hist, hist_len, params)
    run_logits(z, None, None, None, ids, vals, blen)
    run_logits(z, None, None, None, None, None, None, mask, out_mode="none")
    for mode in ("own", "in place"):
        run_logits(z, hist, hist_len, params, ids, vals, blen, mask, mode, stride_pad=0 if n == 1 else 5)


def test_logits_ties_masks_and_special_values():
    v = 5000
    z = np.zeros((6, v), np.float32)
    z[1, [77, 3000]] = 4                                            # ties: the lowest token
    z[2] = np.nan
    z[3, :] = -np.inf
    z[4, 9] = np.inf
    z[4, 4000] = np.nan
    mask = np.full((6, -(-v // 32)), -1, np.int32)
    mask[5] = 0                                                     # nothing allowed
    run_logits(z, mask=mask)
    _, out, idx = run_logits(z)
    assert idx.tolist() == [0, 77, -1, -1, 9, 0]
    z = np.full((1, v), np.finfo(np.float32).min, np.float32)       # the lowest value is a value, not a mask
    mask = np.zeros((1, -(-v // 32)), np.int32)
    mask[0, 100] = 4
    _, _, idx = run_logits(z, mask=mask)
    assert idx.tolist() == [3202]


def test_logits_captured_and_after_the_vocabulary_product():
    rng = np.random.default_rng(3)
    v, n = 4096, 3
    z = rng.standard_normal((n, v)).astype(np.float32)
    hist = rng.integers(0, v, (n, 64)).astype(np.int32)
    params = np.tile(np.array([[1.2, 0.1, 0.2]], np.float32), (n, 1))
    args, out, idx = run_logits(z, hist, np.full(n, 64, np.int32), params)
    zd = args._held[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.logits_argmax(args)
    for seed in range(3):
        z = np.random.default_rng(seed).standard_normal((n, v)).astype(np.float32)
        zd.copy_(dev(z))
        graph.replay()
        want, want_idx = ref.logits(z, hist, np.full(n, 64, np.int32), params)
        assert np.array_equal(out.cpu().numpy(), want) and idx.tolist() == want_idx.tolist()

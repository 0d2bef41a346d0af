"""The cache and logits operators at the edges of their variants, captured, on other streams, and together
with the weight products as a decode loop uses them; plain 64-bit forms in step_ref.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_decode_superblocks_b200 as q
import step_ref as ref
import test_step_gpu as base
from quantized_decode_superblocks_b200 import synth
from test_step_gpu import check_attn, dev, make_tables, run_attn, run_evict, run_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    q.build()
    q.qmv_check()
    yield
    assert q.qmv_check() == 0


# ----------------------------------------------------------------------------------------------------- attention --
@pytest.mark.parametrize("kind,dim,n_kv,group,n_tok", [
    ("f16", 64, 1, 1, 1), ("bf16", 64, 1, 4, 1), ("q8", 64, 1, 2, 2), ("f16", 128, 1, 4, 1), ("bf16", 128, 1, 2, 8),
    ("q8", 128, 1, 8, 2), ("f16", 256, 1, 3, 1), ("q8", 256, 1, 8, 4), ("bf16", 16, 1, 1, 1)])
def test_attn_one_head_over_every_cta(kind, dim, n_kv, group, n_tok):
    """One head cut into as many parts as there are CTAs: few rows are joined by two threads each, more by one."""
    check_attn(kind, dim, n_kv, group, n_tok, 16, [20011], seed=dim + group, score=dim == 128)


@pytest.mark.parametrize("n_seq", [31, 32, 33, 127, 128, 129, 300])
def test_attn_numbers_of_sequences(n_seq):
    """Up to 32 sequences are looked up in registers, more in shared memory, 128 at a time; ragged ones of them may
    each have whole CTAs, or share them."""
    rng = np.random.default_rng(n_seq)
    check_attn("f16", 32, 1, 2, 1, 16, [int(x) for x in rng.integers(0, 900, n_seq)], seed=n_seq)
    check_attn("q8", 64, 2, 2, 2, 48, [int(x) for x in rng.integers(1, 200, n_seq)], seed=n_seq, layout="token")


@pytest.mark.parametrize("page", [8, 16, 17, 32, 80])
@pytest.mark.parametrize("kind,dim", [("f16", 64), ("q8", 64), ("q8", 128), ("bf16", 128)])
def test_attn_windows_that_start_and_end_inside_tiles(kind, dim, page):
    """Window starts around the 16 and 32 slots of a tile, first tokens that end before, in and after them."""
    for window, n_sink in ((15, 0), (16, 1), (31, 16), (33, 17), (48, 31), (64, 33)):
        check_attn(kind, dim, 1, 3, 3, page, [159, 96, 65, 33], window=window, n_sink=n_sink, score=True, seed=window)


def test_attn_scale_signs():
    """A negative scale is the scale of negated queries; with none every visible slot weighs the same."""
    for kind in ("f16", "bf16", "q8"):
        rng = np.random.default_rng(9)
        lens = [300, 17]
        table, n_pages = make_tables(rng, lens, 16)
        cache = ref.Cache(rng, kind, n_pages, 2, 16, 64)
        x = rng.standard_normal((2, 1, 4 * 64)).astype(np.float32)
        plus, _ = run_attn(cache, x, 4, table, lens, 0.2)
        minus, _ = run_attn(cache, -x, 4, table, lens, -0.2)
        assert np.array_equal(plus, minus)
        even, _ = run_attn(cache, x, 4, table, lens, 0.0)
        for s, n in enumerate(lens):
            for h in range(2):
                v = cache.rows(1, table[s], n, h)
                mean, bound = v.mean(0), 2 * ref.U * (n + 64) * np.abs(v).mean(0)
                got = even[s, 0].reshape(2, 2, 64)[h]
                assert (np.abs(got - mean) <= bound).all()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_attn_scores_captured_and_replayed_on_another_stream(kind):
    rng = np.random.default_rng(12)
    room, page, n_kv, n_head, n_tok, dim = [700, 260], 16, 2, 8, 2, 64
    table, n_pages = make_tables(rng, room, page)
    cache = ref.Cache(rng, kind, n_pages, n_kv, page, dim)
    k, v, ks, vs = cache.device()
    c = q.KvCache(base.KINDS[kind], k, v, ks, vs)
    x = rng.standard_normal((2, n_tok, n_head * dim)).astype(np.float32)
    tab, lens, out = dev(table), dev(np.zeros(2, np.int32)), torch.zeros(2, n_tok, n_head * dim, device="cuda")
    slots = table.shape[1] * page
    score = torch.zeros(2, n_kv, slots, device="cuda")
    ws = torch.zeros(q.attn_ws_bytes(c, n_head, 2, n_tok, table.shape[1], True), dtype=torch.uint8, device="cuda")
    args = q.AttnArgs(c, dev(x), out, tab, lens, ws, 0.125, 300, 4, score)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q.attn_decode(args)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q.attn_decode(args)
    want = np.zeros((2, n_kv, slots))
    stol = np.zeros_like(want)
    score.zero_()
    for now in ([0, 1], [500, 3], [502, 5], [700, 260]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        expect, tol, want, t = ref.attn(cache, x, n_head, table, now, 0.125, 300, 4, want)
        stol += t
        assert (np.abs(out.double().cpu().numpy() - expect) <= tol).all()
        assert (np.abs(score.double().cpu().numpy() - want) <= stol).all()


def test_attn_lengths_beyond_the_scores_and_tables_far_beyond_the_lengths():
    rng = np.random.default_rng(14)
    lens, page, n_kv, dim = [50, 20], 16, 2, 64
    table, n_pages = make_tables(rng, lens, page)
    cache = ref.Cache(rng, "f16", n_pages, n_kv, page, dim)
    x = rng.standard_normal((2, 1, 4 * dim)).astype(np.float32)
    score = rng.random((2, n_kv, 32)).astype(np.float32)         # room for 32 slots only
    out, got = run_attn(cache, x, 4, table, lens, 0.125, score=score)
    assert q.qmv_check() == q.DEVERR_SEQ_LEN
    want, tol, want_score, stol = ref.attn(cache, x, 4, table, [32, 20], 0.125, score=score)
    assert (np.abs(out - want) <= tol).all() and (np.abs(got - want_score) <= stol).all()
    wide = np.full((2, 40000), -1, np.int32)                      # 640000 slots that a later step may reach
    wide[:, :table.shape[1]] = table
    score = rng.random((2, n_kv, 640000)).astype(np.float32)
    out, got = run_attn(cache, x, 4, wide, lens, 0.125, score=score)
    want, tol, want_score, stol = ref.attn(cache, x, 4, table, lens, 0.125, score=score[:, :, :64])
    assert (np.abs(out - want) <= tol).all() and (np.abs(got[:, :, :64] - want_score) <= stol).all()
    assert np.array_equal(got[:, :, 64:].astype(np.float32), score[:, :, 64:])


# ------------------------------------------------------------------------------------------------------- eviction --
@pytest.mark.parametrize("n,budget", [(40959, 1000), (40961, 40000), (50000, 12345)])
def test_evict_beyond_the_keys_that_shared_memory_holds(n, budget):
    rng = np.random.default_rng(n)
    run_evict("f16", 16, 1, 64, [n, 100], 3, 50, budget, rng.random((2, 1, n)).astype(np.float32))
    run_evict("f16", 16, 1, 64, [n], 3, 50, budget, rng.integers(0, 5, (1, 1, n)).astype(np.float32))      # ties


def test_evict_long_caches_of_few_and_of_many_heads():
    """Several CTAs choose for a head where there are few; one does where there are many."""
    rng = np.random.default_rng(8)
    lens = [17000, 0, 1, 16384, 8193, 300]
    for kind, first, last, budget in (("f16", 4, 100, 5000), ("bf16", 0, 0, 1), ("q8", 250, 50, 300)):
        for score in (rng.standard_normal((6, 2, 17000)), rng.integers(-2, 3, (6, 2, 17000))):
            run_evict(kind, 64, 2, 64, lens, first, last, budget, score.astype(np.float32), "token")
    score = rng.standard_normal((1, 20, 41500)).astype(np.float32)
    score[rng.random(score.shape) < 0.2] = np.nan
    run_evict("f16", 16, 20, 64, [41500], 1, 1, 41000, score)
    run_evict("f16", 16, 20, 64, [41500], 1, 1, 900, score)


def test_evict_nothing_between_the_ends_and_everything():
    rng = np.random.default_rng(1)
    score = rng.standard_normal((3, 2, 400)).astype(np.float32)
    run_evict("q8", 64, 2, 16, [400, 30, 31], 10, 20, 30, score, "token")
    run_evict("bf16", 32, 2, 16, [400, 399, 2], 0, 0, 399, score)
    run_evict("bf16", 256, 2, 5, [400, 399, 2], 0, 0, 400, score)


def test_evict_captured_and_replayed():
    rng = np.random.default_rng(3)
    n, budget, page, n_kv, dim = 300, 64, 16, 2, 64
    table, n_src = make_tables(rng, [n], page)
    dst = np.arange(4, dtype=np.int32)[None] + n_src
    cache = ref.Cache(rng, "bf16", n_src + 4, n_kv, page, dim)
    k, v, _, _ = cache.device()
    score, lens = torch.zeros(1, n_kv, n, device="cuda"), dev(np.array([n], np.int32))
    kept, so = torch.zeros(1, n_kv, budget, dtype=torch.int32, device="cuda"), torch.zeros(1, n_kv, budget, device="cuda")
    n_out = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = q.EvictArgs(q.KvCache(q.KV_BF16, k, v), score, dev(table), lens, dev(dst), kept, so, n_out, 2, 8, budget)
    q.kv_evict(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.kv_evict(args)
    for step, now in enumerate((300, 257, 64, 40)):
        z = np.random.default_rng(step).random((1, n_kv, n)).astype(np.float32)
        score.copy_(dev(z))
        lens.fill_(now)
        k[n_src:] = 0
        graph.replay()
        want = ref.evict(z, [now], 2, 8, budget)[0]
        assert n_out.item() == min(now, budget)
        for h in range(n_kv):
            w = want[h]
            assert kept[0, h, :len(w)].tolist() == w and np.array_equal(so[0, h, :len(w)].cpu().numpy(), z[0, h, w])
            got = k[n_src:, h].cpu().reshape(-1, dim)
            old = cache.kv[0][table[0].clip(0)][:, h].reshape(-1, dim)
            assert torch.equal(got[:len(w)], old[w]) and not got[len(w):].any()


# --------------------------------------------------------------------------------------------------------- logits --
@pytest.mark.parametrize("v", [5, 1023, 1025, 8193, 20001])
def test_logits_most_tokens_pushed(v):
    """More pushed tokens than a slice's list holds, and entries in neither order nor range."""
    rng = np.random.default_rng(v)
    z = rng.standard_normal((3, v)).astype(np.float32)
    hist = np.concatenate([rng.permutation(v) for _ in range(2)])[None].repeat(3, 0).astype(np.int32)
    hist_len = np.array([2 * v, v // 2, v + 1], np.int32)
    params = np.array([[1.1, 0.2, 0.3], [0.7, -0.5, 0.0], [1.0, 0.0, 0.0]], np.float32)
    ids = rng.integers(-1, v + 1, (3, 2 * v)).astype(np.int32)
    vals = rng.standard_normal(ids.shape).astype(np.float32)
    mask = rng.integers(-2**31, 2**31, (3, -(-v // 32))).astype(np.int32)
    for mode in ("own", "in place", "none"):
        run_logits(z, hist, hist_len, params, ids, vals, np.array([2 * v, v, 1], np.int32), mask, mode, stride_pad=3)


def test_logits_histories_and_biases_beyond_16_bits():
    """Counts and entries that need more than 16 bits."""
    rng = np.random.default_rng(1)
    v, n = 3001, 70001
    z = rng.standard_normal((2, v)).astype(np.float32)
    hist = np.full((2, n), 7, np.int32)                 # one token 70000 times
    hist[:, ::1000] = rng.integers(0, v, (2, 71))
    params = np.array([[1.3, 1e-4, 0.1], [1.0, 1e-4, 0.0]], np.float32)
    ids = rng.integers(0, v, (2, n)).astype(np.int32)
    vals = rng.standard_normal((2, n)).astype(np.float32)
    blen = np.array([n, 66000], np.int32)
    run_logits(z, hist, np.array([n, n - 5], np.int32), params, ids, vals, blen)
    run_logits(z, hist, np.array([n, n - 5], np.int32), params)
    run_logits(z, None, None, None, ids, vals, blen, out_mode="in place")
    run_logits(z, hist[:, :65535], np.array([65535, 65535], np.int32), params, ids[:, :65534], vals[:, :65534], np.array([65534, 65534], np.int32))


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_logits_rows_at_any_alignment(offset):
    """Rows and outputs whose 16-byte boundaries lie apart."""
    rng = np.random.default_rng(offset)
    n, v = 3, 2050
    z = rng.standard_normal((n, v)).astype(np.float32)
    hist = rng.integers(0, v, (n, 50)).astype(np.int32)
    params = np.tile(np.array([[1.2, 0.1, 0.2]], np.float32), (n, 1))
    mask = rng.integers(-2**31, 2**31, (n, -(-v // 32))).astype(np.int32)
    want, idx_want = ref.logits(z, hist, np.full(n, 50, np.int32), params, mask=mask)
    for out_offset in range(4):
        store = torch.full((n * (v + 7) + 8,), 5.0, device="cuda")
        zd = torch.as_strided(store, (n, v), (v + 7, 1), offset)
        zd.copy_(dev(z))
        hold = torch.full((n * (v + 9) + 8,), 9.0, device="cuda")
        out = torch.as_strided(hold, (n, v), (v + 9, 1), out_offset)
        idx = torch.zeros(n, dtype=torch.int32, device="cuda")
        ws = torch.zeros(q.logits_ws_bytes(n), dtype=torch.uint8, device="cuda")
        q.logits_argmax(q.LogitsArgs(zd, dev(hist), dev(np.full(n, 50, np.int32)), dev(params), out, idx, ws, mask=dev(mask)))
        assert np.array_equal(out.cpu().numpy(), want) and idx.tolist() == idx_want.tolist()
        used = torch.zeros_like(hold, dtype=torch.bool)
        torch.as_strided(used, (n, v), (v + 9, 1), out_offset).fill_(True)
        assert bool((hold[~used] == 9.0).all())


def test_arguments_of_another_operator_are_refused():
    z = torch.zeros(1, 8, device="cuda")
    args = q.LogitsArgs(z, None, None, None, None, torch.zeros(1, dtype=torch.int32, device="cuda"),
                        torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="logits_argmax"):
        q.attn_decode(args)
    q.logits_argmax(args)
    with pytest.raises(TypeError, match="logits_argmax"):
        q.kv_evict(args)


# ------------------------------------------------------------------------------------------------------- together --
@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
def test_a_decode_loop_with_the_weight_products(kind, pdl):
    """Fused QKV product -> kv_append -> attn_decode with weights accumulated -> O product -> vocabulary product ->
    logits_argmax, captured once and replayed as the sequences grow; then kv_evict, and on over the smaller cache.
    Every operator is held to its 64-bit form on the inputs that the one before it really gave."""
    rng = np.random.default_rng(21)
    hidden, n_head, n_kv, dim, vocab, n_seq, page, room = 256, 8, 2, 64, 4000, 2, 16, 160
    group, wide = n_head // n_kv, (n_head + 2 * n_kv) * dim
    weights = [dev(synth.gen_blocks(synth.Q8_0, rows, cols, 5, i)) for i, (rows, cols) in
               enumerate([(wide, hidden), (hidden, n_head * dim), (vocab, hidden)])]
    lens = [40, 23]
    table, n_src = make_tables(rng, [room, room], page)
    new_pages = 2 * 3
    cache = ref.Cache(rng, kind, n_src + new_pages, n_kv, page, dim)
    k, v, ks, vs = cache.device()
    c = q.KvCache(base.KINDS[kind], k, v, ks, vs)
    slots = table.shape[1] * page
    inv = (10000.0 ** (-2.0 * np.arange(dim // 2) / dim)).astype(np.float32)
    x, y = torch.empty(n_seq, hidden, device="cuda"), torch.empty(n_seq, wide, device="cuda")
    qr, out = torch.empty(n_seq, 1, n_head * dim, device="cuda"), torch.empty(n_seq, 1, n_head * dim, device="cuda")
    h, z = torch.empty(n_seq, hidden, device="cuda"), torch.empty(n_seq, vocab, device="cuda")
    adj, idx = torch.empty(n_seq, vocab, device="cuda"), torch.empty(n_seq, dtype=torch.int32, device="cuda")
    n_dev, tab = dev(np.array(lens, np.int32)), dev(table)
    pos = torch.zeros(n_seq, 1, dtype=torch.int32, device="cuda")
    score = torch.zeros(n_seq, n_kv, slots, device="cuda")
    hist, hist_len = torch.zeros(n_seq, 32, dtype=torch.int32, device="cuda"), torch.zeros(n_seq, dtype=torch.int32, device="cuda")
    params = dev(np.tile(np.array([[1.2, 0.1, 0.3]], np.float32), (n_seq, 1)))
    ws = torch.zeros(q.attn_ws_bytes(c, n_head, n_seq, 1, table.shape[1], True), dtype=torch.uint8, device="cuda")
    lws = torch.zeros(q.logits_ws_bytes(n_seq), dtype=torch.uint8, device="cuda")
    qs, kn, vn = y.view(n_seq, 1, wide).split([n_head * dim, n_kv * dim, n_kv * dim], -1)
    append = q.AppendArgs(c, qs, kn, vn, qr, tab, n_dev, pos=pos, inv_freq=dev(inv), rope_dim=dim)
    attn = q.AttnArgs(c, qr, out, tab, n_dev, ws, dim ** -0.5, score=score)
    choose = q.LogitsArgs(z, hist, hist_len, params, adj, idx, lws)

    def step():
        q.qmv_batched(synth.Q8_0, weights[0], wide, hidden, x, y, n_seq)
        q.kv_append(append)
        q.attn_decode(attn)
        q.qmv_batched(synth.Q8_0, weights[1], hidden, n_head * dim, out.view(n_seq, -1), h, n_seq)
        q.qmv_batched(synth.Q8_0, weights[2], vocab, hidden, h, z, n_seq)
        q.logits_argmax(choose)

    def stored():
        """The cache as it is now, as a plain one."""
        now = ref.Cache(np.random.default_rng(0), kind, 1, n_kv, page, dim)
        now.kv, now.scale = [k.cpu(), v.cpu()], [] if ks is None else [ks.cpu(), vs.cpu()]
        return now

    was = q.qmv_get_pdl()
    q.qmv_set_pdl(pdl)
    try:
        x.normal_()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        score.zero_()
        weights_sum, weights_tol = np.zeros((n_seq, n_kv, slots)), np.zeros((n_seq, n_kv, slots))
        at = [n + 1000 for n in lens]                   # positions run on when the cache shrinks
        evicted = False
        for t in range(6):
            if t == 4:                                  # both caches down to their budget
                budget = 40
                dst = (n_src + np.arange(new_pages, dtype=np.int32)).reshape(2, 3)
                kept = torch.zeros(n_seq, n_kv, budget, dtype=torch.int32, device="cuda")
                so, n_out = torch.zeros(n_seq, n_kv, budget, device="cuda"), torch.zeros(n_seq, dtype=torch.int32, device="cuda")
                before = stored()
                z32 = score.cpu().numpy()
                q.kv_evict(q.EvictArgs(c, score, tab, n_dev, dev(dst), kept, so, n_out, 4, 8, budget))
                want = ref.evict(z32, lens, 4, 8, budget)
                after = stored()
                for s in range(n_seq):
                    m = min(lens[s], budget)
                    for hd in range(n_kv):
                        assert kept[s, hd, :m].tolist() == want[s][hd]
                        for i in range(2):
                            assert np.array_equal(after.rows(i, dst[s], m, hd), before.rows(i, table[s], lens[s], hd)[want[s][hd]])
                    lens[s] = m
                table = np.full_like(table, -1)
                table[:, :3] = dst
                tab.copy_(dev(table))
                score.zero_()
                score[:, :, :budget] = so
                weights_sum, weights_tol = score.double().cpu().numpy(), np.zeros_like(weights_tol)
                evicted = True
            lens = [n + 1 for n in lens]
            at = [n + 1 for n in at]
            x.copy_(torch.from_numpy(rng.standard_normal((n_seq, hidden)).astype(np.float32)))
            n_dev.copy_(torch.tensor(lens, dtype=torch.int32))
            pos.copy_(torch.tensor(at, dtype=torch.int32)[:, None])
            if t % 2:
                graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            now = stored()
            got = qr.double().cpu().numpy()
            rows = y.cpu().numpy().reshape(n_seq, n_head + 2 * n_kv, dim)
            half = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}.get(kind)
            for s in range(n_seq):
                turned = ref.rope(rows[s, :n_head + n_kv], at[s], inv, dim, False)
                assert (np.abs(got[s, 0].reshape(n_head, dim) - turned[:n_head]) <= 2 * ref.U * np.abs(turned[:n_head]) + 1e-10 * np.abs(rows[s]).max()).all()
                for hd in range(n_kv):
                    for i, new in enumerate((turned[n_head + hd], rows[s, n_head + n_kv + hd].astype(np.float64))):
                        kept_value = now.rows(i, table[s], lens[s], hd)[-1]
                        if half:
                            lim = np.abs(new) * (half + 2 * ref.U) + 2.0 ** -25 + 1e-10 * np.abs(rows[s]).max()
                        else:                           # half a step of a block of 32, whose scale is rounded to f16
                            lim = np.repeat(np.abs(new.reshape(-1, 32)).max(1) / 127 * (0.5 + 127 * 2.0 ** -11 + 1e-3), 32)
                        assert (np.abs(kept_value - new) <= lim).all()
            expect, tol, weights_sum, st = ref.attn(now, qr.cpu().numpy(), n_head, table, lens, float(np.float32(dim ** -0.5)), score=weights_sum)
            # a weight below f32's smallest normal value, 2^-126, may be cut to zero (2^x flushes what is subnormal):
            # each head of a group then gives that much less, here where the products make scores tens of units apart
            weights_tol += st + group * 2.0 ** -126
            assert (np.abs(out.double().cpu().numpy() - expect) <= tol).all()
            assert (np.abs(score.double().cpu().numpy() - weights_sum) <= weights_tol).all()
            want_z, want_idx = ref.logits(z.cpu().numpy(), hist.cpu().numpy(), hist_len.cpu().numpy(), params.cpu().numpy())
            assert np.array_equal(adj.cpu().numpy(), want_z) and idx.tolist() == want_idx.tolist()
            hist[:, t] = idx
            hist_len.fill_(t + 1)
        assert evicted
    finally:
        q.qmv_set_pdl(was)

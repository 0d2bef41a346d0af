"""The cache and logits operators where a call's inputs leave the ordinary range: rows of wider tensors, lengths beyond
the table, values that the caches cannot hold; plain 64-bit forms in step_ref.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_decode_superblocks_b200 as q
import step_ref as ref
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

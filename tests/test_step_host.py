"""Argument checks of the cache and logits operators (no GPU needed): every refusal is found on the host
before a device is touched, and the plain forms that the GPU tests compare with hold on cases worked by hand."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import quantized_decode_superblocks_b200 as q
import step_ref as ref

A = 0x10000              # a fake, 256-byte aligned "device" address: never dereferenced on these paths
OK, NULL, FMT, SHAPE, ALIGN, NTOK, CUDA, WS = 0, -1, -2, -3, -4, -5, -7, -9


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def cache(**kw):
    c = q.KvCache.__new__(q.KvCache)
    ctypes.Structure.__init__(c)
    f = dict(type=q.KV_F16, n_kv_head=8, head_dim=64, page_size=16, n_pages=10, page_stride=8 * 16 * 64, head_stride=16 * 64,
             slot_stride=64, k=A, v=A, k_scale=None, v_scale=None)
    f.update(kw)
    for n, x in f.items():
        setattr(c, n, x)
    return c


def filled(cls, base, kw, c):
    a = cls.__new__(cls)
    ctypes.Structure.__init__(a)
    a.cache = c if c is not None else cache()
    for n, x in {**base, **kw}.items():
        setattr(a, n, x)
    return a


def attn(L, c=None, **kw):
    base = dict(q=A, out=2 * A, score=None, q_stride=2048, out_stride=2048, score_stride=0, n_head=32, n_seq=2, n_tok=1, max_pages=4,
                table_stride=4, block_table=A, kv_len=A, scale=0.125, window=0, n_sink=0, workspace=A, workspace_bytes=1 << 40)
    return L.attn_decode(ctypes.byref(filled(q.AttnArgs, base, kw, c)), None)


def append(L, c=None, **kw):
    base = dict(q=A, k_in=A, v_in=A, q_out=2 * A, q_stride=3000, k_stride=3000, v_stride=3000, q_out_stride=2048, n_head=32, n_seq=2,
                n_tok=1, rope_dim=64, rope_style=0, max_pages=4, table_stride=4, block_table=A, kv_len=A, pos=None, inv_freq=A)
    return L.kv_append(ctypes.byref(filled(q.AppendArgs, base, kw, c)), None)


def evict(L, c=None, **kw):
    base = dict(score=A, score_out=2 * A, score_stride=64, score_out_stride=32, n_seq=2, max_pages=4, dst_max_pages=2, keep_first=4,
                keep_last=8, budget=32, table_stride=4, dst_table_stride=2, block_table=A, kv_len=A, dst_table=A, kept=A, len_out=3 * A)
    return L.kv_evict(ctypes.byref(filled(q.EvictArgs, base, kw, c)), None)


def logits(L, **kw):
    a = q.LogitsArgs.__new__(q.LogitsArgs)
    ctypes.Structure.__init__(a)
    base = dict(logits=A, out=A + 4096, logits_stride=1000, out_stride=1000, n_rows=2, vocab=1000, hist=A, hist_len=A, hist_stride=10,
                params=A, bias_ids=A, bias_len=A, bias_vals=A, bias_stride=5, mask=A, mask_stride=32, idx_out=A, workspace=A,
                workspace_bytes=1 << 20)
    for n, x in {**base, **kw}.items():
        setattr(a, n, x)
    return L.logits_argmax(ctypes.byref(a), None)


def good(L, call, **kw):
    """The call passes its checks: the launch that follows is made to fail on the host."""
    L.qmv_debug_fail_next_launches(1)
    rc = call(L, **kw)
    L.qmv_debug_fail_next_launches(0)
    return rc == CUDA


CALLS = [attn, append, evict]


@pytest.mark.parametrize("call", CALLS)
def test_cache_checks(L, call):
    assert good(L, call)
    for name in ("k", "v"):
        assert call(L, cache(**{name: None})) == NULL
        assert call(L, cache(**{name: A + 8})) == ALIGN
    assert call(L, cache(type=3)) == FMT and call(L, cache(type=-1)) == FMT
    for d in (0, 8, 24, 72, 272, -64):
        assert call(L, cache(head_dim=d)) == SHAPE
    for name in ("n_kv_head", "page_size", "n_pages"):
        assert call(L, cache(**{name: 0})) == SHAPE and call(L, cache(**{name: -1})) == SHAPE
    assert call(L, cache(n_kv_head=1025)) == SHAPE and call(L, cache(n_pages=2 ** 31)) == SHAPE
    for name in ("page_stride", "head_stride", "slot_stride"):
        assert call(L, cache(**{name: 0})) == SHAPE and call(L, cache(**{name: -64})) == SHAPE
        assert call(L, cache(**{name: 1028})) == ALIGN and call(L, cache(**{name: 2 ** 62})) == SHAPE
    q8 = dict(type=q.KV_Q8_0, k_scale=A, v_scale=A)
    assert good(L, call, c=cache(**q8))
    assert call(L, cache(**{**q8, "k_scale": None})) == NULL and call(L, cache(**{**q8, "v_scale": None})) == NULL
    assert call(L, cache(**{**q8, "v_scale": A + 2})) == ALIGN
    assert call(L, cache(**q8, head_dim=96)) == SHAPE and call(L, cache(**q8, head_stride=1056)) == ALIGN


@pytest.mark.parametrize("call", CALLS)
def test_table_checks(L, call):
    assert call(L, block_table=None) == NULL and call(L, kv_len=None) == NULL
    assert call(L, block_table=A + 2) == ALIGN and call(L, kv_len=A + 1) == ALIGN
    assert call(L, n_seq=0) == SHAPE and call(L, n_seq=1025) == SHAPE
    assert call(L, max_pages=0) == SHAPE and call(L, table_stride=3) == SHAPE and call(L, table_stride=-4) == SHAPE
    assert call(L, max_pages=2 ** 28, table_stride=2 ** 28) == SHAPE       # slot numbers are 32-bit


def test_attn_checks(L):
    for name in ("q", "out", "workspace"):
        assert attn(L, **{name: None}) == NULL
    assert attn(L, n_tok=0) == NTOK and attn(L, n_tok=9) == NTOK
    assert attn(L, n_head=0) == SHAPE and attn(L, n_head=12) == SHAPE and attn(L, n_head=8200) == SHAPE
    assert attn(L, q_stride=2044) == SHAPE and attn(L, out_stride=2047) == SHAPE and attn(L, q_stride=2050) == ALIGN
    assert attn(L, q=A + 8) == ALIGN and attn(L, out=A + 2) == ALIGN and attn(L, workspace=A + 128) == ALIGN
    assert attn(L, score=A) == SHAPE and attn(L, score=A + 2, score_stride=64) == ALIGN and good(L, attn, score=A, score_stride=64)
    assert attn(L, window=-1) == SHAPE and attn(L, n_sink=-1) == SHAPE
    assert attn(L, scale=float("nan")) == SHAPE and attn(L, scale=float("inf")) == SHAPE
    need = q.attn_ws_bytes(cache(), 32, 2, 1, 4)
    assert attn(L, workspace_bytes=need - 1) == WS and good(L, attn, workspace_bytes=need)
    more = q.attn_ws_bytes(cache(), 32, 2, 1, 4, True)
    assert more > need and attn(L, score=A, score_stride=64, workspace_bytes=need) == WS
    assert q.attn_ws_bytes(cache(), 31, 2, 1, 4) == 0 and q.attn_ws_bytes(cache(), 32, 2, 9, 4) == 0
    assert q.attn_ws_bytes(cache(type=7), 32, 2, 1, 4) == 0
    assert L.attn_decode(None, None) == NULL
    assert "workspace" in q.strerror(WS)
    assert attn(L, out=A) == SHAPE                      # other CTAs may still read the queries


def test_outputs_that_share_memory_with_inputs_are_refused(L):
    assert append(L, q_out=A, q_stride=3000, q_out_stride=2048) == SHAPE and good(L, append, q_out=A, q_stride=2048, q_out_stride=2048)
    rows = 2 * 8                                        # scores of 64 floats a row, the last one whole
    assert evict(L, score_out=A) == SHAPE and evict(L, score_out=A + rows * 64 * 4 - 4) == SHAPE
    assert good(L, evict, score_out=A + rows * 64 * 4)
    assert evict(L, score=2 * A + rows * 32 * 4 - 4) == SHAPE and good(L, evict, score=2 * A + rows * 32 * 4)
    assert evict(L, len_out=A) == SHAPE and evict(L, len_out=A + 4) == SHAPE and good(L, evict, len_out=A + 8)
    assert evict(L, kv_len=3 * A + 4) == SHAPE and good(L, evict, kv_len=3 * A + 8)


def test_append_checks(L):
    for name in ("k_in", "v_in", "inv_freq"):
        assert append(L, **{name: None}) == NULL
    assert append(L, q=None) == NULL and append(L, q_out=None) == NULL and good(L, append, q=None, q_out=None, n_head=0)
    assert good(L, append, inv_freq=None, rope_dim=0)
    assert append(L, n_tok=0) == NTOK and append(L, n_tok=9) == NTOK
    for r in (-2, 3, 66):
        assert append(L, rope_dim=r) == SHAPE
    assert append(L, rope_style=2) == SHAPE and append(L, n_head=0) == SHAPE
    for name in ("q_stride", "k_stride", "v_stride", "q_out_stride"):
        assert append(L, **{name: 511}) == SHAPE
    for name in ("q", "k_in", "v_in", "q_out", "pos", "inv_freq"):
        assert append(L, **{name: A + 2}) == ALIGN
    assert L.kv_append(None, None) == NULL


def test_evict_checks(L):
    for name in ("score", "score_out", "dst_table", "kept", "len_out"):
        assert evict(L, **{name: None}) == NULL and evict(L, **{name: A + 2}) == ALIGN
    assert evict(L, keep_first=-1) == SHAPE and evict(L, keep_last=-1) == SHAPE and evict(L, keep_first=25) == SHAPE
    assert evict(L, budget=0) == SHAPE and evict(L, budget=33) == SHAPE and evict(L, score_out_stride=31) == SHAPE
    assert evict(L, dst_max_pages=0) == SHAPE and evict(L, dst_table_stride=1) == SHAPE and evict(L, score_stride=0) == SHAPE
    assert good(L, evict, keep_first=24) and L.kv_evict(None, None) == NULL


def test_logits_checks(L):
    assert good(L, logits)
    assert good(L, logits, hist=None, bias_ids=None, mask=None, out=None)
    for name in ("logits", "idx_out", "workspace", "hist_len", "params", "bias_len", "bias_vals"):
        assert logits(L, **{name: None}) == NULL
    assert logits(L, n_rows=0) == SHAPE and logits(L, n_rows=65536) == SHAPE and logits(L, vocab=0) == SHAPE
    assert logits(L, logits_stride=999) == SHAPE and logits(L, out_stride=999) == SHAPE and logits(L, mask_stride=31) == SHAPE
    assert logits(L, out=A, out_stride=1001) == SHAPE and good(L, logits, out=A)
    assert logits(L, hist_stride=-1) == SHAPE and logits(L, bias_stride=-1) == SHAPE
    for name in ("logits", "out", "hist", "hist_len", "params", "bias_ids", "bias_len", "bias_vals", "mask", "idx_out"):
        assert logits(L, **{name: A + 2}) == ALIGN
    assert logits(L, workspace=A + 4) == ALIGN and logits(L, workspace_bytes=31) == WS and good(L, logits, workspace_bytes=32)
    assert q.logits_ws_bytes(0) == 0 and L.logits_argmax(None, None) == NULL


def test_argument_objects_check_their_tensors():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        q.KvCache(q.KV_F16, k, k)
    with pytest.raises(ValueError, match="expected bfloat16"):
        q.KvCache(q.KV_BF16, k, k)
    with pytest.raises(ValueError, match="dimensions"):
        q.KvCache(q.KV_F16, k[0], k[0])
    with pytest.raises(ValueError, match="unknown cache type"):
        q.KvCache(9, k, k)


# ------------------------------------------------------------------- the plain forms on cases worked by hand --
def test_plain_attention_by_hand():
    c = ref.Cache(np.random.default_rng(0), "f16", 2, 1, 2, 16)
    for i in range(2):
        c.kv[i][:] = 0
    c.kv[1][1, 0, :, 0] = 1.0                            # page 1 holds slots 0 and 1: values 1 and 3
    c.kv[1][1, 0, 1, 0] = 3.0
    c.kv[1][0, 0, 0, 0] = 8.0                            # page 0 holds slot 2
    x = np.zeros((1, 2, 16), np.float32)
    out, tol, score, _ = ref.attn(c, x, 1, [[1, 0]], [3], 1.0, score=np.full((1, 1, 4), 5.0))
    assert out[0, 0, 0] == 2.0 and abs(out[0, 1, 0] - 4.0) < 1e-15 and (tol[0, :, 0] > 0).all()
    assert np.allclose(score[0, 0], [5 + 1 / 2 + 1 / 3, 1 / 2 + 1 / 3, 1 / 3, 5])    # the newest two are set
    out, _, _, _ = ref.attn(c, x, 1, [[1, 0]], [3], 1.0, window=1)
    assert out[0, 0, 0] == 3.0 and out[0, 1, 0] == 8.0
    out, _, _, _ = ref.attn(c, x, 1, [[1, 0]], [3], 1.0, window=1, n_sink=1)
    assert out[0, 0, 0] == 2.0 and out[0, 1, 0] == 4.5
    out, _, _, _ = ref.attn(c, x, 1, [[1, 0]], [1], 1.0)
    assert out[0, 0, 0] == 0.0 and out[0, 1, 0] == 1.0   # the first query sits before the sequence


def test_plain_rope_evict_and_logits_by_hand():
    y = ref.rope(np.array([[1.0, 0.0, 0.0, 2.0]]), 1, np.array([np.pi / 2, np.pi], np.float64), 4, True)
    assert np.allclose(y, [[0, 1, 0, -2]])
    y = ref.rope(np.array([[1.0, 0.0, 0.0, 2.0]]), 1, np.array([np.pi / 2, np.pi], np.float64), 4, False)
    assert np.allclose(y, [[0, 0, 1, -2]])
    s = np.array([[[9, 1, 2, 2, np.nan, 5, 0, 0]]], np.float32)
    assert ref.evict(s, [8], 1, 1, 4) == [[[0, 2, 5, 7]]]
    assert ref.evict(s, [8], 0, 0, 7) == [[[0, 1, 2, 3, 5, 6, 7]]] and ref.evict(s, [3], 1, 1, 4) == [[[0, 1, 2]]]
    z, i = ref.logits(np.array([[2.0, -2.0, 1.0]]), np.array([[0, 1, 0, 9]]), [4], [[2.0, 0.25, 0.5]], np.array([[2, 2]]), np.array([[5.0, 1.5]]), [2])
    assert z.tolist() == [[0.0, -4.75, 2.5]] and i.tolist() == [2]
    z, i = ref.logits(np.array([[2.0, -2.0, 1.0]]), mask=np.array([[0]]))
    assert (z == -np.inf).all() and i.tolist() == [-1]

"""Calls at the edges of what the cache and logits operators take, as far as they show without a GPU: what an
argument object lets a call touch, and which mistakes the tests' bounds tell apart."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import quantized_decode_superblocks_b200 as q
import step_ref as ref
import step_tight as tight
import test_step_host as host
from test_step_host import A, SHAPE, L, attn, evict, good  # noqa: F401


class Fake:
    """A CPU tensor that says it lies on cuda:0: for argument objects that no call gets."""

    def __init__(self, t):
        self.t, self.device, self.dtype, self.shape = t, torch.device("cuda", 0), t.dtype, t.shape

    def dim(self):
        return self.t.dim()

    def stride(self, *i):
        return self.t.stride(*i)

    def data_ptr(self):
        return self.t.data_ptr()

    def numel(self):
        return self.t.numel()

    def is_contiguous(self):
        return self.t.is_contiguous()


def zeros(*shape, dtype=torch.float32):
    return Fake(torch.zeros(*shape, dtype=dtype))


def small_cache():
    return q.KvCache(q.KV_F16, zeros(80, 2, 16, 64, dtype=torch.float16), zeros(80, 2, 16, 64, dtype=torch.float16))


def attn_args(score):
    return q.AttnArgs(small_cache(), zeros(2, 1, 512), zeros(2, 1, 512), zeros(2, 40, dtype=torch.int32), zeros(2, dtype=torch.int32),
                      zeros(1 << 22, dtype=torch.uint8), 0.125, score=score)


def evict_args(score):
    return q.EvictArgs(small_cache(), score, zeros(2, 40, dtype=torch.int32), zeros(2, dtype=torch.int32), zeros(2, 2, dtype=torch.int32),
                       zeros(2, 2, 32, dtype=torch.int32), zeros(2, 2, 32), zeros(2, dtype=torch.int32), 4, 8, 32)


@pytest.mark.parametrize("make", [attn_args, evict_args])
@pytest.mark.parametrize("lo,hi", [(0, 1000), (900, 1000), (0, 100), (999, 1000)])
def test_rows_of_a_wider_score_end_where_the_tensor_ends(make, lo, hi):
    """640 slots a sequence: whatever the lengths are, no entry behind a row's last one is reached."""
    whole = torch.zeros(2, 2, 1000)
    args = make(Fake(whole[:, :, lo:hi]))
    reach = min(640, getattr(args, "score_slots", 0) or args.score_stride)
    assert args.score_stride == 1000 and reach == min(640, hi - lo)
    assert args.score + (3 * 1000 + reach) * 4 <= whole.data_ptr() + whole.numel() * 4


@pytest.mark.parametrize("make", [attn_args, evict_args])
def test_a_score_without_entries_is_refused(make):
    with pytest.raises(ValueError, match="entry a row"):
        make(Fake(torch.zeros(2, 2, 0)))


def test_score_rows_may_not_reach_into_each_other(L):  # noqa: F811
    for call, kw in ((attn, dict(score=A)), (evict, {})):
        assert good(L, call, score_stride=64, score_slots=64, **kw) and good(L, call, score_stride=64, score_slots=1, **kw)
        assert good(L, call, score_stride=64, score_slots=0, **kw)
        assert call(L, score_stride=64, score_slots=65, **kw) == SHAPE and call(L, score_stride=64, score_slots=-1, **kw) == SHAPE
    # outputs may lie between the rows' entries' end and the buffer's
    end = A + (15 * 64 + 20) * 4
    assert evict(L, score_slots=20, score_out=end - 4) == SHAPE and good(L, evict, score_slots=20, score_out=end)


def test_attn_steps_leave_room_for_padding(L):  # noqa: F811
    """Step numbers are 32-bit; a CTA's share may grow by an eighth and one to end with a sequence."""
    def padded(steps, ctas):
        share = -(-steps // ctas)
        return (share + share // 8 + 1) * ctas
    assert padded(2 ** 31 - 1, 444) >= 2 ** 31 and padded(2 ** 30, 444) < 2 ** 31
    c = host.cache(n_kv_head=1024, head_dim=16, page_stride=1024 * 16 * 16, head_stride=256, slot_stride=16)
    assert q.attn_ws_bytes(c, 1024, 1, 1, 2 ** 22) == 0        # 1024 heads, 2^26 slots, 64 a step
    assert q.attn_ws_bytes(c, 1024, 1, 1, 2 ** 22 - 2 ** 12) > 0
    kw = dict(c=c, n_head=1024, n_seq=1, q_stride=16384, out_stride=16384)
    assert attn(L, max_pages=2 ** 22, table_stride=2 ** 22, **kw) == SHAPE
    assert good(L, attn, max_pages=2 ** 21, table_stride=2 ** 21, **kw)


# --------------------------------------------------------------- the bounds that the GPU tests hold the kernels to --
@pytest.mark.parametrize("kind,dim", [("f16", 16), ("f16", 128), ("bf16", 64), ("bf16", 256), ("q8", 64), ("q8", 256)])
@pytest.mark.parametrize("slip", ["q", "weights"])
def test_a_lost_part_of_queries_or_weights_breaks_the_bound(kind, dim, slip):
    rng = np.random.default_rng(dim)
    cache, table, lens, x = tight.two_slots(rng, kind, dim, 50, 3)
    want, tol = tight.attn(cache, x, table, lens, 1.0)
    wrong, _ = tight.attn(cache, x, table, lens, 1.0, slip)
    beyond = np.abs(wrong - want) > 2 * tol
    # f16 parts: 2^-12 against some 40 roundings of 2^-24; the third bf16 part: 2^-16 against some 20
    assert beyond.mean() > (0.2 if kind == "bf16" else 0.7)


@pytest.mark.parametrize("kind", ["f16", "q8"])
def test_a_long_tail_cut_at_the_second_parts_last_bit_breaks_the_bound(kind):
    cache, table, lens, x = tight.long_tail(kind, 64, 700)
    want, tol = tight.attn(cache, x, table, lens, 1.0, depth=100)
    p = 2.0 ** 9 * np.exp(np.float64(x[0, 0, 3]))
    hi = tight.high_part(p, "f16")
    kept = (hi + tight.high_part(p - hi, "f16")) / p
    assert (np.abs(want * kept - want) > 5 * tol).all()
    scaled = (hi + tight.high_part(p - hi, "f16", 2048)) / p
    assert (np.abs(want * scaled - want) < 0.01 * tol).all()


def test_plain_one_hot_attention_agrees_with_the_general_form():
    for kind in ("f16", "bf16", "q8"):
        rng = np.random.default_rng(4)
        cache, table, lens, x = tight.two_slots(rng, kind, 64, 6, 2)
        a, small = tight.attn(cache, x, table, lens, 1.0)
        b, large, _, _ = ref.attn(cache, x, 2, table, lens, 1.0)
        assert np.abs(a - b).max() < 1e-14 and (small <= large + 1e-30).all()

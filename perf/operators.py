"""The decode step's operators between and after the weight products, with their sizes.

  kv_append      rotary embedding of the new tokens' q and k; k and v written into a paged key-value cache
  attn_decode    attention of a sequence's newest 1-8 tokens over that cache: grouped heads, a sliding window
                 with first tokens that stay visible, and the weights accumulated per slot where asked
  kv_evict       a smaller cache per sequence: the first, the last and the highest-scored slots of every kv head
  logits_argmax  penalties for repeated tokens, biases and a grammar mask on logits, and the greedy choice

``run`` computes each in plain torch operations, or through the framework where ``own`` is true.  Caches are pools of
pages indexed by a block table; activations are f32 as everywhere in the framework; caches hold f16, bf16 or 8-bit
blocks of 32 values with an f16 scale ("q8").
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "q8": torch.int8}


# --------------------------------------------------------------------------------------------------- the cases --
def _append(name, **kw):
    c = dict(op="kv_append", type="f16", n_head=32, n_kv_head=8, head_dim=64, page=16, layout="head", n_seq=1, n_tok=1,
             len_min=100, len_max=100, rope_dim=64, style="halves", pos=5000)
    c.update(kw)
    return dict(c, name=name) if name else c


def _attn(name, **kw):
    c = dict(op="attn_decode", type="f16", n_head=32, n_kv_head=8, head_dim=64, page=16, layout="head", n_seq=1, n_tok=1,
             len_min=1000, len_max=1000, window=0, n_sink=0, score=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def _evict(name, **kw):
    c = dict(op="kv_evict", type="f16", n_kv_head=8, head_dim=64, page=16, layout="head", n_seq=1, len_min=4352,
             len_max=4352, first=4, last=256, budget=4096)
    c.update(kw)
    return dict(c, name=name) if name else c


def _logits(name, **kw):
    c = dict(op="logits_argmax", vocab=128000, n_rows=1, hist=512, bias=0, mask=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token: the 32 query / 8 kv heads of 64 of the framework's own fused QKV projection
        _append("append_step"),
        # a served batch with speculative tokens, far positions, part of each head rotated in neighbouring pairs
        _append("append_batch", type="bf16", head_dim=128, layout="token", n_seq=64, n_tok=4, len_min=9, len_max=200,
                rope_dim=96, style="pairs", pos=120000),
        # one user's next token over a short conversation: latency
        _attn("attn_step"),
        # the same over a long document
        _attn("attn_long", page=64, len_min=131071, len_max=131071),
        # a served batch of ragged conversations
        _attn("attn_batch", type="bf16", head_dim=128, layout="token", n_seq=32, len_min=1001, len_max=16384),
        # eight speculative tokens checked at once, 8-bit cache, a sliding window with four first tokens kept visible
        _attn("attn_verify", type="q8", head_dim=128, page=32, n_seq=4, n_tok=8, len_min=3000, len_max=8191, window=4096,
              n_sink=4),
        # the weights accumulated for eviction, wider groups of heads
        _attn("attn_score", type="bf16", n_head=40, head_dim=128, page=32, n_seq=4, len_min=6001, len_max=12003,
              score=True),
        # one user's cache brought back to its budget
        _evict("evict_step"),
        # a batch of long caches cut to a quarter
        _evict("evict_batch", type="bf16", head_dim=128, layout="token", n_seq=16, len_min=8000, len_max=16384, last=512),
        # one user's next token: penalties only, the framework's vocabulary
        _logits("logits_step"),
        # eight speculative tokens under a grammar, with biases
        _logits("logits_verify", n_rows=8, hist=4096, bias=300, mask=True),
        # a served batch, an odd vocabulary
        _logits("logits_batch", vocab=151937, n_rows=128, hist=2000, bias=17, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["kv_append", "attn_decode", "attn_decode", "attn_decode", "kv_evict", "logits_argmax"])
    if op == "logits_argmax":
        while True:
            c = _logits("", vocab=_log(rng, 100, 260000), n_rows=_log(rng, 1, 256), hist=rng.choice([0, _log(rng, 1, 8192)]),
                        bias=rng.choice([0, _log(rng, 1, 1000)]), mask=rng.random() < 0.5)
            if c["vocab"] * c["n_rows"] <= 151937 * 128:
                return c
    kind = rng.choice(["f16", "bf16", "q8"])
    dim = rng.choice([64, 128, 192, 256] if kind == "q8" else [32, 64, 80, 96, 112, 128, 256])
    n_kv = rng.choice([1, 2, 3, 4, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8, 16])
    common = dict(type=kind, n_kv_head=n_kv, head_dim=dim, page=rng.choice([1, 7, 16, 16, 32, 48, 64, 128, 256]),
                  layout=rng.choice(["head", "token"]))
    while True:
        n_seq, longest = _log(rng, 1, 64), _log(rng, 1, 65536)
        least = rng.randint(1, longest)
        if op == "kv_append":
            longest = min(longest, 1 + longest % 300)
            least = min(least, longest)
            rope = rng.choice([0, dim, dim // 4 * 2])
            c = _append("", n_head=n_kv * group, n_seq=n_seq, n_tok=rng.randint(1, 8), len_min=least, len_max=longest,
                        rope_dim=rope, style=rng.choice(["halves", "pairs"]), pos=_log(rng, 1, 1000000), **common)
            if n_seq * longest * n_kv * dim <= 20_000_000:
                return c
        elif op == "attn_decode":
            n_tok = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
            c = _attn("", n_head=n_kv * group, n_seq=n_seq, n_tok=n_tok, len_min=least, len_max=longest,
                      window=rng.choice([0, 0, _log(rng, 1, longest)]), n_sink=rng.choice([0, 0, 4, rng.randint(1, 100)]),
                      score=rng.random() < 0.25, **common)
            if n_seq * longest * n_kv * dim <= 100_000_000 and n_seq * longest * n_kv * group * n_tok <= 100_000_000:
                return c
        else:
            budget = _log(rng, 1, longest)
            first = rng.choice([0, min(4, budget)])
            c = _evict("", n_seq=n_seq, len_min=least, len_max=longest, first=first,
                       last=rng.randint(0, budget - first), budget=budget, **common)
            if n_seq * longest * n_kv * dim <= 100_000_000:
                return c


# -------------------------------------------------------------------------------------------------- the inputs --
def _lens(case):
    """Ragged lengths from len_min to len_max, spread over the sequences; the longest is always there."""
    n, lo, hi = case["n_seq"], case["len_min"], case["len_max"]
    return [hi - (hi - lo) * ((i * 7) % n) // n for i in range(n)]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g, dtype=dtype)


def _quantise(x):
    """Blocks of 32 along the last dimension: an f16 scale amax / 127 and whole values of at most 127."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    d = (b.abs().amax(-1) / 127).clamp(max=65504.0).half()
    df = d.float()[..., None]
    q = torch.where(df > 0, torch.round(b / df), torch.zeros_like(b)).clamp(-127, 127)
    return q.reshape(x.shape).to(torch.int8), d


def _pool(case, g, n_pages, empty=False):
    """One pool [n_pages, n_kv_head, page, head_dim] (for the "token" layout a page's tokens come before its heads) and,
    for q8, its scales [n_pages, n_kv_head, page, head_dim / 32], laid out alike."""
    h, p, d = case["n_kv_head"], case["page"], case["head_dim"]
    shape = (n_pages, h, p, d) if case["layout"] == "head" else (n_pages, p, h, d)
    scale = None
    if case["type"] == "q8":
        pool = torch.zeros(shape, dtype=torch.int8, device=DEV)
        scale = torch.zeros(*shape[:-1], d // 32, dtype=torch.float16, device=DEV)
        if not empty:
            step = max(1, (1 << 26) // (h * p * d))
            for i in range(0, n_pages, step):
                pool[i:i + step], scale[i:i + step] = _quantise(_randn(g, min(step, n_pages - i), *shape[1:]))
    elif empty:
        pool = torch.zeros(shape, dtype=TYPES[case["type"]], device=DEV)
    else:
        pool = _randn(g, *shape, dtype=TYPES[case["type"]])
    if case["layout"] != "head":
        pool = pool.transpose(1, 2)
        scale = scale.transpose(1, 2) if scale is not None else None
    return pool, scale


def _table(case, g, lens, first=0):
    """A block table with every sequence's pages scattered over the pool, and how many pages it names."""
    most = max(1, max(-(-n // case["page"]) for n in lens))
    total = case["n_seq"] * most
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32) + first
    return order.reshape(case["n_seq"], most).contiguous(), total


def _scores(g, n_seq, n_kv, most):
    """Accumulated weights: a few heavy slots, many light ones, some that never got any."""
    x = torch.exp(2.0 * _randn(g, n_seq, n_kv, most) - 6.0)
    return torch.where(_randn(g, n_seq, n_kv, most) > 2.0, torch.zeros_like(x), x)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "logits_argmax":
        n, v = case["n_rows"], case["vocab"]
        s["logits"] = 3.0 * _randn(g, n, v)
        # text repeats itself: low ids more often than high ones
        u = torch.rand(n, max(1, case["hist"]), device=DEV, generator=g)
        s["hist"] = (u * u * u * v).to(torch.int32).clamp(max=v - 1)
        cut = torch.rand(n, device=DEV, generator=g)
        s["hist_len"] = (case["hist"] * (0.5 + 0.5 * cut)).round().to(torch.int32)
        pen = torch.rand(n, 3, device=DEV, generator=g)
        s["params"] = torch.stack([1.0 + 0.3 * pen[:, 0], 0.5 * pen[:, 1], 0.5 * pen[:, 2]], 1).contiguous()
        if case["bias"]:
            s["bias_ids"] = torch.randint(0, v, (n, case["bias"]), device=DEV, generator=g, dtype=torch.int32)
            s["bias_vals"] = 2.0 * _randn(g, n, case["bias"])
            s["bias_len"] = torch.full((n,), case["bias"], dtype=torch.int32, device=DEV)
        if case["mask"]:
            # a grammar lets a small part of the vocabulary through
            w = [torch.randint(-2**31, 2**31, (n, -(-v // 32)), device=DEV, generator=g, dtype=torch.int64) for _ in range(3)]
            s["mask"] = (w[0] & w[1] & w[2]).to(torch.int32)
        s["out"] = torch.empty(n, v, device=DEV)
        s["idx"] = torch.empty(n, dtype=torch.int32, device=DEV)
        return s

    lens = _lens(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["table"], n_pages = _table(case, g, lens)
    more = 0
    if op == "kv_evict":
        s["dst_table"], more = _table(case, g, [min(n, case["budget"]) for n in lens], n_pages)
    s["n_src"] = n_pages
    s["k"], s["k_scale"] = _pool(case, g, n_pages + more, op == "kv_append")
    s["v"], s["v_scale"] = _pool(case, g, n_pages + more, op == "kv_append")
    d, h = case["head_dim"], case["n_kv_head"]
    if op == "kv_evict":
        s["score"] = _scores(g, case["n_seq"], h, max(lens))
        s["kept"] = torch.zeros(case["n_seq"], h, case["budget"], dtype=torch.int32, device=DEV)
        s["score_out"] = torch.zeros(case["n_seq"], h, case["budget"], device=DEV)
        s["len_out"] = torch.zeros(case["n_seq"], dtype=torch.int32, device=DEV)
        return s
    n_tok, nh = case["n_tok"], case["n_head"]
    # the fused projection's output: a token's q, k and v next to each other
    s["qkv"] = _randn(g, case["n_seq"], n_tok, (nh + 2 * h) * d)
    if op == "kv_append":
        s["pos"] = (case["pos"] + s["lens"][:, None] - n_tok + torch.arange(n_tok, device=DEV)).clamp(min=0).to(torch.int32)
        if case["rope_dim"]:
            i = torch.arange(case["rope_dim"] // 2, device=DEV, dtype=torch.float64)
            s["inv_freq"] = (10000.0 ** (-2.0 * i / case["rope_dim"])).float()
        s["q_out"] = torch.empty(case["n_seq"], n_tok, nh * d, device=DEV)
    else:
        s["q"] = 1.5 * s["qkv"][..., :nh * d].contiguous()
        del s["qkv"]
        s["out"] = torch.empty(case["n_seq"], n_tok, nh * d, device=DEV)
        if case["score"]:
            s["score"] = _scores(g, case["n_seq"], h, max(lens))
    return s


# ------------------------------------------------------------------------------------------------- plain forms --
def _places(s, table, n):
    """Page, and place in the page, of slots 0..n-1 of every sequence (slots past its table's end: its last page)."""
    p = s["case"]["page"]
    slot = torch.arange(n, device=DEV)
    return table.long()[:, (slot // p).clamp(max=table.shape[1] - 1)], (slot % p)[None].expand(table.shape[0], n)


def _read(s, which, n):
    """[n_seq, n, n_kv_head, head_dim] in f32."""
    page, off = _places(s, s["table"], n)
    x = s[which][page, :, off].float()
    if s["case"]["type"] == "q8":
        x = (x.unflatten(-1, (-1, 32)) * s[which + "_scale"][page, :, off].float()[..., None]).flatten(-2)
    return x


def _plain_attn(s):
    case = s["case"]
    b, t, h, d = case["n_seq"], case["n_tok"], case["n_kv_head"], case["head_dim"]
    n = case["len_max"]
    q = s["q"].reshape(b, t, h, -1, d)
    score = torch.einsum("bthgd,bjhd->bhgtj", q, _read(s, "k", n)) * d ** -0.5
    slot = torch.arange(n, device=DEV)
    at = s["lens"][:, None] - t + torch.arange(t, device=DEV)                      # [b, t]
    seen = slot <= at[..., None]
    if case["window"]:
        seen = seen & ((slot > at[..., None] - case["window"]) | (slot < case["n_sink"]))
    seen = seen[:, None, None]                                                     # [b, 1, 1, t, j]
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))))
    total = w.sum(-1, keepdim=True)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    v = _read(s, "v", n)
    s["out"].copy_(torch.einsum("bhgtj,bjhd->bthgd", w, v).reshape(s["out"].shape))
    if not case["score"]:
        return s["out"]
    given = w.sum((2, 3))                                                          # [b, h, j]
    newest = (slot >= s["lens"][:, None] - t)[:, None]
    inside = (slot < s["lens"][:, None])[:, None]
    s["score"].copy_(torch.where(inside, torch.where(newest, given, s["score"] + given), s["score"]))
    return s["out"], s["score"]


def _plain_append(s):
    case = s["case"]
    b, t, h, d, nh = case["n_seq"], case["n_tok"], case["n_kv_head"], case["head_dim"], case["n_head"]
    x = s["qkv"].reshape(b, t, nh + 2 * h, d)
    qk, v = x[:, :, :nh + h].double(), x[:, :, nh + h:]
    if case["rope_dim"]:
        r = case["rope_dim"]
        angle = s["pos"].double()[..., None] * s["inv_freq"].double()
        c, sn = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
        rot = qk[..., :r].reshape(b, t, nh + h, 2, r // 2).transpose(-1, -2) if case["style"] == "halves" else \
            qk[..., :r].reshape(b, t, nh + h, r // 2, 2)
        turned = torch.stack([rot[..., 0] * c - rot[..., 1] * sn, rot[..., 0] * sn + rot[..., 1] * c], -1)
        if case["style"] == "halves":
            turned = turned.transpose(-1, -2)
        qk = torch.cat([turned.reshape(b, t, nh + h, r), qk[..., r:]], -1)
    qk = qk.float()
    s["q_out"].copy_(qk[:, :, :nh].reshape(s["q_out"].shape))
    slot = (s["lens"][:, None] - t + torch.arange(t, device=DEV)).long()           # [b, t]
    real = slot >= 0
    page = s["table"].long().gather(1, (slot.clamp(min=0) // case["page"]))[real]
    off = (slot.clamp(min=0) % case["page"])[real]
    for which, new in (("k", qk[:, :, nh:]), ("v", v)):
        new = new[real]
        if case["type"] == "q8":
            new, scale = _quantise(new)
            s[which + "_scale"][page, :, off] = scale
        s[which][page, :, off] = new.to(s[which].dtype)


def _cache_values(s, first=0):
    """The cache's pages from `first` on, as the values that they stand for."""
    got = []
    for which in ("k", "v"):
        x = s[which][first:]
        if s["case"]["type"] == "q8":
            x = (x.float().unflatten(-1, (-1, 32)) * s[which + "_scale"][first:].float()[..., None]).flatten(-2)
        got.append(x)
    return got


def _plain_evict(s):
    case = s["case"]
    n, budget = case["len_max"], case["budget"]
    lens = s["lens"][:, None, None]
    slot = torch.arange(n, device=DEV)
    rank = torch.where((slot < case["first"]) | (slot >= lens - case["last"]), math.inf, s["score"])
    rank = torch.where(slot < lens, rank, -math.inf)
    m = min(n, budget)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :m]  # ties: the lower slot first
    best = torch.where(torch.gather(rank, -1, best) > -math.inf, best, n)
    keep = torch.sort(best, dim=-1).values                                         # [b, h, m], n where there is none
    real = keep < n
    s["kept"][..., :m] = torch.where(real, keep.int(), s["kept"][..., :m])
    at = keep.clamp(max=n - 1)
    s["score_out"][..., :m] = torch.where(real, torch.gather(s["score"], -1, at), s["score_out"][..., :m])
    s["len_out"].copy_(s["lens"].clamp(max=budget))
    p = case["page"]
    b_at, h_at, i_at = torch.nonzero(real, as_tuple=True)
    src = keep[real]
    from_page, from_off = s["table"].long()[b_at, src // p], src % p
    to_page, to_off = s["dst_table"].long()[b_at, i_at // p], i_at % p
    for which in ("k", "v", "k_scale", "v_scale"):
        if s[which] is not None:
            s[which][to_page, h_at, to_off] = s[which][from_page, h_at, from_off]


def _plain_logits(s):
    case = s["case"]
    n, v = case["n_rows"], case["vocab"]
    z = s["logits"]
    here = torch.arange(s["hist"].shape[1], device=DEV) < s["hist_len"][:, None]
    count = torch.zeros(n, v, device=DEV).scatter_add_(1, s["hist"].long(), here.float())
    rep, freq, pres = (s["params"][:, i:i + 1] for i in range(3))
    pushed = torch.where(z > 0, z / rep, z * rep) - (freq * count + pres)
    z = torch.where(count > 0, pushed, z)
    if case["bias"]:
        # of several entries for one token the last one counts
        entry = torch.arange(case["bias"], device=DEV).expand(n, -1)
        last = torch.full((n, v), -1, device=DEV).scatter_reduce_(1, s["bias_ids"].long(), entry, "amax")
        z = z + torch.where(last >= 0, torch.gather(s["bias_vals"], 1, last.clamp(min=0)), torch.zeros_like(z))
    if case["mask"]:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        z = torch.where(bits.reshape(n, -1)[:, :v] != 0, z, -math.inf)
    s["out"].copy_(z)
    top = z.amax(1, keepdim=True)
    first = torch.where(z == top, torch.arange(v, device=DEV), v).amin(1)
    s["idx"].copy_(torch.where(top[:, 0] > -math.inf, first, -1))
    return s["out"], s["idx"]


# ----------------------------------------------------------------------------------------- through the framework --
def _call(s):
    """The call's arguments as a program lays them down once for its buffers, and its workspace."""
    import quantized_decode_superblocks_b200 as qd
    case, op = s["case"], s["case"]["op"]
    if op == "logits_argmax":
        ws = torch.zeros(qd.logits_ws_bytes(case["n_rows"]), dtype=torch.uint8, device=DEV)
        return qd.logits_argmax, qd.LogitsArgs(s["logits"], s["hist"], s["hist_len"], s["params"], s["out"], s["idx"], ws,
                                               bias_ids=s.get("bias_ids"), bias_vals=s.get("bias_vals"),
                                               bias_len=s.get("bias_len"), mask=s.get("mask"))
    kind = {"f16": qd.KV_F16, "bf16": qd.KV_BF16, "q8": qd.KV_Q8_0}[case["type"]]
    cache = qd.KvCache(kind, s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "kv_append":
        d, nh, h = case["head_dim"], case["n_head"], case["n_kv_head"]
        q, k, v = s["qkv"].split([nh * d, h * d, h * d], -1)
        return qd.kv_append, qd.AppendArgs(cache, q, k, v, s["q_out"], s["table"], s["lens"], pos=s["pos"],
                                           inv_freq=s.get("inv_freq"), rope_dim=case["rope_dim"],
                                           rope_style=qd.ROPE_HALVES if case["style"] == "halves" else qd.ROPE_PAIRS)
    if op == "kv_evict":
        return qd.kv_evict, qd.EvictArgs(cache, s["score"], s["table"], s["lens"], s["dst_table"], s["kept"],
                                         s["score_out"], s["len_out"], keep_first=case["first"], keep_last=case["last"],
                                         budget=case["budget"])
    ws = torch.zeros(qd.attn_ws_bytes(cache, case["n_head"], case["n_seq"], case["n_tok"], s["table"].shape[1],
                                      case["score"]), dtype=torch.uint8, device=DEV)
    return qd.attn_decode, qd.AttnArgs(cache, s["q"], s["out"], s["table"], s["lens"], ws, scale=case["head_dim"] ** -0.5,
                                       window=case["window"], n_sink=case["n_sink"], score=s.get("score"))


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if "call" not in s:
            s["call"] = _call(s)
        call, args = s["call"]
        call(args)
    elif op == "logits_argmax":
        return _plain_logits(s)
    elif op == "attn_decode":
        return _plain_attn(s)
    elif op == "kv_append":
        _plain_append(s)
    else:
        _plain_evict(s)
    if op == "logits_argmax":
        return s["out"], s["idx"]
    if op == "attn_decode":
        return (s["out"], s["score"]) if s["case"]["score"] else s["out"]
    if op == "kv_append":
        return s["q_out"], _cache_values(s)
    return s["kept"], s["score_out"], s["len_out"], _cache_values(s, s["n_src"])


# ---------------------------------------------------------------------------------------------- bytes and flops --
def _slot_bytes(case):
    """Bytes of one head's k and v in one slot."""
    return 2 * case["head_dim"] * (1.0625 if case["type"] == "q8" else 2)


def work(case):
    op = case["op"]
    if op == "logits_argmax":
        n, v = case["n_rows"], case["vocab"]
        return {"bytes": n * (8 * v + 3 * case["hist"] + 8 * case["bias"] + (v / 8 if case["mask"] else 0) + 20),
                "flops": 2 * n * v}
    h, d, lens = case["n_kv_head"], case["head_dim"], _lens(case)
    if op == "kv_evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": h * (sum(lens) * 4 + kept * (8 + 2 * _slot_bytes(case))), "flops": h * sum(lens)}
    nh, t = case["n_head"], case["n_tok"]
    if op == "kv_append":
        n = case["n_seq"] * t
        return {"bytes": n * ((2 * nh + 2 * h) * d * 4 + h * _slot_bytes(case) + 8), "flops": n * 3 * (nh + h) * case["rope_dim"]}
    slots = pairs = 0
    for n in lens:
        first, win = case["n_sink"], case["window"]
        seen = [(max(0, p + 1 - win) if win else 0, p + 1) for p in range(n - t, n) if p >= 0]
        pairs += sum(hi - lo + min(first, lo) for lo, hi in seen)
        slots += n - seen[0][0] + min(first, seen[0][0]) if seen else 0
    return {"bytes": slots * h * (_slot_bytes(case) + (8 if case["score"] else 0)) + case["n_seq"] * t * nh * d * 8,
            "flops": pairs * nh * 4 * d}


# -------------------------------------------------------------------------------------- the definition in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    return {"kv_append": _exact_append, "attn_decode": _exact_attn, "kv_evict": _exact_evict,
            "logits_argmax": _exact_logits}[case["op"]](case, s)


def _rows(s, which, b, h, n):
    """Slots 0..n-1 of sequence b, head h, in 64 bits, page by page of its table."""
    p = s["case"]["page"]
    pages = s["table"][b, :-(-n // p)].long()
    x = s[which][pages, h].reshape(-1, s["case"]["head_dim"])[:n].double()
    if s["case"]["type"] == "q8":
        x = x * s[which + "_scale"][pages, h].reshape(-1, s["case"]["head_dim"] // 32)[:n].double().repeat_interleave(32, -1)
    return x


def _exact_attn(case, s):
    d, t, group = case["head_dim"], case["n_tok"], case["n_head"] // case["n_kv_head"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    score = s["score"].double() if case["score"] else None
    for b, n in enumerate(_lens(case)):
        for h in range(case["n_kv_head"]):
            k, v = _rows(s, "k", b, h, n), _rows(s, "v", b, h, n)
            if score is not None:
                score[b, h, max(0, n - t):n] = 0
            for i in range(t):
                p = n - t + i
                if p < 0:
                    continue
                cols = slice(h * group * d, (h + 1) * group * d)
                lo = max(0, p + 1 - case["window"]) if case["window"] else 0
                first = min(case["n_sink"], lo)
                kk, vv = (torch.cat([x[:first], x[lo:p + 1]]) for x in (k, v))
                w = torch.softmax(q[b, i, cols].reshape(group, d) @ kk.T / math.sqrt(d), -1)
                out[b, i, cols] = (w @ vv).reshape(-1)
                if score is not None:
                    score[b, h, :first] += w[:, :first].sum(0)
                    score[b, h, lo:p + 1] += w[:, first:].sum(0)
    return (out, score) if case["score"] else out


def _exact_append(case, s):
    d, nh, h, t = case["head_dim"], case["n_head"], case["n_kv_head"], case["n_tok"]
    x = s["qkv"].double().reshape(case["n_seq"], t, nh + 2 * h, d)
    r = case["rope_dim"]
    if r:
        turn = torch.exp(1j * s["pos"].double()[:, :, None, None] * s["inv_freq"].double())
        first = torch.arange(r // 2, device=DEV) * (1 if case["style"] == "halves" else 2)
        second = first + (r // 2 if case["style"] == "halves" else 1)
        z = torch.complex(x[:, :, :nh + h][..., first], x[:, :, :nh + h][..., second]) * turn
        x[:, :, :nh + h, first], x[:, :, :nh + h, second] = z.real, z.imag
    cache = None
    if case["type"] != "q8":                      # rounded values of 16 bits: what they are rounded from
        cache = [s["k"].double(), s["v"].double()]
        for b, n in enumerate(_lens(case)):
            for i in range(t):
                slot = n - t + i
                if slot >= 0:
                    page = int(s["table"][b, slot // case["page"]])
                    cache[0][page, :, slot % case["page"]] = x[b, i, nh:nh + h]
                    cache[1][page, :, slot % case["page"]] = x[b, i, nh + h:]
    return x[:, :, :nh].reshape(case["n_seq"], t, -1), cache


def _exact_evict(case, s):
    return None                                    # whole numbers and copies


def _exact_logits(case, s):
    z = s["logits"].double()
    for r in range(case["n_rows"]):
        rep, freq, pres = (float(x) for x in s["params"][r].double())
        ids, count = torch.unique(s["hist"][r, :int(s["hist_len"][r])].long(), return_counts=True)
        old = z[r, ids]
        z[r, ids] = torch.where(old > 0, old / rep, old * rep) - freq * count.double() - pres
        if case["bias"]:
            last = dict(zip(s["bias_ids"][r].tolist(), s["bias_vals"][r].tolist()))
            z[r, torch.tensor(list(last), device=DEV)] += torch.tensor(list(last.values()), device=DEV, dtype=torch.float64)
    if case["mask"]:
        ids = torch.arange(case["vocab"], device=DEV)
        z[(s["mask"][:, ids // 32].long() >> (ids % 32)) & 1 == 0] = -math.inf
    return z, None

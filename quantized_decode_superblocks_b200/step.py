"""The decode step's operators around the weight products: a paged key-value
cache (``kv_append``, ``attn_decode``, ``kv_evict``) and the adjusted greedy
choice (``logits_argmax``).  See ``include/qmv.h`` for what each computes.

A call's arguments are one C structure.  The classes here fill it from tensors
once -- shapes, strides and addresses -- and keep the tensors alive; a decode
loop builds them for its buffers and then only calls::

    cache = KvCache(KV_F16, k, v)                   # pools [n_pages, n_kv_head, page_size, head_dim]
    args = AttnArgs(cache, q, out, table, kv_len, workspace, scale=0.125)
    attn_decode(args)                               # every step

The tensors must not be resized or freed behind an argument object's back.
A call runs on the device of its tensors, on the given stream or that device's
current one.
"""
from __future__ import annotations

import ctypes

KV_F16, KV_BF16, KV_Q8_0 = 0, 1, 2
ROPE_HALVES, ROPE_PAIRS = 0, 1

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


def _fail(what: str):
    raise ValueError(what)


def _take(self, name, t, dtype, dims, shape=None, like=None):
    """Checks tensor `t` and notes it: its address goes into field `name`."""
    if t is None:
        return
    if str(t.dtype) != "torch." + dtype:
        _fail(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != dims or (dims and t.shape[-1] > 1 and t.stride(-1) != 1):
        _fail(f"{name}: expected {dims} dimensions, the last one contiguous, got {tuple(t.shape)} with strides {t.stride()}")
    if shape is not None and any(w is not None and n != w for n, w in zip(t.shape, shape)):
        _fail(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _same_device(self, name, t.device)
    self._held.append(t)
    setattr(self, name, t.data_ptr())


def _same_device(self, name, device):
    if device.type != "cuda":
        _fail(f"{name}: expected a CUDA tensor, got one on {device}")
    if self._device is None:
        self._device = device.index
    elif self._device != device.index:
        _fail(f"{name}: on {device}, the other tensors are on cuda:{self._device}")


def _rows(self, name, t, n_seq, n_tok):
    """Floats between the tokens of [n_seq, n_tok, width], which must be evenly spaced."""
    stride = t.stride(1) if n_tok > 1 else t.stride(0)
    if n_seq > 1 and n_tok > 1 and t.stride(0) != n_tok * t.stride(1):
        _fail(f"{name}: tokens must be evenly spaced, got strides {t.stride()}")
    return stride if n_seq * n_tok > 1 else t.shape[2]


def _lines(t):
    """Stride between the rows of a 2-D tensor."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _heads(name, t):
    """Stride between the (sequence, head) rows of a [n_seq, n_kv_head, n] tensor."""
    s, h, n = t.shape
    if n < 1:
        _fail(f"{name}: needs an entry a row, got {tuple(t.shape)}")
    stride = t.stride(1) if h > 1 else t.stride(0)
    if s > 1 and h > 1 and t.stride(0) != h * t.stride(1):
        _fail(f"{name}: rows must be evenly spaced, got strides {t.stride()}")
    return stride if s * h > 1 else n


class KvCache(ctypes.Structure):
    """A pool of pages: ``k`` and ``v`` [n_pages, n_kv_head, page_size, head_dim] (any order of the first
    three in memory; float16, bfloat16 or int8), for KV_Q8_0 with their f16 scales [.., head_dim / 32]."""
    _fields_ = [("type", _i32), ("n_kv_head", _i32), ("head_dim", _i32), ("page_size", _i32), ("n_pages", _i64),
                ("page_stride", _i64), ("head_stride", _i64), ("slot_stride", _i64),
                ("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp)]

    def __init__(self, type, k, v, k_scale=None, v_scale=None):
        super().__init__()
        self._held, self._device = [], None
        if type not in (KV_F16, KV_BF16, KV_Q8_0):
            _fail(f"unknown cache type {type}")
        self.type = type
        dtype = {KV_F16: "float16", KV_BF16: "bfloat16", KV_Q8_0: "int8"}[type]
        _take(self, "k", k, dtype, 4)
        _take(self, "v", v, dtype, 4, k.shape)
        if v.stride() != k.stride():
            _fail(f"k and v must be laid out alike, got strides {k.stride()} and {v.stride()}")
        self.n_pages, self.n_kv_head, self.page_size, self.head_dim = k.shape
        # a dimension of one slot is never stepped over: any stride would do
        strides = [st if n > 1 else self.head_dim for st, n in zip(k.stride(), k.shape)]
        self.page_stride, self.head_stride, self.slot_stride = strides[:3]
        if type == KV_Q8_0:
            if k_scale is None or v_scale is None:
                _fail("KV_Q8_0 needs k_scale and v_scale")
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                _take(self, name, t, "float16", 4, (*k.shape[:3], self.head_dim // 32))
                if any(n > 1 and 32 * a != b for n, a, b in zip(k.shape[:3], t.stride(), k.stride())):
                    _fail(f"{name}: must be laid out as the quants, one scale per 32, got strides {t.stride()} for {k.stride()}")
        elif k_scale is not None or v_scale is not None:
            _fail("scales belong to KV_Q8_0 only")


class _Args(ctypes.Structure):
    _name = None

    def _begin(self, cache=None):
        self._held, self._device, self._entry = [], None, None
        if cache is not None:
            self._held.append(cache)
            self._device = cache._device
            self.cache = cache

    def _tables(self, table, kv_len, name="block_table"):
        n = kv_len.shape[0] if kv_len is not None else None
        _take(self, name, table, "int32", 2, (n, None))
        return table.shape[1], _lines(table)


class AppendArgs(_Args):
    """kv_append: q [n_seq, n_tok, n_head * head_dim] or None, k and v [.., n_kv_head * head_dim] (f32; slices
    of one fused product are fine) into the cache; q_out as q, or q itself to rotate in place."""
    _name = "kv_append"
    _fields_ = [("cache", KvCache), ("q", _vp), ("k_in", _vp), ("v_in", _vp), ("q_out", _vp), ("q_stride", _i64),
                ("k_stride", _i64), ("v_stride", _i64), ("q_out_stride", _i64), ("n_head", _i32), ("n_seq", _i32),
                ("n_tok", _i32), ("rope_dim", _i32), ("rope_style", _i32), ("max_pages", _i32), ("table_stride", _i64),
                ("block_table", _vp), ("kv_len", _vp), ("pos", _vp), ("inv_freq", _vp)]

    def __init__(self, cache, q, k, v, q_out, block_table, kv_len, pos=None, inv_freq=None, rope_dim=0,
                 rope_style=ROPE_HALVES):
        super().__init__()
        self._begin(cache)
        self.n_seq, self.n_tok = k.shape[0], k.shape[1] if k.dim() == 3 else 0
        lead = (self.n_seq, self.n_tok)
        width = cache.n_kv_head * cache.head_dim
        _take(self, "k_in", k, "float32", 3, (*lead, width))
        _take(self, "v_in", v, "float32", 3, (*lead, width))
        self.k_stride, self.v_stride = _rows(self, "k", k, *lead), _rows(self, "v", v, *lead)
        if (q is None) != (q_out is None):
            _fail("q and q_out go together")
        if q is not None:
            _take(self, "q", q, "float32", 3, lead)
            _take(self, "q_out", q_out, "float32", 3, q.shape)
            if q.shape[2] % cache.head_dim:
                _fail(f"q: width {q.shape[2]} is not a multiple of head_dim {cache.head_dim}")
            self.n_head = q.shape[2] // cache.head_dim
            self.q_stride, self.q_out_stride = _rows(self, "q", q, *lead), _rows(self, "q_out", q_out, *lead)
        _take(self, "kv_len", kv_len, "int32", 1, (self.n_seq,))
        self.max_pages, self.table_stride = self._tables(block_table, kv_len)
        if pos is not None and not pos.is_contiguous():
            _fail("pos: must be contiguous")
        _take(self, "pos", pos, "int32", 2, lead)
        self.rope_dim, self.rope_style = rope_dim, rope_style
        _take(self, "inv_freq", inv_freq, "float32", 1, (rope_dim // 2,))


class AttnArgs(_Args):
    """attn_decode: q and out [n_seq, n_tok, n_head * head_dim] f32, score [n_seq, n_kv_head, slots] f32 or None,
    workspace: a zeroed uint8 tensor of at least attn_ws_bytes()."""
    _name = "attn_decode"
    _fields_ = [("cache", KvCache), ("q", _vp), ("out", _vp), ("score", _vp), ("q_stride", _i64), ("out_stride", _i64),
                ("score_stride", _i64), ("n_head", _i32), ("n_seq", _i32), ("n_tok", _i32), ("max_pages", _i32),
                ("table_stride", _i64), ("block_table", _vp), ("kv_len", _vp), ("scale", _f32), ("window", _i32),
                ("n_sink", _i32), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("score_slots", _i64)]

    def __init__(self, cache, q, out, block_table, kv_len, workspace, scale, window=0, n_sink=0, score=None):
        super().__init__()
        self._begin(cache)
        _take(self, "q", q, "float32", 3)
        _take(self, "out", out, "float32", 3, q.shape)
        self.n_seq, self.n_tok = q.shape[:2]
        if q.shape[2] % cache.head_dim:
            _fail(f"q: width {q.shape[2]} is not a multiple of head_dim {cache.head_dim}")
        self.n_head = q.shape[2] // cache.head_dim
        self.q_stride = _rows(self, "q", q, self.n_seq, self.n_tok)
        self.out_stride = _rows(self, "out", out, self.n_seq, self.n_tok)
        _take(self, "kv_len", kv_len, "int32", 1, (self.n_seq,))
        self.max_pages, self.table_stride = self._tables(block_table, kv_len)
        if score is not None:
            _take(self, "score", score, "float32", 3, (self.n_seq, cache.n_kv_head, None))
            self.score_stride, self.score_slots = _heads("score", score), score.shape[2]
        self.scale, self.window, self.n_sink = scale, window, n_sink
        _take(self, "workspace", workspace, "uint8", 1)
        self.workspace_bytes = workspace.numel()


class EvictArgs(_Args):
    """kv_evict: score [n_seq, n_kv_head, slots], kept int32 and score_out f32 [n_seq, n_kv_head, budget],
    len_out int32 [n_seq]; the kept slots go to the pages of dst_table."""
    _name = "kv_evict"
    _fields_ = [("cache", KvCache), ("score", _vp), ("score_out", _vp), ("score_stride", _i64),
                ("score_out_stride", _i64), ("n_seq", _i32), ("max_pages", _i32), ("dst_max_pages", _i32),
                ("keep_first", _i32), ("keep_last", _i32), ("budget", _i32), ("table_stride", _i64),
                ("dst_table_stride", _i64), ("block_table", _vp), ("kv_len", _vp), ("dst_table", _vp), ("kept", _vp),
                ("len_out", _vp), ("score_slots", _i64)]

    def __init__(self, cache, score, block_table, kv_len, dst_table, kept, score_out, len_out, keep_first, keep_last,
                 budget):
        super().__init__()
        self._begin(cache)
        self.n_seq = kv_len.shape[0]
        _take(self, "kv_len", kv_len, "int32", 1)
        _take(self, "score", score, "float32", 3, (self.n_seq, cache.n_kv_head, None))
        _take(self, "score_out", score_out, "float32", 3, (self.n_seq, cache.n_kv_head, None))
        if score_out.shape[2] < budget:
            _fail(f"score_out: {score_out.shape[2]} entries a head, the budget is {budget}")
        self.score_stride, self.score_out_stride = _heads("score", score), _heads("score_out", score_out)
        self.score_slots = score.shape[2]
        _take(self, "kept", kept, "int32", 3, (self.n_seq, cache.n_kv_head, budget))
        if not kept.is_contiguous():
            _fail("kept: must be contiguous")
        _take(self, "len_out", len_out, "int32", 1, (self.n_seq,))
        self.max_pages, self.table_stride = self._tables(block_table, kv_len)
        self.dst_max_pages, self.dst_table_stride = self._tables(dst_table, kv_len, "dst_table")
        self.keep_first, self.keep_last, self.budget = keep_first, keep_last, budget


class LogitsArgs(_Args):
    """logits_argmax: logits and out [n_rows, vocab] f32 (out may be logits itself, or None), hist int32
    [n_rows, n] with hist_len [n_rows] and params [n_rows, 3] (or all None), bias_ids / bias_vals [n_rows, n]
    with bias_len, mask int32 [n_rows, >= ceil(vocab / 32)] of bits, idx_out int32 [n_rows], workspace: a
    zeroed uint8 tensor of at least logits_ws_bytes(n_rows)."""
    _name = "logits_argmax"
    _fields_ = [("logits", _vp), ("out", _vp), ("logits_stride", _i64), ("out_stride", _i64), ("n_rows", _i32),
                ("vocab", _i32), ("hist", _vp), ("hist_len", _vp), ("hist_stride", _i64), ("params", _vp),
                ("bias_ids", _vp), ("bias_len", _vp), ("bias_vals", _vp), ("bias_stride", _i64), ("mask", _vp),
                ("mask_stride", _i64), ("idx_out", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]

    def __init__(self, logits, hist, hist_len, params, out, idx_out, workspace, bias_ids=None, bias_vals=None,
                 bias_len=None, mask=None):
        super().__init__()
        self._begin()
        _take(self, "logits", logits, "float32", 2)
        n, v = self.n_rows, self.vocab = logits.shape
        self.logits_stride = _lines(logits)
        if out is not None:
            _take(self, "out", out, "float32", 2, (n, v))
            self.out_stride = _lines(out)
        if hist is not None:
            _take(self, "hist", hist, "int32", 2, (n, None))
            self.hist_stride = hist.stride(0) if n > 1 else hist.shape[1]
            if n > 1 and hist.stride(0) != hist.shape[1]:
                _fail("hist: must be contiguous")
            _take(self, "hist_len", hist_len, "int32", 1, (n,))
            if params is None or not params.is_contiguous():
                _fail("params: must be given with hist, and contiguous")
            _take(self, "params", params, "float32", 2, (n, 3))
        if bias_ids is not None:
            _take(self, "bias_ids", bias_ids, "int32", 2, (n, None))
            _take(self, "bias_vals", bias_vals, "float32", 2, bias_ids.shape)
            if not bias_ids.is_contiguous() or not bias_vals.is_contiguous():
                _fail("bias_ids and bias_vals: must be contiguous")
            self.bias_stride = bias_ids.shape[1]
            _take(self, "bias_len", bias_len, "int32", 1, (n,))
        if mask is not None:
            _take(self, "mask", mask, "int32", 2, (n, None))
            if mask.shape[1] < -(-v // 32):
                _fail(f"mask: {mask.shape[1]} words a row, {v} tokens need {-(-v // 32)}")
            self.mask_stride = _lines(mask)
        _take(self, "idx_out", idx_out, "int32", 1, (n,))
        _take(self, "workspace", workspace, "uint8", 1)
        self.workspace_bytes = workspace.numel()


def _call(name, args, stream):
    if args._entry is None:                            # the entry point and its argument, looked up once
        from . import lib
        import torch
        if args._name != name:
            raise TypeError(f"{name}: got the arguments of {args._name}")
        args._entry = name, getattr(lib(), name), ctypes.byref(args), torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    what, fn, ref, current, current_stream = args._entry
    if what != name:
        raise TypeError(f"{name}: got the arguments of {what}")
    dev = args._device
    if dev != current():
        import torch
        with torch.cuda.device(dev):
            return _call(name, args, stream)
    rc = fn(ref, current_stream(dev) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream)
    if rc:
        from . import _check
        _check(rc, name)


def kv_append(args: AppendArgs, stream=None):
    """The new tokens' rotated keys and values into the cache, their rotated queries to q_out."""
    _call("kv_append", args, stream)


def attn_decode(args: AttnArgs, stream=None):
    """Attention of each sequence's newest tokens over its cache."""
    _call("attn_decode", args, stream)


def kv_evict(args: EvictArgs, stream=None):
    """The kept slots of every sequence and kv head into the pages of dst_table."""
    _call("kv_evict", args, stream)


def logits_argmax(args: LogitsArgs, stream=None):
    """Penalties, biases and mask on the logits, and the greedy choice."""
    _call("logits_argmax", args, stream)


def attn_ws_bytes(cache, n_head, n_seq, n_tok, max_pages, with_score=False) -> int:
    """Workspace bytes of attn_decode; 0 when the sizes are outside its limits."""
    from . import lib
    return lib().attn_ws_bytes(ctypes.byref(cache), n_head, n_seq, n_tok, max_pages, 1 if with_score else 0)


def logits_ws_bytes(n_rows) -> int:
    """Workspace bytes of logits_argmax; 0 when n_rows is outside its limits."""
    from . import lib
    return lib().logits_ws_bytes(n_rows)

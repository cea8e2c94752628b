"""ctypes binding of the attention side of libqlora (include/qlora.h): rotary
positions, the paged key/value cache that is quantized as it is written, and
attention of new tokens over it.  Argument marshalling only, as in qlora.py.
"""

from __future__ import annotations

import ctypes

from .qlora import Heads, KVCacheDesc, _check, _dev, _empty, _need, _p, _stream, _torch, _workspace, lib

KV_TYPES = {"bf16": 0, "int8": 1, "nf4": 2, "int4": 3, "fp4": 4}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "bands": 3}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _choice(table, value, name):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}")
    return table[value]


def _heads(t, name):
    """qlora_heads of a [tokens, heads, dim] bf16 tensor with contiguous dims."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim]")
    n, h, d = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    # The stride of an axis of one element is never used.
    return Heads(t.data_ptr(), st if n > 1 else 0, sh if h > 1 else 0, h)


def _new_heads(like, stream):
    """A contiguous tensor like this one, and its view."""
    torch = _torch()
    t = (torch.empty_like(like, memory_format=torch.contiguous_format) if stream is None
         else _empty(like.shape, like.dtype, like.device, stream))
    _, heads, dim = t.shape
    return t, Heads(t.data_ptr(), heads * dim, dim, heads)


def _index(t, n, dtype, name):
    return _need(_dev(t, dtype, name), n, name)


def _given(t, shape, dtype, name):
    """A given output: it holds what is written, and where it has the output's
    axes they are in its order (rows of a longer buffer, not [heads, tokens, dim])."""
    n = 1
    for x in shape:
        n *= x
    _need(_dev(t, dtype, name), n, name)
    if t.dim() == len(shape) and tuple(t.shape[1:]) != tuple(shape[1:]):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def rope_table(positions, rot, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0, high=32.0,
               amplitude=1.0, device="cuda", stream=None):
    """Table of rotations, fp32 [positions, rot/2, 2] (see qlora_rope_table).

    scaling: "none", "linear" (every frequency divided by factor), "base" (the
    base raised so that the slowest pair is slowed by factor), "bands" (pairs
    that turn at least `high` times over `original` positions keep their
    frequency, those that turn at most `low` times get it divided)."""
    torch = _torch()
    table = _empty((positions, rot // 2, 2), torch.float32, device, stream)
    _check(lib().qlora_rope_table(positions, rot, float(base), _choice(ROPE_SCALINGS, scaling, "scaling"),
                                  float(factor), float(original), float(low), float(high), float(amplitude),
                                  _p(table), _stream(stream)))
    return table


def _table(table, positions, T):
    torch = _torch()
    _dev(table, torch.float32, "table")
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be [positions, rot/2, 2]")
    _index(positions, T, torch.int32, "positions")
    return table.shape[0], 2 * table.shape[1]


def rope(q, k, table, positions, layout="half", inverse=False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q and k (k may be None): [tokens, heads, dim] bf16,
    dims contiguous, heads and tokens with any strides that are multiples of 8.

    table: fp32 [positions, rot/2, 2] of rope_table; positions: int32 [tokens].
    layout "half" pairs dims i and i + rot/2, "interleaved" 2i and 2i + 1; dims
    from rot on are copied.  inverse=True is the transpose: the gradient of q
    and k from those of the rotated ones.  q_out, k_out: outputs (q and k
    themselves for in place); allocated when absent.  Returns (q_out, k_out)."""
    T, _, D = q.shape
    rows, rot = _table(table, positions, T)
    qv = _heads(q, "q")
    if q_out is None:
        q_out, qo = _new_heads(q, stream)
    else:
        qo = _heads(q_out, "q_out")
    kv = ko = None
    if k is not None:
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError("q and k must have the same tokens and dim")
        kv = _heads(k, "k")
        if k_out is None:
            k_out, ko = _new_heads(k, stream)
        else:
            ko = _heads(k_out, "k_out")
        if k_out.shape != k.shape:
            raise ValueError("outputs must have their input's shape")
    if q_out.shape != q.shape:
        raise ValueError("outputs must have their input's shape")
    _check(lib().qlora_rope(T, D, rot, _choice(ROPE_LAYOUTS, layout, "layout"), 1 if inverse else 0, table.data_ptr(),
                            rows, positions.data_ptr(), qv, qo, kv, ko, _stream(stream)))
    return q_out, k_out


class KVCache:
    """A paged key/value cache over the caller's tensors (see qlora_kv_cache).

    k, v: [pages, heads, page_size, row]: bf16 rows of dim, int8 rows of dim, or
    uint8 rows of dim/2 (nf4, int4, fp4: two codes a byte).  k_scale, v_scale:
    fp32 [pages, heads, page_size], None for bf16.  KVCache.empty allocates
    them."""

    def __init__(self, k, v, k_scale=None, v_scale=None, kv_type="int8"):
        torch = _torch()
        code = _choice(KV_TYPES, kv_type, "kv_type")
        dtype = torch.bfloat16 if code == 0 else torch.int8 if code == 1 else torch.uint8
        _dev(k, dtype, "k")
        _dev(v, dtype, "v")
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v must be [pages, heads, page_size, row]")
        if code != 0:
            for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if _dev(t, torch.float32, nm).shape != k.shape[:3]:
                    raise ValueError(f"{nm} must be [pages, heads, page_size]")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale, self.kv_type = k, v, k_scale, v_scale, kv_type
        self.pages, self.heads, self.page_size, row = k.shape
        self.dim = row * 2 if code >= 2 else row
        self._desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if code else None,
                                 v_scale.data_ptr() if code else None, self.pages, code, self.heads, self.dim,
                                 self.page_size)

    @classmethod
    def empty(cls, pages, heads, page_size, dim, kv_type="int8", device="cuda"):
        torch = _torch()
        code = _choice(KV_TYPES, kv_type, "kv_type")
        row, dtype = (dim, torch.bfloat16) if code == 0 else (dim, torch.int8) if code == 1 else (dim // 2, torch.uint8)
        codes = [torch.empty(pages, heads, page_size, row, dtype=dtype, device=device) for _ in range(2)]
        scales = [torch.empty(pages, heads, page_size, dtype=torch.float32, device=device) if code else None
                  for _ in range(2)]
        return cls(*codes, *scales, kv_type=kv_type)


def kv_write(cache, k, v, slots, table=None, positions=None, layout="half", stream=None):
    """Store the keys and values of T tokens ([T, heads, dim] bf16) in the
    cache, quantized as they are written.  slots: int64 [T]; a negative one is
    skipped.  With a table of rope_table and int32 positions [T] the keys are
    rotated first (in fp32, not rounded in between)."""
    torch = _torch()
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1:] != (cache.heads, cache.dim):
        raise ValueError("k and v must be [tokens, heads, dim] of the cache")
    _index(slots, T, torch.int64, "slots")
    rows, rot = (0, 0) if table is None else _table(table, positions, T)
    kh, vh = _heads(k, "k"), _heads(v, "v")
    _check(lib().qlora_kv_write(cache._desc, T, kh, vh, slots.data_ptr(), None if table is None else table.data_ptr(),
                                rows, None if table is None else positions.data_ptr(), rot,
                                _choice(ROPE_LAYOUTS, layout, "layout"), _stream(stream)))


def kv_read(cache, slots, k_out=None, v_out=None, stream=None):
    """(k, v) bf16 [T, heads, dim]: the values that the rows at `slots` (int64
    [T]; a negative one gives zeros) stand for."""
    torch = _torch()
    T = slots.numel()
    _dev(slots, torch.int64, "slots")
    shape = (T, cache.heads, cache.dim)
    if k_out is None:
        k_out = (cache.k.new_empty(shape, dtype=torch.bfloat16) if stream is None
                 else _empty(shape, torch.bfloat16, cache.k.device, stream))
    else:
        _given(k_out, shape, torch.bfloat16, "k_out")
    if v_out is None:
        v_out = (cache.k.new_empty(shape, dtype=torch.bfloat16) if stream is None
                 else _empty(shape, torch.bfloat16, cache.k.device, stream))
    else:
        _given(v_out, shape, torch.bfloat16, "v_out")
    _check(lib().qlora_kv_read(cache._desc, T, slots.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), _stream(stream)))
    return k_out, v_out


def attend_paged_workspace_bytes(cache, tokens, q_heads, batch, max_new, max_len, causal=True, window=0):
    return int(lib().qlora_attend_paged_workspace_bytes(cache._desc, tokens, q_heads, batch, max_new,
                                                        max_len, 1 if causal else 0, window))


def attend_paged(q, cache, pages, starts, lengths, max_new, max_len, scale=None, causal=True, window=0, out=None,
                 lse=False, workspace=None, stream=None):
    """Attention of new tokens over a paged cache that already holds them (see
    qlora_attend_paged).

    q: [tokens, q_heads, dim] bf16 (dims contiguous); pages: int32 [batch,
    pages_per_seq]; starts: int32 [batch + 1], the first new token of each
    sequence and the end (0 and q's tokens at both ends; padding is a last
    sequence of length 0); lengths: int32 [batch], stored tokens with the new
    ones; max_new, max_len: host bounds of both.  scale defaults to dim**-0.5.
    out: bf16 [tokens, q_heads, dim]; lse: True, or an fp32 [tokens, q_heads]
    tensor, to have the log-sums too.  Returns (out, lse or None)."""
    torch = _torch()
    T, Hq, D = q.shape
    if D != cache.dim:
        raise ValueError("q and the cache must have the same dim")
    B = lengths.numel()
    _dev(pages, torch.int32, "pages")
    if pages.dim() != 2 or pages.shape[0] != B:
        raise ValueError("pages must be [batch, pages_per_seq]")
    _index(starts, B + 1, torch.int32, "starts")
    _dev(lengths, torch.int32, "lengths")
    if T > 0 and (B == 0 or max_new == 0):
        raise ValueError("tokens of no sequence: batch and max_new must be positive where q has tokens")
    if out is None:
        out = (torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None
               else _empty(q.shape, q.dtype, q.device, stream))
    else:
        _given(out, (T, Hq, D), torch.bfloat16, "out")
    if lse is True:
        lse = q.new_empty((T, Hq), dtype=torch.float32) if stream is None else _empty((T, Hq), torch.float32, q.device, stream)
    elif lse is False or lse is None:
        lse = None
    else:
        _given(lse, (T, Hq), torch.float32, "lse")
    nbytes = attend_paged_workspace_bytes(cache, T, Hq, B, max_new, max_len, causal, window)
    workspace = _workspace(nbytes, q.device, workspace, stream)
    _check(lib().qlora_attend_paged(cache._desc, T, _heads(q, "q"), B, pages.data_ptr(), pages.shape[1],
                                    starts.data_ptr(), lengths.data_ptr(), max_new, max_len,
                                    D ** -0.5 if scale is None else scale, 1 if causal else 0, window, out.data_ptr(),
                                    None if lse is None else lse.data_ptr(),
                                    None if workspace is None else workspace.data_ptr(), nbytes, _stream(stream)))
    return out, lse

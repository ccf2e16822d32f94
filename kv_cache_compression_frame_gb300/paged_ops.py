"""Operators over paged caches of keys and values, and a draft's verification,
on the caller's tensors.

Thin marshalling over the handle-free entry points of include/statekv.h, which
states the mathematics, limits and errors of each; tensors, streams, status
word and errors as in text_ops.  A pool is a CUDA tensor
[pages][heads][page_rows][head_dim] (page_rows a multiple of 16) of any strides
with a contiguous last dimension and rows on 16-byte boundaries; row i of batch
entry n is row i % page_rows of page table[n][i // page_rows], table int32
[n][entries].  Without a table (None) batch entry n is page n: a plain cache
[n][heads][rows][head_dim].  lengths (int, or int32 [sequences]) and counts
(int32 [sequences]; None: all tokens) have one entry per sequence, the batch is
sequences x layers.
"""

from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import _native as N
from .text_ops import (_BF16, _DTYPES, _F32, _I32, _I64, _On, _call, _elsewhere, _lengths, _no_grad, _no_tangents,
                       _out, _shape4, _status_ptr, _vector, _view)


def _table(table, name: str, batch: int, pages: int, rows: int, dev: int) -> tuple[int, int, int, int]:
    """(pointer, stride, entries, rows that a sequence can hold) of a table
    over `pages` pages of `rows` rows."""
    if table is None:
        if pages < batch:
            raise ValueError(f"without a {name} the pages are the batch: {pages} for {batch} entries")
        return 0, 0, 0, rows
    s = table.shape
    if table.dtype is not _I32 or len(s) != 2 or s[0] != batch or table.get_device() != dev or \
            (s[1] > 1 and table.stride(1) != 1) or (s[0] > 1 and table.stride(0) < s[1]):
        raise ValueError(f"{name}: want int32 [{batch}][entries] on cuda:{dev} with contiguous rows, got "
                         f"{table.dtype} {tuple(s)} strides {table.stride()} on {table.device}")
    # (a table of no entries has no memory, but is not the same as none)
    return table.data_ptr() or 16, table.stride(0) if s[0] > 1 else s[1], s[1], s[1] * rows


def _counts(counts, layers: int, batch: int, dev: int) -> tuple[int, int]:
    """(pointer, layers) of a counts argument; layers 0: not known yet."""
    if counts is None:
        return 0, layers or 1
    p = _vector(counts, "counts", _I32, dev)
    seqs = counts.shape[0]
    if (seqs * layers != batch) if layers else (seqs == 0 or batch % seqs):
        if not batch == seqs == 0:
            raise ValueError(f"counts: {seqs} for a batch of {batch}" + (f" of {layers} layers" if layers else ""))
    return p, layers or (batch // seqs if seqs else 1) or 1


def paged_append(k_new, v_new, k_pages, v_pages, table, lengths, counts=None, *, stream=None):
    """Rows i < counts of k_new and v_new [n][Hkv][tokens][d] become cache rows
    lengths + i.  Returns the new lengths (int32 [sequences], or an int where
    lengths is an int and counts None)."""
    n, hkv, tok, d = ns = _shape4(k_new, "k_new")
    pages, _, rows, _ = _shape4(k_pages, "k_pages")
    dt, dev = k_new.dtype, k_new.get_device()
    if forward_ad._current_level >= 0:
        _no_tangents(k_new=k_new, v_new=v_new, k_pages=k_pages, v_pages=v_pages)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return paged_append(k_new, v_new, k_pages, v_pages, table, lengths, counts)
    if dt not in _DTYPES:
        raise ValueError(f"k_new: {dt}, want one of {list(_DTYPES)}")
    ps = (pages, hkv, rows, d)
    views = (*_view(k_new, "k_new", ns, dt, dev), *_view(v_new, "v_new", ns, dt, dev),
             *_view(k_pages, "k_pages", ps, dt, dev), *_view(v_pages, "v_pages", ps, dt, dev))
    tp, ts, entries, _ = _table(table, "table", n, pages, rows, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    cnt, layers = _counts(counts, layers, n, dev)
    status = _status_ptr(dev)
    new, to = None, 0
    if lens or cnt or isinstance(lengths, torch.Tensor) or counts is not None:
        new = torch.empty(n // layers, dtype=_I32, device=k_new.device)
        to = new.data_ptr()
    _call("statekv_paged_append", N.PACK_PAGED_APPEND, dev,
              *views, tp, lens, cnt, to, status, length, ts, entries, pages, rows, n, layers, hkv, tok, d,
              _DTYPES[dt])
    return length + tok if new is None else new


def paged_attention(q, k_pages, v_pages, table, lengths, counts=None, *, scale: float, with_lse: bool = False,
                    out=None, lse=None, workspace=None, stream=None):
    """Attention of the last `counts` tokens of each sequence, q
    [n][Hq][tokens][d] at cache rows lengths - counts + j, over the cache up to
    themselves.  bf16.  Tokens from counts on give zeros.  Returns out like q,
    or (out, lse) with_lse: the rows' log-sum-exps, float32 [n][Hq][tokens].
    workspace: a uint8 CUDA tensor of paged_attention_workspace() bytes
    (default: allocated)."""
    n, hq, tok, d = qs = _shape4(q, "q")
    pages, hkv, rows, _ = _shape4(k_pages, "k_pages")
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return paged_attention(q, k_pages, v_pages, table, lengths, counts, scale=scale, with_lse=with_lse,
                                   out=out, lse=lse, workspace=workspace)
    if forward_ad._current_level >= 0:
        _no_tangents(q=q, k_pages=k_pages, v_pages=v_pages)
    ps = (pages, hkv, rows, d)
    qv = _view(q, "q", qs, _BF16, dev)
    kv_ = (*_view(k_pages, "k_pages", ps, _BF16, dev), *_view(v_pages, "v_pages", ps, _BF16, dev))
    tp, ts, entries, cap = _table(table, "table", n, pages, rows, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    cnt, layers = _counts(counts, layers, n, dev)
    status = _status_ptr(dev)
    out, ov = _out(out, "out", qs, _BF16, q, dev)
    lp = 0
    if lse is not None or with_lse:
        if lse is None:
            lse = torch.empty((n, hq, tok), dtype=_F32, device=q.device)
        elif lse.shape != (n, hq, tok):
            raise ValueError(f"lse: want {(n, hq, tok)}, got {tuple(lse.shape)}")
        lp = _vector(lse, "lse", _F32, dev, 3)
    ws = size = 0
    if workspace is None:
        size = N.load().statekv_paged_attention_workspace(n, hq, hkv, tok, d, cap if cap < 1 << 31 else -1)
        if size > 0:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        ws, size = _vector(workspace, "workspace", torch.uint8, dev), workspace.shape[0]
    _call("statekv_paged_attention", N.PACK_PAGED_ATTENTION, dev,
              *qv, *ov, *kv_, tp, lens, cnt, lp, status, ws, size, scale,
              length, ts, entries, pages, rows, n, layers, hq, hkv, tok, d)
    return (out, lse) if with_lse else out


def paged_attention_workspace(batch: int, q_heads: int, kv_heads: int, tokens: int, head_dim: int,
                              cache_rows: int) -> int:
    """Bytes of workspace paged_attention needs on the current device (0 for a
    few short caches), cache_rows the most that a sequence can hold.  With the
    same kv_heads it never falls as another argument rises."""
    size = N.load().statekv_paged_attention_workspace(batch, q_heads, kv_heads, tokens, head_dim, cache_rows)
    if size < 0:
        raise N.StateKVError(N.E_UNSUPPORTED, "statekv_paged_attention_workspace")
    return size


def attention_weights(q, lse, k_pages, table, lengths, counts=None, *, scale: float, before=None, out=None,
                      stream=None):
    """Attention that each cache row received from the tokens of a
    paged_attention call (the same q, lengths and counts, and its lse), summed
    over the tokens and the query heads of each KV head, added to `before`
    (float32 [n][Hkv][rows], rows at least what a sequence can hold; None:
    zeros).  bf16.  Returns out, like before; out may be before."""
    n, hq, tok, d = qs = _shape4(q, "q")
    pages, hkv, rows, _ = _shape4(k_pages, "k_pages")
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return attention_weights(q, lse, k_pages, table, lengths, counts, scale=scale, before=before, out=out)
    if forward_ad._current_level >= 0:
        _no_tangents(q=q, lse=lse, k_pages=k_pages, before=before)
    views = (*_view(q, "q", qs, _BF16, dev), *_view(k_pages, "k_pages", (pages, hkv, rows, d), _BF16, dev))
    tp, ts, entries, cap = _table(table, "table", n, pages, rows, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    cnt, layers = _counts(counts, layers, n, dev)
    if lse.shape != (n, hq, tok):
        raise ValueError(f"lse: want {(n, hq, tok)}, got {tuple(lse.shape)}")
    _no_grad(lse, "lse")
    lp = _vector(lse, "lse", _F32, dev, 3)
    status = _status_ptr(dev)
    shape = (n, hkv, cap) if before is None and out is None else (before if before is not None else out).shape
    if out is None:
        out = torch.empty(shape, dtype=_F32, device=q.device)
    ptrs = [0, 0]
    for i, (t, name) in enumerate(((before, "before"), (out, "out"))):
        if t is not None:
            if t.shape != shape or shape[:2] != (n, hkv):
                raise ValueError(f"{name}: want ({n}, {hkv}, rows), got {tuple(t.shape)}")
            _no_grad(t, name)
            ptrs[i] = _vector(t, name, _F32, dev, 3)
    _call("statekv_attention_weights", N.PACK_WEIGHTS, dev,
              *views, tp, lens, cnt, lp, *ptrs, status, scale,
              length, ts, entries, pages, rows, shape[2], n, layers, hq, hkv, tok, d)
    return out


def evict_rows(k_pages, v_pages, table, lengths, weights, keep: int, out_table, *, sinks: int = 0, recent: int = 0,
               k_out=None, v_out=None, weights_out=None, kept=None, stream=None):
    """Each batch entry and KV head keeps min(lengths, keep) rows: those below
    `sinks`, the last `recent`, and of the others those of the largest weight
    (float32 [n][Hkv][rows], as attention_weights returns them), ties to the
    lower row.  They move, in their order, to the pages of k_out and v_out
    (default: k_pages and v_pages themselves; of any page size) that out_table
    names; those pages are in no entry's table.  Returns (new lengths, weights_out float32
    [n][Hkv][rows of out_table], the kept rows' weights and then zeros, kept
    int32 [n][Hkv][keep], their old rows and then -1)."""
    pages, hkv, rows, d = ps = _shape4(k_pages, "k_pages")
    k_out, v_out = k_pages if k_out is None else k_out, v_pages if v_out is None else v_out
    out_pages, _, out_rows, _ = _shape4(k_out, "k_out")
    dt, dev = k_pages.dtype, k_pages.get_device()
    if forward_ad._current_level >= 0:
        _no_tangents(k_pages=k_pages, v_pages=v_pages, weights=weights)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return evict_rows(k_pages, v_pages, table, lengths, weights, keep, out_table, sinks=sinks, recent=recent,
                              k_out=k_out, v_out=v_out, weights_out=weights_out, kept=kept)
    if dt not in _DTYPES:
        raise ValueError(f"k_pages: {dt}, want one of {list(_DTYPES)}")
    os_ = (out_pages, hkv, out_rows, d)
    views = (*_view(k_pages, "k_pages", ps, dt, dev), *_view(v_pages, "v_pages", ps, dt, dev),
             *_view(k_out, "k_out", os_, dt, dev), *_view(v_out, "v_out", os_, dt, dev))
    wp = _vector(weights, "weights", _F32, dev, 3)
    _no_grad(weights, "weights")
    n, _, weight_rows = ws = weights.shape
    if ws[1] != hkv:
        raise ValueError(f"weights: want (n, {hkv}, rows), got {tuple(ws)}")
    tp, ts, entries, _ = _table(table, "table", n, pages, rows, dev)
    otp, ots, out_entries, out_cap = _table(out_table, "out_table", n, out_pages, out_rows, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    layers = layers or 1
    keep = int(keep)
    status = _status_ptr(dev)
    if weights_out is None:
        weights_out = torch.empty((n, hkv, out_cap), dtype=_F32, device=k_pages.device)
    elif weights_out.dim() != 3 or weights_out.shape[:2] != (n, hkv):
        raise ValueError(f"weights_out: want ({n}, {hkv}, rows), got {tuple(weights_out.shape)}")
    _no_grad(weights_out, "weights_out")
    if kept is None:
        kept = torch.empty((n, hkv, max(0, keep)), dtype=_I32, device=k_pages.device)
    elif kept.shape != (n, hkv, keep):
        raise ValueError(f"kept: want {(n, hkv, keep)}, got {tuple(kept.shape)}")
    new, to = None, 0
    if isinstance(lengths, torch.Tensor):
        new = torch.empty(n // layers, dtype=_I32, device=k_pages.device)
        to = new.data_ptr()
    _call("statekv_evict_rows", N.PACK_EVICT, dev,
              *views, tp, otp, lens, wp, _vector(weights_out, "weights_out", _F32, dev, 3),
              _vector(kept, "kept", _I32, dev, 3), to, status, length, ts, entries, pages, rows, weight_rows,
              ots, out_entries, out_pages, out_rows, weights_out.shape[2], keep, int(sinks), int(recent),
              n, layers, hkv, d, _DTYPES[dt])
    return min(length, keep) if new is None else new, weights_out, kept


def _rows3(t, name: str, shape, dev: int) -> tuple[int, int, int]:
    """(pointer, sequence stride, row stride) of probabilities [sequences][rows][vocab]."""
    if t.dtype is not _F32 or t.shape != shape or t.get_device() != dev or (t.stride(2) != 1 and shape[2] != 1):
        raise ValueError(f"{name}: want float32 {tuple(shape)} on cuda:{dev} with a contiguous last dimension, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    _no_grad(t, name)
    return t.data_ptr(), t.stride(0), t.stride(1)


def verify_tree(target, draft, drafted, tree, uniforms, *, stream=None):
    """Which path of a drafted tree (tree_masks) stands against the target's
    probabilities (float32 [sequences][tokens + 1][vocab]: row 0 after the text
    so far, row i + 1 after node i), and the token after it.  draft: the
    probabilities that the nodes' children were drawn from, likewise, or None:
    the children are proposals without probabilities.  drafted: int32
    [sequences][tokens]; uniforms: float32 [sequences][tokens + 1] in [0, 1),
    one per node and one for the last token.  Returns (path int32
    [sequences][tokens], -1 past its end, counts int32 [sequences], as
    append_accepted takes them, next token int32 [sequences])."""
    if target.dim() != 3 or not target.is_cuda or target.shape[1] < 2:
        raise ValueError(f"target: want a CUDA tensor [sequences][tokens + 1][vocab], got {tuple(target.shape)} on "
                         f"{target.device}")
    s, rows, vocab = shape = target.shape
    tok, dev = rows - 1, target.get_device()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return verify_tree(target, draft, drafted, tree, uniforms)
    if forward_ad._current_level >= 0:
        _no_tangents(target=target, draft=draft, uniforms=uniforms)
    tv = _rows3(target, "target", shape, dev)
    dv = (0, 0, 0) if draft is None else _rows3(draft, "draft", shape, dev)
    if drafted.shape != (s, tok) or uniforms.shape != (s, rows):
        raise ValueError(f"drafted and uniforms: want {(s, tok)} and {(s, rows)}, got {tuple(drafted.shape)} and "
                         f"{tuple(uniforms.shape)}")
    _no_grad(uniforms, "uniforms")
    dims = tree.dim()
    masks = _vector(tree, "tree", _I64, dev, dims if dims == 2 else 1)
    if tree.shape[-1] != tok or (dims == 2 and tree.shape[0] not in (1, s)):
        raise ValueError(f"tree: want ({tok},) or ({s}, {tok}), got {tuple(tree.shape)}")
    dp, up = _vector(drafted, "drafted", _I32, dev, 2), _vector(uniforms, "uniforms", _F32, dev, 2)
    status = _status_ptr(dev)
    whole = torch.empty(s * (tok + 2), dtype=_I32, device=target.device)
    path, counts, after = whole[:s * tok].view(s, tok), whole[s * tok:s * rows], whole[s * rows:]
    at = whole.data_ptr()
    _call("statekv_verify_tree", N.PACK_VERIFY, dev,
              tv[0], dv[0], dp, masks, up, at, at + 4 * s * tok, at + 4 * s * rows, status, *tv[1:], *dv[1:],
              tok if dims == 2 and tree.shape[0] != 1 else 0, s, tok, vocab)
    return path, counts, after

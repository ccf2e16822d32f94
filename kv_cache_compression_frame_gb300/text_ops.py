"""Text operators over a cache of keys and values, on the caller's tensors.

Thin marshalling over the handle-free entry points of include/statekv.h, which
states the mathematics, limits and errors of each.  Tensors are CUDA tensors
[batch][heads][tokens][head_dim] of any strides with a contiguous last
dimension and rows on 16-byte boundaries (expanded ones are inputs only, and
not tree attention's keys and values); the batch is sequences x layers, and
lengths, trees, paths and destination rows have one entry per sequence.

Work is enqueued on `stream` (default: the current stream of the tensors'
device).  Outputs and workspaces that are not passed in are allocated there.
Failures that only the device can see (a length out of range, a wait that gave
up) are kept in one status word per device, which check_status() reads; a
device's first call allocates it and must not be inside a graph capture.
There is no derivative: inputs that require grad are refused while grad mode is
on, and inputs with a forward-mode tangent always.
"""

from __future__ import annotations

import struct
import threading

import torch
from torch.autograd import forward_ad

from . import _native as N

_BF16, _F32, _I32, _I64, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.int8
_DTYPES = {_BF16: N.BF16, _F32: N.F32}
_NO_VIEW = (0, 0, 0, 0)
_status: dict[int, tuple] = {}              # device -> (status word, its address)
_status_lock = threading.Lock()
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _status_ptr(dev: int) -> int:
    try:
        return _status[dev][1]
    except KeyError:
        pass
    if torch.cuda.is_current_stream_capturing():
        # its zeros would be part of the graph, and its memory the graph's
        raise RuntimeError("call a text operator once on this device before capturing one")
    # one word per device, whichever thread comes first: kernels keep its address
    with _status_lock:
        if dev not in _status:
            t = torch.zeros(4, dtype=_I32, device=torch.device("cuda", dev))
            torch.cuda.synchronize(dev)     # any stream may use it from here on
            _status[dev] = (t, t.data_ptr())
        return _status[dev][1]


def check_status(device: int | torch.device | None = None) -> None:
    """Synchronise the device and raise if a text operator recorded a failure
    there since the last check."""
    dev = device if isinstance(device, int) else None if device is None else torch.device(device).index
    if dev is None:
        dev = torch.cuda.current_device()
    if dev not in _status:
        return
    t = _status[dev][0]
    torch.cuda.synchronize(dev)
    code = int(t[0])
    if code:
        site = t[1:].tolist()
        t.zero_()
        torch.cuda.synchronize(dev)
        raise N.StateKVError(code, f"device status (site, block, value) = {site}")


def tree_masks(parents, device=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Masks and depths of drafted trees from parent lists: parents[i] < i is
    node i's parent, -1 for a root.  One list, or one per sequence (all of one
    length).  Returns (masks int64 [sequences][tokens] for tree_attention,
    depths int32 [sequences][tokens], what each node adds to the position of
    the first)."""
    rows = [list(p) for p in parents] if len(parents) and not isinstance(parents[0], int) else [list(parents)]
    masks, depths = [], []
    for row in rows:
        if not 1 <= len(row) <= 64 or len(row) != len(rows[0]):
            raise ValueError("a tree has 1 to 64 nodes, the same number in each sequence")
        bits, depth = [], []
        for i, p in enumerate(row):
            if not -1 <= p < i:
                raise ValueError(f"node {i}: parent {p} is not an earlier node or -1")
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(depth[p] + 1 if p >= 0 else 0)
        masks.append([b - (1 << 64) if b >> 63 else b for b in bits])
        depths.append(depth)
    return (torch.tensor(masks, dtype=_I64, device=device),
            torch.tensor(depths, dtype=_I32, device=device))


def _view(t: torch.Tensor, name: str, shape, dtype, dev: int) -> tuple:
    """(pointer, batch, head and token stride) of a checked argument."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or (st[3] != 1 and shape[3] != 1):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on cuda:{dev} with a contiguous last dimension, "
                         f"got {t.dtype} {tuple(t.shape)} strides {st} on {t.device}")
    if t.requires_grad:
        _no_grad(t, name)
    return t.data_ptr(), st[0], st[1], st[2]


def _no_grad(t: torch.Tensor, name: str) -> None:
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: the text operators have no backward pass")


def _no_tangents(**inputs) -> None:
    # (called inside of a dual level only: outside no tensor has a tangent)
    for name, t in inputs.items():
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{name} has a tangent: the text operators have no forward-mode derivative")


def _shape4(t: torch.Tensor, name: str):
    s = t.shape
    if len(s) != 4 or not t.is_cuda:
        raise ValueError(f"{name}: want a CUDA tensor [batch][heads][tokens][head_dim], got "
                         f"{tuple(s)} on {t.device}")
    return s


def _vector(t: torch.Tensor, name: str, dtype, dev: int, dims: int = 1) -> int:
    if t.dtype is not dtype or t.dim() != dims or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dims}-D {dtype} tensor on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _lengths(lengths, batch: int, dev: int) -> tuple[int, int, int]:
    """(pointer, common value, layers; 0: not known) of a lengths argument."""
    if isinstance(lengths, torch.Tensor):
        p = _vector(lengths, "lengths", _I32, dev)
        seqs = lengths.shape[0]
        if seqs == 0 or batch % seqs:
            if batch == seqs == 0:
                return 0, 0, 1
            raise ValueError(f"lengths: {seqs} sequences do not divide a batch of {batch}")
        return p, 0, batch // seqs or 1
    return 0, int(lengths), 0


def _layers(found: int, rows: int, batch: int, name: str) -> int:
    """Batch entries per sequence, from the lengths (found > 0) or from an
    array of `rows` rows; one row may serve all sequences."""
    if found:
        if rows not in (1, batch // found):
            raise ValueError(f"{name}: {rows} rows for {batch // found} sequences")
        return found
    if rows == batch == 0:
        return 1
    if rows == 0 or batch % rows:
        raise ValueError(f"{name}: {rows} rows do not divide a batch of {batch}")
    return max(1, batch // rows)


class _On:
    """Makes the tensors' device and the call's stream current."""

    def __init__(self, dev: int, stream):
        self.guards = [torch.cuda.device(dev)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _elsewhere(dev: int, stream) -> bool:
    """Whether a call needs _On around it."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream: of device {stream.device_index}, the tensors are on cuda:{dev}")
    return stream is not None or _current_device() != dev


def _call(name: str, pack: struct.Struct, dev: int, *values) -> None:
    if not N.packed:
        N.load()
    try:
        args = pack.pack(*values)
    except struct.error as e:
        raise ValueError(f"{name}: a size is out of range ({e})") from None
    status = N.packed[name](args, _raw_stream(dev))
    if status:
        N.check(status, name)


def _out(t, name: str, shape, dtype, like: torch.Tensor, dev: int) -> tuple:
    """(tensor, its view): the caller's checked, or a new contiguous one."""
    if t is not None:
        return t, _view(t, name, shape, dtype, dev)
    t = torch.empty(shape, dtype=dtype, device=like.device)
    row = shape[3]
    head = shape[2] * row
    return t, (t.data_ptr(), shape[1] * head, head, row)


def qk_norm_rope(q, k, positions, omega, q_weight=None, k_weight=None, *, v=None, eps: float = 1e-6,
                 q_out=None, k_out=None, v_out=None, out_rows=None, stream=None):
    """RMS norm of every head of q [n][Hq][t][d] and k [n][Hkv][t][d] with
    weights [d] or [layers][d] (the batch is sequences x layers; no norm where
    the weight is None), rotation at `positions` (int32 [t] or [rows][t]
    with rows dividing n, or an int: that and the following ones) with omega
    float64 [d/2], in one pass.  v is copied.  k and v go to rows out_rows
    (int32 [sequences]) + t of k_out and v_out (default: new tensors, row t).
    Returns (q_out, k_out) or (q_out, k_out, v_out)."""
    n, hq, t, d = qs = _shape4(q, "q")
    hkv = _shape4(k, "k")[1]
    dt, dev = q.dtype, q.get_device()
    if forward_ad._current_level >= 0:
        _no_tangents(q=q, k=k, v=v, q_weight=q_weight, k_weight=k_weight, omega=omega)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return qk_norm_rope(q, k, positions, omega, q_weight, k_weight, v=v, eps=eps, q_out=q_out,
                                k_out=k_out, v_out=v_out, out_rows=out_rows)
    if dt not in _DTYPES:
        raise ValueError(f"q: {dt}, want one of {list(_DTYPES)}")
    ks = (n, hkv, t, d)
    qv, kv_ = _view(q, "q", qs, dt, dev), _view(k, "k", ks, dt, dev)
    wd, w_rows, w_ptr = None, 1, [0, 0]
    for i, w in enumerate((q_weight, k_weight)):
        if w is not None:
            rows = w.shape[0] if w.dim() == 2 else 1
            if w.dim() not in (1, 2) or w.shape[-1] != d or w.dtype not in _DTYPES or rows < 1 or n % rows or \
                    (wd is not None and (wd is not w.dtype or rows != w_rows)):
                raise ValueError(f"{'qk'[i]}_weight: want [{d}] or [layers][{d}] of one of {list(_DTYPES)}, the "
                                 "same for both weights, layers dividing the batch")
            _no_grad(w, f"{'qk'[i]}_weight")
            wd, w_rows = w.dtype, rows
            w_ptr[i] = _vector(w, f"{'qk'[i]}_weight", wd, dev, w.dim())
    if omega.shape != (d // 2,):
        raise ValueError(f"omega: want [{d // 2}]")
    _no_grad(omega, "omega")
    om = _vector(omega, "omega", torch.float64, dev)
    pos = p0 = p_stride = 0
    p_layers = layers = 1
    if isinstance(positions, torch.Tensor):
        dims = positions.dim()
        pos = _vector(positions, "positions", _I32, dev, dims if dims == 2 else 1)
        if positions.shape[-1] != t:
            raise ValueError(f"positions: want {t} per row")
        if dims == 2 and positions.shape[0] != 1:
            rows = positions.shape[0]
            if n and (rows == 0 or n % rows):
                raise ValueError(f"positions: {rows} rows do not divide a batch of {n}")
            p_stride, p_layers = t, max(1, n // max(1, rows))
    else:
        p0 = int(positions)
    at = 0
    if out_rows is not None:
        if not isinstance(out_rows, torch.Tensor):
            raise ValueError("out_rows: want int32 [sequences]")
        at, _, layers = _lengths(out_rows, n, dev)
        if k_out is None or (v is not None and v_out is None):
            raise ValueError("out_rows needs k_out (and v_out)")
    if v is None and v_out is not None:
        raise ValueError("v_out without v")
    status = _status_ptr(dev)
    cap = t if k_out is None else k_out.shape[2] if k_out.dim() == 4 else -1
    os_ = (n, hkv, cap, d)
    q_out, qo = _out(q_out, "q_out", qs, dt, q, dev)
    k_out, ko = _out(k_out, "k_out", os_, dt, q, dev)
    vv = vo = _NO_VIEW
    if v is not None:
        vv = _view(v, "v", ks, dt, dev)
        v_out, vo = _out(v_out, "v_out", os_, dt, q, dev)
    _call("statekv_norm_rope", N.PACK_NORM_ROPE, dev,
              *qv, *kv_, *vv, *qo, *ko, *vo,
              w_ptr[0], w_ptr[1], om, pos, at, status, p0, p_stride, p_layers, n, layers, hq, hkv, t, d, cap,
              w_rows, _DTYPES[dt], _DTYPES[wd or dt], eps)
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def tree_attention(q, k_new, v_new, tree, k_cache, v_cache, lengths, *, scale: float, out=None,
                   workspace=None, stream=None):
    """Attention of drafted tokens q [n][Hq][tokens][d], k_new and v_new
    [n][Hkv][tokens][d] over the first `lengths` rows (int, or int32
    [sequences]) of k_cache and v_cache [n][Hkv][rows][d] and, among
    themselves, where tree (int64 masks [tokens] or [sequences][tokens], see
    tree_masks) says.  bf16.  Returns out like q.  workspace: a uint8 CUDA
    tensor of tree_attention_workspace() bytes (default: allocated)."""
    n, hq, tok, d = qs = _shape4(q, "q")
    _, hkv, rows, _ = _shape4(k_cache, "k_cache")
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return tree_attention(q, k_new, v_new, tree, k_cache, v_cache, lengths, scale=scale, out=out,
                                  workspace=workspace)
    if forward_ad._current_level >= 0:
        _no_tangents(q=q, k_new=k_new, v_new=v_new, k_cache=k_cache, v_cache=v_cache)
    ns, cs = (n, hkv, tok, d), (n, hkv, rows, d)
    views = (*_view(q, "q", qs, _BF16, dev), *_view(k_new, "k_new", ns, _BF16, dev),
             *_view(v_new, "v_new", ns, _BF16, dev), *_view(k_cache, "k_cache", cs, _BF16, dev),
             *_view(v_cache, "v_cache", cs, _BF16, dev))
    lens, length, layers = _lengths(lengths, n, dev)
    dims = tree.dim()
    masks = _vector(tree, "tree", _I64, dev, dims if dims == 2 else 1)
    if tree.shape[-1] != tok:
        raise ValueError(f"tree: want {tok} masks per row")
    t_stride = 0
    if dims == 2 and tree.shape[0] != 1:
        layers = _layers(layers, tree.shape[0], n, "tree")
        t_stride = tok
    status = _status_ptr(dev)
    out, ov = _out(out, "out", qs, _BF16, q, dev)
    ws = size = 0
    if workspace is None:
        size = N.load().statekv_tree_attention_workspace(n, hq, hkv, tok, d, rows)
        if size > 0:
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        ws, size = _vector(workspace, "workspace", torch.uint8, dev), workspace.shape[0]
    _call("statekv_tree_attention", N.PACK_TREE, dev,
              *views[:4], *ov, *views[4:], masks, lens, status, ws, size, scale,
              t_stride, length, n, layers or 1, hq, hkv, tok, d, rows)
    return out


def tree_attention_workspace(batch: int, q_heads: int, kv_heads: int, tokens: int, head_dim: int,
                             cache_rows: int) -> int:
    """Bytes of workspace tree_attention needs on the current device (0 for a
    few short caches).  With the same kv_heads it never falls as another
    argument rises; with more KV heads it may."""
    size = N.load().statekv_tree_attention_workspace(batch, q_heads, kv_heads, tokens, head_dim, cache_rows)
    if size < 0:
        raise N.StateKVError(N.E_UNSUPPORTED, "statekv_tree_attention_workspace")
    return size


def append_accepted(k_new, v_new, path, counts, k_cache, v_cache, lengths, *, stream=None):
    """Rows path (int32 [steps] or [sequences][steps]) of k_new and v_new
    [n][Hkv][tokens][d] become cache rows lengths + i, i < counts (int32
    [sequences], or None: all steps).  Returns the new lengths (int32
    [sequences], or an int where lengths is an int and counts None)."""
    n, hkv, tok, d = ns = _shape4(k_new, "k_new")
    rows = _shape4(k_cache, "k_cache")[2]
    dt, dev = k_new.dtype, k_new.get_device()
    if forward_ad._current_level >= 0:
        _no_tangents(k_new=k_new, v_new=v_new, k_cache=k_cache, v_cache=v_cache)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return append_accepted(k_new, v_new, path, counts, k_cache, v_cache, lengths)
    if dt not in _DTYPES:
        raise ValueError(f"k_new: {dt}, want one of {list(_DTYPES)}")
    cs = (n, hkv, rows, d)
    views = (*_view(k_new, "k_new", ns, dt, dev), *_view(v_new, "v_new", ns, dt, dev),
             *_view(k_cache, "k_cache", cs, dt, dev), *_view(v_cache, "v_cache", cs, dt, dev))
    lens, length, layers = _lengths(lengths, n, dev)
    dims = path.dim()
    pp = _vector(path, "path", _I32, dev, dims if dims == 2 else 1)
    steps = path.shape[-1]
    p_stride = cnt = 0
    if dims == 2 and path.shape[0] != 1:
        layers = _layers(layers, path.shape[0], n, "path")
        p_stride = steps
    if counts is not None:
        cnt = _vector(counts, "counts", _I32, dev)
        if layers and counts.shape[0] * layers != n:
            raise ValueError(f"counts: {counts.shape[0]} for {n // layers} sequences")
        layers = layers or _layers(0, counts.shape[0], n, "counts")
    layers = layers or 1
    status = _status_ptr(dev)
    new, to = None, 0
    if counts is not None or isinstance(lengths, torch.Tensor):
        new = torch.empty(n // layers, dtype=_I32, device=k_new.device)
        to = new.data_ptr()
    _call("statekv_append_accepted", N.PACK_APPEND, dev,
              *views, pp, cnt, lens, to, status, p_stride, steps, length, n, layers, hkv, tok, d, rows,
              _DTYPES[dt])
    return length + steps if new is None else new


def block_summaries(k_cache, codes, scales, lengths, *, appended: int | None = None, stream=None) -> None:
    """Brings codes (int8 [n][Hkv][blocks][d]) and scales (float32
    [n][Hkv][blocks]) up to date for the complete 64-row blocks of k_cache
    [n][Hkv][rows][d] that the last `appended` rows (None: all) of the first
    `lengths` completed.  blocks >= rows // 64."""
    n, hkv, rows, d = cs = _shape4(k_cache, "k_cache")
    dev = k_cache.get_device()
    if forward_ad._current_level >= 0:
        _no_tangents(k_cache=k_cache, scales=scales)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return block_summaries(k_cache, codes, scales, lengths, appended=appended)
    view = _view(k_cache, "k_cache", cs, _BF16, dev)
    pc, ps, blocks = _summary_ptrs(codes, scales, n, hkv, d, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    appended = rows if appended is None else min(int(appended), rows)
    _call("statekv_block_summaries", N.PACK_SUMMARY, dev,
              *view, pc, ps, lens, _status_ptr(dev), length, appended, blocks, n, layers or 1, hkv, d, rows)


def _summary_ptrs(codes, scales, n: int, hkv: int, d: int, dev: int) -> tuple[int, int, int]:
    pc = _vector(codes, "codes", _I8, dev, 4)
    _no_grad(scales, "scales")
    ps = _vector(scales, "scales", _F32, dev, 3)
    blocks = codes.shape[2]
    if codes.shape != (n, hkv, blocks, d) or scales.shape != (n, hkv, blocks):
        raise ValueError(f"codes and scales: want ({n}, {hkv}, blocks, {d}) and ({n}, {hkv}, blocks), got "
                         f"{tuple(codes.shape)} and {tuple(scales.shape)}")
    return pc, ps, blocks


def sparse_attention(q, k_cache, v_cache, codes, scales, lengths, top: int, *, scale: float, out=None,
                     selected=None, stream=None):
    """Attention of the last tokens of each sequence, q [n][Hq][tokens][d] at
    cache rows lengths - tokens + j, over the `top` blocks of k_cache and
    v_cache [n][Hkv][rows][d] that codes and scales (block_summaries) score
    best for each token and KV head, and the rows since the last complete
    block.  bf16.  Returns (out like q, selected int32 [n][Hkv][tokens][top]:
    the chosen blocks in ascending order, then -1)."""
    n, hq, tok, d = qs = _shape4(q, "q")
    _, hkv, rows, _ = _shape4(k_cache, "k_cache")
    dev = q.get_device()
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return sparse_attention(q, k_cache, v_cache, codes, scales, lengths, top, scale=scale, out=out,
                                    selected=selected)
    if forward_ad._current_level >= 0:
        _no_tangents(q=q, k_cache=k_cache, v_cache=v_cache, scales=scales)
    top = int(top)
    cs = (n, hkv, rows, d)
    qv = _view(q, "q", qs, _BF16, dev)
    kc, vc = _view(k_cache, "k_cache", cs, _BF16, dev), _view(v_cache, "v_cache", cs, _BF16, dev)
    pc, ps, blocks = _summary_ptrs(codes, scales, n, hkv, d, dev)
    lens, length, layers = _lengths(lengths, n, dev)
    status = _status_ptr(dev)
    out, ov = _out(out, "out", qs, _BF16, q, dev)
    ss = (n, hkv, tok, max(0, top))
    if selected is None:
        selected = torch.empty(ss, dtype=_I32, device=q.device)
    elif selected.shape != ss:
        raise ValueError(f"selected: want {ss}, got {tuple(selected.shape)}")
    _call("statekv_sparse_attention", N.PACK_SPARSE, dev,
              *qv, *ov, *kc, *vc, pc, ps, lens,
              _vector(selected, "selected", _I32, dev, 4), status, scale, length, top, blocks, n, layers or 1, hq,
              hkv, tok, d, rows)
    return out, selected

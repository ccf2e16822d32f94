"""Text operators over a cache of keys and values, on the caller's tensors.

Thin marshalling over the handle-free entry points of include/statekv.h, which
states the mathematics, limits and errors of each.  Tensors are CUDA tensors
[batch][heads][tokens][head_dim] of any strides with a contiguous last
dimension and rows on 16-byte boundaries; the batch is sequences x layers, and
lengths, trees, paths and destination rows have one entry per sequence.

Work is enqueued on `stream` (default: the current stream of the tensors'
device).  Outputs and workspaces that are not passed in are allocated there.
Failures that only the device can see (a length out of range, a wait that gave
up) are kept in one status word per device, which check_status() reads.
There is no backward pass: inputs that require grad are refused while grad
mode is on.
"""

from __future__ import annotations

import ctypes as C

import torch

from . import _native as N

_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_DTYPES = {_BF16: N.BF16, _F32: N.F32}
_NO_VIEW = N.View(None, 0, 0, 0)
_status: dict[int, torch.Tensor] = {}
_raw_stream = torch._C._cuda_getCurrentRawStream


def _status_ptr(dev: int) -> int:
    t = _status.get(dev)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            # its zeros would be part of the graph, and its memory the graph's
            raise RuntimeError("call a text operator once on this device before capturing one")
        t = _status[dev] = torch.zeros(4, dtype=_I32, device=torch.device("cuda", dev))
        torch.cuda.synchronize(dev)         # any stream may use it from here on
    return t.data_ptr()


def check_status(device: int | torch.device | None = None) -> None:
    """Synchronise the device and raise if a text operator recorded a failure
    there since the last check."""
    dev = torch.cuda.current_device() if device is None else torch.device("cuda", device).index \
        if isinstance(device, int) else torch.device(device).index
    if dev is None:
        dev = torch.cuda.current_device()
    t = _status.get(dev)
    if t is None:
        return
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


def _view(t: torch.Tensor, name: str, shape, dtype, dev) -> N.View:
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.device != dev or (st[3] != 1 and shape[3] != 1):
        raise ValueError(f"{name}: want {dtype} {tuple(shape)} on {dev} with a contiguous last dimension, "
                         f"got {t.dtype} {tuple(t.shape)} strides {st} on {t.device}")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad: the text operators have no backward pass")
    return N.View(t.data_ptr(), st[0], st[1], st[2])


def _shape4(t: torch.Tensor, name: str):
    if t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name}: want a CUDA tensor [batch][heads][tokens][head_dim], got "
                         f"{tuple(t.shape)} on {t.device}")
    return t.shape


def _vector(t: torch.Tensor, name: str, dtype, dev, dims: int = 1) -> int:
    if t.dtype is not dtype or t.dim() != dims or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {dims}-D {dtype} tensor on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _lengths(lengths, batch: int, dev) -> tuple[int | None, int, int]:
    """(pointer, common value, layers) of a lengths argument."""
    if isinstance(lengths, torch.Tensor):
        p = _vector(lengths, "lengths", _I32, dev)
        seqs = lengths.shape[0]
        if seqs == 0 or batch % seqs:
            if batch == seqs == 0:
                return None, 0, 1
            raise ValueError(f"lengths: {seqs} sequences do not divide a batch of {batch}")
        return p, 0, batch // seqs or 1
    return None, int(lengths), 0


def _layers(found: int, rows: int, batch: int, name: str) -> int:
    """Batch entries per sequence, from the lengths (found > 0) or from an
    array of `rows` rows; one row may serve all sequences."""
    if found:
        if rows not in (1, batch // found):
            raise ValueError(f"{name}: {rows} rows for {batch // found} sequences")
        return found
    if rows == 0 or batch % rows:
        raise ValueError(f"{name}: {rows} rows do not divide a batch of {batch}")
    return max(1, batch // rows)


class _On:
    """The tensors' device and the stream of a call made current."""

    def __init__(self, dev: torch.device, stream):
        self.dev = dev.index
        self.away = torch.cuda.current_device() != self.dev
        self.stream = stream

    def __enter__(self) -> int:
        self.guards = []
        if self.away:
            self.guards.append(torch.cuda.device(self.dev))
        if self.stream is not None:
            self.guards.append(torch.cuda.stream(self.stream))
        for g in self.guards:
            g.__enter__()
        return _raw_stream(self.dev)

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def qk_norm_rope(q, k, positions, omega, q_weight=None, k_weight=None, *, v=None, eps: float = 1e-6,
                 q_out=None, k_out=None, v_out=None, out_rows=None, stream=None):
    """RMS norm of every head of q [n][Hq][t][d] and k [n][Hkv][t][d] with
    weights [d] or [layers][d] (the batch is sequences x layers; no norm where
    the weight is None), rotation at `positions` (int32 [t] or [rows][t]
    with rows dividing n, or an int: that and the following ones) with omega
    float64 [d/2], in one pass.  v is copied.  k and v go to rows out_rows
    (int32 [sequences]) + t of k_out and v_out (default: new tensors, row t).
    Returns (q_out, k_out) or (q_out, k_out, v_out)."""
    n, hq, t, d = _shape4(q, "q")
    hkv = _shape4(k, "k")[1]
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise ValueError(f"q: {dt}, want one of {list(_DTYPES)}")
    a = N.NormRopeArgs()
    a.q = _view(q, "q", (n, hq, t, d), dt, dev)
    a.k = _view(k, "k", (n, hkv, t, d), dt, dev)
    wd = None
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            wd = wd or w.dtype
            rows = w.shape[0] if w.dim() == 2 else 1
            if w.shape[-1:] != (d,) or wd not in _DTYPES or rows < 1 or n % rows or a.weight_rows not in (0, rows):
                raise ValueError(f"{name}: want [{d}] or [layers][{d}] of one of {list(_DTYPES)}, the same for "
                                 "both weights, layers dividing the batch")
            setattr(a, name, _vector(w, name, wd, dev, w.dim()))
            a.weight_rows = rows
    a.weight_rows = a.weight_rows or 1
    if omega.shape != (d // 2,):
        raise ValueError(f"omega: want [{d // 2}]")
    a.omega = _vector(omega, "omega", torch.float64, dev)
    a.position_layers = 1
    if isinstance(positions, torch.Tensor):
        a.positions = _vector(positions, "positions", _I32, dev, positions.dim() if positions.dim() == 2 else 1)
        if positions.shape[-1] != t:
            raise ValueError(f"positions: want {t} per row")
        if positions.dim() == 2 and positions.shape[0] != 1:
            if n and (positions.shape[0] == 0 or n % positions.shape[0]):
                raise ValueError(f"positions: {positions.shape[0]} rows do not divide a batch of {n}")
            a.position_stride, a.position_layers = t, max(1, n // max(1, positions.shape[0]))
    else:
        a.position0 = int(positions)
    a.layers = 1
    if out_rows is not None:
        a.out_rows, _, a.layers = _lengths(out_rows, n, dev)
        if k_out is None or (v is not None and v_out is None):
            raise ValueError("out_rows needs k_out (and v_out)")
    with _On(dev, stream) as st:
        a.status = _status_ptr(dev.index)
        if q_out is None:
            q_out = torch.empty((n, hq, t, d), dtype=dt, device=dev)
        if k_out is None:
            k_out = torch.empty((n, hkv, t, d), dtype=dt, device=dev)
        a.q_out = _view(q_out, "q_out", (n, hq, t, d), dt, dev)
        cap = k_out.shape[2] if k_out.dim() == 4 else -1
        a.k_out = _view(k_out, "k_out", (n, hkv, cap, d), dt, dev)
        if v is not None:
            a.v = _view(v, "v", (n, hkv, t, d), dt, dev)
            if v_out is None:
                v_out = torch.empty((n, hkv, cap, d), dtype=dt, device=dev)
            a.v_out = _view(v_out, "v_out", (n, hkv, cap, d), dt, dev)
        elif v_out is not None:
            raise ValueError("v_out without v")
        a.batch, a.q_heads, a.kv_heads, a.tokens, a.head_dim = n, hq, hkv, t, d
        a.out_capacity, a.dtype, a.weight_dtype, a.eps = cap, _DTYPES[dt], _DTYPES[wd or dt], eps
        N.check(N.load().statekv_norm_rope(C.byref(a), st), "statekv_norm_rope")
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def tree_attention(q, k_new, v_new, tree, k_cache, v_cache, lengths, *, scale: float, out=None,
                   workspace=None, stream=None):
    """Attention of drafted tokens q [n][Hq][tokens][d], k_new and v_new
    [n][Hkv][tokens][d] over the first `lengths` rows (int, or int32
    [sequences]) of k_cache and v_cache [n][Hkv][rows][d] and, among
    themselves, where tree (int64 masks [tokens] or [sequences][tokens], see
    tree_masks) says.  bf16.  Returns out like q.  workspace: a uint8 CUDA
    tensor of tree_attention_workspace() bytes (default: allocated)."""
    n, hq, tok, d = _shape4(q, "q")
    hkv, rows = _shape4(k_cache, "k_cache")[1:3]
    dev = q.device
    a = N.TreeArgs()
    a.q = _view(q, "q", (n, hq, tok, d), _BF16, dev)
    a.k_new = _view(k_new, "k_new", (n, hkv, tok, d), _BF16, dev)
    a.v_new = _view(v_new, "v_new", (n, hkv, tok, d), _BF16, dev)
    a.k_cache = _view(k_cache, "k_cache", (n, hkv, rows, d), _BF16, dev)
    a.v_cache = _view(v_cache, "v_cache", (n, hkv, rows, d), _BF16, dev)
    a.lengths, a.length, layers = _lengths(lengths, n, dev)
    dims = tree.dim()
    a.tree = _vector(tree, "tree", _I64, dev, dims if dims == 2 else 1)
    if tree.shape[-1] != tok:
        raise ValueError(f"tree: want {tok} masks per row")
    if dims == 2 and tree.shape[0] != 1:
        layers = _layers(layers, tree.shape[0], n, "tree")
        a.tree_stride = tok
    lib = N.load()
    with _On(dev, stream) as st:
        a.status = _status_ptr(dev.index)
        if out is None:
            out = torch.empty((n, hq, tok, d), dtype=_BF16, device=dev)
        a.out = _view(out, "out", (n, hq, tok, d), _BF16, dev)
        if workspace is None:
            size = lib.statekv_tree_attention_workspace(n, hq, hkv, tok, d)
            if size > 0:
                workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        if workspace is not None:
            a.workspace = _vector(workspace, "workspace", torch.uint8, dev)
            a.workspace_bytes = workspace.shape[0]
        a.scale, a.layers = scale, layers or 1
        a.batch, a.q_heads, a.kv_heads, a.tokens, a.head_dim, a.cache_rows = n, hq, hkv, tok, d, rows
        N.check(lib.statekv_tree_attention(C.byref(a), st), "statekv_tree_attention")
    return out


def tree_attention_workspace(batch: int, q_heads: int, kv_heads: int, tokens: int, head_dim: int) -> int:
    """Bytes of workspace tree_attention needs on the current device."""
    size = N.load().statekv_tree_attention_workspace(batch, q_heads, kv_heads, tokens, head_dim)
    if size < 0:
        raise N.StateKVError(N.E_UNSUPPORTED, "statekv_tree_attention_workspace")
    return size


def append_accepted(k_new, v_new, path, counts, k_cache, v_cache, lengths, *, stream=None):
    """Rows path (int32 [steps] or [sequences][steps]) of k_new and v_new
    [n][Hkv][tokens][d] become cache rows lengths + i, i < counts (int32
    [sequences], or None: all steps).  Returns the new lengths (int32
    [sequences], or an int where lengths is an int and counts None)."""
    n, hkv, tok, d = _shape4(k_new, "k_new")
    rows = _shape4(k_cache, "k_cache")[2]
    dev, dt = k_new.device, k_new.dtype
    if dt not in _DTYPES:
        raise ValueError(f"k_new: {dt}, want one of {list(_DTYPES)}")
    a = N.AppendArgs()
    a.k_new = _view(k_new, "k_new", (n, hkv, tok, d), dt, dev)
    a.v_new = _view(v_new, "v_new", (n, hkv, tok, d), dt, dev)
    a.k_cache = _view(k_cache, "k_cache", (n, hkv, rows, d), dt, dev)
    a.v_cache = _view(v_cache, "v_cache", (n, hkv, rows, d), dt, dev)
    a.lengths, a.length, layers = _lengths(lengths, n, dev)
    dims = path.dim()
    a.path = _vector(path, "path", _I32, dev, dims if dims == 2 else 1)
    a.path_len = path.shape[-1]
    if dims == 2 and path.shape[0] != 1:
        layers = _layers(layers, path.shape[0], n, "path")
        a.path_stride = a.path_len
    if counts is not None:
        a.counts = _vector(counts, "counts", _I32, dev)
        if layers and counts.shape[0] * layers != n:
            raise ValueError(f"counts: {counts.shape[0]} for {n // layers} sequences")
        layers = layers or _layers(0, counts.shape[0], n, "counts")
    layers = layers or 1
    with _On(dev, stream) as st:
        a.status = _status_ptr(dev.index)
        new = None
        if a.lengths or a.counts:
            new = torch.empty(n // layers, dtype=_I32, device=dev)
            a.new_lengths = new.data_ptr()
        a.layers, a.batch, a.kv_heads, a.tokens, a.head_dim = layers, n, hkv, tok, d
        a.cache_rows, a.dtype = rows, _DTYPES[dt]
        N.check(N.load().statekv_append_accepted(C.byref(a), st), "statekv_append_accepted")
    return int(lengths) + path.shape[-1] if new is None else new


def block_summaries(k_cache, codes, scales, lengths, *, appended: int | None = None, stream=None) -> None:
    """Brings codes (int8 [n][Hkv][blocks][d]) and scales (float32
    [n][Hkv][blocks]) up to date for the complete 64-row blocks of k_cache
    [n][Hkv][rows][d] that the last `appended` rows (None: all) of the first
    `lengths` completed.  blocks >= rows // 64."""
    n, hkv, rows, d = _shape4(k_cache, "k_cache")
    dev = k_cache.device
    a = N.SummaryArgs()
    a.k_cache = _view(k_cache, "k_cache", (n, hkv, rows, d), _BF16, dev)
    a.codes, a.scales, a.blocks = _summary_ptrs(codes, scales, n, hkv, d, dev)
    a.lengths, a.length, layers = _lengths(lengths, n, dev)
    a.appended = rows if appended is None else min(int(appended), rows)
    with _On(dev, stream) as st:
        a.status = _status_ptr(dev.index)
        a.layers, a.batch, a.kv_heads, a.head_dim, a.cache_rows = layers or 1, n, hkv, d, rows
        N.check(N.load().statekv_block_summaries(C.byref(a), st), "statekv_block_summaries")


def _summary_ptrs(codes, scales, n: int, hkv: int, d: int, dev) -> tuple[int, int, int]:
    pc = _vector(codes, "codes", torch.int8, dev, 4)
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
    n, hq, tok, d = _shape4(q, "q")
    hkv, rows = _shape4(k_cache, "k_cache")[1:3]
    dev, top = q.device, int(top)
    a = N.SparseArgs()
    a.q = _view(q, "q", (n, hq, tok, d), _BF16, dev)
    a.k_cache = _view(k_cache, "k_cache", (n, hkv, rows, d), _BF16, dev)
    a.v_cache = _view(v_cache, "v_cache", (n, hkv, rows, d), _BF16, dev)
    a.codes, a.scales, a.blocks = _summary_ptrs(codes, scales, n, hkv, d, dev)
    a.lengths, a.length, layers = _lengths(lengths, n, dev)
    with _On(dev, stream) as st:
        a.status = _status_ptr(dev.index)
        if out is None:
            out = torch.empty((n, hq, tok, d), dtype=_BF16, device=dev)
        a.out = _view(out, "out", (n, hq, tok, d), _BF16, dev)
        if selected is None:
            selected = torch.empty((n, hkv, tok, max(0, top)), dtype=_I32, device=dev)
        elif selected.shape != (n, hkv, tok, top):
            raise ValueError(f"selected: want {(n, hkv, tok, top)}, got {tuple(selected.shape)}")
        a.selected = _vector(selected, "selected", _I32, dev, 4)
        a.scale, a.top, a.layers = scale, top, layers or 1
        a.batch, a.q_heads, a.kv_heads, a.tokens, a.head_dim, a.cache_rows = n, hq, hkv, tok, d, rows
        N.check(N.load().statekv_sparse_attention(C.byref(a), st), "statekv_sparse_attention")
    return out, selected

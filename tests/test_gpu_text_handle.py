"""The handle's text operators over its detailed state D: per-head norm in
every rotation, tree verification and acceptance, block-sparse decode.

Rotated values are checked against fp64 within half a bf16 step of the result
and 2^-20 of the pair's magnitude (fp32 arithmetic); attention outputs against
fp64 attention over the GPU's own D rows and rotated queries, within the bf16
roundings of P and of the output (2^-8 of A = sum p |v| / sum p and of the
value, and 2^-12 A for fp32 scores)."""

import pytest
import torch

import kv_cache_compression_frame_gb300 as kv
import oracle.statekv_oracle as orc
from test_text_ops import DEV, check_sparse, gen, randn, ref_attend, ref_summaries, seen, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_compression_frame_gb300 import build_lib
    build_lib.build()


def handle(**over):
    cfg = dict(num_q_heads=6, num_kv_heads=2, head_dim=128, frame_tokens=64, budget=96, max_frames=6, num_streams=2,
               num_layers=3, rope_theta=1e6, rope_alpha=4.0, rope_orig_ctx=128, position_offset=1000)
    cfg.update(over)
    h = kv.StateKV(kv.StateKVConfig(**cfg))
    om, ms = orc.rope_frequencies(cfg["head_dim"], cfg["rope_theta"], cfg["rope_alpha"], cfg["rope_orig_ctx"])
    h.omega64 = torch.tensor(om, dtype=torch.float64, device=DEV)
    h.scale64 = orc.logit_scale(cfg["head_dim"], ms)
    return h


def text(h, g, tok):
    c = h.cfg
    return [randn(g, c.num_streams, c.num_layers, n, tok, c.head_dim, dtype=h.torch_dtype)
            for n in (c.num_q_heads, c.num_kv_heads, c.num_kv_heads)]


def rotated(x, pos, omega, w=None, eps=0.0):
    """x [S][L][H][t][d], pos [S][t], w [L][d]: fp64 result and pair magnitude."""
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()[None, :, None, None, :]
    a, b = x.chunk(2, -1)
    ang = pos.double()[:, None, None, :, None] * omega
    return (torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1),
            (a.abs() + b.abs()).repeat(1, 1, 1, 1, 2))


def check_rotated(got, x, pos, omega, w=None, eps=0.0):
    ref, mag = rotated(x, pos, omega, w, eps)
    within(got, ref, torch.finfo(got.dtype).eps / 2 * ref.abs() + 2.0 ** -20 * mag)


def rows_of(h, name):
    """D's keys or values as [S][L][Hkv][pitch][d]."""
    c = h.cfg
    return torch.stack([torch.stack([h.detailed(s, l)[0 if name == "k" else 1] for l in range(c.num_layers)])
                        for s in range(c.num_streams)])


def check_attention(h, q_rot, k, v, mask, o):
    """q_rot, o [S][L][Hq][t][d] over k, v [S][L][Hkv][m][d] with mask [S][t][m]."""
    c = h.cfg
    G, d = c.num_q_heads // c.num_kv_heads, c.head_dim
    for s in range(c.num_streams):
        for l in range(c.num_layers):
            for hk in range(c.num_kv_heads):
                sl = slice(hk * G, hk * G + G)
                ref, a = ref_attend(q_rot[s, l, sl].reshape(-1, d), k[s, l, hk], v[s, l, hk],
                                    mask[s].repeat(G, 1), h.scale64)
                within(o[s, l, sl].reshape(-1, d), ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a,
                       f"unit {s} {l} {hk}")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
def test_qk_norm_in_prefill_and_decode(dtype, d):
    h = handle(dtype=dtype, head_dim=d)
    c, g = h.cfg, gen(1)
    plain = handle(dtype=dtype, head_dim=d)
    qw, kw = (1 + randn(g, c.num_layers, d, dtype=torch.float32) / 4 for _ in range(2))
    h.set_qk_norm(qw, kw, 1e-5)
    T = c.frame_tokens
    for n in range(3):
        q, k, v = (3 * x for x in text(h, g, T))
        o = h.prefill_frame(q, k, v)
        h.check_device_status()
        pos = (c.position_offset + n * T + torch.arange(T, device=DEV)).expand(c.num_streams, T)
        check_rotated(h.rotated_query(), q, pos, h.omega64, qw, 1e-5)
        check_rotated(rows_of(h, "k")[..., n * T:(n + 1) * T, :], k, pos, h.omega64, kw, 1e-5)
        assert torch.equal(rows_of(h, "v")[..., n * T:(n + 1) * T, :], v)
        assert o.isfinite().all()
    if dtype == "bf16" and d == 128:
        q, k, v = text(h, g, 4)
        q_in = q.clone()
        h.decode(q, k, v)
        pos = (c.position_offset + 3 * T + torch.arange(4, device=DEV)).expand(c.num_streams, 4)
        qr = h.rotated_query().reshape(-1)[:q.numel()].view(q.shape)
        check_rotated(qr, q_in, pos, h.omega64, qw, 1e-5)
    # off again: bit-equal to a handle that never had it
    h.set_qk_norm(None, None)
    h.reset()
    q, k, v = text(h, g, T)
    assert torch.equal(h.prefill_frame(q, k, v), plain.prefill_frame(q, k, v))
    assert torch.equal(h.rotated_query(), plain.rotated_query())


@pytest.mark.parametrize("shape", [(), (1,), (3, 1), (1, 128), (3, 1, 128), (128, 3)])
def test_qk_norm_weights_of_other_shapes_are_refused(shape):
    h = handle()
    right, wrong = torch.ones(128), torch.ones(shape)
    with pytest.raises(ValueError, match="q_weight"):
        h.set_qk_norm(wrong, right)
    with pytest.raises(ValueError, match="k_weight"):
        h.set_qk_norm(right, wrong)
    h.set_qk_norm(right, right.expand(3, 128))


@pytest.mark.parametrize("d,norm", [(128, False), (128, True), (64, True)])
def test_tree_step_and_acceptance(d, norm):
    h = handle(head_dim=d)
    c, g = h.cfg, gen(2)
    qw = kw = None
    if norm:
        qw, kw = (1 + randn(g, c.num_layers, d, dtype=torch.float32) / 4 for _ in range(2))
        h.set_qk_norm(qw, kw)
    for n in range(4):
        h.prefill_frame(*text(h, g, c.frame_tokens))
    parents = [[-1, 0, 0, 1, 1, 2, 5, 5, 3], [-1, 0, 1, 2, 3, 4, 5, 6, 7]]
    tree, depth = kv.tree_masks(parents, DEV)
    paths = [torch.tensor([[0, 2, 5], [0, 1, 2]], dtype=torch.int32, device=DEV),
             torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=DEV)]
    first = 4 * c.frame_tokens
    for path in paths:
        q, k, v = text(h, g, 9)
        dk, dv = rows_of(h, "k"), rows_of(h, "v")
        o = h.decode_tree(q, k, v, tree, depth)
        h.check_device_status()
        again = h.decode_tree(q, k, v, tree, depth)
        assert torch.equal(o, again)
        # D as it was
        assert torch.equal(rows_of(h, "k"), dk) and torch.equal(rows_of(h, "v"), dv)
        assert h.frame_index == 4 and h.detailed(0, 0)[2] == first
        pos = c.position_offset + first + depth
        qr = h.rotated_query().reshape(-1)[:q.numel()].view(q.shape).clone()
        check_rotated(qr, q, pos, h.omega64, qw, 1e-6)
        h.accept(path)
        h.check_device_status()
        cnt = path.shape[1]
        assert h.detailed(0, 0)[2] == first + cnt
        nk, nv = rows_of(h, "k"), rows_of(h, "v")
        at = path.long()[:, None, None, :, None].expand(*k.shape[:3], cnt, d)
        check_rotated(nk[..., first:first + cnt, :], k.gather(3, at), pos.gather(1, path.long()), h.omega64, kw, 1e-6)
        assert torch.equal(nv[..., first:first + cnt, :], v.gather(3, at))
        nk[..., first:first + cnt, :], nv[..., first:first + cnt, :] = \
            dk[..., first:first + cnt, :], dv[..., first:first + cnt, :]
        assert torch.equal(nk, dk) and torch.equal(nv, dv)
        # the step's output over the drafted keys as the handle-free operator
        # rotates them (the same kernel; its values are checked above)
        kf = k.flatten(0, 1)
        kr = kv.qk_norm_rope(kf, kf, pos.repeat_interleave(c.num_layers, 0).to(torch.int32), h.omega64, kw, kw)[1]
        kr = kr.view(k.shape)
        mask = torch.cat([torch.ones(2, 9, first, dtype=torch.bool, device=DEV), seen(tree, 9)], 2)
        check_attention(h, qr, torch.cat([dk[..., :first, :], kr], 3), torch.cat([dv[..., :first, :], v], 3), mask, o)
        first += cnt
    # text continues after the accepted rows
    assert h.text_tokens == 5


def test_tree_rules():
    h = handle(max_frames=2)
    c, g = h.cfg, gen(3)
    path = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    tree, depth = kv.tree_masks([[-1, 0, 1]] * 2, DEV)
    x = text(h, g, 3)
    with pytest.raises(kv.StateKVError) as e:
        h.accept(path)                                # nothing drafted
    assert e.value.status == -1
    h.decode_tree(*x, tree, depth)                    # before any frame: only the tree
    h.accept(path[:, :0])                             # dropped
    with pytest.raises(kv.StateKVError):
        h.accept(path)
    h.decode_tree(*x, tree, depth)
    with pytest.raises(kv.StateKVError):
        h.accept(torch.zeros(2, 4, dtype=torch.int32, device=DEV))    # more than drafted
    h.prefill_frame(*text(h, g, c.frame_tokens))      # a frame drops the draft
    with pytest.raises(kv.StateKVError):
        h.accept(path)
    h.prefill_frame(*text(h, g, c.frame_tokens))      # D is full
    o = h.decode_tree(*x, tree, depth)
    assert o.isfinite().all()
    with pytest.raises(kv.StateKVError) as e:
        h.accept(path)
    assert e.value.status == -3
    h.reset()
    h.decode_tree(*x, tree, depth)
    before = rows_of(h, "k")
    h.accept(torch.tensor([[0, 3], [0, -1]], dtype=torch.int32, device=DEV))   # no such nodes
    with pytest.raises(kv.StateKVError) as e:
        h.check_device_status()
    assert e.value.status == -7
    after = rows_of(h, "k")
    assert torch.equal(after[..., 1, :], before[..., 1, :])
    with pytest.raises(ValueError, match="depth"):
        h.decode_tree(*x, tree, depth[:1])
    with pytest.raises(kv.StateKVError) as e:
        h.accept(path)                                # taken over already
    assert e.value.status == -1
    f = handle(dtype="f32", num_streams=1)
    with pytest.raises(kv.StateKVError) as e:
        f.decode_tree(*text(f, g, 3), tree[:1].contiguous(), depth[:1].contiguous())
    assert e.value.status == -2


@pytest.mark.parametrize("restart", [False, True])
@pytest.mark.parametrize("frames,merged", [(6, False), (20, True)])
def test_a_frame_behind_a_tree_step_waits_for_it(frames, merged, restart):
    """The rotation of a frame rewrites Q' and, after a restart, D's first rows:
    the tree step enqueued just before still reads them as they were.  Short
    caches have no merging kernel between the two."""
    h = handle(max_frames=frames, num_layers=4)
    c, g = h.cfg, gen(20)
    T = c.frame_tokens
    assert (frames * T > 896) == merged
    frame = text(h, g, T)
    out = [torch.empty(h.q_shape, dtype=h.torch_dtype, device=DEV) for _ in range(2)]
    tok = 21                                          # more than one copy of Q per thread
    tree, depth = kv.tree_masks([[-1] + list(range(tok - 1))] * 2, DEV)
    x = text(h, g, tok)
    rows = [text(h, g, T) for _ in range(frames - 1)]
    o = torch.empty_like(x[0])

    def step(wait):
        h.reset()
        for r in rows:
            h.prefill_frame(*r, out[0])
        torch.cuda.synchronize()
        h.decode_tree(*x, tree, depth, o=o)
        if wait:
            torch.cuda.synchronize()
        if restart:
            h.reset()
        h.prefill_frame(*frame, out[1])
        torch.cuda.synchronize()
        return o.clone(), out[1].clone()

    want = step(True)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(step(False), want))
    h.check_device_status()


def test_first_calls_on_a_stream_of_their_own():
    """Buffers allocated on first use hold what the call's stream writes, whatever
    is pending on the default stream."""
    g = gen(21)
    outs = []
    for side in (False, True):
        g.manual_seed(21)
        h = handle(max_frames=20)
        c, T = h.cfg, h.cfg.frame_tokens
        qw, kw = (1 + randn(g, c.num_layers, c.head_dim, dtype=torch.float32) / 4 for _ in range(2))
        frames = [text(h, g, T) for _ in range(18)]
        xs = [text(h, g, tok) for tok in (1, 4, 2, 3)]
        tree, depth = kv.tree_masks([[-1, 0, 0, 2]] * 2, DEV)
        path = torch.tensor([[0, 2], [0, 1]], dtype=torch.int32, device=DEV)
        got = []

        def run():
            h.set_qk_norm(qw, kw)
            for f in frames:
                h.prefill_frame(*f)
            got.append(h.decode_sparse(*xs[0], 3))
            got.append(h.decode_tree(*xs[1], tree, depth))
            h.accept(path)
            got.append(h.decode(*xs[2]))
            got.append(h.decode_sparse(*xs[3], 3))

        torch.cuda.synchronize()
        if side:
            torch.cuda._sleep(400_000_000)            # about 0.2 s of the default stream
            with torch.cuda.stream(torch.cuda.Stream()):
                run()
        else:
            run()
        torch.cuda.synchronize()
        got += [h.decode_sparse(*xs[3], 3), rows_of(h, "k"), rows_of(h, "v")]
        h.check_device_status()
        outs.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert all(o.float().abs().sum() > 0 for o in outs[0])


@pytest.mark.parametrize("d", [64, 128])
def test_sparse_decode(d):
    """After frames, after decoded text and after an accepted draft; the same
    bits as the handle-free operators over D."""
    h = handle(head_dim=d, max_frames=12, frame_tokens=100)
    c, g = h.cfg, gen(4)
    for n in range(9):
        h.prefill_frame(*text(h, g, 100))
    tree, depth = kv.tree_masks([[-1, 0, 1, 2]] * 2, DEV)
    rows = 900
    for step, tok in enumerate((1, 5, 70, 3)):
        q, k, v = text(h, g, tok)
        o = h.decode_sparse(q, k, v, 4)
        h.check_device_status()
        pos = (c.position_offset + rows + torch.arange(tok, device=DEV)).expand(2, tok)
        qr = h.rotated_query().reshape(-1)[:q.numel()].view(q.shape).clone()
        check_rotated(qr, q, pos, h.omega64)
        dk, dv = rows_of(h, "k"), rows_of(h, "v")
        check_rotated(dk[..., rows:rows + tok, :], k, pos, h.omega64)
        rows += tok
        assert h.detailed(0, 0)[2] == rows
        flat = [x.flatten(0, 1).contiguous() for x in (qr, dk, dv)]
        codes, scales = ref_summaries(flat[1][:, :, :c.max_frames * 100 // 64 * 64])
        got, sel = kv.sparse_attention(*flat, codes, scales, rows, 4, scale=h.scale64)
        assert torch.equal(got.view(o.shape), o)
        if step < 2:
            check_sparse(*flat, codes, scales, rows, 4, h.scale64, got, sel)
        if step == 1:                                   # rows that come in another way
            h.decode_tree(*text(h, g, 4), tree, depth)
            h.accept(torch.tensor([[0, 1, 2], [0, 1, 2]], dtype=torch.int32, device=DEV))
            rows += 3
    # enough blocks: every row, as in dense decode
    q, k, v = text(h, g, 2)
    o = h.decode_sparse(q, k, v, 64)
    qr = h.rotated_query().reshape(-1)[:q.numel()].view(q.shape).clone()
    rows += 2
    mask = (torch.arange(rows, device=DEV) <= rows - 2 + torch.arange(2, device=DEV)[:, None]).expand(2, 2, rows)
    check_attention(h, qr, rows_of(h, "k")[..., :rows, :], rows_of(h, "v")[..., :rows, :], mask, o)
    # after a reset the summaries are built anew
    h.reset()
    for n in range(7):
        h.prefill_frame(*text(h, g, 100))
    q, k, v = text(h, g, 1)
    o = h.decode_sparse(q, k, v, 3)
    flat = [x.flatten(0, 1).contiguous() for x in
            (h.rotated_query().reshape(-1)[:q.numel()].view(q.shape), rows_of(h, "k"), rows_of(h, "v"))]
    codes, scales = ref_summaries(flat[1][:, :, :c.max_frames * 100 // 64 * 64])
    assert torch.equal(kv.sparse_attention(*flat, codes, scales, 701, 3, scale=h.scale64)[0].view(o.shape), o)
    with pytest.raises(kv.StateKVError) as e:
        h.decode_sparse(*text(h, g, 1), 1025)
    assert e.value.status == -2
    with pytest.raises(kv.StateKVError):
        h.decode_sparse(*text(h, g, 1), 0)
    f = handle(dtype="f32", num_streams=1)
    with pytest.raises(kv.StateKVError) as e:
        f.decode_sparse(*text(f, g, 1), 4)
    assert e.value.status == -2


def test_tree_step_captured_on_another_stream():
    """After a first call (which allocates), a tree step can be captured."""
    h = handle()
    c, g = h.cfg, gen(5)
    for n in range(5):
        h.prefill_frame(*text(h, g, c.frame_tokens))
    tree, depth = kv.tree_masks([[-1, 0, 0, 2]] * 2, DEV)
    x = text(h, g, 4)
    want = h.decode_tree(*x, tree, depth)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        h.decode_tree(*x, tree, depth, o=out)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        for t in x:
            t.copy_(randn(g, *t.shape))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        assert torch.equal(out, h.decode_tree(*x, tree, depth))
    h.check_device_status()

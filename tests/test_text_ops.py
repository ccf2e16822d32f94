"""The text operators against their definitions in 64 bits: per-head norm with
rotation, attention of drafted trees, the accepted path's append, block
summaries, and a chain of them.

Tolerances, all derived beforehand.
 * Stored values: half a step of the storage type, 2^-8 |x| (bf16) or 2^-24
   |x| (fp32).
 * norm_rope adds the fp32 arithmetic: a result is a sum of two products of
   norm factor (rsqrtf, two ulp), weight and cosine (two ulp, angle rounded to
   2^-24 half turns): below 2^-20 of the pair's magnitude |y_k| + |y_k+h|.
 * Attention with P rounded to bf16: each term p v is off by at most 2^-8 of
   itself, so the output by 2^-8 A with A = sum p |v| / sum p.  Scores are sums
   of 128 exact products in fp32, each step at worst 2^-23 of sum |q k| scale
   (about 7 here): 1.1e-4 on the exponent, twice that on a quotient: 2^-12 A.
"""

import ctypes as C
import math

import pytest
import torch

import kv_cache_compression_frame_gb300 as kv
from kv_cache_compression_frame_gb300 import _native as N

gpu = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kv_cache_compression_frame_gb300 import build_lib
    build_lib.build()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def within(got, ref, tol, what=""):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    bad &= ~(got.isnan() & ref.isnan()) & ~((got == ref) & ref.isinf())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, worst "
                           f"{float((got - ref).abs()[bad].max()):.3g}")


# ---------------------------------------------------------------- norm_rope
def ref_norm_rope(x, pos, omega, w, eps):
    """x [n][H][t][d], pos [n][t]: the result and each pair's magnitude."""
    x = x.double()
    h = x.shape[-1] // 2
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    a, b = x[..., :h], x[..., h:]
    ang = pos.double()[:, None, :, None] * omega
    c, s = ang.cos(), ang.sin()
    return torch.cat([a * c - b * s, b * c + a * s], -1), (a.abs() + b.abs()).repeat(1, 1, 1, 2)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def omega_of(d, theta=1e6):
    return theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)


@gpu
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("n,hq,hkv,t,d", [(1, 16, 8, 1, 128), (1, 14, 2, 3, 64), (3, 5, 1, 33, 128),
                                          (4, 12, 2, 256, 128), (2, 1, 1, 7, 64)])
def test_norm_rope_projection_layout(dtype, n, hq, hkv, t, d):
    """Heads of q, k and v side by side, tokens outermost; far positions."""
    g = gen(n * 100 + t)
    qkv = 3 * randn(g, n, t, hq + 2 * hkv, d, dtype=dtype)
    q, k, v = (x.transpose(1, 2) for x in qkv.split([hq, hkv, hkv], 2))
    qw, kw = (1 + randn(g, d, dtype=dtype) / 4 for _ in range(2))
    pos = torch.randint(0, 1 << 20, (n, t), generator=g, device=DEV).to(torch.int32)
    omega = omega_of(d)
    qo, ko, vo = kv.qk_norm_rope(q, k, pos, omega, qw, kw, v=v, eps=1e-5)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        ref, mag = ref_norm_rope(x, pos, omega, w, 1e-5)
        within(got, ref, half_step(dtype) * ref.abs() + 2.0 ** -20 * mag)
    assert torch.equal(vo, v)
    kv.check_status()


@gpu
def test_norm_rope_positions_weights_and_zero_rows():
    g = gen(5)
    q, k = randn(g, 2, 4, 9, 64), randn(g, 2, 2, 9, 64)
    q[0, 1, 3] = 0                                   # a zero row stays zero
    w = 1 + randn(g, 64, dtype=torch.float32) / 4    # fp32 weights with bf16 tensors
    omega = omega_of(64)
    for first in (0, -3, 131072, (1 << 31) - 20):
        pos = first + torch.arange(9, device=DEV)
        got = {"int": kv.qk_norm_rope(q, k, first, omega, w, None)}
        got["row"] = kv.qk_norm_rope(q, k, pos.to(torch.int32), omega, w, None)
        got["rows"] = kv.qk_norm_rope(q, k, pos.to(torch.int32).expand(2, 9).contiguous(), omega, w, None)
        for qo, ko in got.values():
            # fp64 p * omega itself is off by 2^-53 p
            far = 2.0 ** -52 * (abs(first) + 9)
            ref, mag = ref_norm_rope(q, pos.expand(2, 9), omega, w, 1e-6)
            within(qo, ref, 2.0 ** -8 * ref.abs() + (2.0 ** -20 + far) * mag, f"q at {first}")
            ref, mag = ref_norm_rope(k, pos.expand(2, 9), omega, None, 0)   # no norm: rotation alone
            within(ko, ref, 2.0 ** -8 * ref.abs() + (2.0 ** -20 + far) * mag, f"k at {first}")
            assert torch.equal(qo[0, 1, 3], torch.zeros_like(qo[0, 1, 3]))


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, torch.float32), (torch.float32, torch.float32)])
def test_norm_rope_weights_per_layer(dtype, wdtype):
    g = gen(7)
    seqs, layers, t, d = 2, 3, 6, 64
    q, k = randn(g, seqs * layers, 3, t, d, dtype=dtype), randn(g, seqs * layers, 2, t, d, dtype=dtype)
    qw, kw = (1 + randn(g, layers, d, dtype=wdtype) / 4 for _ in range(2))
    pos = torch.randint(0, 5000, (t,), generator=g, device=DEV).to(torch.int32)
    qo, ko = kv.qk_norm_rope(q, k, pos, omega_of(d), qw, kw)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        for n in range(seqs * layers):
            ref, mag = ref_norm_rope(x[n:n + 1], pos[None], omega_of(d), w[n % layers], 1e-6)
            within(got[n:n + 1], ref, half_step(dtype) * ref.abs() + 2.0 ** -20 * mag)
    with pytest.raises(ValueError, match="weight"):
        kv.qk_norm_rope(q, k, pos, omega_of(d), qw, kw[:2].contiguous())


@gpu
def test_norm_rope_weights_of_other_shapes_are_refused():
    g = gen(63)
    q, k, om = randn(g, 4, 2, 3, 64), randn(g, 4, 1, 3, 64), omega_of(64)
    for shape in ((2, 1, 64), (1, 1, 64), (1,), (4, 1), (3, 64), (0, 64), (2, 128), ()):
        w = torch.ones(shape, dtype=BF16, device=DEV)
        with pytest.raises(ValueError, match="q_weight"):
            kv.qk_norm_rope(q, k, 0, om, w)
        with pytest.raises(ValueError, match="k_weight"):
            kv.qk_norm_rope(q, k, 0, om, None, w)


@gpu
def test_norm_rope_into_a_cache_and_in_place():
    """K and V land at each sequence's rows; every other row stays as it was."""
    g = gen(6)
    seqs, layers, t, d = 3, 2, 5, 128
    n = seqs * layers
    q, k, v = randn(g, n, 4, t, d), randn(g, n, 2, t, d), randn(g, n, 2, t, d)
    kc, vc = randn(g, n, 2, 40, d), randn(g, n, 2, 40, d)
    kc0, vc0 = kc.clone(), vc.clone()
    rows = torch.tensor([0, 35, 17], dtype=torch.int32, device=DEV)
    pos = (rows[:, None] + torch.arange(t, device=DEV)).to(torch.int32)
    w = 1 + randn(g, d) / 4
    q0 = q.clone()
    ref, mag = ref_norm_rope(k, pos.repeat_interleave(layers, 0), omega_of(d), w, 1e-6)
    out = kv.qk_norm_rope(q, k, pos, omega_of(d), w, w, v=v, q_out=q, k_out=kc, v_out=vc, out_rows=rows)
    assert out[0] is q and out[1] is kc
    for i in range(n):
        r = int(rows[i // layers])
        within(kc[i, :, r:r + t], ref[i], 2.0 ** -8 * ref[i].abs() + 2.0 ** -20 * mag[i])
        assert torch.equal(vc[i, :, r:r + t], v[i])
        kc[i, :, r:r + t], vc[i, :, r:r + t] = kc0[i, :, r:r + t], vc0[i, :, r:r + t]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    ref, mag = ref_norm_rope(q0, pos.repeat_interleave(layers, 0), omega_of(d), w, 1e-6)
    within(q, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag)
    kv.check_status()
    # rows that do not fit: recorded, and nothing of that sequence is stored
    kv.qk_norm_rope(q, k, pos, omega_of(d), w, w, v=v, k_out=kc, v_out=vc,
                    out_rows=torch.tensor([36, -1, 40], dtype=torch.int32, device=DEV))
    with pytest.raises(kv.StateKVError) as e:
        kv.check_status()
    assert e.value.status == N.E_DEVICE
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    kv.check_status()                                # cleared


# --------------------------------------------------------------------- tree
def seen(tree, tok):
    """int64 masks [..., tok] -> bool [..., tok, tok]"""
    return ((tree[..., None] >> torch.arange(tok, device=tree.device)) & 1).bool()


def ref_attend(q, k, v, mask, scale):
    """One unit: q [r][d], k, v [m][d], mask [r][m] -> output and A.  A key that
    is masked contributes nothing whatever it holds."""
    x = (q.double() @ k.double().T) * scale
    x = torch.where(mask, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.where(mask, torch.exp(x - torch.where(top == -math.inf, 0.0, top)), 0.0)
    den = p.sum(-1, keepdim=True)
    den = torch.where(mask.any(-1, keepdim=True), den, 1.0)
    v = v.double()
    if not bool(v.isfinite().all()):
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        for r in range(q.shape[0]):
            o[r] = (p[r, mask[r], None] * v[mask[r]]).sum(0) / den[r]
        return o, o.nan_to_num(0, 0, 0).abs() + 8
    return p @ v / den, p @ v.abs() / den


def check_tree(q, kn, vn, tree, kc, vc, lengths, scale, got, what=""):
    n, hq, tok, d = q.shape
    hkv = kc.shape[1]
    G = hq // hkv
    for i in range(n):
        rows = lengths if isinstance(lengths, int) else int(lengths[i * len(lengths) // n])
        mask = seen(tree if tree.dim() == 1 else tree[i * tree.shape[0] // n], tok)
        mask = torch.cat([torch.ones(tok, rows, dtype=torch.bool, device=DEV), mask], 1).repeat(G, 1)
        for h in range(hkv):
            ref, a = ref_attend(q[i, h * G:(h + 1) * G].reshape(-1, d), torch.cat([kc[i, h, :rows], kn[i, h]]),
                                torch.cat([vc[i, h, :rows], vn[i, h]]), mask, scale)
            within(got[i, h * G:(h + 1) * G].reshape(-1, d), ref,
                   2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a, f"{what} entry {i} head {h}")


def random_tree(tok, seqs, seed):
    import random
    r = random.Random(seed)
    return kv.tree_masks([[-1] + [r.randrange(max(0, i - 4), i) for i in range(1, tok)] for _ in range(seqs)],
                         DEV)[0]


def tree_inputs(seed, n, hq, hkv, tok, d, cap):
    g = gen(seed)
    return (randn(g, n, hq, tok, d), randn(g, n, hkv, tok, d), randn(g, n, hkv, tok, d),
            randn(g, n, hkv, cap, d), randn(g, n, hkv, cap, d))


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,tok,rows", [
    (1, 1, 1, 0), (1, 1, 1, 1), (4, 2, 3, 127), (4, 2, 5, 128), (14, 2, 7, 129), (14, 2, 7, 300),
    (12, 2, 16, 2000),           # 96 rows
    (2, 1, 64, 700),             # 128 rows: the last size of one row tile
    (3, 1, 43, 513),             # 129 rows: two tiles, one live row in the second
    (12, 2, 42, 5000),           # 252 rows
    (4, 1, 64, 256),             # 256 rows
    (8, 1, 33, 400),             # 264 rows: two row blocks
    (16, 1, 64, 1000),           # 1024 rows: four
])
def test_tree_sizes(d, hq, hkv, tok, rows):
    x = tree_inputs(rows * 7 + tok, 2, hq, hkv, tok, d, rows + 3)
    tree = random_tree(tok, 2, rows)
    scale = 1 / math.sqrt(d)
    got = kv.tree_attention(*x[:3], tree, *x[3:], rows, scale=scale)
    check_tree(*x[:3], tree, *x[3:], rows, scale, got)
    kv.check_status()


@gpu
@pytest.mark.parametrize("layers", [1, 3])
def test_tree_ragged_lengths(layers):
    lens = [0, 1, 900, 128, 4097, 64, 255]
    n = len(lens) * layers
    x = tree_inputs(3, n, 4, 2, 9, 128, 4100)
    tree = random_tree(9, len(lens), 1)
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = kv.tree_attention(*x[:3], tree, *x[3:], lengths, scale=0.09)
    check_tree(*x[:3], tree, *x[3:], lengths, 0.09, got)
    kv.check_status()
    again = kv.tree_attention(*x[:3], tree, *x[3:], lengths, scale=0.09)
    assert torch.equal(got, again)


@gpu
@pytest.mark.parametrize("hq,tok", [(16, 32), (16, 43), (32, 64)])    # 64, 86 and 256 rows
def test_tree_long_ragged_caches(hq, tok):
    """A CTA's share holds the end of one long unit and the start of the next."""
    n = 16
    lengths = torch.randint(3000, 20000, (n,), generator=gen(2), device=DEV).to(torch.int32)
    x = tree_inputs(5, n, hq, 8, tok, 128, 20000)
    tree = random_tree(tok, n, 1)
    got = [kv.tree_attention(*x[:3], tree, *x[3:], lengths, scale=0.09) for _ in range(10)]
    check_tree(*x[:3], tree, *x[3:], lengths, 0.09, got[0])
    for o in got[1:]:
        assert torch.equal(o, got[0])


@gpu
def test_tree_many_sequences():
    """More sequences than a warp's lanes, more units than SMs."""
    n = 70
    lengths = torch.randint(0, 600, (n,), generator=gen(1), device=DEV).to(torch.int32)
    x = tree_inputs(4, n, 6, 3, 4, 64, 600)
    tree = random_tree(4, n, 1)
    got = kv.tree_attention(*x[:3], tree, *x[3:], lengths, scale=0.125)
    check_tree(*x[:3], tree, *x[3:], lengths, 0.125, got)


@gpu
@pytest.mark.parametrize("tok,hq", [(6, 4), (40, 8)])
def test_tree_masked_places_may_hold_anything(tok, hq):
    """Stale rows past the length, masked nodes and rows that see nothing."""
    rows = 200
    q, kn, vn, kc, vc = tree_inputs(8, 2, hq, 2, tok, 128, rows + 60)
    for c in (kc, vc):
        c[:, :, rows:] = float("nan")
        c[0, :, rows + 1] = float("inf")
    tree = random_tree(tok, 2, 3)
    tree[:, 4] = 0                                    # sees no node, only the cache
    # node 2 is seen by itself alone; its key and value are not numbers
    tree &= ~(1 << 2)
    tree[:, 2] |= 1 << 2
    kn[:, :, 2] = float("nan")
    vn[:, 0, 2, 5] = float("inf")
    vn[:, 1, 2] = float("nan")
    # a value of a node that others see too
    vn[1, 0, 1, 7] = -float("inf")
    tree[:, 3] |= 1 << 1
    got = kv.tree_attention(q, kn, vn, tree, kc, vc, rows, scale=0.1)
    G = hq // 2
    out = got.view(2, 2, G, tok, 128)
    assert out[:, :, :, 2].isnan().all()
    mask = seen(tree, tok)
    for i in range(2):
        for j in range(tok):
            if j == 2:
                continue
            o = out[i, :, :, j].clone()
            if i == 1 and mask[1, j, 1]:
                assert (o[0, :, 7] == -math.inf).all()
                o[0, :, 7] = 0
            assert o.isfinite().all(), (i, j)
    # the finite rows against the definition
    keep = [j for j in range(tok) if j != 2]
    vn2 = vn.nan_to_num(0, 0, 0)
    vn2[1, 0, 1, 7] = 0
    kn2 = kn.nan_to_num(0)
    # rows that see node 2 are left out, so its key and value do not matter
    ref = torch.zeros_like(out).double()
    a = torch.zeros_like(ref)
    for i in range(2):
        for h in range(2):
            m = torch.cat([torch.ones(tok, rows, dtype=torch.bool, device=DEV), mask[i]], 1).repeat(G, 1)
            r, aa = ref_attend(q[i, h * G:(h + 1) * G].reshape(-1, 128), torch.cat([kc[i, h, :rows], kn2[i, h]]),
                               torch.cat([vc[i, h, :rows], vn2[i, h]]), m, 0.1)
            ref[i, h], a[i, h] = r.view(G, tok, 128), aa.view(G, tok, 128)
    o = out.clone()
    o[1, 0, ..., 7] = ref[1, 0, ..., 7].to(BF16)
    within(o[:, :, :, keep], ref[:, :, :, keep], (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a)[:, :, :, keep])
    # nothing at all to see: zeros
    tree = torch.zeros(tok, dtype=torch.int64, device=DEV)
    got = kv.tree_attention(q, kn, vn, tree, kc, vc, 0, scale=0.1)
    assert torch.equal(got, torch.zeros_like(got))
    kv.check_status()


@gpu
def test_tree_large_scores_and_order():
    """Rising maxima (the reference is raised many times) and a huge common part."""
    tok, rows, d = 5, 1500, 64
    q, kn, vn, kc, vc = tree_inputs(9, 1, 4, 2, tok, d, rows)
    ramp = torch.linspace(0.1, 12, rows, device=DEV)[None, None, :, None]
    for order in (1, -1):
        k = (kc.float() * (ramp if order == 1 else ramp.flip(2))).to(BF16)
        tree = random_tree(tok, 1, 2)
        got = kv.tree_attention(q, kn, vn, tree, k, vc, rows, scale=0.2)
        # scores reach 12 * 7 * 1.6 of the derivation's 7: 2^-12 grows with them
        for h in range(2):
            m = torch.cat([torch.ones(tok, rows, dtype=torch.bool, device=DEV), seen(tree[0], tok)], 1).repeat(2, 1)
            ref, a = ref_attend(q[0, 2 * h:2 * h + 2].reshape(-1, d), torch.cat([k[0, h], kn[0, h]]),
                                torch.cat([vc[0, h], vn[0, h]]), m, 0.2)
            within(got[0, 2 * h:2 * h + 2].reshape(-1, d), ref,
                   2.0 ** -8 * ref.abs() + (2.0 ** -8 + 20 * 2.0 ** -12) * a, f"order {order}")


@gpu
def test_tree_views_workspace_stream_and_shared_tree():
    """Token-major caches and queries, one tree for all, own workspace, another stream."""
    g = gen(11)
    n, hq, hkv, tok, d, rows = 2, 6, 3, 8, 128, 1333
    q = randn(g, n, tok, hq + 2 * hkv, d).transpose(1, 2)
    q, kn, vn = q.split([hq, hkv, hkv], 1)
    pool = randn(g, n, rows, 2, hkv, d)
    kc, vc = pool[:, :, 0].transpose(1, 2), pool[:, :, 1].transpose(1, 2)
    tree = random_tree(tok, 1, 5)[0]
    ws = torch.full((kv.tree_attention_workspace(n, hq, hkv, tok, d, 5000),), 255, dtype=torch.uint8, device=DEV)
    out = torch.zeros(n, tok, hq, d, dtype=BF16, device=DEV).transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kv.tree_attention(q, kn, vn, tree, kc, vc, rows - 2, scale=0.1, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert got is out
    check_tree(q, kn, vn, tree, kc, vc, rows - 2, 0.1, got)
    assert torch.equal(got, kv.tree_attention(q.contiguous(), kn.contiguous(), vn.contiguous(), tree,
                                              kc.contiguous(), vc.contiguous(), rows - 2, scale=0.1))


@gpu
@pytest.mark.parametrize("kv_heads", [1, 2, 8])
def test_tree_workspace_rises_with_all_but_kv_heads(kv_heads):
    """One workspace for the largest arguments serves every call of a model."""
    base = dict(batch=3, q_heads=16, kv_heads=kv_heads, tokens=8, head_dim=64, cache_rows=2000)
    for name, values in dict(batch=range(0, 200), q_heads=range(kv_heads, 64 * kv_heads + 1, kv_heads),
                             tokens=range(1, 65), head_dim=(64, 128), cache_rows=range(0, 4000, 50)).items():
        for other in (dict(), dict(batch=40), dict(tokens=40), dict(cache_rows=600)):
            sizes = [kv.tree_attention_workspace(**{**base, **other, name: x}) for x in values]
            assert sizes == sorted(sizes), (name, other)


@gpu
def test_tree_units_that_fill_the_device_exactly():
    """One share per unit: nothing to merge, and what follows on the stream
    still waits for the whole call."""
    n = torch.cuda.get_device_properties(0).multi_processor_count
    x = tree_inputs(13, n, 2, 1, 5, 128, 3000)
    tree = random_tree(5, n, 1)
    want = kv.tree_attention(*x[:3], tree, *x[3:], 3000, scale=0.1)
    check_tree(*x[:3], tree, *x[3:], 3000, 0.1, want)
    torch.cuda.synchronize()
    got = kv.tree_attention(*x[:3], tree, *x[3:], 3000, scale=0.1)
    x[3].fill_(7)
    x[4].fill_(float("nan"))
    assert torch.equal(got, want)


@gpu
def test_offsets_past_32_bits():
    """The second batch entry of a cache lies 2^32 elements behind the first."""
    far, rows, d = 1 << 32, 1500, 64
    g = gen(14)
    flat = torch.empty(far + rows * d, dtype=BF16, device=DEV)
    cache = flat.as_strided((2, 1, rows, d), (far, rows * d, d, 1))
    for i in range(2):
        cache[i] = randn(g, 1, rows, d)
    small = cache.contiguous()
    q, k, v = randn(g, 2, 2, 6, d), randn(g, 2, 1, 6, d), randn(g, 2, 1, 6, d)
    tree = random_tree(6, 2, 1)
    assert torch.equal(kv.tree_attention(q, k, v, tree, cache, cache, rows, scale=0.1),
                       kv.tree_attention(q, k, v, tree, small, small, rows, scale=0.1))
    codes, scales = (torch.zeros((2, 1, 24, d), dtype=torch.int8, device=DEV), torch.zeros((2, 1, 24), device=DEV))
    kv.block_summaries(cache, codes, scales, rows)
    c, s = ref_summaries(small[:, :, :23 * 64])
    assert torch.equal(codes[:, :, :23], c) and torch.equal(scales[:, :, :23], s)
    for a, b in zip(kv.sparse_attention(q, cache, cache, codes, scales, rows, 3, scale=0.1),
                    kv.sparse_attention(q, small, small, codes, scales, rows, 3, scale=0.1)):
        assert torch.equal(a, b)
    path = torch.tensor([5, 0], dtype=torch.int32, device=DEV)
    kv.append_accepted(v, v, path, None, cache, cache, 700)
    assert torch.equal(cache[:, :, 700:702], v[:, :, [5, 0]])
    out = kv.qk_norm_rope(cache[:, :, :6], cache[:, :, 6:12], 3, omega_of(d))
    want = kv.qk_norm_rope(cache[:, :, :6].contiguous(), cache[:, :, 6:12].contiguous(), 3, omega_of(d))
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    kv.check_status()


@gpu
def test_tree_lengths_out_of_range_are_recorded():
    x = tree_inputs(12, 2, 2, 1, 3, 64, 50)
    tree = random_tree(3, 1, 1)[0]
    lengths = torch.tensor([51, -1], dtype=torch.int32, device=DEV)
    kv.check_status()
    got = kv.tree_attention(*x[:3], tree, *x[3:], lengths, scale=0.1)
    with pytest.raises(kv.StateKVError) as e:
        kv.check_status()
    assert e.value.status == N.E_DEVICE
    # clamped
    check_tree(*x[:3], tree, *x[3:], torch.tensor([50, 0]), 0.1, got)


# ------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (torch.float32, 64)])
@pytest.mark.parametrize("layers", [1, 2])
def test_append_accepted(dtype, d, layers):
    g = gen(21)
    seqs, hkv, tok, cap = 4, 3, 11, 60
    n = seqs * layers
    kn, vn = randn(g, n, tok, 2, hkv, d, dtype=dtype).unbind(2)   # token-major drafts
    kn, vn = kn.transpose(1, 2), vn.transpose(1, 2)
    kc, vc = randn(g, n, hkv, cap, d, dtype=dtype), randn(g, n, hkv, cap, d, dtype=dtype)
    k0, v0 = kc.clone(), vc.clone()
    path = torch.tensor([[0, 2, 5, 10], [0, 1, 2, 3], [0, 9, 10, 10], [10, 0, 3, 3]], dtype=torch.int32, device=DEV)
    counts = torch.tensor([4, 1, 0, 3], dtype=torch.int32, device=DEV)
    lengths = torch.tensor([0, 59, 60, 7], dtype=torch.int32, device=DEV)
    new = kv.append_accepted(kn, vn, path, counts, kc, vc, lengths)
    assert new.tolist() == [4, 60, 60, 10]
    for i in range(n):
        s = i // layers
        for j in range(int(counts[s])):
            k0[i, :, int(lengths[s]) + j] = kn[i, :, int(path[s, j])]
            v0[i, :, int(lengths[s]) + j] = vn[i, :, int(path[s, j])]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    kv.check_status()
    # one path for all, common length
    assert kv.append_accepted(kn, vn, path[0].contiguous(), None, kc, vc, 20) == 24
    for j in range(4):
        k0[:, :, 20 + j], v0[:, :, 20 + j] = kn[:, :, int(path[0, j])], vn[:, :, int(path[0, j])]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    # what does not fit or does not exist is recorded and left out
    new = kv.append_accepted(kn, vn, path, torch.tensor([4, 2, 1, 5], dtype=torch.int32, device=DEV), kc, vc,
                             torch.tensor([57, 59, 60, 7], dtype=torch.int32, device=DEV))
    assert new.tolist() == [57, 59, 60, 7]
    with pytest.raises(kv.StateKVError):
        kv.check_status()
    bad = torch.tensor([-1, tok, 4], dtype=torch.int32, device=DEV)
    kv.append_accepted(kn, vn, bad, None, kc, vc, 30)
    with pytest.raises(kv.StateKVError):
        kv.check_status()
    k0[:, :, 32], v0[:, :, 32] = kn[:, :, 4], vn[:, :, 4]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


@gpu
def test_append_of_more_units_than_32_bits_count():
    """One head's K and V rows are more than 2^31 units of 16 bytes: 34 GB."""
    g = gen(32)
    steps, d = (1 << 23) + 5001, 512
    kn, vn = (randn(g, 1, 1, 2, d, dtype=torch.float32) for _ in range(2))
    kc, vc = (torch.empty(1, 1, steps + 3, d, device=DEV) for _ in range(2))
    for c in (kc, vc):
        c[:, :, :1] = c[:, :, -2:] = 7
    path = torch.arange(steps, device=DEV, dtype=torch.int32) % 2
    assert 2 * steps * (d * 4 // 16) > 1 << 31
    assert kv.append_accepted(kn, vn, path, None, kc, vc, 1) == steps + 1
    kv.check_status()
    for c, x in ((kc, kn), (vc, vn)):
        assert (c[:, :, 0] == 7).all() and (c[:, :, -2:] == 7).all()
        for part in (c[:, :, 1:-2:997], c[:, :, -1003:-2]):
            first = (steps - 1001 if part.shape[2] == 1001 else 0)
            at = (first + torch.arange(part.shape[2], device=DEV) * (1 if first else 997)) % 2
            assert torch.equal(part, x[:, :, at])


# ---------------------------------------------------------------- summaries
def ref_summaries(k):
    """[..., blocks * 64, d] -> int8 codes and scales, as the header defines them."""
    m = (k.unflatten(-2, (-1, 64)).double().sum(-2)).float() / 64
    top = m.abs().amax(-1)
    # quotients in fp64, rounded: the correctly rounded fp32 quotient (torch
    # multiplies by a rounded reciprocal where one side is a plain number)
    inv = torch.where(top > 0, (127 / top.double()).float(), torch.zeros_like(top))
    return torch.round(m * inv[..., None]).to(torch.int8), (top.double() / 127).float()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("token_major", [False, True])
def test_block_summaries(d, token_major):
    g = gen(31)
    seqs, layers, hkv, cap = 3, 2, 2, 700
    n = seqs * layers
    k = randn(g, n, cap, hkv, d).transpose(1, 2)
    # values of very different sizes, cancelling sums, a zero block
    k[0, :, :64] *= torch.logspace(-20, 10, 64, device=DEV)[:, None]
    k[1, 0, 64:96] = -k[1, 0, 96:128]
    k[2, :, 64:128] = 0
    k[3, 1, :64] *= 1e30
    if not token_major:
        k = k.contiguous()
    blocks = cap // 64 + 1
    codes = torch.full((n, hkv, blocks, d), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((n, hkv, blocks), 7.0, device=DEV)
    c, s = ref_summaries(k[:, :, :cap // 64 * 64])
    lens = [700, 63, 129]
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kv.block_summaries(k, codes, scales, lengths)
    for i in range(n):
        b = lens[i // layers] // 64
        assert torch.equal(codes[i, :, :b], c[i, :, :b]) and torch.equal(scales[i, :, :b], s[i, :, :b])
        assert (codes[i, :, b:] == 77).all() and (scales[i, :, b:] == 7).all()
    # later: 60 more rows of the second sequence, the last ones alone
    codes.fill_(77)
    kv.block_summaries(k, codes, scales, torch.tensor([700, 128, 129], dtype=torch.int32, device=DEV), appended=65)
    for i in range(n):
        fresh = {0: range(9, 10), 1: range(0, 2), 2: range(1, 2)}[i // layers]
        for b in range(blocks):
            want = c[i, :, b] if b in fresh else torch.full_like(c[i, :, 0], 77)
            assert torch.equal(codes[i, :, b], want), (i, b)
    kv.block_summaries(k, codes, scales, 640, appended=0)
    kv.check_status()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_codes_of_tiny_keys(d):
    """Blocks whose factor 127 / max |mean| would pass fp32's range: the codes of
    the same block times 2^64, and zeros for zeros."""
    g = gen(33)
    sizes = [2.0 ** e for e in (-99, -100, -101, -110, -119, -121, -122, -126, -131, -133)]
    nb = len(sizes)
    k = randn(g, 1, 2, nb, 64, d, dtype=torch.float32) + 2 * randn(g, 1, 2, nb, 1, d, dtype=torch.float32)
    k[..., ::3] = 0
    k = (k * torch.tensor(sizes, device=DEV)[:, None, None]).flatten(2, 3).to(BF16)
    codes, scales = torch.zeros(1, 2, nb, d, dtype=torch.int8, device=DEV), torch.zeros(1, 2, nb, device=DEV)
    kv.block_summaries(k, codes, scales, nb * 64)
    m = k.unflatten(-2, (-1, 64)).double().sum(-2).float() / 64
    top = m.abs().amax(-1)
    up = torch.where(top < 2.0 ** -100, 2.0 ** 64, 1.0)
    want = torch.round(m * up[..., None] * (127 / (top * up).double()).float()[..., None]).to(torch.int8)
    assert torch.equal(codes, want) and torch.equal(scales, (top.double() / 127).float())
    assert (codes[..., ::3] == 0).all() and (codes.abs().amax(-1) == 127).all()


# ------------------------------------------------------------------- sparse
def ref_choice(q, codes, scales, nb, top):
    """q [g][d] of one token and KV head -> the chosen blocks, ascending."""
    big = q.float().abs().max()
    qi = torch.round(q.float() * (127 / big.double()).float()) if big > 0 else torch.zeros_like(q.float())
    s = (qi.double() @ codes[:nb].double().T).amax(0).float() * scales[:nb]
    return sorted(sorted(range(nb), key=lambda b, v=s.tolist(): (-v[b], b))[:top])


def check_sparse(q, kc, vc, codes, scales, lengths, top, scale, got, selected):
    n, hq, tok, d = q.shape
    hkv = kc.shape[1]
    G = hq // hkv
    for i in range(n):
        rows = lengths if isinstance(lengths, int) else int(lengths[i * len(lengths) // n])
        nb = max(0, rows - tok) // 64
        for h in range(hkv):
            for t in range(tok):
                at = rows - tok + t
                if at < 0:
                    assert (got[i, h * G:(h + 1) * G, t] == 0).all() and (selected[i, h, t] == -1).all()
                    continue
                qs = q[i, h * G:(h + 1) * G, t]
                keep = ref_choice(qs, codes[i, h], scales[i, h], nb, top)
                assert selected[i, h, t].tolist() == keep + [-1] * (top - len(keep)), (i, h, t)
                idx = torch.cat([64 * torch.tensor(keep, dtype=torch.int64)[:, None].expand(-1, 64).reshape(-1)
                                 + torch.arange(64).repeat(len(keep)), torch.arange(64 * nb, at + 1)]).to(DEV)
                ref, a = ref_attend(qs, kc[i, h, idx], vc[i, h, idx],
                                    torch.ones(G, len(idx), dtype=torch.bool, device=DEV), scale)
                within(got[i, h * G:(h + 1) * G, t], ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a,
                       f"entry {i} head {h} token {t}")


def sparse_inputs(seed, n, hq, hkv, tok, d, cap):
    g = gen(seed)
    kc, vc = randn(g, n, hkv, cap, d), randn(g, n, hkv, cap, d)
    kc[:, :, :cap // 64 * 64].view(n, hkv, -1, 64, d).add_(randn(g, n, hkv, cap // 64, 1, d) / 2)
    codes, scales = ref_summaries(kc[:, :, :cap // 64 * 64])
    return randn(g, n, hq, tok, d), kc, vc, codes, scales


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,hq,hkv,tok,rows,top", [
    (1, 1, 1, 1, 1, 1), (1, 2, 1, 1, 64, 1), (1, 2, 1, 1, 65, 1), (1, 4, 2, 3, 190, 2), (1, 12, 2, 1, 4100, 5),
    (2, 16, 8, 2, 2000, 31),      # cluster of 4
    (3, 16, 8, 5, 1000, 7),       # 120 items: no cluster
    (1, 32, 2, 1, 9001, 64),      # 16 query heads per KV head
    (1, 14, 2, 70, 700, 4),       # more tokens than a block has rows
    (1, 6, 2, 1, 40000, 1),       # 624 blocks, one kept
])
def test_sparse_sizes(d, n, hq, hkv, tok, rows, top):
    x = sparse_inputs(rows + tok, n, hq, hkv, tok, d, rows + 5)
    got, sel = kv.sparse_attention(*x, rows, top, scale=0.1)
    check_sparse(*x, rows, top, 0.1, got, sel)
    kv.check_status()


@gpu
@pytest.mark.parametrize("layers", [1, 2])
def test_sparse_ragged(layers):
    lens = [3, 0, 1, 700, 64, 129, 650, 2]
    n = len(lens) * layers
    x = sparse_inputs(7, n, 6, 2, 3, 128, 705)
    # what a sequence has not reached yet may hold anything
    for i in range(n):
        for c in x[1:3]:
            c[i, :, lens[i // layers]:] = float("nan")
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    got, sel = kv.sparse_attention(*x, lengths, 4, scale=0.1)
    check_sparse(*x, lengths, 4, 0.1, got, sel)
    kv.check_status()


@gpu
def test_sparse_ties_and_full_attention():
    """Equal scores keep the lower blocks; enough blocks make it full attention."""
    x = list(sparse_inputs(8, 1, 4, 2, 2, 64, 64 * 40 + 10))
    x[3][:, :, 5:] = x[3][:, :, 5:6]
    x[4][:, :, 5:] = x[4][:, :, 5:6]
    for top in (1, 7, 30):
        got, sel = kv.sparse_attention(*x, 64 * 40 + 10, top, scale=0.1)
        check_sparse(*x, 64 * 40 + 10, top, 0.1, got, sel)
    zero = [torch.zeros_like(x[0])] + x[1:]              # no query: every score is 0
    got, sel = kv.sparse_attention(*zero, 64 * 40 + 10, 9, scale=0.1)
    assert (sel == torch.arange(9, device=DEV)).all()
    check_sparse(*zero, 64 * 40 + 10, 9, 0.1, got, sel)
    q, kc, vc, rows = x[0], x[1], x[2], 64 * 40 + 10
    got, sel = kv.sparse_attention(*x, rows, 1024, scale=0.1)
    assert (sel[..., :40] == torch.arange(40, device=DEV)).all() and (sel[..., 40:] == -1).all()
    tree = kv.tree_masks([-1, 0], DEV)[0]
    full = kv.tree_attention(q, kc[:, :, rows - 2:rows].contiguous(), vc[:, :, rows - 2:rows].contiguous(), tree,
                             kc, vc, rows - 2, scale=0.1)
    # two results, each within its tolerance of the same value (|v| < 8)
    assert (got.double() - full.double()).abs().max() < 2 * (2 * 2.0 ** -8 + 2.0 ** -12) * 8


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_sparse_choice_of_tiny_queries(d):
    """A power of two times a query chooses the same blocks, and a query's zeros
    stay zeros, as small as it may be."""
    q, kc, vc, codes, scales = sparse_inputs(34, 1, 4, 2, 3, d, 2000)
    q[..., ::2] = 0
    for e in (-90, -101, -120, -126):
        tiny = (q.float() * 2.0 ** e).to(BF16)
        selected = kv.sparse_attention(tiny, kc, vc, codes, scales, 2000, 5, scale=0.1)[1]
        for h in range(2):
            for t in range(3):
                qs = (tiny[0, 2 * h:2 * h + 2, t].float() * 2.0 ** 64).to(BF16)
                assert selected[0, h, t].tolist() == ref_choice(qs, codes[0, h], scales[0, h], (2000 - 3) // 64, 5), e


@gpu
def test_sparse_many_blocks_views_and_stream():
    """The largest number of blocks, token-major cache, another stream, captured."""
    g = gen(61)
    rows = 32768 * 64 + 40
    pool = torch.randn(1, rows, 2, 1, 64, generator=g, device=DEV, dtype=BF16)
    kc, vc = pool[:, :, 0].transpose(1, 2), pool[:, :, 1].transpose(1, 2)
    codes = torch.empty((1, 1, 32768, 64), dtype=torch.int8, device=DEV)
    scales = torch.empty((1, 1, 32768), device=DEV)
    kv.block_summaries(kc, codes, scales, rows)
    c, s = ref_summaries(kc[:, :, :32768 * 64])
    assert torch.equal(codes, c) and torch.equal(scales, s)
    q = randn(g, 1, 2, 4, 64).transpose(1, 2).contiguous().transpose(1, 2).view(1, 2, 4, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, sel = kv.sparse_attention(q, kc, vc, codes, scales, rows, 100, scale=0.1, stream=st)
    st.synchronize()
    check_sparse(q, kc, vc, codes, scales, rows, 100, 0.1, got, sel)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = kv.sparse_attention(q, kc, vc, codes, scales, rows, 100, scale=0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[0], got) and torch.equal(again[1], sel)
    kv.check_status()


# ------------------------------------------------------------------- chains
@gpu
def test_speculative_step_as_used_and_captured():
    """Norm and rotate the drafted tokens, attend as a tree, append the accepted
    path, summarise: eager against the definitions, then captured and replayed."""
    g = gen(41)
    seqs, layers, hq, hkv, d, cap = 2, 2, 6, 2, 128, 600
    n = seqs * layers
    parents = [[-1, 0, 0, 1, 1, 2, 5], [-1, 0, 1, 2, 3, 4, 5]]
    tree, depth = kv.tree_masks(parents, DEV)
    tok = tree.shape[1]
    kc, vc = randn(g, n, hkv, cap, d), randn(g, n, hkv, cap, d)
    lengths = torch.tensor([500, 317], dtype=torch.int32, device=DEV)
    w = 1 + randn(g, d) / 4
    omega = omega_of(d)
    path = torch.tensor([[0, 2, 5, 6], [0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    counts = torch.tensor([4, 2], dtype=torch.int32, device=DEV)
    codes = torch.zeros((n, hkv, cap // 64, d), dtype=torch.int8, device=DEV)
    scales = torch.zeros((n, hkv, cap // 64), device=DEV)
    x = randn(g, n, tok, hq + 2 * hkv, d)

    def step():
        q, k, v = x.transpose(1, 2).split([hq, hkv, hkv], 1)
        pos = lengths[:, None] + depth
        qr, kr, vr = kv.qk_norm_rope(q, k, pos, omega, w, w, v=v)
        o = kv.tree_attention(qr, kr, vr, tree, kc, vc, lengths, scale=0.09)
        new = kv.append_accepted(kr, vr, path, counts, kc, vc, lengths)
        kv.block_summaries(kc, codes, scales, new, appended=4)
        return qr, kr, vr, o, new

    kv.block_summaries(kc, codes, scales, lengths)
    for round_ in range(2):
        k0, v0 = kc.clone(), vc.clone()
        qr, kr, vr, o, new = step()
        check_tree(qr, kr, vr, tree, k0, v0, lengths, 0.09, o, f"round {round_}")
        assert (new - lengths).tolist() == [4, 2]
        for i in range(n):
            at, cnt = int(lengths[i // layers]), int(counts[i // layers])
            sel = path[i // layers, :cnt].long()
            assert torch.equal(kc[i, :, at:at + cnt], kr[i][:, sel])
            c, s = ref_summaries(kc[i, :, :int(new[i // layers]) // 64 * 64])
            assert torch.equal(codes[i, :, :c.shape[1]], c)
        lengths.copy_(new)
    kv.check_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        lengths_next = out[4]
    for round_ in range(3):
        x.copy_(randn(g, *x.shape))
        k0, v0 = kc.clone(), vc.clone()
        graph.replay()
        got = [t.clone() for t in out]
        kc.copy_(k0), vc.copy_(v0)
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        lengths.copy_(lengths_next)
    kv.check_status()


@gpu
def test_two_captured_graphs_at_once():
    """Two graphs on two streams: each has a workspace of its own."""
    xs = [tree_inputs(50 + i, 1, 12, 2, 8, 128, 9000) for i in range(2)]
    tree = random_tree(8, 1, 1)
    want = [kv.tree_attention(*x[:3], tree, *x[3:], 9000, scale=0.09) for x in xs]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kv.tree_attention(*x[:3], tree, *x[3:], 9000, scale=0.09))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    kv.check_status()


# ----------------------------------------------------------------- refusals
def test_tree_masks_on_the_host():
    m, d = kv.tree_masks([-1, 0, 0, 1])
    assert m.tolist() == [[1, 3, 5, 11]] and d.tolist() == [[0, 1, 1, 2]]
    m, _ = kv.tree_masks([[-1] + list(range(63))] * 2)
    assert m.shape == (2, 64) and m[1, 63] == -1
    for bad in ([], [0], [-1, 1], [-1, -2], [-1] * 65, [[-1], [-1, 0]]):
        with pytest.raises(ValueError):
            kv.tree_masks(bad)


def view(p=16, b=1024, h=512, t=128):
    return N.View(p, b, h, t)


def tree_args(**kw):
    a = dict(q=view(), out=view(), k_new=view(), v_new=view(), k_cache=view(), v_cache=view(), tree=16, status=16,
             workspace=16, workspace_bytes=1 << 40, scale=0.1, tree_stride=0, length=2, batch=2, layers=1, q_heads=4,
             kv_heads=2, tokens=3, head_dim=128, cache_rows=4)
    a.update(kw)
    return N.TreeArgs(**a)


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=0), N.E_INVALID_ARG), (dict(tokens=65), N.E_UNSUPPORTED), (dict(head_dim=96), N.E_UNSUPPORTED),
    (dict(q_heads=3), N.E_INVALID_ARG), (dict(kv_heads=0), N.E_INVALID_ARG), (dict(layers=3), N.E_INVALID_ARG),
    (dict(layers=0), N.E_INVALID_ARG), (dict(batch=-1), N.E_INVALID_ARG), (dict(scale=0.0), N.E_INVALID_ARG),
    (dict(scale=math.nan), N.E_INVALID_ARG), (dict(scale=math.inf), N.E_INVALID_ARG), (dict(scale=1e-40), N.E_INVALID_ARG),
    (dict(length=5), N.E_CAPACITY), (dict(length=-1), N.E_INVALID_ARG), (dict(status=None), N.E_INVALID_ARG),
    (dict(status=18), N.E_INVALID_ARG), (dict(tree=None), N.E_INVALID_ARG), (dict(tree=20), N.E_INVALID_ARG),
    (dict(q=view(8)), N.E_INVALID_ARG), (dict(q=view(t=4)), N.E_INVALID_ARG), (dict(out=view(h=-512)), N.E_INVALID_ARG),
    (dict(k_cache=view(None)), N.E_INVALID_ARG), (dict(k_cache=view(t=0)), N.E_INVALID_ARG),
    (dict(k_new=view(h=0)), N.E_INVALID_ARG), (dict(batch=0), N.OK),
])
def test_tree_refusals_before_device_work(bad, want):
    assert N.load().statekv_tree_attention(tree_args(**bad), None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(dtype=5), N.E_INVALID_ARG), (dict(weight_dtype=5), N.E_INVALID_ARG), (dict(head_dim=96), N.E_UNSUPPORTED),
    (dict(omega=None), N.E_INVALID_ARG), (dict(omega=20), N.E_INVALID_ARG), (dict(status=None), N.E_INVALID_ARG),
    (dict(q=view(8)), N.E_INVALID_ARG), (dict(k_out=view(b=4)), N.E_INVALID_ARG), (dict(v_out=view(None)), N.E_INVALID_ARG),
    (dict(layers=0), N.E_INVALID_ARG), (dict(position_layers=0), N.E_INVALID_ARG), (dict(weight_rows=0), N.E_INVALID_ARG), (dict(q_weight=8), N.E_INVALID_ARG), (dict(batch=3, layers=2), N.E_INVALID_ARG),
    (dict(out_capacity=2), N.E_CAPACITY), (dict(eps=-1.0), N.E_INVALID_ARG), (dict(eps=math.nan), N.E_INVALID_ARG),
    (dict(tokens=-1), N.E_INVALID_ARG), (dict(q_heads=17000), N.E_UNSUPPORTED), (dict(tokens=0, out_capacity=0), N.OK),
    (dict(batch=0), N.OK),
])
def test_norm_rope_refusals_before_device_work(bad, want):
    a = dict(q=view(), k=view(), v=view(), q_out=view(), k_out=view(), v_out=view(), omega=16, status=16,
             position_layers=1, weight_rows=1, batch=2, layers=1, q_heads=4, kv_heads=2, tokens=3, head_dim=128, out_capacity=3,
             dtype=0, weight_dtype=0, eps=1e-6)
    a.update(bad)
    assert N.load().statekv_norm_rope(N.NormRopeArgs(**a), None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(dtype=5), N.E_INVALID_ARG), (dict(head_dim=4), N.E_UNSUPPORTED), (dict(head_dim=100), N.E_UNSUPPORTED),
    (dict(path=None), N.E_INVALID_ARG), (dict(k_new=view(8)), N.E_INVALID_ARG), (dict(v_cache=view(None)), N.E_INVALID_ARG),
    (dict(length=3), N.E_CAPACITY), (dict(new_lengths=64, lengths=64), N.E_INVALID_ARG),
    (dict(new_lengths=64, counts=64), N.E_INVALID_ARG), (dict(status=None), N.E_INVALID_ARG),
    (dict(layers=0), N.E_INVALID_ARG), (dict(path_len=-1), N.E_INVALID_ARG), (dict(batch=0), N.OK),
])
def test_append_refusals_before_device_work(bad, want):
    a = dict(k_new=view(), v_new=view(), k_cache=view(), v_cache=view(), path=16, status=16, path_len=2, length=2,
             batch=2, layers=1, kv_heads=2, tokens=3, head_dim=128, cache_rows=4, dtype=0)
    a.update(bad)
    assert N.load().statekv_append_accepted(N.AppendArgs(**a), None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(head_dim=96), N.E_UNSUPPORTED), (dict(blocks=1), N.E_CAPACITY), (dict(codes=20), N.E_INVALID_ARG),
    (dict(scales=None), N.E_INVALID_ARG), (dict(k_cache=view(8)), N.E_INVALID_ARG), (dict(appended=-1), N.E_INVALID_ARG),
    (dict(status=None), N.E_INVALID_ARG), (dict(batch=0), N.OK), (dict(cache_rows=63, blocks=0), N.OK),
])
def test_summary_refusals_before_device_work(bad, want):
    a = dict(k_cache=view(), codes=16, scales=16, status=16, length=128, appended=64, blocks=2, batch=2, layers=1,
             kv_heads=2, head_dim=128, cache_rows=128)
    a.update(bad)
    assert N.load().statekv_block_summaries(N.SummaryArgs(**a), None) == want


@pytest.mark.parametrize("bad,want", [
    (dict(head_dim=96), N.E_UNSUPPORTED), (dict(q_heads=34), N.E_UNSUPPORTED), (dict(q_heads=3), N.E_INVALID_ARG),
    (dict(top=0), N.E_INVALID_ARG), (dict(top=1025), N.E_UNSUPPORTED), (dict(blocks=1), N.E_CAPACITY),
    (dict(length=257), N.E_CAPACITY), (dict(codes=24), N.E_INVALID_ARG), (dict(scales=None), N.E_INVALID_ARG),
    (dict(selected=18), N.E_INVALID_ARG), (dict(status=None), N.E_INVALID_ARG), (dict(scale=-1.0), N.E_INVALID_ARG),
    (dict(q=view(8)), N.E_INVALID_ARG), (dict(k_cache=view(None)), N.E_INVALID_ARG), (dict(out=view(t=4)), N.E_INVALID_ARG),
    (dict(cache_rows=64 * 32769, blocks=40000), N.E_UNSUPPORTED), (dict(batch=1 << 28), N.E_UNSUPPORTED),
    (dict(layers=3), N.E_INVALID_ARG), (dict(batch=0), N.OK), (dict(tokens=0), N.OK),
])
def test_sparse_refusals_before_device_work(bad, want):
    a = dict(q=view(), out=view(), k_cache=view(), v_cache=view(), codes=16, scales=16, selected=16, status=16,
             scale=0.1, length=256, top=2, blocks=4, batch=2, layers=1, q_heads=4, kv_heads=2, tokens=3, head_dim=128,
             cache_rows=256)
    a.update(bad)
    assert N.load().statekv_sparse_attention(N.SparseArgs(**a), None) == want


def test_arrays_that_reach_past_their_rows_or_lie_between_words_are_refused():
    """Rows of an array closer together than they are long would be read past the
    array's end; an odd address faults on the device."""
    lib, g = N.load(), view(b=4096, h=512)
    sizes = dict(batch=2, layers=1, kv_heads=2, tokens=3, head_dim=128, status=16)
    norm = dict(sizes, **{f: g for f in ("q", "k", "v", "q_out", "k_out", "v_out")}, omega=16, position_layers=1,
                weight_rows=1, q_heads=4, out_capacity=3, eps=1e-6, positions=16)
    tree = dict(sizes, **{f: g for f in ("q", "out", "k_new", "v_new", "k_cache", "v_cache")}, tree=16, workspace=16,
                workspace_bytes=1 << 40, scale=0.1, length=2, q_heads=4, cache_rows=4)
    append = dict(sizes, **{f: g for f in ("k_new", "v_new", "k_cache", "v_cache")}, path=16, path_len=2, length=2,
                  cache_rows=4)
    summary = dict({k: x for k, x in sizes.items() if k != "tokens"}, k_cache=g, codes=16, scales=16, length=128,
                   appended=64, blocks=2, cache_rows=128)
    sparse = dict(sizes, **{f: g for f in ("q", "out", "k_cache", "v_cache")}, codes=16, scales=16, scale=0.1,
                  length=256, top=2, blocks=4, q_heads=4, cache_rows=256)
    for f, args, good, bads in (
            (lib.statekv_norm_rope, N.NormRopeArgs, norm,
             [dict(position_stride=2), dict(positions=18), dict(out_rows=18)]),
            (lib.statekv_tree_attention, N.TreeArgs, tree, [dict(tree_stride=2), dict(lengths=18)]),
            (lib.statekv_append_accepted, N.AppendArgs, append,
             [dict(path_stride=1), dict(path=18), dict(counts=18), dict(lengths=18), dict(new_lengths=18)]),
            (lib.statekv_block_summaries, N.SummaryArgs, summary, [dict(lengths=18)]),
            (lib.statekv_sparse_attention, N.SparseArgs, sparse, [dict(lengths=18)])):
        for bad in bads:
            assert f(args(**{**good, **bad}), None) == N.E_INVALID_ARG, bad
    # a stride that belongs to no array is not looked at
    assert lib.statekv_norm_rope(N.NormRopeArgs(**{**norm, "positions": None, "position_stride": 2, "batch": 0}),
                                 None) == N.OK


@pytest.mark.parametrize("pack,args", [(N.PACK_NORM_ROPE, N.NormRopeArgs), (N.PACK_TREE, N.TreeArgs),
                                       (N.PACK_APPEND, N.AppendArgs), (N.PACK_SUMMARY, N.SummaryArgs),
                                       (N.PACK_SPARSE, N.SparseArgs)])
def test_packed_arguments_are_the_structures(pack, args):
    flat, n = [], 0

    def leaf(t):
        nonlocal n
        n += 1
        flat.append(n / 2 if t in (C.c_float, C.c_double) else n)
        return flat[-1]

    a = args(**{f: N.View(*(leaf(x) for _, x in N.View._fields_)) if t is N.View else leaf(t) for f, t in args._fields_})
    assert pack.size == C.sizeof(args) and pack.pack(*flat) == bytes(a)


@pytest.mark.parametrize("where", [dict(b=0), dict(h=0), dict(t=0)])
def test_outputs_that_share_memory_are_refused(where):
    """Entries of an output that lie on one another, where there are several."""
    lib, bad = N.load(), view(**where)
    ins = {f: view() for f in ("q", "k", "v", "k_new", "v_new", "k_cache", "v_cache")}
    sizes = dict(batch=2, layers=1, q_heads=4, kv_heads=2, tokens=3, head_dim=128, status=16)
    of = lambda args, **kw: args(**{f: x for f, x in {**ins, **sizes, **kw}.items()  # noqa: E731
                                    if f in dict(args._fields_)})
    for name in ("q_out", "k_out", "v_out"):
        outs = {**{f: view() for f in ("q_out", "k_out", "v_out")}, name: bad}
        a = of(N.NormRopeArgs, **outs, omega=16, position_layers=1, weight_rows=1, out_capacity=3, eps=1e-6)
        assert lib.statekv_norm_rope(a, None) == N.E_INVALID_ARG, name
    assert lib.statekv_tree_attention(tree_args(out=bad), None) == N.E_INVALID_ARG
    for name in ("k_cache", "v_cache"):
        a = of(N.AppendArgs, **{name: bad}, path=16, path_len=2, length=2, cache_rows=4)
        assert lib.statekv_append_accepted(a, None) == N.E_INVALID_ARG, name
    a = of(N.SparseArgs, out=bad, codes=16, scales=16, scale=0.1, length=256, top=2, blocks=4, cache_rows=256)
    assert lib.statekv_sparse_attention(a, None) == N.E_INVALID_ARG


@pytest.mark.parametrize("where", [dict(t=64), dict(h=256), dict(h=0), dict(b=896), dict(h=128, t=128, b=1 << 20),
                                   dict(h=128, t=248), dict(b=128, h=248), dict(b=1 << 62, h=1 << 62)])
def test_outputs_whose_rows_overlap_are_refused(where):
    """Rows of 128 that reach into one another with strides that need not be 0:
    2 batch entries of 4 heads (K and V: 2) of 3 tokens (of a cache: 4)."""
    lib, good = N.load(), view(b=4096, h=512)
    bad = view(**{**dict(b=4096, h=512), **where})
    sizes = dict(batch=2, layers=1, q_heads=4, kv_heads=2, tokens=3, head_dim=128, status=16)
    views = {f: good for f in ("q", "k", "v", "k_new", "v_new", "k_cache", "v_cache", "out", "q_out", "k_out", "v_out")}

    def of(args, **kw):
        return args(**{f: x for f, x in {**views, **sizes, **kw}.items() if f in dict(args._fields_)})

    for name in ("q_out", "k_out", "v_out"):
        a = of(N.NormRopeArgs, **{name: bad}, omega=16, position_layers=1, weight_rows=1, out_capacity=4, eps=1e-6)
        assert lib.statekv_norm_rope(a, None) == N.E_INVALID_ARG, name
    a = of(N.TreeArgs, out=bad, tree=16, workspace=16, workspace_bytes=1 << 40, scale=0.1, length=2, cache_rows=4)
    assert lib.statekv_tree_attention(a, None) == N.E_INVALID_ARG
    for name in ("k_cache", "v_cache"):
        a = of(N.AppendArgs, **{name: bad}, path=16, path_len=2, length=2, cache_rows=4)
        assert lib.statekv_append_accepted(a, None) == N.E_INVALID_ARG, name
    a = of(N.SparseArgs, out=bad, codes=16, scales=16, scale=0.1, length=256, top=2, blocks=4, cache_rows=256)
    assert lib.statekv_sparse_attention(a, None) == N.E_INVALID_ARG


@gpu
def test_inputs_may_repeat_their_entries():
    """Expanded inputs give what their copies give."""
    g = gen(62)
    q, k, v = (randn(g, 1, 1, 5, 64).expand(2, h, 5, 64) for h in (6, 2, 2))
    om = omega_of(64)
    for a, b in zip(kv.qk_norm_rope(q, k, 7, om, v=v),
                    kv.qk_norm_rope(q.contiguous(), k.contiguous(), 7, om, v=v.contiguous())):
        assert torch.equal(a, b)
    path = torch.tensor([4, 1], dtype=torch.int32, device=DEV)
    caches = [torch.zeros(2, 2, 9, 64, dtype=BF16, device=DEV) for _ in range(4)]
    kv.append_accepted(k, v, path, None, *caches[:2], 3)
    kv.append_accepted(k.contiguous(), v.contiguous(), path, None, *caches[2:], 3)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    cache = randn(g, 1, 1, 1000, 64).expand(2, 2, 1000, 64)
    codes, scales = torch.zeros(2, 2, 15, 64, dtype=torch.int8, device=DEV), torch.zeros(2, 2, 15, device=DEV)
    kv.block_summaries(cache, codes, scales, 1000)
    assert torch.equal(codes, codes[:1, :1].expand_as(codes)) and scales.min() == scales[0, 0].min() > 0
    got = kv.sparse_attention(q, cache, cache, codes, scales, 1000, 4, scale=0.1)
    want = kv.sparse_attention(q.contiguous(), cache.contiguous(), cache.contiguous(), codes, scales, 1000, 4,
                               scale=0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    tree = random_tree(5, 1, 1)[0]
    new = k.contiguous()
    assert torch.equal(kv.tree_attention(q, new, new, tree, *caches[:2], 9, scale=0.1),
                       kv.tree_attention(q.contiguous(), new, new, tree, *caches[:2], 9, scale=0.1))
    kv.check_status()


def test_first_calls_of_two_threads_share_a_status_word(monkeypatch):
    """The address a thread gets is that of the word that is kept."""
    import threading
    import time

    from kv_cache_compression_frame_gb300 import text_ops

    def zeros(*a, **kw):
        time.sleep(0.05)                            # another thread runs meanwhile
        return torch.empty(4, dtype=torch.int32)

    monkeypatch.setattr(text_ops, "_status", {})
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: time.sleep(0.05))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    got, start = [], threading.Barrier(4)

    def call():
        start.wait()
        got.append(text_ops._status_ptr(5))

    threads = [threading.Thread(target=call) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert got == [text_ops._status[5][0].data_ptr()] * 4


def test_a_half_loaded_library_is_not_seen(monkeypatch):
    """A thread that finds packed entry points finds all of them."""
    seen_while_loading, cdll = [], C.CDLL

    class Lib:
        def __init__(self, path):
            self.lib = cdll(path)

        def __getattr__(self, name):
            return getattr(self.lib, name)

        def __getitem__(self, name):
            seen_while_loading.append(len(N.packed))
            return self.lib[name]

    N.load()
    monkeypatch.setattr(N, "packed", {})
    monkeypatch.setattr(N, "_lib", None)
    monkeypatch.setattr(N.C, "CDLL", Lib)
    N.load()
    assert seen_while_loading == [0] * len(N.PACKED) and sorted(N.packed) == sorted(N.PACKED)


@gpu
def test_empty_batches_and_tokens():
    """Nothing to do: outputs of the right shape and type, and no error."""
    z, c = (torch.zeros(0, 2, t, 64, dtype=BF16, device=DEV) for t in (3, 640))
    none, two = torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    codes, scales = torch.zeros(0, 2, 10, 64, dtype=torch.int8, device=DEV), torch.zeros(0, 2, 10, device=DEV)
    for lengths in (3, none):
        for counts in (None, none):
            got = kv.append_accepted(z, z, two, counts, c, c, lengths)
            if lengths is none or counts is none:
                assert got.shape == (0,) and got.dtype == torch.int32
            else:
                assert got == 5
        for tree in (torch.ones(3, dtype=torch.int64, device=DEV), torch.ones(0, 3, dtype=torch.int64, device=DEV)):
            assert kv.tree_attention(z, z, z, tree, c, c, lengths, scale=0.1).shape == z.shape
        kv.block_summaries(c, codes, scales, lengths)
        out, sel = kv.sparse_attention(z, c, c, codes, scales, lengths, 4, scale=0.1)
        assert out.shape == z.shape and sel.shape == (0, 2, 3, 4)
    for q in (z, torch.zeros(2, 2, 0, 64, dtype=BF16, device=DEV)):
        got = kv.qk_norm_rope(q, q, 7, omega_of(64), v=q)
        assert all(x.shape == q.shape for x in got)
    q = torch.zeros(2, 2, 0, 64, dtype=BF16, device=DEV)
    c = torch.zeros(2, 2, 640, 64, dtype=BF16, device=DEV)
    codes, scales = torch.zeros(2, 2, 10, 64, dtype=torch.int8, device=DEV), torch.zeros(2, 2, 10, device=DEV)
    assert kv.sparse_attention(q, c, c, codes, scales, 9, 4, scale=0.1)[0].shape == q.shape
    assert kv.append_accepted(q, q, two[:0], None, c, c, 9) == 9
    kv.check_status()


@gpu
def test_streams_of_another_device_are_refused():
    """They would leave the work on the current stream of the tensors' device."""
    class Elsewhere(torch.cuda.Stream):
        device_index = 1

    s = Elsewhere()
    z, path = torch.zeros(1, 1, 1, 64, dtype=BF16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    codes, scales = torch.zeros(1, 1, 0, 64, dtype=torch.int8, device=DEV), torch.zeros(1, 1, 0, device=DEV)
    for call in (lambda: kv.qk_norm_rope(z, z, 0, omega_of(64), stream=s),
                 lambda: kv.tree_attention(z, z, z, path.long(), z, z, 1, scale=0.1, stream=s),
                 lambda: kv.append_accepted(z, z, path, None, z.clone(), z.clone(), 0, stream=s),
                 lambda: kv.block_summaries(z, codes, scales, 1, stream=s),
                 lambda: kv.sparse_attention(z, z, z, codes, scales, 1, 1, scale=0.1, stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call()


@gpu
def test_strides_of_single_entries_do_not_matter():
    """One token, one head or one batch entry may have any stride: what contiguous
    copies give."""
    g = gen(65)
    d, rows = 64, 300

    def odd(x):                                     # the same values, odd strides where a dimension is 1
        st = [s if n > 1 else 3 + 2 * i for i, (n, s) in enumerate(zip(x.shape, x.stride()))]
        return x.as_strided(x.shape, (*st[:3], 1))

    for n, hq, hkv, tok in ((1, 1, 1, 1), (2, 1, 1, 1), (1, 4, 2, 1), (1, 2, 1, 3), (1, 1, 1, 5)):
        q, k, v = (randn(g, n, h, tok, d) for h in (hq, hkv, hkv))
        kc, vc = randn(g, n, hkv, rows, d), randn(g, n, hkv, rows, d)
        assert any(a != b for a, b in zip(odd(q).stride(), q.stride()))
        out = torch.zeros_like(q)
        om, tree = omega_of(d), random_tree(tok, 1, 1)[0]
        for a, b in zip(kv.qk_norm_rope(odd(q), odd(k), 9, om, v=odd(v), q_out=odd(out)),
                        kv.qk_norm_rope(q, k, 9, om, v=v)):
            assert torch.equal(a, b)
        assert torch.equal(kv.tree_attention(odd(q), odd(k), odd(v), tree, odd(kc), odd(vc), rows, scale=0.1,
                                             out=odd(out)),
                           kv.tree_attention(q, k, v, tree, kc, vc, rows, scale=0.1))
        codes, scales = (torch.zeros(n, hkv, 4, d, dtype=torch.int8, device=DEV), torch.zeros(n, hkv, 4, device=DEV))
        kv.block_summaries(odd(kc), codes, scales, rows)
        c, s = ref_summaries(kc[:, :, :256])
        assert torch.equal(codes, c) and torch.equal(scales, s)
        assert torch.equal(kv.sparse_attention(odd(q), odd(kc), odd(vc), codes, scales, rows, 2, scale=0.1,
                                               out=odd(out))[0],
                           kv.sparse_attention(q, kc, vc, codes, scales, rows, 2, scale=0.1)[0])
        path = torch.tensor([tok - 1], dtype=torch.int32, device=DEV)
        kv.append_accepted(odd(k), odd(v), path, None, odd(kc), odd(vc), 7)
        assert torch.equal(kc[:, :, 7], k[:, :, -1]) and torch.equal(vc[:, :, 7], v[:, :, -1])
    # a cache of one row
    one = torch.zeros(1, 1, 1, d, dtype=BF16, device=DEV)
    kv.append_accepted(odd(k), odd(v), path, None, odd(one), odd(one.clone()), 0)
    assert torch.equal(one[0, 0, 0], k[0, 0, -1])
    kv.check_status()


def test_null_arguments():
    lib = N.load()
    for f in ("norm_rope", "tree_attention", "append_accepted", "block_summaries", "sparse_attention"):
        assert getattr(lib, "statekv_" + f)(None, None) == N.E_INVALID_ARG
    assert lib.statekv_tree_attention_workspace(1, 4, 2, 65, 128, 100) == -1
    assert lib.statekv_tree_attention_workspace(1, 3, 2, 4, 128, 100) == -1


@gpu
def test_derivatives_are_refused():
    """Reverse mode while grad mode is on, forward mode always, for every input
    that could have one."""
    from torch.autograd import forward_ad as fw
    g = gen(64)
    q, k, v = (randn(g, 2, h, 3, 64) for h in (4, 2, 2))
    kc, vc = randn(g, 2, 2, 256, 64), randn(g, 2, 2, 256, 64)
    codes, scales = ref_summaries(kc)
    om, w = omega_of(64), torch.ones(64, device=DEV)
    path = torch.zeros(1, dtype=torch.int32, device=DEV)
    tree = random_tree(3, 1, 1)[0]
    calls = [
        (kv.qk_norm_rope, dict(q=q, k=k, omega=om, q_weight=w, k_weight=w, v=v), dict(positions=0)),
        (kv.tree_attention, dict(q=q, k_new=k, v_new=v, k_cache=kc, v_cache=vc),
         dict(tree=tree, lengths=256, scale=0.1)),
        (kv.append_accepted, dict(k_new=k, v_new=v), dict(path=path, counts=None, k_cache=kc.clone(),
                                                          v_cache=vc.clone(), lengths=3)),
        (kv.block_summaries, dict(k_cache=kc), dict(codes=codes.clone(), scales=scales.clone(), lengths=256)),
        (kv.sparse_attention, dict(q=q, k_cache=kc, v_cache=vc, scales=scales),
         dict(codes=codes, lengths=256, top=1, scale=0.1)),
    ]
    for f, ins, rest in calls:
        for name, x in ins.items():
            with pytest.raises(ValueError, match=f"{name} requires grad"):
                f(**{**ins, **rest, name: x.clone().requires_grad_()})
            with fw.dual_level():
                dual = fw.make_dual(x, torch.ones_like(x))
                with torch.no_grad(), pytest.raises(ValueError, match=f"{name} has a tangent"):
                    f(**{**ins, **rest, name: dual})
                f(**ins, **rest)                    # no tangent: as outside
    kv.check_status()


@gpu
def test_python_checks_name_the_argument():
    q, kn, vn, kc, vc = tree_inputs(1, 2, 4, 2, 3, 64, 10)
    tree = random_tree(3, 1, 1)
    call = lambda **kw: kv.tree_attention(**{**dict(q=q, k_new=kn, v_new=vn, tree=tree, k_cache=kc, v_cache=vc,  # noqa: E731
                                                    lengths=4, scale=0.1), **kw})
    for name, bad in (("k_new", kn[:1]), ("k_new", kn.float()), ("v_cache", vc.transpose(2, 3)), ("tree", tree.int()),
                      ("tree", tree[:, :2].contiguous()), ("q", q[0]), ("q", q.cpu()),
                      ("lengths", torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)),
                      ("lengths", torch.tensor([1, 2], device=DEV)), ("q", q.clone().requires_grad_())):
        with pytest.raises(ValueError, match=name):
            call(**{name: bad})
    with torch.no_grad():
        call(q=q.clone().requires_grad_())
    with pytest.raises(kv.StateKVError):
        call(lengths=11)
    call(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))     # none needed: short caches
    long = [torch.zeros(2, 2, 1200, 64, dtype=BF16, device=DEV) for _ in range(2)]
    with pytest.raises(kv.StateKVError):
        call(k_cache=long[0], v_cache=long[1], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(kv.StateKVError):
        call(k_cache=kc[:, :1].expand(2, 2, 10, 64))

"""The operators over paged caches, and a draft's verification, against their
definitions in 64 bits: append, attention of a chunk, accumulated weights,
eviction, and a chain of them.

Pools are filled with NaN but for the rows in use, and table entries past the
last page in use with numbers of no page.

Tolerances, all derived beforehand.
 * Moved rows, kept weights, paths, tokens: equal.
 * Attention with P rounded to bf16 (2^-8 of each term p v): 2^-8 A with A = sum
   p |v| / sum p, and 2^-8 |o| for the output's rounding.  Scores are sums of 128
   exact products in fp32, each step at worst 2^-23 of sum |q k| scale (about 7
   here): 1.1e-4 on the exponent, twice that on a quotient: 2^-12 A.
 * Log-sum-exp: the exponent's 1.1e-4 < 2^-13, and 2^-20 |lse| for its own arithmetic.
 * Weights: each exponential is off by the scores' 2^-13 and its log-sum-exp's
   rounding, 2^-20 of at most 2^5: 2^-12 of itself; a sum of up to N in fp32 by N
   2^-24 of itself, N <= 2^12; 2^-22 of the result for `before`.
"""

import ctypes as C
import math
import random

import numpy as np
import pytest
import torch

import kv_cache_compression_frame_gb300 as kv
from kv_cache_compression_frame_gb300 import _native as N
from test_text_ops import BF16, DEV, _built, gen, randn, ref_attend, view, within  # noqa: F401

gpu = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32


def ints(*x):
    return torch.tensor(x, dtype=I32, device=DEV)


class Cache:
    """Dense rows [n][heads][rows][d] per sequence length, as pages of one
    shuffled pool (page 0: a plain cache)."""

    def __init__(self, g, n, heads, lengths, page, d, dtype=BF16, cap=None, pools=2, strided=False):
        self.page, self.lengths = page, lengths
        cap = cap or max([1, *lengths])
        self.cap = -(-cap // page) * page if page else cap
        self.dense = [randn(g, n, heads, self.cap, d, dtype=dtype) for _ in range(pools)]
        if page:
            per = self.cap // page
            order = torch.randperm(n * per + 2, generator=g, device=DEV)[:n * per].view(n, per)
            shape = (n * per + 2, heads, page, d)
            self.table = torch.full((n, per + 3), 1 << 30, dtype=I32, device=DEV)
            self.table[:, :per] = order.to(I32)
            for i in range(n):
                used = -(-lengths[i] // page)
                self.table[i, used:] = -7
            self.full = order
        else:
            shape, self.table, self.full = (n, heads, self.cap, d), None, None
        self.pools = []
        for x in self.dense:
            if strided:                              # rows before heads, and a gap behind each page
                p = torch.full((shape[0], shape[2] + 1, shape[1], d), math.nan, dtype=dtype, device=DEV)
                p = p[:, :shape[2]].transpose(1, 2)
            else:
                p = torch.full(shape, math.nan, dtype=dtype, device=DEV)
            for i in range(n):
                self.write(p, i, 0, x[i, :, :lengths[i]])
            self.pools.append(p)

    def write(self, pool, i, row0, rows):
        if not self.page:
            pool[i, :, row0:row0 + rows.shape[1]] = rows
            return
        at = torch.arange(row0, row0 + rows.shape[1], device=DEV)
        pool[self.full[i, at // self.page], :, at % self.page] = rows.transpose(0, 1)

    def rows(self, pool, i, count, table=None):
        if not self.page:
            return pool[i, :, :count]
        t = self.full[i] if table is None else table[i].long()
        at = torch.arange(count, device=DEV)
        return pool[t[at // self.page], :, at % self.page].transpose(0, 1)


def check_attention(q, cache, lengths, counts, scale, out, lse, layers=1, what=""):
    n, hq, tok, d = q.shape
    k, v = cache.dense
    G = hq // k.shape[1]
    for i in range(n):
        rows, new = lengths[i // layers], counts[i // layers]
        mask = torch.ones(new, rows, dtype=torch.bool, device=DEV).tril(rows - new).repeat(G, 1)
        if new == 0:
            assert not out[i].any() and (lse is None or bool((lse[i] == -math.inf).all()))
            continue
        for h in range(k.shape[1]):
            qs = q[i, h * G:(h + 1) * G, :new].reshape(-1, d)
            ref, a = ref_attend(qs, k[i, h, :rows], v[i, h, :rows], mask, scale)
            got = out[i, h * G:(h + 1) * G]
            within(got[:, :new].reshape(-1, d), ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a,
                   f"{what} entry {i} head {h}")
            assert not got[:, new:].any()
            if lse is not None:
                x = torch.where(mask, qs.double() @ k[i, h, :rows].double().T * scale, -math.inf)
                want = torch.logsumexp(x, -1).view(G, new)
                within(lse[i, h * G:(h + 1) * G, :new], want, 2.0 ** -13 + 2.0 ** -20 * want.abs(), f"{what} lse")
                assert bool((lse[i, h * G:(h + 1) * G, new:] == -math.inf).all())


# ---------------------------------------------------------------- attention
@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,tok,rows,page", [
    (1, 1, 1, 1, 16), (1, 1, 1, 1, 0), (4, 2, 3, 3, 16), (4, 2, 1, 127, 32), (14, 2, 1, 128, 64), (14, 2, 2, 129, 16),
    (12, 2, 21, 2000, 48),       # 126 rows; pages of three boxes
    (2, 1, 64, 700, 128),        # 128 rows: the last size of one row tile
    (3, 1, 43, 513, 256),        # 129 rows: two tiles, one live row in the second
    (12, 2, 42, 5000, 64),       # 252 rows
    (4, 1, 64, 64, 32),          # 256 rows, no cache before them
    (7, 1, 77, 377, 16),         # 539 rows: three blocks
    (1, 1, 300, 1111, 112),      # blocks of 256 tokens over a diagonal of several tiles
    (1, 1, 257, 257, 0),
    (64, 1, 9, 900, 64),
    (2, 2, 1, 40000, 64),        # one row over many parts
    (12, 2, 38, 20000, 256),     # 228 rows over many parts
    (12, 2, 130, 3333, 0),
])
def test_attention_sizes(d, hq, hkv, tok, rows, page):
    g = gen(rows * 7 + tok + d)
    c = Cache(g, 2, hkv, [rows, rows], page, d)
    q, scale = randn(g, 2, hq, tok, d), 1 / math.sqrt(d)
    out, lse = kv.paged_attention(q, *c.pools, c.table, rows, scale=scale, with_lse=True)
    check_attention(q, c, [rows] * 2, [tok] * 2, scale, out, lse)
    kv.check_status()


@gpu
@pytest.mark.parametrize("layers,page,hq,hkv,tok", [(1, 64, 4, 2, 9), (3, 16, 4, 2, 9), (1, 0, 2, 1, 1), (2, 32, 6, 1, 50),
                                                    (1, 128, 16, 2, 33)])
def test_attention_ragged(layers, page, hq, hkv, tok):
    """Lengths and counts of their own, also none; every row of a padded token."""
    lens = [0, 1, 900, 128, 4097, 64, 255, 50]
    counts = [min(x, y, tok) for x, y in zip(lens, (0, 1, tok, 0, tok, 3, 8, tok))]
    n = len(lens) * layers
    g = gen(layers + page)
    c = Cache(g, n, hkv, [x for x in lens for _ in range(layers)], page, 128)
    q = randn(g, n, hq, tok, 128)
    for i in range(n):
        q[i, :, counts[i // layers]:] = math.nan
    for _ in range(2):
        out, lse = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.1, with_lse=True)
        check_attention(q, c, lens, counts, 0.1, out, lse, layers)
    again = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.1)
    assert torch.equal(again, out)
    kv.check_status()


@gpu
def test_attention_many_units_and_blocks():
    """More units than CTAs, blocks of a prompt cut between CTAs."""
    lens = [1000, 333, 640, 2222, 17, 1, 129]
    counts = [700, 333, 1, 555, 17, 1, 100]
    g = gen(11)
    c = Cache(g, 7, 4, lens, 64, 64)
    q = randn(g, 7, 12, 700, 64)
    out, lse = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.125, with_lse=True)
    check_attention(q, c, lens, counts, 0.125, out, lse)
    kv.check_status()


@gpu
def test_attention_strided_views_and_outputs():
    g = gen(12)
    c = Cache(g, 3, 2, [200, 77, 130], 32, 128, strided=True)
    qkv = randn(g, 3, 20, 8, 128)
    q = qkv[:, :, :6].transpose(1, 2)                # the projection's output
    buf = torch.full((3, 22, 6, 128), 7.0, dtype=BF16, device=DEV)
    out, lse = buf[:, 1:21].transpose(1, 2), torch.full((3, 6, 20), 7.0, device=DEV)
    lens, counts = [200, 77, 130], [20, 5, 11]
    got = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.09, out=out, lse=lse)
    assert got is out
    check_attention(q, c, lens, counts, 0.09, out, lse)
    assert bool((buf[:, 0] == 7).all()) and bool((buf[:, 21] == 7).all())
    # one query for all entries, and one table for all
    q1 = randn(g, 1, 6, 4, 128).expand(3, 6, 4, 128)
    t = c.table[:1].expand(3, -1).contiguous()
    out = kv.paged_attention(q1, *c.pools, t, 200, scale=0.09)
    for i in range(1, 3):
        assert torch.equal(out[i], out[0])
    kv.check_status()


@gpu
@pytest.mark.parametrize("hq,tok,rows", [(2, 40, 170), (1, 200, 260), (4, 90, 90)])
def test_attention_infinities_and_nan_in_masked_places(hq, tok, rows):
    """A new row that is not finite reaches the tokens from its own on, no other."""
    g = gen(tok)
    for bad in (math.nan, math.inf, -math.inf):
        c = Cache(g, 1, 1, [rows], 16, 128)
        at = rows - tok + tok // 2
        c.dense[1][0, 0, at, 5] = bad
        c.write(c.pools[1], 0, 0, c.dense[1][0, :, :rows])
        q = randn(g, 1, hq, tok, 128)
        out = kv.paged_attention(q, *c.pools, c.table, rows, scale=0.1)
        check_attention(q, c, [rows], [tok], 0.1, out, None, what=str(bad))
        assert bool(out[0, :, :tok // 2].isfinite().all())
        # the same in K: the token's own score, and those after it
        c = Cache(g, 1, 1, [rows], 16, 128)
        c.dense[0][0, 0, at, 5] = bad
        c.write(c.pools[0], 0, 0, c.dense[0][0, :, :rows])
        out = kv.paged_attention(q, *c.pools, c.table, rows, scale=0.1)
        ref = kv.paged_attention(q[:, :, :tok // 2].contiguous(), *c.pools, c.table, at, scale=0.1)
        check_attention(q[:, :, :tok // 2], c, [at], [tok // 2], 0.1, out[:, :, :tok // 2], None, what=str(bad))
        assert bool(out[0, :, :tok // 2].isfinite().all()) and bool(ref.isfinite().all())
    kv.check_status()


@gpu
def test_attention_extreme_scores():
    """Scores of hundreds, equal scores, and a reference that has to rise."""
    g = gen(21)
    c = Cache(g, 1, 1, [700], 64, 64)
    q = randn(g, 1, 4, 5, 64)
    k = c.dense[0]
    k[0, 0, :300] = 0
    k[0, 0, 300:600] *= torch.linspace(0.1, 30, 300, device=DEV)[:, None].to(BF16)
    c.write(c.pools[0], 0, 0, k[0, :, :700])
    out, lse = kv.paged_attention(q, *c.pools, c.table, 700, scale=0.5, with_lse=True)
    i = torch.ones(5, 700, dtype=torch.bool, device=DEV).tril(695).repeat(4, 1)
    x = torch.where(i, q[0].reshape(-1, 64).double() @ k[0, 0, :700].double().T * 0.5, -math.inf)
    # sums of 64 products of magnitude up to 30 * 16 each: 64 steps of 2^-24 of at most 1000
    tol = 64 * 2.0 ** -24 * 1000
    within(lse[0].reshape(-1), torch.logsumexp(x, -1), tol + 2.0 ** -20 * x.amax(-1).abs())
    ref, a = ref_attend(q[0].reshape(-1, 64), k[0, 0, :700], c.dense[1][0, 0, :700], i, 0.5)
    within(out[0].reshape(-1, 64), ref, 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * tol) * a)
    kv.check_status()


@gpu
def test_attention_bad_lengths_counts_and_pages_are_recorded():
    g = gen(13)
    c = Cache(g, 3, 2, [100, 100, 100], 16, 64, cap=112)
    q = randn(g, 3, 2, 4, 64)
    good = kv.paged_attention(q, *c.pools, c.table, 100, scale=0.1)
    for lens, counts, table in ((ints(100, -5, 100), None, c.table), (ints(100, 1 << 20, 100), None, c.table),
                                (ints(100, 100, 100), ints(4, -1, 4), c.table),
                                (ints(100, 100, 100), ints(4, 5, 4), c.table), (ints(100, 3, 100), None, c.table),
                                (ints(100, 100, 100), None, torch.where(c.table == c.table[1, 3], 1 << 20, c.table)),
                                (ints(100, 100, 100), None, torch.where(c.table == c.table[1, 6], -1, c.table))):
        out = kv.paged_attention(q, *c.pools, table.contiguous(), lens, counts, scale=0.1)
        with pytest.raises(kv.StateKVError) as e:
            kv.check_status()
        assert e.value.status == N.E_DEVICE
        # the other sequences are as they were
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    kv.check_status()


@gpu
def test_attention_offsets_past_32_bits():
    g = gen(14)
    pages = (1 << 31) // (2 * 256 * 128) + 40            # elements pass 2^31
    pools = [torch.zeros((pages, 2, 256, 128), dtype=BF16, device=DEV) for _ in range(2)]
    c = Cache(g, 1, 2, [1000], 256, 128)
    t = torch.tensor([[pages - 1, 3, pages - 7, pages - 20]], dtype=I32, device=DEV)
    at = torch.arange(1000, device=DEV)
    for p, x in zip(pools, c.dense):
        p[t[0].long()[at // 256], :, at % 256] = x[0, :, :1000].transpose(0, 1)
    q = randn(g, 1, 4, 30, 128)
    out, lse = kv.paged_attention(q, *pools, t, 1000, scale=0.1, with_lse=True)
    check_attention(q, c, [1000], [30], 0.1, out, lse)
    w = kv.attention_weights(q, lse, pools[0], t, 1000, scale=0.1)
    check_weights(q, lse, c, [1000], [30], 0.1, None, w)
    new = kv.paged_append(c.dense[0][:, :, :24], c.dense[1][:, :, :24], *pools, t, 1000)
    assert new == 1024
    assert torch.equal(pools[0][pages - 20, :, 232:], c.dense[0][0, :, :24])
    assert torch.equal(pools[1][pages - 20, :, 232:], c.dense[1][0, :, :24])
    kv.check_status()


# ------------------------------------------------------------------ weights
def check_weights(q, lse, cache, lengths, counts, scale, before, got, layers=1):
    n, hq, tok, d = q.shape
    k = cache.dense[0]
    G = hq // k.shape[1]
    for i in range(n):
        rows, new = lengths[i // layers], counts[i // layers]
        mask = torch.ones(new, rows, dtype=torch.bool, device=DEV).tril(rows - new)
        for h in range(k.shape[1]):
            x = torch.einsum("gtd,kd->gtk", q[i, h * G:(h + 1) * G, :new].double(), k[i, h, :rows].double()) * scale
            at = lse[i, h * G:(h + 1) * G, :new, None].double()
            add = torch.where(mask & (at != -math.inf), torch.exp(x - at), 0.0).sum((0, 1))
            b = before[i, h] if before is not None else torch.zeros(got.shape[2], device=DEV)
            ref = b[:rows].double() + add
            within(got[i, h, :rows], ref, 2.0 ** -11 * add + 2.0 ** -22 * ref.abs(), f"entry {i} head {h}")
            assert torch.equal(got[i, h, rows if new else 0:], b[rows if new else 0:])


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,tok,rows,page", [
    (1, 1, 1, 1, 16), (14, 2, 1, 300, 16), (12, 2, 1, 5000, 64), (12, 2, 21, 2000, 48), (2, 1, 64, 700, 128),
    (7, 1, 77, 377, 16), (1, 1, 300, 1111, 112), (1, 1, 129, 129, 0), (64, 1, 9, 900, 64), (33, 1, 7, 257, 32),
    (12, 2, 130, 3333, 0), (5, 1, 256, 256, 256)])
def test_weights_sizes(d, hq, hkv, tok, rows, page):
    g = gen(rows + tok + d)
    c = Cache(g, 2, hkv, [rows, rows], page, d)
    q, scale = randn(g, 2, hq, tok, d), 1 / math.sqrt(d)
    _, lse = kv.paged_attention(q, *c.pools, c.table, rows, scale=scale, with_lse=True)
    cap = c.cap if c.table is None else c.table.shape[1] * page
    before = torch.rand((2, hkv, cap + 5), generator=g, device=DEV)
    got = kv.attention_weights(q, lse, c.pools[0], c.table, rows, scale=scale, before=before)
    check_weights(q, lse, c, [rows] * 2, [tok] * 2, scale, before, got)
    # every query's probabilities sum to 1
    w = kv.attention_weights(q, lse, c.pools[0], c.table, rows, scale=scale)
    assert w.shape == (2, hkv, cap)
    within(w.sum(-1), torch.full((2, hkv), hq // hkv * tok, dtype=torch.float64, device=DEV),
           2.0 ** -11 * hq // hkv * tok + 2.0 ** -11 * hq / hkv * tok)
    got2 = kv.attention_weights(q, lse, c.pools[0], c.table, rows, scale=scale, before=before, out=before)
    assert got2 is before and torch.equal(got2, got)
    kv.check_status()


@gpu
@pytest.mark.parametrize("layers,page,tok", [(1, 64, 9), (3, 16, 33), (2, 0, 70)])
def test_weights_ragged(layers, page, tok):
    lens = [0, 1, 900, 128, 4097, 64, 255, 90]
    counts = [min(x, y) for x, y in zip(lens, (0, 1, tok, 0, tok, 3, 8, tok))]
    n = len(lens) * layers
    g = gen(layers + page)
    c = Cache(g, n, 2, [x for x in lens for _ in range(layers)], page, 128)
    q = randn(g, n, 4, tok, 128)
    for i in range(n):
        q[i, :, counts[i // layers]:] = math.nan
    _, lse = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.1, with_lse=True)
    lse[:, 1, 0] = -math.inf                         # a query that adds nothing
    cap = c.cap if c.table is None else c.table.shape[1] * page
    before = torch.rand((n, 2, cap), generator=g, device=DEV)
    got = kv.attention_weights(q, lse, c.pools[0], c.table, ints(*lens), ints(*counts), scale=0.1, before=before)
    check_weights(q, lse, c, lens, counts, 0.1, before, got, layers)
    again = kv.attention_weights(q, lse, c.pools[0], c.table, ints(*lens), ints(*counts), scale=0.1, before=before)
    assert torch.equal(again, got)
    kv.check_status()


@gpu
@pytest.mark.parametrize("seqs,layers,page,hq,tok", [(33, 1, 64, 4, 3), (77, 2, 16, 4, 9), (40, 1, 64, 4, 300),
                                                     (70, 2, 0, 2, 150)])
def test_attention_and_weights_of_many_sequences(seqs, layers, page, hq, tok):
    """More sequences than a warp has lanes, one block of query rows each or
    several (padded prompts), ragged, some without tokens."""
    r = random.Random(seqs)
    lens = [r.choice([0, 1, r.randrange(2, 400), r.randrange(300, 1500)]) for _ in range(seqs - 1)] + [3000]
    counts = [r.choice([0, 1, min(x, tok), r.randrange(0, min(x, tok) + 1)]) if x else 0 for x in lens[:-1]] + [tok]
    n = seqs * layers
    g = gen(seqs)
    c = Cache(g, n, 2, [x for x in lens for _ in range(layers)], page, 64)
    q = randn(g, n, hq, tok, 64)
    out, lse = kv.paged_attention(q, *c.pools, c.table, ints(*lens), ints(*counts), scale=0.125, with_lse=True)
    check_attention(q, c, lens, counts, 0.125, out, lse, layers)
    cap = c.cap if c.table is None else c.table.shape[1] * page
    before = torch.rand((n, 2, cap), generator=g, device=DEV)
    got = kv.attention_weights(q, lse, c.pools[0], c.table, ints(*lens), ints(*counts), scale=0.125, before=before)
    check_weights(q, lse, c, lens, counts, 0.125, before, got, layers)
    kv.check_status()


@gpu
def test_weights_of_rows_that_are_not_finite_stay_their_own():
    g = gen(31)
    c = Cache(g, 1, 1, [400], 16, 64)
    q = randn(g, 1, 3, 50, 64)
    _, lse = kv.paged_attention(q, *c.pools, c.table, 400, scale=0.1, with_lse=True)
    want = kv.attention_weights(q, lse, c.pools[0], c.table, 400, scale=0.1)
    c.dense[0][0, 0, 7, 3] = math.nan
    c.dense[0][0, 0, 390, 3] = math.inf
    c.write(c.pools[0], 0, 0, c.dense[0][0, :, :400])
    got = kv.attention_weights(q, lse, c.pools[0], c.table, 400, scale=0.1)
    assert bool(got[0, 0, 7].isnan())
    for r in (7, 390):
        got[0, 0, r] = want[0, 0, r]
    assert torch.equal(got, want)
    kv.check_status()
    bad = c.table.clone()
    bad[0, 5] = 1 << 20
    kv.attention_weights(q, lse, c.pools[0], bad, 400, scale=0.1)
    with pytest.raises(kv.StateKVError):
        kv.check_status()


@gpu
def test_weights_in_an_array_of_the_most_rows():
    """Rows behind the length are zeros up to the last of 2^31 - 1 (copied in pieces of 512)."""
    g = gen(54)
    c = Cache(g, 1, 1, [40], 16, 64)
    q = randn(g, 1, 1, 3, 64)
    _, lse = kv.paged_attention(q, *c.pools, c.table, 40, scale=0.1, with_lse=True)
    out = torch.full((1, 1, 2 ** 31 - 1), 9.0, device=DEV)
    kv.attention_weights(q, lse, c.pools[0], c.table, 40, scale=0.1, out=out)
    assert torch.equal(out[:, :, :40], kv.attention_weights(q, lse, c.pools[0], c.table, 40, scale=0.1)[:, :, :40])
    assert int(out.count_nonzero()) == 40
    kv.check_status()


# ------------------------------------------------------------------- append
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layers,page,tok,d", [(1, 16, 1, 128), (2, 64, 40, 64), (1, 0, 7, 96), (3, 32, 100, 128)])
def test_append(dtype, layers, page, tok, d):
    lens = [0, 16, 37, 100]
    counts = [tok, 0, min(tok, 5), max(1, tok - 1)]
    n = 4 * layers
    g = gen(page + tok)
    c = Cache(g, n, 2, [x + y for x, y in zip(lens, counts) for _ in range(layers)], page, d, dtype, cap=100 + tok)
    before = [p.clone() for p in c.pools]
    k, v = randn(g, n, 2, tok, d, dtype=dtype), randn(g, n, tok, 2, d, dtype=dtype).transpose(1, 2)
    new = kv.paged_append(k, v, *c.pools, c.table, ints(*lens), ints(*counts))
    assert new.tolist() == [x + y for x, y in zip(lens, counts)]
    for pool, old, x in zip(c.pools, before, (k, v)):
        for i in range(n):
            c.write(old, i, lens[i // layers], x[i, :, :counts[i // layers]])
        assert torch.equal(pool.view(torch.int16), old.view(torch.int16))
    kv.check_status()


@gpu
def test_append_that_does_not_fit_is_recorded():
    g = gen(41)
    c = Cache(g, 3, 2, [48, 48, 48], 16, 64)
    t = c.table[:, :3].contiguous()
    k = randn(g, 3, 2, 4, 64)
    old = [p.clone() for p in c.pools]
    bad = t.clone()
    bad[2, 2] = 99
    for lens, counts, table in ((ints(40, 45, 3), None, t), (ints(40, -1, 3), ints(4, 0, 4), t),
                                (ints(40, 20, 3), ints(4, 9, 4), t), (ints(40, 20, 32), ints(4, 4, 4), bad)):
        new = kv.paged_append(k, k, *c.pools, table, lens, counts)
        with pytest.raises(kv.StateKVError) as e:
            kv.check_status()
        assert e.value.status == N.E_DEVICE
        assert new[0] == 44
        assert torch.equal(c.rows(c.pools[0], 0, 44)[:, 40:], k[0])
        for p, x in zip(c.pools, old):
            p.copy_(x)
    assert kv.paged_append(k, k, *c.pools, t, 44) == 48
    with pytest.raises(kv.StateKVError):
        kv.paged_append(k, k, *c.pools, t, 45)
    kv.check_status()


@gpu
def test_append_of_a_tensor_of_the_most_tokens():
    """Fewer rows than `tokens`, whose blocks of 32 are counted past 2^31 - 1."""
    k = torch.arange(8, dtype=F32, device=DEV).expand(1, 1, 2 ** 31 - 1, 8)
    pools = [torch.zeros((1, 1, 100, 8), device=DEV) for _ in range(2)]
    new = kv.paged_append(k, k, *pools, None, ints(7), ints(80))
    assert new.tolist() == [87]
    for p in pools:
        assert torch.equal(p[0, 0, 7:87], k[0, 0, :80]) and not p[0, 0, :7].any() and not p[0, 0, 87:].any()
    kv.check_status()


# ----------------------------------------------------------------- eviction
def kept_rows(w, rows, keep, sinks, recent):
    """The rows that stay, by sorting."""
    if rows <= keep:
        return list(range(rows))
    w = w.tolist()
    key = lambda r: (w[r] == w[r], w[r] if w[r] == w[r] else 0, -r)  # noqa: E731  (NaN below all)
    free = sorted(range(sinks, rows - recent), key=key, reverse=True)[:keep - sinks - recent]
    return sorted([*range(sinks), *free, *range(rows - recent, rows)])


def check_evict(c, lens, layers, w, keep, sinks, recent, old, pools, out_table, got, out_page):
    new, w_out, kept = got
    n, hkv = w.shape[:2]
    assert (new if isinstance(new, int) else new.tolist()) == (min(lens[0], keep) if isinstance(new, int) else
                                                               [min(x, keep) for x in lens])
    for i in range(n):
        rows = lens[i // layers]
        for h in range(hkv):
            want = kept_rows(w[i, h], rows, keep, sinks, recent)
            m = len(want)
            assert kept[i, h].tolist() == want + [-1] * (keep - m)
            at = torch.tensor(want, dtype=torch.int64, device=DEV)
            assert torch.equal(w_out[i, h, :m].nan_to_num(-3), w[i, h, at].nan_to_num(-3))
            assert not w_out[i, h, m:].any()
            for src, dst in zip(old, pools):
                to = torch.arange(m, device=DEV)
                moved = dst[out_table[i].long()[to // out_page], h, to % out_page] if out_page else dst[i, h, :m]
                assert torch.equal(moved, c.rows(src, i, rows)[h, at])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layers,page,rows,keep,sinks,recent", [
    (1, 16, 1, 1, 0, 0), (1, 64, 1000, 1, 0, 0), (2, 32, 1000, 500, 4, 100), (1, 16, 4500, 4096, 4, 128),
    (1, 0, 777, 333, 0, 10), (1, 64, 300, 300, 0, 0), (1, 64, 300, 100, 60, 40), (1, 128, 70000, 200, 1, 1),
    (1, 16, 50, 64, 3, 5)])
def test_evict(dtype, layers, page, rows, keep, sinks, recent):
    g = gen(rows + keep)
    lens = [rows, max(1, rows // 2), 0, rows - rows // 5]
    n = 4 * layers
    c = Cache(g, n, 2, [x for x in lens for _ in range(layers)], page, 64, dtype)
    cap = c.cap if c.table is None else c.table.shape[1] * page
    w = torch.rand((n, 2, cap), generator=g, device=DEV)
    w[0] = (w[0] * 8).floor()                        # many ties
    w[-1] = -w[-1]
    w[-1, 0, ::3] = 0.0
    w[-1, 0, 1::3] = -0.0                            # equal to 0
    w[1, 1, ::5] = math.nan
    w[1, 1, 1::7] = math.inf
    w[1, 1, 2::7] = -math.inf
    per = -(-keep // page) if page else 0
    order = torch.randperm(n * per, generator=g, device=DEV).view(n, per).to(I32) if page else None
    out = [torch.full((n * per, 2, page, 64) if page else (n, 2, keep, 64), 9.0, dtype=dtype, device=DEV)
           for _ in range(2)]
    lengths = torch.tensor(lens, dtype=I32, device=DEV)
    got = kv.evict_rows(*c.pools, c.table, lengths, w, keep, order, sinks=sinks, recent=recent, k_out=out[0],
                        v_out=out[1])
    check_evict(c, lens, layers, w, keep, sinks, recent, c.pools, out, order, got, page)
    if page:
        # rows of the last page past the kept ones stay as they were
        m = min(rows, keep)
        if m % page:
            assert bool((out[0][order[0, m // page].long(), :, m % page:] == 9).all())
    kv.check_status()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,out_page,keep", [(64, 16, 333), (16, 128, 100), (48, 32, 600), (0, 16, 200), (0, 64, 77),
                                                (32, 0, 150), (16, 0, 500)])
def test_evict_between_pages_of_two_sizes(page, out_page, keep, dtype):
    """Pools of their own page sizes, and a plain cache (0) on one side."""
    g = gen(page + out_page)
    lens, n = [600, 31, 0, 599], 4
    c = Cache(g, n, 2, lens, page, 64, dtype)
    cap = c.cap if c.table is None else c.table.shape[1] * page
    w = torch.rand((n, 2, cap), generator=g, device=DEV)
    per = -(-keep // out_page) if out_page else 0
    order = torch.randperm(n * per, generator=g, device=DEV).view(n, per).to(I32) if out_page else None
    out = [torch.full((n * per, 2, out_page, 64) if out_page else (n, 2, keep + 3, 64), 9.0, dtype=dtype, device=DEV)
           for _ in range(2)]
    got = kv.evict_rows(*c.pools, c.table, ints(*lens), w, keep, order, sinks=3, recent=20, k_out=out[0], v_out=out[1])
    assert got[1].shape == (n, 2, per * out_page if out_page else keep + 3)
    check_evict(c, lens, 1, w, keep, 3, 20, c.pools, out, order, got, out_page)
    kv.check_status()


@gpu
def test_evict_within_one_pool():
    """Source and destination pages of one pool; a page of the source that two
    sequences share stays as it is."""
    g = gen(51)
    c = Cache(g, 2, 2, [200, 200], 16, 128, cap=208)
    c.table[1, 0] = c.table[0, 0]
    c.full[1, 0] = c.full[0, 0]
    more = [torch.cat([p, torch.full((20, 2, 16, 128), math.nan, dtype=BF16, device=DEV)]) for p in c.pools]
    fresh = (len(c.pools[0]) + torch.randperm(14, generator=g, device=DEV)).view(2, 7).to(I32)
    old = [p.clone() for p in more]
    w = torch.rand((2, 2, c.table.shape[1] * 16), generator=g, device=DEV)
    got = kv.evict_rows(*more, c.table, 200, w, 100, fresh, sinks=16, recent=20)
    assert got[1].shape == (2, 2, 112)
    check_evict(c, [200, 200], 1, w, 100, 16, 20, old, more, fresh, got, 16)
    for p, x in zip(more, old):
        assert torch.equal(p[:len(c.pools[0])].view(torch.int16), x[:len(c.pools[0])].view(torch.int16))
    kv.check_status()
    # nothing stays
    new, w_out, kept = kv.evict_rows(*more, c.table, ints(200, 3), w, 0, fresh)
    assert new.tolist() == [0, 0] and kept.shape == (2, 2, 0) and not w_out.any()
    # lengths and pages out of range
    for lens, table in ((ints(200, 5000), c.table), (ints(200, -1), c.table),
                        (ints(200, 200), torch.where(c.table == c.table[1, 5], -1, c.table))):
        kv.evict_rows(*more, table, lens, w, 100, fresh)
        with pytest.raises(kv.StateKVError):
            kv.check_status()
    kv.check_status()


@gpu
def test_evict_long_rows():
    """More rows than a cluster's shared memory holds."""
    g = gen(52)
    rows = 700_001
    k = torch.arange(rows, device=DEV, dtype=F32)[None, None, :, None].expand(1, 1, rows, 8).contiguous()
    w = torch.rand((1, 1, rows), generator=g, device=DEV)
    out = [torch.zeros((1, 1, 5000, 8), device=DEV) for _ in range(2)]
    new, w_out, kept = kv.evict_rows(k, k, None, rows, w, 5000, None, recent=7, k_out=out[0], v_out=out[1])
    want = torch.cat([w[0, 0, :-7].topk(4993).indices.sort().values, torch.arange(rows - 7, rows, device=DEV)])
    assert torch.equal(kept[0, 0].long(), want) and new == 5000
    assert torch.equal(out[1][0, 0, :, 0].long(), want)
    kv.check_status()


@gpu
def test_evict_into_an_array_of_the_most_weights():
    """Zeros up to the last of 2^31 - 1 entries (counted in steps of a cluster's threads)."""
    k = torch.arange(40, device=DEV, dtype=F32)[None, None, :, None].expand(1, 1, 40, 8).contiguous()
    w = torch.rand((1, 1, 40), generator=gen(53), device=DEV)
    out = [torch.zeros((1, 1, 3, 8), device=DEV) for _ in range(2)]
    w_out = torch.full((1, 1, 2 ** 31 - 1), 9.0, device=DEV)
    new, _, kept = kv.evict_rows(k, k.clone(), None, 40, w, 3, None, k_out=out[0], v_out=out[1], weights_out=w_out)
    want = w[0, 0].topk(3).indices.sort().values
    assert new == 3 and torch.equal(kept[0, 0].long(), want) and torch.equal(w_out[0, 0, :3], w[0, 0, want])
    assert int(w_out.count_nonzero()) == 3
    kv.check_status()


# ------------------------------------------------------------- verification
def plain_verify(target, draft, drafted, masks, uniforms):
    """One sequence, from the definition: the residual after each refusal is a
    distribution of its own."""
    tok = len(drafted)
    parent = [((m & ((1 << 64) - 1)) & ((1 << i) - 1)).bit_length() - 1 for i, m in enumerate(masks)]
    at, path = -1, []
    while True:
        p = target[at + 1].double()
        rest, left, done = p.clone(), 1.0, False
        for i in (i for i in range(tok) if parent[i] == at):
            x, u = drafted[i], uniforms[i]
            if draft is None:
                if u * left < float(rest[x]):
                    done = True
                    break
                left = max(0.0, left - float(rest[x]))
                rest[x] = 0.0
            else:
                q = draft[at + 1].double()
                if u * float(q[x]) * left < float(rest[x]):
                    done = True
                    break
                rest = (rest - left * q).clamp(min=0.0)
                left = float(rest.sum())
        if not done:
            break
        at = i
        path.append(i)
    if float(rest.sum()) == 0.0:
        rest = p
    upto = rest.cumsum(0)
    return path, int((upto <= uniforms[tok] * upto[-1]).sum())


def verify_case(g, seqs, tok, vocab, seed, spread=2.0):
    r = random.Random(seed)
    parents = [[r.randrange(-1 if i < 3 else max(0, i - 5), i) if i else -1 for i in range(tok)] for _ in range(seqs)]
    tree, _ = kv.tree_masks(parents, DEV)
    x = spread * torch.randn((seqs, tok + 1, vocab), generator=g, device=DEV)
    p = torch.softmax(x, -1)
    q = torch.softmax(x + torch.randn(x.shape, generator=g, device=DEV), -1)
    rows = torch.tensor(parents, device=DEV) + 1
    drafted = torch.multinomial(q[torch.arange(seqs, device=DEV)[:, None], rows].flatten(0, 1), 1, generator=g)
    return p, q, drafted.view(seqs, tok).to(I32), tree, torch.rand((seqs, tok + 1), generator=g, device=DEV)


@gpu
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("seqs,tok,vocab", [(1, 1, 2), (3, 7, 100), (40, 5, 33), (2, 64, 4097), (16, 42, 10007), (1, 9, 150001),
                                            (200, 3, 1), (1, 5, 1_000_003), (160, 4, 40001), (24, 6, 150000)])
def test_verify(seqs, tok, vocab, with_draft):
    g = gen(seqs + tok)
    p, q, drafted, tree, u = verify_case(g, seqs, tok, vocab, seqs * tok)
    q = q if with_draft else None
    path, counts, after = kv.verify_tree(p, q, drafted, tree, u)
    for s in range(seqs):
        want, token = plain_verify(p[s], None if q is None else q[s], drafted[s].tolist(), tree[s].tolist(),
                                   u[s].double().tolist())
        assert path[s].tolist() == want + [-1] * (tok - len(want)), s
        assert int(counts[s]) == len(want) and int(after[s]) == token, s
    kv.check_status()


@gpu
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_keeps_the_target_distribution(with_draft):
    """The first token after the text is distributed as the target's row 0
    whatever the draft: three siblings, 60000 sequences, each frequency within 5
    standard deviations."""
    g = gen(77)
    seqs, vocab = 60000, 6
    p = torch.softmax(torch.randn((1, 1, vocab), generator=g, device=DEV), -1).expand(seqs, 4, vocab)
    q = torch.softmax(torch.randn((1, 1, vocab), generator=g, device=DEV), -1).expand(seqs, 4, vocab)
    if with_draft:
        drafted = torch.multinomial(q[:, 0].contiguous(), 3, replacement=True, generator=g).to(I32)
    else:
        drafted = torch.tensor([4, 0, 2], dtype=I32, device=DEV).expand(seqs, 3).contiguous()
    tree, _ = kv.tree_masks([-1, -1, -1], DEV)
    u = torch.rand((seqs, 4), generator=g, device=DEV)
    path, counts, after = kv.verify_tree(p, q if with_draft else None, drafted, tree, u)
    first = torch.where(counts > 0, drafted.gather(1, path[:, :1].clamp(min=0).long())[:, 0], after)
    want = p[0, 0].double()
    got = torch.bincount(first, minlength=vocab).double() / seqs
    assert bool(((got - want).abs() <= 5 * (want * (1 - want) / seqs).sqrt()).all())
    assert 0.1 < float((counts > 0).double().mean()) < 1
    kv.check_status()


@gpu
def test_verify_edges():
    tree, _ = kv.tree_masks([-1, 0, 0, -1], DEV)
    one = lambda *x: torch.tensor(x, dtype=F32, device=DEV)  # noqa: E731
    p = one(0.5, 0.25, 0.25, 0.0).expand(1, 5, 4).contiguous()
    t = torch.tensor([[0, 0, 1, 0]], dtype=I32, device=DEV)
    # equal distributions: everything stands, u = 0 picks the first token that can be
    got = kv.verify_tree(p, p, t, tree, torch.full((1, 5), 0.999, device=DEV))
    assert got[0].tolist() == [[0, 1, -1, -1]] and got[1].tolist() == [2] and got[2].tolist() == [2]
    z = p.roll(1, -1).contiguous()
    assert kv.verify_tree(z, None, t, tree, torch.zeros((1, 5), device=DEV))[2].tolist() == [1]
    # nothing is left after a refusal (the draft is above the target everywhere): the target's row
    q = one(1.0, 1.0, 1.0, 1.0).expand(1, 5, 4).contiguous()
    got = kv.verify_tree(p, q, t, tree, torch.full((1, 5), 0.6, device=DEV))
    assert got[1].tolist() == [0] and got[2].tolist() == [1]
    # rows of zeros, NaN and negative values count as 0
    got = kv.verify_tree(torch.zeros_like(p), None, t, tree, torch.full((1, 5), 0.6, device=DEV))
    assert got[1].tolist() == [0] and got[2].tolist() == [0]
    bad = one(math.nan, -1.0, 0.0, 1.0).expand(1, 5, 4).contiguous()
    got = kv.verify_tree(bad, None, t, tree, torch.full((1, 5), 0.3, device=DEV))
    assert got[1].tolist() == [0] and got[2].tolist() == [3]
    # uniforms out of range are clamped
    for u, tok in ((1.5, 2), (-3.0, 0), (math.nan, 0)):
        got = kv.verify_tree(p, None, torch.full_like(t, 3), tree, torch.full((1, 5), u, device=DEV))
        assert got[1].tolist() == [0] and got[2].tolist() == [tok], u
    # the same token twice among siblings
    got = kv.verify_tree(p, None, torch.tensor([[1, 1, 1, 1]], dtype=I32, device=DEV),
                         kv.tree_masks([-1, -1, -1, -1], DEV)[0], torch.full((1, 5), 0.5, device=DEV))
    assert got[1].tolist() == [0] and got[2].tolist() == [0]
    kv.check_status()
    # a token that is none: refused and recorded
    got = kv.verify_tree(p, None, torch.tensor([[4, 0, 0, -1]], dtype=I32, device=DEV), tree,
                         torch.zeros((1, 5), device=DEV))
    assert got[1].tolist() == [0] and got[2].tolist() == [0]
    with pytest.raises(kv.StateKVError):
        kv.check_status()


@gpu
def test_verify_of_rows_that_are_no_probabilities_gives_some_token():
    """Rows whose sums leave 64 bits in units of 2^-52 (16 warps of 128 entries of
    14.95 each), infinities, and the largest numbers."""
    tree, t = kv.tree_masks([-1, 0], DEV)[0], torch.zeros((1, 2), dtype=I32, device=DEV)
    for vocab, value, u in [(2048, 14.95, 0.999), (2048, 3e38, 0.7), (150001, 1.0, 0.9), (150001, 7.3, 0.6),
                            (5000, math.inf, 0.5), (150001, math.inf, 0.99)]:
        p = torch.full((1, 3, vocab), value, device=DEV)
        for q in (None, p, p.roll(1, -1) / 3):
            torch.full((4,), -7, dtype=I32, device=DEV)          # what the outputs' memory holds
            path, counts, after = kv.verify_tree(p, q, t, tree, torch.full((1, 3), u, device=DEV))
            n = int(counts)
            assert 0 <= int(after) < vocab and 0 <= n <= 2, (vocab, value)
            assert path[0].tolist() == list(range(n)) + [-1] * (2 - n), (vocab, value)
    kv.check_status()


@gpu
def test_verify_sums_what_a_tiny_residual_leaves():
    """After a residual R1 <= 2^-24 the whole of c = 1 + R1 counts, not what fp32 holds of it."""
    f = lambda *x: torch.tensor(x, dtype=F32, device=DEV)  # noqa: E731
    # residuals 2^-24, 2^-25, 2^-26, all of token 0: it is next whatever the last uniform
    e = 2.0 ** -24
    p, q = (f(*x).expand(4, 4, 2).contiguous() for x in ((0.5 + e, 0.5 - e), (0.5, 0.5)))
    u = f(1 - e).expand(4, 4).contiguous()
    u[:, 3] = f(0.0, 0.4, 0.75, 1 - e)
    path, counts, after = kv.verify_tree(p, q, torch.ones((4, 3), dtype=I32, device=DEV),
                                         kv.tree_masks([-1, -1, -1], DEV)[0], u)
    assert not counts.any() and not after.any()
    # one token drafted twice that the target never has, and two others to choose from
    n, g = 1000, gen(61)
    q = [5e-8, 0.25, 1e-4, 0.74989995]
    p = torch.tensor([[0.0, 0.25, 1e-4 + 2e-8, 0.7498]], device=DEV)
    p[0, 1] = torch.nextafter(p[0, 1], torch.ones_like(p[0, 1]))
    p, q = p.expand(n, 3, 4).contiguous(), f(*q).expand(n, 3, 4).contiguous()
    u = torch.rand((n, 3), generator=g, device=DEV)
    t, tree = torch.zeros((n, 2), dtype=I32, device=DEV), kv.tree_masks([-1, -1], DEV)[0]
    path, counts, after = kv.verify_tree(p, q, t, tree, u)
    pc, qc = p[0].cpu(), q[0].cpu()
    want = [plain_verify(pc, qc, [0, 0], tree[0].tolist(), x)[1] for x in u.cpu().double().tolist()]
    assert not counts.any() and after.tolist() == want and len(set(want)) == 2
    kv.check_status()


def near_boundary(seed, vocab, with_draft):
    """Rows p, q (float32 [vocab]) whose residual after the refused token 5 has
    sums that pass half of the whole by 2^-48 at entry v, or miss it by that:
    (p, q, token).  Every entry is 0 or at least 2^-36, a whole number of 2^-60 then,
    so the sums here are exact."""
    r = np.random.default_rng(seed)
    units = lambda x: (x.astype(np.float64) * 2.0 ** 60).astype(np.int64)  # noqa: E731
    p = np.exp(r.standard_normal(vocab))
    p[:3] = 1e-2 * p.sum(), 2.0 ** -20, 2.0 ** -30
    q = np.where(np.arange(vocab) % 7 < 3, 0.9, 1.3) * p
    p = np.maximum(p / p.sum(), 2.0 ** -36).astype(np.float32)
    q = np.maximum(q / q.sum(), 2.0 ** -36).astype(np.float32)
    p[1:3] = 2.0 ** -20, 2.0 ** -30
    q[:3] = 2.0 ** -36
    p[5], q[5] = 2.0 ** -34, 2.0 ** -8                       # refused

    def rest():
        x = units(p) - units(q) if with_draft else units(p)
        x = np.maximum(x, 0)
        x[5] = 0
        return x

    upto = rest().cumsum()
    v = int(np.searchsorted(2 * upto, upto[-1]))
    sign = 1 if seed % 2 else -1
    for i in range(3):
        # what twice the sum up to v passes the whole by, by the entry i <= v alone
        x = rest()
        over = 2 * int(x[:v + 1].sum()) - int(x.sum()) - sign * 2 ** 13
        p[i] = np.float32(float(p[i]) - over * 2.0 ** -60)
        assert p[i] > 2.0 ** -35
    x = rest()
    over = 2 * int(x[:v + 1].sum()) - int(x.sum())
    assert v > 100 and abs(over - sign * 2 ** 13) <= 2 ** 8
    return p, q, v if sign > 0 else v + 1 + int(np.flatnonzero(x[v + 1:])[0])


@gpu
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("vocab", [20011, 40009])
def test_verify_next_to_a_boundary_in_any_batch(vocab, with_draft):
    """The token changes where its sum passes u times the whole, however many
    CTAs the row is cut over: margins of 2^-48 of it, alone and in larger batches.
    (p - c q with c = 1 is exact as two fp32 numbers, and half the whole is off by 2^-54.)"""
    n = 128
    cases = [near_boundary(i, vocab, with_draft) for i in range(n)]
    p = torch.tensor(np.stack([c[0] for c in cases]), device=DEV)[:, None].expand(n, 2, vocab)
    q = torch.tensor(np.stack([c[1] for c in cases]), device=DEV)[:, None].expand(n, 2, vocab) if with_draft else None
    want = [c[2] for c in cases]
    t = torch.full((n, 1), 5, dtype=I32, device=DEV)
    u = torch.tensor([[0.999, 0.5]], device=DEV).repeat(n, 1)
    tree = kv.tree_masks([-1], DEV)[0]
    for batch in (128, 40, 16, 1):
        for s in range(0, n, batch):
            e = min(n, s + batch)
            _, counts, after = kv.verify_tree(p[s:e], None if q is None else q[s:e], t[s:e], tree, u[s:e])
            assert not counts.any() and after.tolist() == want[s:e], batch
    kv.check_status()


# ------------------------------------------------------------------- chains
@gpu
def test_a_served_text_eager_and_replayed():
    """A prompt, then tokens one by one, with eviction when the cache is full:
    append, attention, weights, eviction, each step against the definition; a
    step captured into a graph gives the same bits."""
    g = gen(61)
    n, hq, hkv, d, page, keep = 3, 8, 2, 128, 32, 96
    lens = [70, 0, 33]
    c = Cache(g, n, hkv, lens, page, d, cap=256)
    pools = [torch.cat([p, torch.full_like(p, math.nan)]) for p in c.pools]
    table = c.full.to(I32).contiguous()
    spare = (len(c.pools[0]) + torch.arange(n * table.shape[1], device=DEV)).view(n, -1).to(I32)
    lengths = ints(*lens)
    weights = torch.zeros((n, hkv, 256), device=DEV)
    dense = [x.clone() for x in c.dense]

    def step(q, k, v, counts, table, lengths, weights, pools):
        new = kv.paged_append(k, v, *pools, table, lengths, counts)
        out, lse = kv.paged_attention(q, *pools, table, new, counts, scale=0.09, with_lse=True)
        return new, out, lse, kv.attention_weights(q, lse, pools[0], table, new, counts, scale=0.09, before=weights)

    for turn, counts in enumerate(([40, 64, 7], [1, 1, 1], [1, 0, 1], [3, 1, 2], [1, 1, 1])):
        t = max(counts)
        q, k, v = randn(g, n, hq, t, d), randn(g, n, hkv, t, d), randn(g, n, hkv, t, d)
        cnt = ints(*counts)
        before = [p.clone() for p in pools]
        w0 = weights
        new, out, lse, weights = step(q, k, v, cnt, table, lengths, w0, pools)
        assert new.tolist() == [a + b for a, b in zip(lens, counts)]
        for i in range(n):
            dense[0][i, :, lens[i]:lens[i] + counts[i]] = k[i, :, :counts[i]]
            dense[1][i, :, lens[i]:lens[i] + counts[i]] = v[i, :, :counts[i]]
        lens = new.tolist()
        c.dense = dense
        check_attention(q, c, lens, counts, 0.09, out, lse)
        check_weights(q, lse, c, lens, counts, 0.09, w0, weights)
        # the same step captured and replayed on the state before it
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = step(q, k, v, cnt, table, lengths, w0, before)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[1], out) and torch.equal(again[2], lse) and torch.equal(again[3], weights)
        lengths = new
        if max(lens) > keep:
            lengths, w, kept = kv.evict_rows(*pools, table, new, weights, keep, spare, sinks=2, recent=16)
            for i in range(n):
                for h in range(hkv):
                    want = kept_rows(weights[i, h], lens[i], keep, 2, 16)
                    assert kept[i, h, :len(want)].tolist() == want
                    for x in dense:
                        x[i, h, :len(want)] = x[i, h, torch.tensor(want, dtype=torch.int64, device=DEV)].clone()
            weights = w
            table, spare = spare, table
            lens = [min(x, keep) for x in lens]
            assert lengths.tolist() == lens
    kv.check_status()


@gpu
def test_a_draft_verified_and_appended():
    """Tree attention, verification of its logits, and the accepted path into
    the cache, as one step without the host."""
    g = gen(62)
    n, hq, hkv, tok, d, vocab = 4, 4, 2, 6, 64, 500
    kc, vc = randn(g, n, hkv, 300, d), randn(g, n, hkv, 300, d)
    q, kn, vn = randn(g, n, hq, tok, d), randn(g, n, hkv, tok, d), randn(g, n, hkv, tok, d)
    p, dr, drafted, tree, u = verify_case(g, n, tok, vocab, 3)
    lens = ints(100, 0, 250, 31)
    out = kv.tree_attention(q, kn, vn, tree, kc, vc, lens, scale=0.1)
    head = randn(g, hq * d, vocab, dtype=F32) / 8
    probs = torch.softmax(out.transpose(1, 2).reshape(n, tok, -1).float() @ head, -1)
    target = torch.cat([p[:, :1], probs], 1)
    path, counts, after = kv.verify_tree(target, dr, drafted, tree, u)
    new = kv.append_accepted(kn, vn, path, counts, kc, vc, lens)
    assert torch.equal(new, lens + counts)
    for s in range(n):
        want, token = plain_verify(target[s], dr[s], drafted[s].tolist(), tree[s].tolist(), u[s].double().tolist())
        assert path[s, :len(want)].tolist() == want and int(after[s]) == token
        for j, node in enumerate(want):
            assert torch.equal(kc[s, :, int(lens[s]) + j], kn[s, :, node])
    kv.check_status()


@gpu
def test_another_stream_and_workspaces():
    """On a stream that is not the tensors' own, with workspaces of the caller;
    two captured calls with their own run at once."""
    g = gen(63)
    c = Cache(g, 2, 2, [5000, 3000], 64, 128)
    q = [randn(g, 2, 4, 3, 128) for _ in range(2)]
    lens = ints(5000, 3000)
    want = [kv.paged_attention(x, *c.pools, c.table, lens, scale=0.1) for x in q]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kv.paged_attention(q[0], *c.pools, c.table, lens, scale=0.1, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])
    size = kv.paged_attention_workspace(2, 4, 2, 3, 128, c.table.shape[1] * 64)
    graphs, outs = [], []
    for x in q:
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(x)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            kv.paged_attention(x, *c.pools, c.table, lens, scale=0.1, out=out, workspace=ws)
        graphs.append((graph, ws))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(20):
        for st, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    with pytest.raises(kv.StateKVError):
        kv.paged_attention(q[0], *c.pools, c.table, lens, scale=0.1,
                           workspace=torch.empty(size - 16, dtype=torch.uint8, device=DEV))
    kv.check_status()


@gpu
def test_every_operator_captured_and_on_other_streams():
    """One step of all five, eager on a stream of its own, and as two graphs that
    are replayed at once: the same bits as eager calls on the default stream."""
    g = gen(64)
    c = Cache(g, 3, 2, [700, 90, 333], 32, 64, cap=800)
    wide = torch.full((3, 40), 1 << 30, dtype=I32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    table = wide[:, :c.full.shape[1]]                    # rows of a larger table
    table.copy_(c.full)
    lens, counts = ints(700, 90, 333), ints(17, 2, 5)
    q, k, v = randn(g, 3, 8, 17, 64), randn(g, 3, 2, 17, 64), randn(g, 3, 2, 17, 64)
    p, dr, drafted, tree, u = verify_case(g, 5, 6, 3001, 9)
    fresh = torch.arange(3 * 4, device=DEV, dtype=I32).view(3, 4)

    def step(pools, out_pools, stream=None):
        new = kv.paged_append(k, v, *pools, table, lens, counts, stream=stream)
        out, lse = kv.paged_attention(q, *pools, table, new, counts, scale=0.1, with_lse=True, stream=stream)
        w = kv.attention_weights(q, lse, pools[0], table, new, counts, scale=0.1, stream=stream)
        e = kv.evict_rows(*pools, table, new, w, 100, fresh, sinks=3, recent=20, k_out=out_pools[0],
                          v_out=out_pools[1], stream=stream)
        return [new, out, lse, w, *e, *out_pools, *kv.verify_tree(p, dr, drafted, tree, u, stream=stream)]

    def state():
        return [x.clone() for x in c.pools], [torch.zeros(12, 2, 32, 64, dtype=BF16, device=DEV) for _ in range(2)]

    want = step(*state())
    c.dense = [x.clone() for x in c.dense]
    for i, (n0, n1) in enumerate(zip((700, 90, 333), (17, 2, 5))):
        c.dense[0][i, :, n0:n0 + n1], c.dense[1][i, :, n0:n0 + n1] = k[i, :, :n1], v[i, :, :n1]
    check_attention(q, c, [717, 92, 338], [17, 2, 5], 0.1, want[1], want[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = state()
    torch.cuda.synchronize()
    got = step(*args, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        args = state()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(*args)
        graphs.append((graph, got, torch.cuda.Stream()))
    for _ in range(10):
        for graph, _, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, _ in graphs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    kv.check_status()


@gpu
def test_empty_batches():
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    pool, none, table = z(4, 2, 16, 64), z(0, dtype=I32), z(0, 3, dtype=I32)
    assert kv.paged_append(z(0, 2, 3, 64), z(0, 2, 3, 64), pool, pool.clone(), table, none).shape == (0,)
    assert kv.paged_attention(z(0, 4, 3, 64), pool, pool, table, none, none, scale=0.1).shape == (0, 4, 3, 64)
    assert kv.attention_weights(z(0, 4, 3, 64), z(0, 4, 3, dtype=F32), pool, table, none, scale=0.1).shape == (0, 2, 48)
    new, w, kept = kv.evict_rows(pool, pool, table, none, z(0, 2, 48, dtype=F32), 5, table)
    assert new.shape == (0,) and kept.shape == (0, 2, 5)
    tree = kv.tree_masks([-1, 0], DEV)[0]
    path, counts, after = kv.verify_tree(z(0, 3, 9, dtype=F32), None, z(0, 2, dtype=I32), tree, z(0, 3, dtype=F32))
    assert path.shape == (0, 2) and counts.shape == (0,) and after.shape == (0,)
    # nothing to append; a sequence of no rows
    one = torch.arange(3, dtype=I32, device=DEV)[None]
    assert kv.paged_append(z(1, 2, 0, 64), z(1, 2, 0, 64), pool, pool.clone(), one, 5) == 5
    out, lse = kv.paged_attention(z(1, 4, 3, 64), pool, pool, one, ints(0), ints(0), scale=0.1, with_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())
    kv.check_status()


# ---------------------------------------------------------------- refusals
@gpu
def test_refusals_of_tensors():
    g = gen(71)
    c = Cache(g, 2, 2, [40, 40], 16, 64)
    q, k = randn(g, 2, 4, 3, 64), randn(g, 2, 2, 3, 64)
    att = lambda **kw: kv.paged_attention(**{**dict(  # noqa: E731
        q=q, k_pages=c.pools[0], v_pages=c.pools[1], table=c.table, lengths=40, scale=0.1), **kw})
    for kw in (dict(q=q.float()), dict(q=q[:, :, :, ::2]), dict(k_pages=c.pools[0][:, :1]), dict(table=c.table[:1]),
               dict(table=c.table.long()), dict(table=c.table.t()), dict(lengths=ints(1, 2, 3)),
               dict(counts=ints(1, 2, 3)), dict(counts=torch.ones(2, device=DEV)), dict(lse=torch.zeros(2, 4, 2, device=DEV)),
               dict(out=q[:, :2]), dict(q=q.clone().requires_grad_()), dict(table=None, q=randn(g, 99, 4, 3, 64)),
               dict(workspace=torch.zeros(64, device=DEV)), dict(q=q[0])):
        with pytest.raises(ValueError):
            att(**kw)
    for kw in (dict(scale=0.0), dict(scale=math.nan), dict(lengths=41 + 999), dict(q=randn(g, 2, 130, 3, 64)),
               dict(out=q.as_strided(q.shape, (0, 64, 256, 1)))):
        with pytest.raises((kv.StateKVError, ValueError)):
            att(**kw)
    with pytest.raises(ValueError, match="tangent"):
        with torch.autograd.forward_ad.dual_level():
            att(q=torch.autograd.forward_ad.make_dual(q, q))
    lse = torch.zeros(2, 4, 3, device=DEV)
    wts = lambda **kw: kv.attention_weights(**{**dict(  # noqa: E731
        q=q, lse=lse, k_pages=c.pools[0], table=c.table, lengths=40, scale=0.1), **kw})
    for kw in (dict(lse=lse[:, :2]), dict(lse=lse.double()), dict(before=torch.zeros(2, 1, 999, device=DEV)),
               dict(before=torch.zeros(2, 2, 999, device=DEV), out=torch.zeros(2, 2, 998, device=DEV)),
               dict(lse=lse.clone().requires_grad_())):
        with pytest.raises(ValueError):
            wts(**kw)
    for kw in (dict(before=torch.zeros(2, 2, 40, device=DEV)), dict(q=q[:, :, :1].expand(2, 4, 3, 64))):
        with pytest.raises(kv.StateKVError):
            wts(**kw)
    with pytest.raises(ValueError):
        kv.paged_append(k, k[:, :1], *c.pools, c.table, 40)
    with pytest.raises(ValueError):
        kv.paged_append(k.half(), k.half(), *c.pools, c.table, 40)
    w = torch.zeros(2, 2, c.table.shape[1] * 16, device=DEV)
    for kw in (dict(keep=10, sinks=6, recent=5), dict(keep=-1), dict(keep=10, out_table=None),
               dict(keep=10, out_table=c.table[:, :0]), dict(keep=10, weights=w[:, :, :40].contiguous())):
        with pytest.raises((kv.StateKVError, ValueError)):
            kv.evict_rows(*c.pools, **{**dict(table=c.table, lengths=40, weights=w, out_table=c.table), **kw})
    p = torch.full((2, 4, 7), 1 / 7, device=DEV)
    tree = kv.tree_masks([-1, 0, 1], DEV)[0]
    t, u = torch.zeros((2, 3), dtype=I32, device=DEV), torch.zeros((2, 4), device=DEV)
    for args in ((p.double(), p, t, tree, u), (p, p[:, :3], t, tree, u), (p, p, t[:, :2], tree, u),
                 (p, p, t, tree[:, :2], u), (p, p, t, tree, u[:, :3]), (p, p, t.long(), tree, u), (p[0], None, t, tree, u),
                 (p.clone().requires_grad_(), p, t, tree, u), (p, None, t, torch.stack([tree[0]] * 3), u)):
        with pytest.raises(ValueError):
            kv.verify_tree(*args)
    kv.check_status()


PAGED = dict(table=16, table_stride=8, table_pages=8, num_pages=20, page_rows=16, status=16, batch=2, layers=1,
             kv_heads=2, head_dim=128)
BAD_PAGING = [
    (dict(table=18), N.E_INVALID_ARG), (dict(table_stride=7), N.E_INVALID_ARG), (dict(table_pages=-1), N.E_INVALID_ARG),
    (dict(num_pages=-1), N.E_INVALID_ARG), (dict(page_rows=8), N.E_INVALID_ARG), (dict(page_rows=24), N.E_UNSUPPORTED),
    (dict(table_pages=1 << 27, table_stride=1 << 27), N.E_UNSUPPORTED), (dict(table=None, num_pages=1), N.E_CAPACITY),
    (dict(status=None), N.E_INVALID_ARG), (dict(layers=0), N.E_INVALID_ARG), (dict(layers=3), N.E_INVALID_ARG),
    (dict(length=-1), N.E_INVALID_ARG), (dict(lengths=18), N.E_INVALID_ARG), (dict(length=129), N.E_CAPACITY)]


@pytest.mark.parametrize("bad,want", BAD_PAGING + [
    (dict(counts=18), N.E_INVALID_ARG), (dict(dtype=5), N.E_INVALID_ARG), (dict(head_dim=100), N.E_UNSUPPORTED),
    (dict(k_new=view(8)), N.E_INVALID_ARG), (dict(v_pages=view(None)), N.E_INVALID_ARG),
    (dict(k_pages=view(t=64)), N.E_INVALID_ARG), (dict(length=126), N.E_CAPACITY), (dict(tokens=-1), N.E_INVALID_ARG),
    (dict(new_lengths=64, lengths=64), N.E_INVALID_ARG), (dict(new_lengths=64, counts=64), N.E_INVALID_ARG),
    (dict(batch=0), N.OK)])
def test_append_refusals_before_device_work(bad, want):
    a = dict(PAGED, k_new=view(), v_new=view(), k_pages=view(b=1 << 20, h=1 << 16), v_pages=view(b=1 << 20, h=1 << 16),
             length=40, tokens=3, dtype=0)
    assert N.load().statekv_paged_append(N.PagedAppendArgs(**{**a, **bad}), None) == want


@pytest.mark.parametrize("bad,want", BAD_PAGING + [
    (dict(counts=18), N.E_INVALID_ARG), (dict(lse=18), N.E_INVALID_ARG), (dict(head_dim=96), N.E_UNSUPPORTED),
    (dict(q_heads=130), N.E_UNSUPPORTED), (dict(q_heads=3), N.E_INVALID_ARG), (dict(tokens=0), N.E_INVALID_ARG),
    (dict(tokens=1 << 26), N.E_UNSUPPORTED), (dict(scale=0.0), N.E_INVALID_ARG), (dict(scale=math.nan), N.E_INVALID_ARG),
    (dict(q=view(8)), N.E_INVALID_ARG), (dict(out=view(None)), N.E_INVALID_ARG), (dict(out=view(t=64)), N.E_INVALID_ARG),
    (dict(k_pages=view(h=0)), N.E_INVALID_ARG), (dict(v_pages=view(b=0)), N.E_INVALID_ARG), (dict(batch=0), N.OK)])
def test_attention_refusals_before_device_work(bad, want):
    pool = view(b=1 << 20, h=1 << 16)
    a = dict(PAGED, q=view(), out=view(), k_pages=pool, v_pages=pool, length=40, tokens=3, q_heads=4, scale=0.1,
             workspace=16, workspace_bytes=1 << 40)
    assert N.load().statekv_paged_attention(N.PagedAttentionArgs(**{**a, **bad}), None) == want


@pytest.mark.parametrize("bad,want", BAD_PAGING + [
    (dict(counts=18), N.E_INVALID_ARG), (dict(lse=None), N.E_INVALID_ARG), (dict(out=None), N.E_INVALID_ARG),
    (dict(before=18), N.E_INVALID_ARG), (dict(head_dim=96), N.E_UNSUPPORTED), (dict(q_heads=130), N.E_UNSUPPORTED),
    (dict(weight_rows=127), N.E_CAPACITY), (dict(scale=-1.0), N.E_INVALID_ARG), (dict(q=view(t=0)), N.E_INVALID_ARG),
    (dict(k_pages=view(b=0)), N.E_INVALID_ARG), (dict(tokens=0), N.E_INVALID_ARG), (dict(batch=0), N.OK)])
def test_weights_refusals_before_device_work(bad, want):
    a = dict(PAGED, q=view(), k_pages=view(b=1 << 20, h=1 << 16), lse=16, out=16, length=40, tokens=3, q_heads=4,
             scale=0.1, weight_rows=128)
    assert N.load().statekv_attention_weights(N.AttentionWeightsArgs(**{**a, **bad}), None) == want


@pytest.mark.parametrize("bad,want", BAD_PAGING + [
    (dict(dtype=5), N.E_INVALID_ARG), (dict(head_dim=100), N.E_UNSUPPORTED), (dict(keep=-1), N.E_INVALID_ARG),
    (dict(sinks=-1), N.E_INVALID_ARG), (dict(sinks=20, recent=13), N.E_INVALID_ARG), (dict(weight_rows=127), N.E_CAPACITY),
    (dict(out_rows=31), N.E_CAPACITY), (dict(out_table_pages=1), N.E_CAPACITY), (dict(out_page_rows=24), N.E_UNSUPPORTED),
    (dict(out_table=18), N.E_INVALID_ARG), (dict(weights=None), N.E_INVALID_ARG), (dict(weights_out=None), N.E_INVALID_ARG),
    (dict(kept=None), N.E_INVALID_ARG), (dict(new_lengths=64, lengths=64), N.E_INVALID_ARG),
    (dict(k_out=view(1 << 20, b=0)), N.E_INVALID_ARG), (dict(v_pages=view(8)), N.E_INVALID_ARG),
    (dict(k_out=view(), out_table=None, out_page_rows=32), N.E_INVALID_ARG),
    (dict(table_pages=1 << 19, table_stride=1 << 19, weight_rows=1 << 24), N.E_UNSUPPORTED), (dict(batch=0), N.OK)])
def test_evict_refusals_before_device_work(bad, want):
    pool, to = view(b=1 << 20, h=1 << 16), view(1 << 20, b=1 << 20, h=1 << 16)
    a = dict(PAGED, k_pages=pool, v_pages=pool, k_out=to, v_out=to, out_table=16, out_table_stride=2, out_table_pages=2,
             out_num_pages=4, out_page_rows=16, out_rows=32, keep=32, sinks=4, recent=8, weights=16, weights_out=16,
             kept=16, weight_rows=128, length=40, dtype=0)
    assert N.load().statekv_evict_rows(N.EvictArgs(**{**a, **bad}), None) == want


@pytest.mark.parametrize("bad", [
    dict(weights_out=1 << 30), dict(weights_out=(1 << 30) + 2044), dict(weights_out=(1 << 30) - 508),
    dict(kept=(1 << 30) + 1024), dict(kept=(1 << 31) + 508)])
def test_evict_arrays_that_share_memory_are_refused(bad):
    """4 units of 128 weights in, 32 out, 32 rows kept: ranges that share one entry at least."""
    pool, to = view(b=1 << 20, h=1 << 16), view(1 << 20, b=1 << 20, h=1 << 16)
    a = dict(PAGED, k_pages=pool, v_pages=pool, k_out=to, v_out=to, out_table=16, out_table_stride=2, out_table_pages=2,
             out_num_pages=4, out_page_rows=16, out_rows=32, keep=32, sinks=4, recent=8, weights=1 << 30,
             weights_out=1 << 31, kept=1 << 32, weight_rows=128, length=40, dtype=0)
    assert N.load().statekv_evict_rows(N.EvictArgs(**{**a, **bad}), None) == N.E_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(v_pages=view(1 << 30, b=1 << 20, h=1 << 16)),                             # the same rows
    dict(v_pages=view((1 << 30) + 256, b=1 << 20, h=1 << 16)),                     # a row on
    dict(v_pages=view((1 << 30) + (1 << 17) + 15 * 256, b=1 << 20, h=1 << 16)),    # its head 0's rows 0.. are head 1's 15..
    dict(v_pages=view((1 << 30) + (19 << 21), b=1 << 20, h=1 << 16)),              # its first page is K's last
    dict(v_pages=view((1 << 30) - (1 << 21), b=1 << 20, h=1 << 16)),
    dict(v_pages=view((1 << 30) + (1 << 17) + 256, b=1 << 20, h=1 << 15)),         # other strides within K's range
    dict(new_lengths=(1 << 33) + 4), dict(new_lengths=(1 << 33) - 4), dict(new_lengths=(1 << 34) + 4)])
def test_append_over_shared_memory_is_refused(bad):
    a = dict(PAGED, k_new=view(), v_new=view(), k_pages=view(1 << 30, b=1 << 20, h=1 << 16),
             v_pages=view(1 << 31, b=1 << 20, h=1 << 16), tokens=3, dtype=0, lengths=1 << 33, counts=1 << 34)
    assert N.load().statekv_paged_append(N.PagedAppendArgs(**{**a, **bad}), None) == N.E_INVALID_ARG


EVICT = dict(PAGED, k_pages=view(1 << 40, b=1 << 20, h=1 << 16), v_pages=view(1 << 41, b=1 << 20, h=1 << 16),
             k_out=view(1 << 42, b=1 << 20, h=1 << 16), v_out=view(1 << 43, b=1 << 20, h=1 << 16), table=1 << 28,
             out_table=1 << 29, out_table_stride=2, out_table_pages=2, out_num_pages=4, out_page_rows=16, out_rows=32, keep=32,
             sinks=4, recent=8, weights=1 << 30, weights_out=1 << 31, kept=1 << 32, new_lengths=1 << 33, lengths=1 << 34,
             weight_rows=128, dtype=0)
PLAIN = dict(table=None, out_table=None, num_pages=2, page_rows=128, out_num_pages=2, out_page_rows=32)


@pytest.mark.parametrize("bad", [
    dict(v_out=view(1 << 42, b=1 << 20, h=1 << 16)),                               # K and V to the same rows
    dict(v_out=view((1 << 42) + 256, b=1 << 20, h=1 << 16)),
    dict(PLAIN, k_out=view((1 << 40) + 16 * 256, b=1 << 20, h=1 << 16)),           # rows 16.. of the source
    dict(PLAIN, k_out=view((1 << 40) + 127 * 256, b=1 << 20, h=1 << 16)),          # its last row
    dict(PLAIN, v_out=view((1 << 40) + 16 * 256, b=1 << 20, h=1 << 16)),           # V over K's rows
    dict(PLAIN, v_out=view((1 << 41) - 31 * 256, b=1 << 20, h=1 << 16)),           # the last row out is its first
    dict(PLAIN, k_out=view((1 << 40) + (1 << 21), b=1 << 21, h=1 << 16)),          # entry 0 goes to the source's entry 1
    dict(out_table=None, out_num_pages=2, out_page_rows=32, k_out=view((1 << 40) + (5 << 21), b=1 << 20, h=1 << 16)),
    dict(table=None, page_rows=128, num_pages=2, k_out=view((1 << 40) - (3 << 21), b=1 << 20, h=1 << 16)),
    dict(new_lengths=(1 << 34) + 4), dict(new_lengths=(1 << 31) + 508), dict(new_lengths=(1 << 32) - 4),
    dict(new_lengths=(1 << 30) + 2044), dict(kept=(1 << 28) - 508), dict(weights_out=(1 << 29) + 12),
    dict(kept=(1 << 34) - 4)])
def test_evict_over_shared_memory_is_refused(bad):
    assert N.load().statekv_evict_rows(N.EvictArgs(**{**EVICT, **bad}), None) == N.E_INVALID_ARG


@gpu
def test_pools_side_by_side_in_one_tensor_are_apart():
    """K and V of each page next to each other, and rows evicted to the other part of one plain cache."""
    g = gen(81)
    lens, n = [40, 3, 0], 3
    c = Cache(g, n, 2, [x + 9 for x in lens], 16, 64)
    for dim in (1, 2, 3):                            # [pages][2][heads][rows][d], ..., [pages][heads][rows][2][d]
        shape = list(c.pools[0].shape)
        both = torch.full((*shape[:dim], 2, *shape[dim:]), 9.0, dtype=BF16, device=DEV)
        pools = both.unbind(dim)
        k, v = randn(g, n, 2, 9, 64), randn(g, n, 2, 9, 64)
        assert kv.paged_append(k, v, *pools, c.table, ints(*lens)).tolist() == [x + 9 for x in lens]
        for pool, x in zip(pools, (k, v)):
            for i in range(n):
                assert torch.equal(c.rows(pool, i, lens[i] + 9)[:, lens[i]:], x[i])
        out = torch.full((*shape[:dim], 2, *shape[dim:]), 9.0, dtype=BF16, device=DEV)
        to = torch.arange(6, dtype=I32, device=DEV).view(3, 2)
        w = torch.rand((n, 2, c.table.shape[1] * 16), generator=g, device=DEV)
        got = kv.evict_rows(*pools, c.table, ints(49, 12, 9), w, 20, to, k_out=out.unbind(dim)[0], v_out=out.unbind(dim)[1])
        check_evict(c, [49, 12, 9], 1, w, 20, 0, 0, pools, out.unbind(dim), to, got, 16)
    wide = randn(g, 2, 2, 2, 300, 64)                # [entry][K, V][head][row][d]: rows 0..199 to rows 200..299
    src, dst = [wide[:, i, :, :200] for i in range(2)], [wide[:, i, :, 200:] for i in range(2)]
    w = torch.rand((2, 2, 200), generator=g, device=DEV)
    p = Cache(g, 2, 2, [200, 200], 0, 64)
    got = kv.evict_rows(*src, None, 200, w, 100, None, k_out=dst[0], v_out=dst[1])
    check_evict(p, [200, 200], 1, w, 100, 0, 0, src, dst, None, got, 0)
    with pytest.raises(kv.StateKVError):
        kv.evict_rows(*src, None, 200, w, 100, None, k_out=wide[:, 0, :, 199:299], v_out=dst[1])
    kv.check_status()


@gpu
def test_pools_of_other_strides_in_one_tensor_are_apart():
    """Each page's K by heads, then its V by rows."""
    g = gen(82)
    n, lens = 2, [30, 5]
    c = Cache(g, n, 2, [x + 4 for x in lens], 16, 64)

    def pair():
        both = torch.full((len(c.pools[0]), 2, 2 * 16 * 64), 9.0, dtype=BF16, device=DEV)
        return both[:, 0].unflatten(1, (2, 16, 64)), both[:, 1].unflatten(1, (16, 2, 64)).transpose(1, 2)

    pools, out = pair(), pair()
    k, v = randn(g, n, 2, 4, 64), randn(g, n, 2, 4, 64)
    assert kv.paged_append(k, v, *pools, c.table, ints(*lens)).tolist() == [34, 9]
    for pool, x in zip(pools, (k, v)):
        for i in range(n):
            assert torch.equal(c.rows(pool, i, lens[i] + 4)[:, lens[i]:], x[i])
    w = torch.rand((n, 2, c.table.shape[1] * 16), generator=g, device=DEV)
    to = torch.arange(4, dtype=I32, device=DEV).view(2, 2)
    got = kv.evict_rows(*pools, c.table, ints(34, 9), w, 20, to, k_out=out[0], v_out=out[1])
    check_evict(c, [34, 9], 1, w, 20, 0, 0, pools, out, to, got, 16)
    kv.check_status()


@pytest.mark.parametrize("bad", [dict(tokens=1 << 26), dict(tokens=1 << 25), dict(tokens=2 ** 31 - 1)])
def test_weights_of_more_queries_than_the_attention_takes_are_refused(bad):
    a = dict(PAGED, q=view(), k_pages=view(b=1 << 20, h=1 << 16), lse=16, out=16, length=40, q_heads=4, scale=0.1,
             weight_rows=128)
    assert N.load().statekv_attention_weights(N.AttentionWeightsArgs(**{**a, **bad}), None) == N.E_UNSUPPORTED


@pytest.mark.parametrize("by", [4, 2044, -4, -2044])
def test_weights_over_a_part_of_what_they_are_added_to_are_refused(by):
    a = dict(PAGED, q=view(), k_pages=view(b=1 << 20, h=1 << 16), lse=16, before=1 << 30, out=(1 << 30) + by, length=40,
             tokens=3, q_heads=4, scale=0.1, weight_rows=128)
    assert N.load().statekv_attention_weights(N.AttentionWeightsArgs(**a), None) == N.E_INVALID_ARG


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=0), N.E_INVALID_ARG), (dict(tokens=65), N.E_UNSUPPORTED), (dict(vocab=0), N.E_INVALID_ARG),
    (dict(vocab=1 << 26), N.E_UNSUPPORTED), (dict(tree_stride=4), N.E_INVALID_ARG), (dict(tree=20), N.E_INVALID_ARG),
    (dict(target=None), N.E_INVALID_ARG), (dict(target=18), N.E_INVALID_ARG), (dict(draft=18), N.E_INVALID_ARG),
    (dict(drafted=None), N.E_INVALID_ARG), (dict(uniforms=None), N.E_INVALID_ARG), (dict(path=None), N.E_INVALID_ARG),
    (dict(counts=None), N.E_INVALID_ARG), (dict(next=None), N.E_INVALID_ARG), (dict(status=None), N.E_INVALID_ARG),
    (dict(target_row=-1), N.E_INVALID_ARG), (dict(sequences=-1), N.E_INVALID_ARG),
    (dict(sequences=1 << 28), N.E_UNSUPPORTED), (dict(sequences=0), N.OK)])
def test_verify_refusals_before_device_work(bad, want):
    a = dict(target=16, draft=16, drafted=16, tree=16, uniforms=16, path=16, counts=16, next=16, status=16,
             target_stride=60, target_row=10, draft_stride=60, draft_row=10, sequences=2, tokens=5, vocab=10)
    assert N.load().statekv_verify_tree(N.VerifyArgs(**{**a, **bad}), None) == want


@pytest.mark.parametrize("pack,args", [(N.PACK_PAGED_APPEND, N.PagedAppendArgs),
                                       (N.PACK_PAGED_ATTENTION, N.PagedAttentionArgs),
                                       (N.PACK_WEIGHTS, N.AttentionWeightsArgs), (N.PACK_EVICT, N.EvictArgs),
                                       (N.PACK_VERIFY, N.VerifyArgs)])
def test_packed_arguments_are_the_structures(pack, args):
    flat, n = [], 0

    def leaf(t):
        nonlocal n
        n += 1
        flat.append(n / 2 if t is C.c_double else n)
        return flat[-1]

    a = args(**{f: N.View(*(leaf(x) for _, x in N.View._fields_)) if t is N.View else leaf(t) for f, t in args._fields_})
    assert pack.size == C.sizeof(args) and pack.pack(*flat) == bytes(a)

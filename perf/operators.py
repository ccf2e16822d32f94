"""Measured cases of the text-decoding operators over the detailed state.

Five operators, used one after the other when a video VLM answers over the
keys and values of a whole video:

  norm_rope  RMS norm of every query and key head, rotation at virtual
             positions, and the store of K and V where the cache wants them
  tree       attention of a tree of drafted tokens over the cache
  append     the accepted path of the tree joins the cache
  summary    int8 mean key and scale of every complete 64-row block
  sparse     attention over the blocks that the summaries select per token

Tensors are [batch, heads, tokens, head_dim]; the batch is sequences x layers,
and lengths, trees and paths have one entry per sequence.
"""

import math

import torch

own = False

BLOCK = 64          # cache rows a summary stands for
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new text token in one layer of the 16/8-head model: pure latency
        dict(name="norm_rope token", op="norm_rope", seqs=1, layers=1, hq=16, hkv=8, t=1, d=128,
             dtype="bf16", p0=131072),
        # a text prompt of odd length, fp32 storage, 64-wide heads
        dict(name="norm_rope f32 prompt", op="norm_rope", seqs=1, layers=3, hq=14, hkv=2, t=77, d=64,
             dtype="f32", p0=16384),
        # one 256-token frame of 16 streams x 4 layers (the batched serving configuration)
        dict(name="norm_rope frame batch", op="norm_rope", seqs=16, layers=4, hq=16, hkv=8, t=256,
             d=128, dtype="bf16", p0=65536),
        # a short chat: one layer, 14/2 heads of 64, a small tree after 300 rows
        dict(name="tree short", op="tree", seqs=1, layers=1, hq=14, hkv=2, d=64, tok=7, rows=300,
             ragged=False),
        # 16 streams of different lengths in one layer, 32 drafted tokens each
        dict(name="tree ragged batch", op="tree", seqs=16, layers=1, hq=16, hkv=8, d=128, tok=32,
             rows=32768, ragged=True),
        # all 28 layers of the 12/2-head model after a 512-frame video, 42 drafted tokens
        dict(name="tree full video", op="tree", seqs=1, layers=28, hq=12, hkv=2, d=128, tok=42,
             rows=131072, ragged=False),
        # the accepted path of a tree, all layers of one stream
        dict(name="append one stream", op="append", seqs=1, layers=28, hkv=2, d=128, tok=16, path=5,
             rows=1000, ragged=False),
        # the accepted paths of 16 streams x 4 layers
        dict(name="append batch", op="append", seqs=16, layers=4, hkv=8, d=128, tok=64, path=13,
             rows=1500, ragged=True),
        # the blocks that one 256-token frame completes, all layers
        dict(name="summary frame", op="summary", seqs=1, layers=28, hkv=2, d=128, rows=4133,
             appended=256, ragged=False),
        # a whole 512-frame video in one layer with 8 KV heads
        dict(name="summary video", op="summary", seqs=1, layers=1, hkv=8, d=128, rows=131072,
             appended=131072, ragged=False),
        # one text token in one layer after a 512-frame video: 64 blocks of 64 rows, the budget of 4096
        dict(name="sparse token", op="sparse", seqs=1, layers=1, hq=12, hkv=2, d=128, tok=1,
             rows=131073, top=64, ragged=False),
        # 16 streams of different lengths, 3 tokens each
        dict(name="sparse ragged batch", op="sparse", seqs=16, layers=1, hq=16, hkv=8, d=128, tok=3,
             rows=32768, top=64, ragged=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "tree", "tree", "append", "summary", "sparse", "sparse"])
    hq, hkv = rng.choice([(14, 2), (12, 2), (16, 8), (4, 2), (8, 8)])
    d = rng.choice([64, 128, 128])
    seqs = _between(rng, 1, 16)
    layers = rng.choice([1, 1, 2, 4])
    ragged = rng.random() < 0.5
    c = dict(op=op, seqs=seqs, layers=layers, hkv=hkv, d=d)
    if op == "norm_rope":
        return dict(c, hq=hq, t=_between(rng, 1, 256), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    p0=rng.randrange(0, 500000))
    rows = _between(rng, 40, 131072)
    if op == "summary":
        rows = max(rows, 64)
    # at most 4 GB of cache
    rows = max(64, min(rows, (4 << 30) // (seqs * layers * hkv * d * 4)))
    c.update(rows=rows, ragged=ragged)
    if op == "summary":
        return dict(c, appended=rng.choice([rows, _between(rng, 1, rows)]))
    if op == "append":
        c["rows"] = min(c["rows"], 20000)
        tok = _between(rng, 1, 64)
        return dict(c, tok=tok, path=rng.randint(1, tok))
    if op == "tree":
        # the plain form keeps a few fp32 score matrices
        tok = _between(rng, 1, 64)
        c["rows"] = max(64, min(rows, (6 << 30) // (seqs * layers * hq * tok * 4)))
        return dict(c, hq=hq, tok=tok)
    tok = min(rows, _between(rng, 1, 16))
    top = _between(rng, 1, 128)
    # the plain form gathers the selected rows in fp32
    while seqs * layers * hkv * tok * top * BLOCK * d * 8 > (2 << 30):
        top = max(1, top // 2)
        tok = max(1, tok - 1)
    return dict(c, hq=hq, tok=tok, top=top)


def _lengths(case, gen, lo):
    """Rows of each sequence in the cache, int32 on the GPU."""
    if not case["ragged"]:
        return torch.full((case["seqs"],), case["rows"], dtype=torch.int32, device=DEV)
    x = torch.randint(lo, case["rows"] + 1, (case["seqs"],), generator=gen, device=DEV)
    x[0] = case["rows"]
    return x.to(torch.int32)


def _tree(case, gen):
    """Parents of a random tree per sequence (node 0 the root, parents before
    children) as bit masks of the nodes each node sees, itself included."""
    tok, seqs = case["tok"], case["seqs"]
    r = torch.rand((seqs, tok), generator=gen, device=DEV).cpu()
    masks = torch.zeros((seqs, tok), dtype=torch.int64)
    for s in range(seqs):
        row = [1]
        for i in range(1, tok):
            # recent nodes are the likelier parents, as in drafted trees
            p = i - 1 - int(float(r[s, i]) ** 2 * i)
            bits = row[p] | (1 << i)
            row.append(bits)
        # bit 63 is the sign of the 64-bit word
        masks[s] = torch.tensor([b - (1 << 64) if b >> 63 else b for b in row], dtype=torch.int64)
    return masks.to(DEV)


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _summaries(k):
    """Codes and scales of every 64-row block of k [..., rows, d] (rows a
    multiple of 64): the block's mean key in fp32 (from an exact sum),
    scale = max |mean| / 127, code = mean * (127 / max |mean|) rounded to even.
    (Tensors on both sides: torch multiplies by a rounded reciprocal where one
    side of a quotient is a plain number.)"""
    m = k.unflatten(-2, (-1, BLOCK)).double().mean(-2).float()
    top = m.abs().amax(-1, keepdim=True)
    inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, torch.zeros_like(top))
    return torch.round(m * inv).to(torch.int8), (top / torch.full_like(top, 127.0)).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, d = case["op"], case["d"]
    n, hkv = case["seqs"] * case["layers"], case["hkv"]
    s = dict(case=case)
    if op == "norm_rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        hq, t = case["hq"], case["t"]
        # the projection's output: tokens outermost, heads of q, k and v side by side
        qkv = _randn(gen, n, t, hq + 2 * hkv, d, dtype=dt) * 2.0
        s["q"] = qkv[:, :, :hq].transpose(1, 2)
        s["k"] = qkv[:, :, hq:hq + hkv].transpose(1, 2)
        s["v"] = qkv[:, :, hq + hkv:].transpose(1, 2)
        s["qw"] = (1.0 + 0.2 * _randn(gen, d, dtype=torch.float32)).to(dt)
        s["kw"] = (1.0 + 0.2 * _randn(gen, d, dtype=torch.float32)).to(dt)
        s["omega"] = 1e6 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
        first = case["p0"] + torch.randint(0, 1000, (n, 1), generator=gen, device=DEV)
        s["positions"] = (first + torch.arange(t, device=DEV)).to(torch.int32)
        s["eps"] = 1e-6
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    if op == "summary":
        cap = (case["rows"] + BLOCK - 1) // BLOCK * BLOCK
        s["k"] = _randn(gen, n, hkv, cap, d)
        s["lengths"] = _lengths(case, gen, 1)
        s["codes"] = torch.zeros((n, hkv, cap // BLOCK, d), dtype=torch.int8, device=DEV)
        s["scales"] = torch.zeros((n, hkv, cap // BLOCK), dtype=torch.float32, device=DEV)
        return s
    tok = case["tok"]
    cap = case["rows"] + 64
    if op == "sparse":
        cap = (case["rows"] + BLOCK - 1) // BLOCK * BLOCK
    kc, vc = _randn(gen, n, hkv, cap, d), _randn(gen, n, hkv, cap, d)
    s["k_cache"], s["v_cache"] = kc, vc
    if op == "append":
        s["k_new"], s["v_new"] = _randn(gen, n, hkv, tok, d), _randn(gen, n, hkv, tok, d)
        a = case["path"]
        order = torch.rand((case["seqs"], tok), generator=gen, device=DEV).argsort(-1)[:, :a]
        s["path"] = order.sort(-1).values.to(torch.int32)
        s["counts"] = torch.randint(1, a + 1, (case["seqs"],), generator=gen, device=DEV).to(torch.int32)
        s["counts"][0] = a
        s["lengths"] = _lengths(case, gen, 0)
        return s
    s["q"] = _randn(gen, n, case["hq"], tok, d)
    if op == "tree":
        s["k_new"], s["v_new"] = _randn(gen, n, hkv, tok, d), _randn(gen, n, hkv, tok, d)
        s["tree"] = _tree(case, gen)
        s["lengths"] = _lengths(case, gen, 0)
        return s
    # keys of a block have a common part, as neighbouring visual tokens do
    kc.view(n, hkv, -1, BLOCK, d).add_(0.5 * _randn(gen, n, hkv, cap // BLOCK, 1, d))
    s["codes"], s["scales"] = _summaries(kc)
    s["lengths"] = _lengths(case, gen, tok)
    return s


# ------------------------------------------------------------- plain forms
def _plain_norm_rope(s):
    ang = s["positions"].double()[:, None, :, None] * s["omega"]
    cos, sin = ang.cos().float(), ang.sin().float()

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        a, b = y.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"]), s["v"].clone(memory_format=torch.contiguous_format)


def _plain_tree(s):
    c = s["case"]
    n, hkv, tok, rows, lay = s["q"].shape[0], c["hkv"], c["tok"], c["rows"], c["layers"]
    q = s["q"].float().reshape(n, hkv, -1, c["d"]) * s["scale"]
    kc, vc = s["k_cache"][:, :, :rows].float(), s["v_cache"][:, :, :rows].float()
    old = q @ kc.transpose(-1, -2)
    if c["ragged"]:
        live = torch.arange(rows, device=DEV) < s["lengths"].repeat_interleave(lay)[:, None]
        old = old.masked_fill(~live[:, None, None, :], float("-inf"))
    new = q @ s["k_new"].float().transpose(-1, -2)
    sees = (s["tree"][:, :, None] >> torch.arange(tok, device=DEV)) & 1
    sees = sees.repeat_interleave(lay, 0).repeat(1, c["hq"] // hkv, 1).bool()
    new = new.masked_fill(~sees[:, None], float("-inf"))
    m = torch.maximum(old.amax(-1, keepdim=True), new.amax(-1, keepdim=True))
    old, new = torch.exp(old - m), torch.exp(new - m)
    o = old @ vc + new @ s["v_new"].float()
    o = o / (old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True))
    return o.reshape(s["q"].shape).to(s["q"].dtype)


def _plain_append(s):
    c = s["case"]
    n, lay = s["k_new"].shape[0], c["layers"]
    # steps past the count write the last accepted node once more
    use = torch.minimum(torch.arange(c["path"], device=DEV), s["counts"][:, None].long() - 1)
    src = s["path"].long().gather(1, use).repeat_interleave(lay, 0)
    dst = (s["lengths"][:, None].long() + use).repeat_interleave(lay, 0)
    b = torch.arange(n, device=DEV)[:, None]
    for cache, new in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        cache[b, :, dst] = new[b, :, src]
    return s["k_cache"], s["v_cache"], s["lengths"] + s["counts"]


def _plain_summary(s):
    c = s["case"]
    n, hkv, nb, d = s["codes"].shape
    lens = s["lengths"].repeat_interleave(c["layers"])
    lo, hi = torch.clamp(lens - c["appended"], min=0) // BLOCK, lens // BLOCK
    # the blocks that the appended rows can have completed
    at = lo[:, None] + torch.arange(min(nb, c["appended"] // BLOCK + 1), device=DEV)
    fresh = (at < hi[:, None])[..., None]
    at = at.clamp(max=nb - 1)
    b = torch.arange(n, device=DEV)[:, None]
    codes, scales = _summaries(s["k"].view(n, hkv, nb, BLOCK, d)[b, :, at].flatten(-3, -2))
    codes, scales = codes.squeeze(-2), scales.squeeze(-1)
    s["codes"][b, :, at] = torch.where(fresh[..., None], codes, s["codes"][b, :, at])
    s["scales"][b, :, at] = torch.where(fresh, scales, s["scales"][b, :, at])
    return s["codes"] * s["scales"][..., None], s["scales"]


def _choose(q, codes, scales, blocks, top):
    """Indices of the `top` best blocks [n, hkv, tok, top], ascending, -1 where
    there are fewer; q [n, hkv, g, tok, d], blocks [n] complete blocks."""
    amax = q.abs().amax((2, 4), keepdim=True)
    inv = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, torch.zeros_like(amax))
    qi = torch.round(q * inv)
    # sums of 128 products of 8-bit numbers stay below 2^24: exact in fp32
    dots = qi.flatten(2, 3) @ codes.float().transpose(-1, -2)
    score = dots.unflatten(2, (q.shape[2], q.shape[3])).amax(2) * scales[:, :, None, :]
    gone = torch.arange(codes.shape[2], device=DEV) >= blocks[:, None]
    score = score.masked_fill(gone[:, None, None, :], float("-inf"))
    val, idx = score.sort(dim=-1, descending=True, stable=True)
    val, idx = val[..., :top], idx[..., :top]
    far = codes.shape[2]
    idx = idx.masked_fill(val == float("-inf"), far).sort(-1).values
    idx = idx.masked_fill(idx == far, -1)
    if idx.shape[-1] < top:
        idx = torch.nn.functional.pad(idx, (0, top - idx.shape[-1]), value=-1)
    return idx


def _plain_sparse(s):
    c = s["case"]
    n, hkv, tok, d, g = s["q"].shape[0], c["hkv"], c["tok"], c["d"], c["hq"] // c["hkv"]
    q = s["q"].float().reshape(n, hkv, g, tok, d)
    lens = s["lengths"].repeat_interleave(c["layers"]).long()
    first = lens - tok                              # rows before the new tokens
    idx = _choose(q, s["codes"], s["scales"], first // BLOCK, c["top"])
    used = idx >= 0
    # rows of the selected blocks, then the rows since the last complete block
    # up to the token itself
    rows = idx.clamp(min=0)[..., None] * BLOCK + torch.arange(BLOCK, device=DEV)
    rows = rows.flatten(-2)
    tail = (first // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK + tok - 1, device=DEV)
    own_row = first[:, None] + torch.arange(tok, device=DEV)
    live = torch.cat([used[..., None].expand(*used.shape, BLOCK).flatten(-2),
                      (tail[:, None, :] <= own_row[:, :, None])[:, None].expand(n, hkv, tok, -1)], -1)
    tail = tail.clamp(max=s["k_cache"].shape[2] - 1)
    rows = torch.cat([rows, tail[:, None, None, :].expand(n, hkv, tok, -1)], -1)
    b = torch.arange(n, device=DEV)[:, None, None, None]
    h = torch.arange(hkv, device=DEV)[None, :, None, None]
    kg, vg = s["k_cache"][b, h, rows].float(), s["v_cache"][b, h, rows].float()
    x = (q.transpose(2, 3) * s["scale"]) @ kg.transpose(-1, -2)
    x = x.masked_fill(~live[:, :, :, None, :], float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = (p @ vg) / p.sum(-1, keepdim=True)
    return o.transpose(2, 3).reshape(s["q"].shape).to(s["q"].dtype), idx.to(torch.int32)


# ---------------------------------------------------------------- one pass
def _own(s):
    import kv_cache_compression_frame_gb300 as kv

    c, op = s["case"], s["case"]["op"]
    if op == "norm_rope":
        return kv.qk_norm_rope(s["q"], s["k"], s["positions"], s["omega"], s["qw"], s["kw"],
                               v=s["v"], eps=s["eps"])
    if op == "tree":
        return kv.tree_attention(s["q"], s["k_new"], s["v_new"], s["tree"], s["k_cache"],
                                 s["v_cache"], s["lengths"], scale=s["scale"])
    if op == "append":
        lengths = kv.append_accepted(s["k_new"], s["v_new"], s["path"], s["counts"], s["k_cache"],
                                     s["v_cache"], s["lengths"])
        return s["k_cache"], s["v_cache"], lengths
    if op == "summary":
        kv.block_summaries(s["k"], s["codes"], s["scales"], s["lengths"], appended=c["appended"])
        return s["codes"] * s["scales"][..., None], s["scales"]
    return kv.sparse_attention(s["q"], s["k_cache"], s["v_cache"], s["codes"], s["scales"],
                               s["lengths"], c["top"], scale=s["scale"])


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "tree": _plain_tree, "append": _plain_append,
            "summary": _plain_summary, "sparse": _plain_sparse}[state["case"]["op"]](state)


def work(case):
    op, d = case["op"], case["d"]
    n, hkv = case["seqs"] * case["layers"], case["hkv"]
    # ragged lengths are uniform up to the largest
    rows = case.get("rows", 0) * (0.5 + 0.5 / case["seqs"] if case.get("ragged") else 1.0)
    if op == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        vals = n * case["t"] * (case["hq"] + 2 * hkv) * d
        return {"bytes": 2 * vals * e + n * case["t"] * 4, "flops": 9 * vals}
    if op == "append":
        a = case["path"]
        return {"bytes": n * hkv * a * d * 2 * 4 + case["seqs"] * (a + 3) * 4, "flops": 0}
    if op == "summary":
        fresh = n * hkv * (min(rows, case["appended"]) // BLOCK)
        # run() returns the decoded values of every block the cache can hold
        held = n * hkv * ((case["rows"] + BLOCK - 1) // BLOCK)
        return {"bytes": fresh * (BLOCK * d * 2 + d + 4) + held * (d + 4 + d * 4),
                "flops": fresh * BLOCK * d}
    tok, hq = case["tok"], case["hq"]
    io = 2 * n * hq * tok * d * 2
    if op == "tree":
        return {"bytes": io + n * hkv * (rows + tok) * d * 4,
                "flops": 4.0 * n * hq * tok * (rows + tok / 2) * d}
    blocks = rows // BLOCK
    keys = min(rows, case["top"] * BLOCK) + BLOCK // 2
    return {"bytes": io + n * hkv * (blocks * (d + 4) + min(rows, tok * keys) * d * 4 + tok * case["top"] * 4),
            "flops": n * hq * tok * (2.0 * blocks * d + 4.0 * keys * d)}


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    lay, hkv = case["layers"], case["hkv"]
    if op == "norm_rope":
        # the pair (x_k, x_{k + d/2}) as a complex number times e^{i p omega_k}
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None, :, None] * s["omega"])

        def one(x, w):
            x = x.double()
            x = x / ((x.pow(2).sum(-1) / d + s["eps"]).sqrt())[..., None] * w.double()
            z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
            return torch.cat([z.real, z.imag], -1)

        return one(s["q"], s["qw"]), one(s["k"], s["kw"]), s["v"].double()
    if op == "append":
        for i in range(s["k_new"].shape[0]):
            q, at = i // lay, int(s["lengths"][i // lay])
            nodes = s["path"][q, :int(s["counts"][q])].long()
            s["k_cache"][i, :, at:at + len(nodes)] = s["k_new"][i][:, nodes]
            s["v_cache"][i, :, at:at + len(nodes)] = s["v_new"][i][:, nodes]
        return s["k_cache"], s["v_cache"], None
    if op == "summary":
        out = torch.zeros(s["codes"].shape, dtype=torch.float64, device=DEV)
        scl = torch.zeros(s["scales"].shape, dtype=torch.float64, device=DEV)
        for i in range(s["k"].shape[0]):
            rows = int(s["lengths"][i // lay])
            lo, hi = max(0, rows - case["appended"]) // BLOCK, rows // BLOCK
            if hi <= lo:
                continue
            x = s["k"][i, :, lo * BLOCK:hi * BLOCK].double().reshape(hkv, hi - lo, BLOCK, d)
            # the 8-bit code is defined on the mean, the factor and their
            # product in fp32
            m = (x.sum(2) / BLOCK).float()
            big = m.abs().max(-1).values
            code = torch.round(m * (127 / big.double()).float()[..., None])
            scl[i, :, lo:hi] = big.double() / 127
            out[i, :, lo:hi] = code.double() * scl[i, :, lo:hi, None]
        return out, scl
    tok, g = case["tok"], case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    if op == "tree":
        for i in range(s["q"].shape[0]):
            rows = int(s["lengths"][i // lay])
            bits = [int(b) & ((1 << 64) - 1) for b in s["tree"][i // lay].tolist()]
            sees = torch.tensor([[b >> j & 1 for j in range(tok)] for b in bits], device=DEV).bool()
            sees = torch.cat([torch.ones((tok, rows), dtype=torch.bool, device=DEV), sees], 1)
            for h in range(hkv):
                k = torch.cat([s["k_cache"][i, h, :rows], s["k_new"][i, h]]).double()
                v = torch.cat([s["v_cache"][i, h, :rows], s["v_new"][i, h]]).double()
                x = torch.einsum("gtd,kd->gtk", s["q"][i, h * g:(h + 1) * g].double(), k) * s["scale"]
                x[:, ~sees] = float("-inf")
                out[i, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
        return out
    if s["q"].shape[0] * hkv * tok > 2000:
        return None
    for i in range(s["q"].shape[0]):
        first = int(s["lengths"][i // lay]) - tok
        nb = first // BLOCK
        for h in range(hkv):
            for t in range(tok):
                q = s["q"][i, h * g:(h + 1) * g, t]
                keep = torch.zeros(first + tok, dtype=torch.bool, device=DEV)
                keep[nb * BLOCK:first + t + 1] = True
                if nb:
                    # whole-number scores of the 8-bit query against the codes
                    big = q.float().abs().max()
                    qi = torch.round(q.float() * (127 / big.double()).float()).double()
                    sc = (qi @ s["codes"][i, h, :nb].double().T).max(0).values.float() * s["scales"][i, h, :nb]
                    best = sorted(range(nb), key=lambda b, v=sc.tolist(): (-v[b], b))[:case["top"]]
                    keep[:nb * BLOCK].view(nb, BLOCK)[torch.tensor(best, device=DEV)] = True
                at = keep.nonzero()[:, 0]
                x = q.double() @ s["k_cache"][i, h, at].double().T * s["scale"]
                out[i, h * g:(h + 1) * g, t] = torch.softmax(x, -1) @ s["v_cache"][i, h, at].double()
    return out, None

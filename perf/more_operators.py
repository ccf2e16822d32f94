"""Measured cases of the operators over a paged cache, and of a draft's verification.

Five operators, used one after the other when a server answers for many streams
whose keys and values lie in pages of one pool:

  append    new rows of K and V go to the pages of their sequences
  attend    attention of a chunk of new tokens (one, or a whole prompt) over the
            cache they now belong to, causal among themselves
  weights   what attention each cache row received, accumulated over the calls
  evict     the rows of least accumulated weight leave: the others move, in
            their order, to fresh pages
  verify    which path of a drafted tree stands against the target's
            probabilities, and the token after it

Tensors are [batch, heads, tokens, head_dim], pages [pages, heads, rows,
head_dim]; the batch is sequences x layers, a page table has one row per batch
entry, and lengths, counts and trees have one entry per sequence.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new row for each of 16 streams x 4 layers, fp32 storage
        dict(name="append token f32", op="append", seqs=16, layers=4, hkv=8, d=128, tok=1, rows=1500, page=64,
             ragged=True, dtype="f32"),
        # a text prompt of 512 tokens, all 28 layers of the 12/2-head model
        dict(name="append prompt", op="append", seqs=1, layers=28, hkv=2, d=128, tok=512, rows=4608, page=64,
             ragged=False, dtype="bf16"),
        # one text token in one layer after a 512-frame video
        dict(name="attend token", op="attend", seqs=1, layers=1, hq=12, hkv=2, d=128, tok=1, rows=131073,
             page=256, ragged=False),
        # a short question after 300 rows, 14/2 heads of 64, small pages: latency
        dict(name="attend short", op="attend", seqs=1, layers=1, hq=14, hkv=2, d=64, tok=77, rows=377, page=16,
             ragged=False),
        # one token each for 16 streams of different lengths in one layer
        dict(name="attend ragged batch", op="attend", seqs=16, layers=1, hq=16, hkv=8, d=128, tok=1, rows=32768,
             page=64, ragged=True),
        # a text prompt of 512 tokens in one layer after a 512-frame video
        dict(name="attend prompt", op="attend", seqs=1, layers=1, hq=12, hkv=2, d=128, tok=512, rows=131584,
             page=64, ragged=False),
        # the weights of one token each for 16 streams of different lengths
        dict(name="weights ragged batch", op="weights", seqs=16, layers=1, hq=16, hkv=8, d=128, tok=1, rows=32768,
             page=64, ragged=True),
        # the weights of the 512-token prompt
        dict(name="weights prompt", op="weights", seqs=1, layers=1, hq=12, hkv=2, d=128, tok=512, rows=131584,
             page=64, ragged=False),
        # every layer falls back to its budget of 4096 rows after a frame and some text
        dict(name="evict frame", op="evict", seqs=1, layers=28, hkv=2, d=128, rows=4429, keep=4096, sinks=4,
             recent=128, page=64, ragged=False, dtype="bf16", apart=True),
        # a whole 512-frame video in one layer with 8 KV heads falls to 4096 rows
        dict(name="evict video", op="evict", seqs=1, layers=1, hkv=8, d=128, rows=131072, keep=4096, sinks=256,
             recent=256, page=64, ragged=False, dtype="bf16", apart=False),
        # a small tree of one stream whose drafts come without probabilities
        dict(name="verify proposals", op="verify", seqs=1, tok=7, vocab=32000, draft=False),
        # 16 streams with 42 drafted tokens each, a large vocabulary of odd size
        dict(name="verify batch", op="verify", seqs=16, tok=42, vocab=150001, draft=True),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weights", "weights", "evict", "verify"])
    seqs = _between(rng, 1, 16)
    if op == "verify":
        return dict(op=op, seqs=seqs, tok=_between(rng, 1, 42), vocab=_between(rng, 1000, 150001),
                    draft=rng.random() < 0.6)
    hq, hkv = rng.choice([(14, 2), (12, 2), (16, 8), (4, 2), (8, 8)])
    d = rng.choice([64, 128, 128])
    layers = rng.choice([1, 1, 2, 4])
    page = rng.choice([16, 32, 64, 128, 256])
    rows = _between(rng, 40, 131072)
    # at most 2 GB of cache
    rows = max(64, min(rows, (2 << 30) // (seqs * layers * hkv * d * 4)))
    c = dict(op=op, seqs=seqs, layers=layers, hkv=hkv, d=d, page=page, rows=rows, ragged=rng.random() < 0.5)
    if op == "evict":
        keep = _between(rng, 16, rows)
        return dict(c, keep=keep, sinks=rng.randrange(0, keep // 4 + 1), recent=rng.randrange(0, keep // 2 + 1),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), apart=rng.random() < 0.5)
    tok = min(rows, rng.choice([1, _between(rng, 1, 16), _between(rng, 1, 512)]))
    if op == "append":
        return dict(c, tok=min(tok, 16) if seqs * layers * hkv > 64 else tok, dtype=rng.choice(["bf16", "bf16", "f32"]))
    # the largest listed case has 8.1e8 pairs of a query row and a key
    while seqs * layers * hq * tok * rows > 8e8:
        tok, rows = max(1, tok // 2), max(64, rows * 3 // 4)
    return dict(c, rows=max(rows, tok), hq=hq, tok=tok)


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _counts(case, gen):
    """New tokens of each sequence (a padded batch where lengths are ragged)."""
    if not case["ragged"]:
        return torch.full((case["seqs"],), case["tok"], dtype=torch.int32, device=DEV)
    x = torch.randint(1, case["tok"] + 1, (case["seqs"],), generator=gen, device=DEV)
    x[0] = case["tok"]
    return x.to(torch.int32)


def _lengths(case, gen, lo):
    """Rows of each sequence in the cache, int32 on the GPU."""
    if not case["ragged"]:
        return torch.full((case["seqs"],), case["rows"], dtype=torch.int32, device=DEV)
    x = torch.randint(lo, case["rows"] + 1, (case["seqs"],), generator=gen, device=DEV)
    x[0] = case["rows"]
    return x.to(torch.int32)


def _tables(gen, page, *rows):
    """Page tables [n, pages] for the rows (int64 [n]) that each batch entry
    needs, in any order of one pool without a page twice; -1 past the last.
    The pool would hold every entry at the longest one's length."""
    need = [(r + page - 1) // page for r in rows]
    pool = sum(len(x) * int(x.max()) for x in need) + 3
    order = torch.randperm(pool, generator=gen, device=DEV)
    out, at = [], 0
    for x in need:
        first = at + x.cumsum(0) - x
        slot = torch.arange(int(x.max()), device=DEV)
        t = order[(first[:, None] + slot).clamp(max=pool - 1)]
        out.append(torch.where(slot < x[:, None], t, -1).to(torch.int32))
        at += int(x.sum())
    return pool, out


def _tree(case, gen):
    """Parents of a random tree per sequence (-1: a root) as a list of lists,
    and the bit masks of the nodes that each node sees, itself included."""
    tok, seqs = case["tok"], case["seqs"]
    r = torch.rand((seqs, tok), generator=gen, device=DEV).cpu()
    parents, masks = [], []
    for s in range(seqs):
        bits, above = [], []
        for i in range(tok):
            # recent nodes are the likelier parents; few roots
            p = i - 1 - int(float(r[s, i]) ** 2 * (i + 1))
            above.append(p)
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        parents.append(above)
        masks.append([b - (1 << 64) if b >> 63 else b for b in bits])
    return parents, torch.tensor(masks, dtype=torch.int64, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, s = case["op"], dict(case=case)
    if op == "verify":
        seqs, tok, vocab = case["seqs"], case["tok"], case["vocab"]
        # distributions as of a language model: a few likely tokens, a long tail;
        # row 0 after the text so far, row i + 1 after node i
        x = 3.0 * torch.randn((seqs, tok + 1, vocab), generator=gen, device=DEV)
        s["target"] = torch.softmax(x, -1)
        x += 1.0 * torch.randn(x.shape, generator=gen, device=DEV)
        q = torch.softmax(x, -1)
        del x
        parents, s["tree"] = _tree(case, gen)
        row = torch.tensor(parents, device=DEV) + 1
        b = torch.arange(seqs, device=DEV)[:, None]
        # each node is drawn from the draft's distribution after its parent
        s["tokens"] = torch.multinomial(q[b, row].flatten(0, 1), 1, generator=gen).view(seqs, tok).to(torch.int32)
        if not case["draft"]:
            # proposals of one parent differ: each token of the vocabulary once
            s["tokens"] = ((s["tokens"][:, :1].long() + torch.arange(tok, device=DEV) * 17) % vocab).to(torch.int32)
            best = s["target"][b, row].argmax(-1)
            first = torch.tensor([[p not in a[:i] for i, p in enumerate(a)] for a in parents], device=DEV)
            clash = (s["tokens"][:, :, None] == best[:, None, :]).any(-1)
            s["tokens"] = torch.where(first & ~clash, best.to(torch.int32), s["tokens"])
        s["draft"] = q if case["draft"] else None
        s["uniforms"] = torch.rand((seqs, tok + 1), generator=gen, device=DEV)
        return s
    n, hkv, d, page = case["seqs"] * case["layers"], case["hkv"], case["d"], case["page"]
    lay = case["layers"]
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    tok = case.get("tok", 0)
    if tok:
        s["counts"] = _counts(case, gen)
    if op == "append":
        s["lengths"] = _lengths(case, gen, 0)
        pool, (s["table"],) = _tables(gen, page, (s["lengths"] + s["counts"]).long().repeat_interleave(lay))
        s["k_new"], s["v_new"] = _randn(gen, n, hkv, tok, d, dtype=dt), _randn(gen, n, hkv, tok, d, dtype=dt)
        s["k_pages"], s["v_pages"] = (torch.zeros((pool, hkv, page, d), dtype=dt, device=DEV) for _ in range(2))
        return s
    if op == "evict":
        s["lengths"] = _lengths(case, gen, 1)
        rows = s["lengths"].long().repeat_interleave(lay)
        kept = rows.clamp(max=case["keep"])
        if case["apart"]:
            pool, (s["table"],) = _tables(gen, page, rows)
            pool_out, (s["out_table"],) = _tables(gen, page, kept)
        else:
            pool, (s["table"], s["out_table"]) = _tables(gen, page, rows, kept)
        s["k_pages"], s["v_pages"] = (_randn(gen, pool, hkv, page, d, dtype=dt) for _ in range(2))
        s["k_out"], s["v_out"] = s["k_pages"], s["v_pages"]
        if case["apart"]:
            s["k_out"], s["v_out"] = (torch.zeros((pool_out, hkv, page, d), dtype=dt, device=DEV) for _ in range(2))
        # few rows with much weight, a tenth that received none at all
        cap = s["table"].shape[1] * page
        w = torch.exp(2.0 * torch.randn((n, hkv, cap), generator=gen, device=DEV))
        s["weights"] = w * (torch.rand(w.shape, generator=gen, device=DEV) > 0.1)
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    # every sequence holds its new tokens
    s["lengths"] = torch.maximum(_lengths(case, gen, 1), s["counts"])
    pool, (s["table"],) = _tables(gen, page, s["lengths"].long().repeat_interleave(lay))
    s["k_pages"] = _randn(gen, pool, hkv, page, d)
    s["q"] = _randn(gen, n, case["hq"], tok, d)
    if op == "attend":
        s["v_pages"] = _randn(gen, pool, hkv, page, d)
        return s
    s["lse"] = _scores(s)[1]
    cap = s["table"].shape[1] * page
    s["before"] = torch.rand((n, hkv, cap), generator=gen, device=DEV)
    return s


# ------------------------------------------------------------- plain forms
def _gather(pages, table):
    """Rows [n, heads, rows, d] in fp32 of the pages that the table names."""
    x = pages[table.long().clamp(min=0)].float()
    return x.transpose(1, 2).flatten(2, 3)


def _scores(s):
    """Masked scores [n, hkv, g * tok, rows] and each query row's log-sum-exp
    [n, hq, tok]."""
    c = s["case"]
    n, hq, tok, d = s["q"].shape
    k = _gather(s["k_pages"], s["table"])
    x = (s["q"].float() * s["scale"]).reshape(n, c["hkv"], -1, d) @ k.transpose(-1, -2)
    first = (s["lengths"] - s["counts"]).repeat_interleave(c["layers"])
    j = torch.arange(tok, device=DEV)
    last = torch.where(j < s["counts"].repeat_interleave(c["layers"])[:, None], first[:, None] + j, -1)
    sees = torch.arange(k.shape[2], device=DEV) <= last[:, :, None]
    x = x.masked_fill_(~sees.repeat(1, hq // c["hkv"], 1)[:, None], float("-inf"))
    return x, torch.logsumexp(x, -1).view(n, hq, tok)


def _plain_append(s):
    c = s["case"]
    n, hkv, tok, d = s["k_new"].shape
    # steps past the count write the last new row once more
    use = torch.minimum(torch.arange(tok, device=DEV), s["counts"][:, None].long() - 1)
    row = (s["lengths"][:, None].long() + use).repeat_interleave(c["layers"], 0)
    use = use.repeat_interleave(c["layers"], 0)
    page = s["table"].long().gather(1, row // c["page"])
    b = torch.arange(n, device=DEV)[:, None]
    s["k_pages"][page, :, row % c["page"]] = s["k_new"][b, :, use]
    s["v_pages"][page, :, row % c["page"]] = s["v_new"][b, :, use]
    return s["k_pages"], s["v_pages"], s["lengths"] + s["counts"]


def _plain_attend(s):
    x, lse = _scores(s)
    n, hkv, r, rows = x.shape
    at = lse.view(n, hkv, r, 1)
    p = x.sub_(at.masked_fill(at == float("-inf"), 0.0)).exp_()
    o = p @ _gather(s["v_pages"], s["table"])
    return o.view(s["q"].shape).to(s["q"].dtype), lse


def _plain_weights(s):
    x, _ = _scores(s)
    n, hkv, r, rows = x.shape
    at = s["lse"].view(n, hkv, r, 1)
    p = x.sub_(at.masked_fill(at == float("-inf"), 0.0)).exp_()
    return s["before"] + p.sum(2)


def _plain_evict(s):
    c = s["case"]
    n, hkv, cap = s["weights"].shape
    keep, page, lay = c["keep"], c["page"], c["layers"]
    lens = s["lengths"].long().repeat_interleave(lay)
    row = torch.arange(cap, device=DEV)
    safe = (row < c["sinks"]) | (row >= lens[:, None] - c["recent"])
    w = s["weights"].masked_fill(safe[:, None], float("inf"))
    w = w.masked_fill((row >= lens[:, None])[:, None], float("-inf"))
    kept = w.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = kept.masked_fill(kept >= lens[:, None, None], cap).sort(-1).values
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=cap)
    gone = kept == cap
    new = s["lengths"].clamp(max=keep)
    # destination slots past the new length write the last kept row once more
    i = torch.arange(keep, device=DEV)
    use = torch.minimum(i, new.long().repeat_interleave(lay)[:, None] - 1)
    src = kept.gather(2, use[:, None].expand(n, hkv, keep))
    b = torch.arange(n, device=DEV)[:, None, None]
    h = torch.arange(hkv, device=DEV)[None, :, None]
    page_in = s["table"].long()[b, src // page]
    page_out = s["out_table"].long().gather(1, use // page)[:, None]
    slot = (use % page)[:, None]
    s["k_out"][page_out, h, slot] = s["k_pages"][page_in, h, src % page]
    s["v_out"][page_out, h, slot] = s["v_pages"][page_in, h, src % page]
    weights = s["weights"].gather(2, kept.clamp(max=cap - 1)).masked_fill(gone, 0.0)
    wide = s["out_table"].shape[1] * page
    weights = torch.nn.functional.pad(weights, (0, max(0, wide - keep)))[..., :wide]
    return s["k_out"], s["v_out"], new, weights, kept.masked_fill(gone, -1).to(torch.int32)


def _plain_verify(s):
    c = s["case"]
    seqs, tok, vocab = c["seqs"], c["tok"], c["vocab"]
    b = torch.arange(seqs, device=DEV)
    node = torch.arange(tok, device=DEV)
    # a node's parent is the highest lower node that it sees; row 0 of the
    # distributions stands before every node
    seen = (s["tree"][:, :, None] >> node) & 1 & (node < node[:, None])
    row = (seen * (node + 1)).amax(-1)
    x, u = s["tokens"].long(), s["uniforms"].double()
    p = s["target"][b[:, None], row, x].double()
    at = torch.zeros(seqs, dtype=torch.int64, device=DEV)           # current row
    left = torch.ones(seqs, dtype=torch.float64, device=DEV)        # R
    path = torch.full((seqs, tok + 1), -1, dtype=torch.int32, device=DEV)
    counts = torch.zeros(seqs, dtype=torch.int64, device=DEV)
    if s["draft"] is not None:
        q = s["draft"][b[:, None], row, x].double()
        used = torch.zeros(seqs, dtype=torch.float64, device=DEV)   # c
    else:
        refused = torch.zeros((seqs, vocab), dtype=torch.bool, device=DEV)
    for i in range(tok):
        tried = row[:, i] == at
        if s["draft"] is not None:
            r = (p[:, i] - used * q[:, i]).clamp(min=0.0)
            yes = tried & (u[:, i] * q[:, i] * left < r)
        else:
            r = p[:, i].masked_fill(refused[b, x[:, i]], 0.0)
            yes = tried & (u[:, i] * left < r)
        no = tried & ~yes
        path[b, torch.where(yes, counts, tok)] = torch.where(yes, i, -1).to(torch.int32)
        counts = counts + yes
        if s["draft"] is not None:
            used = torch.where(no, used + left, used)
            rest = (s["target"][b, at].double() - used[:, None] * s["draft"][b, at].double()).clamp(min=0.0).sum(-1)
            left = torch.where(yes, 1.0, torch.where(no, rest, left))
            used = used.masked_fill(yes, 0.0)
        else:
            left = torch.where(yes, 1.0, torch.where(no, (left - r).clamp(min=0.0), left))
            refused = refused & ~yes[:, None]
            refused[b, x[:, i]] |= no
        at = torch.where(yes, i + 1, at)
    rest = s["target"][b, at].double()
    if s["draft"] is not None:
        rest = (rest - used[:, None] * s["draft"][b, at].double()).clamp(min=0.0)
    else:
        rest = rest.masked_fill(refused, 0.0)
    upto = rest.cumsum(-1)
    # the lowest token whose sum passes u times the whole
    token = (upto <= u[:, tok:] * upto[:, -1:]).sum(-1)
    return path[:, :tok], counts.to(torch.int32), token.to(torch.int32)


# ---------------------------------------------------------------- one pass
def _own(s):
    import kv_cache_compression_frame_gb300 as kv

    op = s["case"]["op"]
    if op == "append":
        lengths = kv.paged_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                                  s["counts"])
        return s["k_pages"], s["v_pages"], lengths
    if op == "attend":
        return kv.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["counts"],
                                  scale=s["scale"], with_lse=True)
    if op == "weights":
        return kv.attention_weights(s["q"], s["lse"], s["k_pages"], s["table"], s["lengths"], s["counts"],
                                    scale=s["scale"], before=s["before"])
    if op == "evict":
        c = s["case"]
        return s["k_out"], s["v_out"], *kv.evict_rows(
            s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["weights"], c["keep"], s["out_table"],
            sinks=c["sinks"], recent=c["recent"], k_out=s["k_out"], v_out=s["v_out"])
    return kv.verify_tree(s["target"], s["draft"], s["tokens"], s["tree"], s["uniforms"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict,
            "verify": _plain_verify}[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "verify":
        # one row of p, and of q where there is one, beside single values
        rows = 2 if case["draft"] else 1
        return {"bytes": case["seqs"] * (rows * case["vocab"] * 4 + case["tok"] * 24), "flops":
                case["seqs"] * case["vocab"] * 3.0}
    n, hkv, d = case["seqs"] * case["layers"], case["hkv"], case["d"]
    e = 4 if case.get("dtype") == "f32" else 2
    # ragged numbers are uniform up to the largest
    part = 0.5 + 0.5 / case["seqs"] if case["ragged"] else 1.0
    if op == "append":
        new = n * hkv * case["tok"] * part
        return {"bytes": new * d * e * 4 + case["seqs"] * 12, "flops": 0}
    rows = case["rows"] * part
    if op == "evict":
        keep = min(rows, case["keep"])
        return {"bytes": n * hkv * (rows * 4 + keep * (d * e * 4 + 8)), "flops": 0}
    new = case["tok"] * part
    pairs = n * case["hq"] * new * max(1.0, rows - new / 2)
    if op == "attend":
        return {"bytes": n * (hkv * rows * d * 4 + case["hq"] * case["tok"] * (d * 4 + 4)), "flops": 4.0 * pairs * d}
    return {"bytes": n * (hkv * rows * (d * 2 + 8) + case["hq"] * case["tok"] * (d * 2 + 4)),
            "flops": 2.0 * pairs * d}


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict" and case["seqs"] * case["layers"] * case["hkv"] * case["rows"] > 4e6:
        return None                                 # (sorted row by row on the host)
    if op == "verify":
        return _exact_verify(case, s)
    lay, hkv, page = case["layers"], case["hkv"], case["page"]
    n = case["seqs"] * lay
    table = s["table"].tolist()

    def rows_of(pages, i, h, count):
        used = torch.tensor(table[i][:(count + page - 1) // page], device=DEV, dtype=torch.int64)
        return pages[used, h].reshape(-1, case["d"])[:count]

    if op == "append":
        for i in range(n):
            at, new = int(s["lengths"][i // lay]), int(s["counts"][i // lay])
            for j in range(new):
                p, slot = table[i][(at + j) // page], (at + j) % page
                s["k_pages"][p, :, slot] = s["k_new"][i, :, j]
                s["v_pages"][p, :, slot] = s["v_new"][i, :, j]
        return s["k_pages"], s["v_pages"], None
    if op == "evict":
        weights = torch.zeros((n, hkv, s["out_table"].shape[1] * page), dtype=torch.float64, device=DEV)
        kept = torch.full((n, hkv, case["keep"]), -1, dtype=torch.int32, device=DEV)
        new = s["lengths"].clone()
        moved = []
        for i in range(n):
            rows = int(s["lengths"][i // lay])
            new[i // lay] = min(rows, case["keep"])
            for h in range(hkv):
                free = range(min(rows, case["sinks"]), max(min(rows, case["sinks"]), rows - case["recent"]))
                w = s["weights"][i, h].tolist()
                drop = sorted(free, key=lambda r, w=w: (w[r], -r))[:max(0, rows - case["keep"])]
                stay = torch.ones(rows, dtype=torch.bool)
                stay[torch.tensor(drop, dtype=torch.int64)] = False
                at = stay.nonzero()[:, 0].to(DEV)
                kept[i, h, :len(at)] = at.to(torch.int32)
                weights[i, h, :len(at)] = s["weights"][i, h, at].double()
                to = s["out_table"][i].long()[torch.arange(len(at), device=DEV) // page]
                moved.append((to, h, torch.arange(len(at), device=DEV) % page,
                              rows_of(s["k_pages"], i, h, rows)[at], rows_of(s["v_pages"], i, h, rows)[at]))
        for to, h, slot, k, v in moved:
            s["k_out"][to, h, slot] = k
            s["v_out"][to, h, slot] = v
        return s["k_out"], s["v_out"], new, weights, kept
    hq, tok = case["hq"], case["tok"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:3], float("-inf"), dtype=torch.float64, device=DEV)
    weights = s["before"].double() if op == "weights" else None
    for i in range(n):
        rows, new = int(s["lengths"][i // lay]), int(s["counts"][i // lay])
        hidden = torch.ones((new, rows), dtype=torch.bool, device=DEV).triu(rows - new + 1)
        for h in range(hkv):
            k = rows_of(s["k_pages"], i, h, rows).double()
            for j in range(h * g, (h + 1) * g):
                x = torch.einsum("td,kd->tk", s["q"][i, j, :new].double(), k) * s["scale"]
                x[hidden] = float("-inf")
                if op == "weights":
                    weights[i, h, :rows] += torch.exp(x - s["lse"][i, j, :new, None].double()).sum(0)
                else:
                    lse[i, j, :new] = torch.logsumexp(x, -1)
                    out[i, j, :new] = torch.softmax(x, -1) @ rows_of(s["v_pages"], i, h, rows).double()
    return (out, lse) if op == "attend" else weights


def _exact_verify(case, s):
    tok = case["tok"]
    paths = torch.full((case["seqs"], tok), -1, dtype=torch.int32)
    counts, tokens = [], []
    for b in range(case["seqs"]):
        bits = [int(x) & ((1 << 64) - 1) for x in s["tree"][b].tolist()]
        parent = [(x & ((1 << i) - 1)).bit_length() - 1 for i, x in enumerate(bits)]
        u, drafted = s["uniforms"][b].tolist(), s["tokens"][b].tolist()
        at, path = -1, []
        while True:
            # the residual after each refusal is a distribution of its own
            rest = s["target"][b, at + 1].double()
            q = s["draft"][b, at + 1].double() if s["draft"] is not None else None
            for child in (i for i in range(tok) if parent[i] == at):
                x = drafted[child]
                if q is None:
                    tried = {drafted[i] for i in range(child) if parent[i] == at}
                    whole = max(0.0, 1.0 - sum(float(s["target"][b, at + 1, t]) for t in tried))
                    if u[child] * whole < float(rest[x]):
                        break
                    rest[x] = 0.0
                else:
                    if u[child] * float(q[x]) < float(rest[x]):
                        break
                    rest = (rest - q).clamp(min=0.0)
                    rest = rest / rest.sum()
            else:
                upto = rest.cumsum(0)
                tokens.append(int(torch.searchsorted(upto, u[tok] * upto[-1], right=True)))
                break
            at = child
            path.append(child)
        counts.append(len(path))
        paths[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
    return (paths.to(DEV), torch.tensor(counts, dtype=torch.int32, device=DEV),
            torch.tensor(tokens, dtype=torch.int32, device=DEV))

"""Cases and plain forms of a serving step with drafted tokens over the paged
e4m3 KV cache: the append with head norms and rotation, the masks and positions
of a tree of drafts, attention under such masks, the drafts' verification, and
the cache's clean-up after it.

``run`` computes either the plain forms (elementary torch operations in 32
bits, 64 where a rounded value decides a code or a token) or, with ``own`` set,
the library's entry points on the same state.
"""

import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def listed():
    return [
        # plain decoding: one new token of each of 64 sequences, pages of 16
        {"name": "rope_append_64x1", "op": "append", "seqs": 64, "new": 1, "context": 2000, "page": 16, "kv_heads": 8,
         "group": 4, "dim": 128, "rot": 128, "norm": False, "pairs": "half", "tree": False, "dtype": "fp16"},
        # drafted trees of a model of narrow heads that rotates half of each, neighbours together
        {"name": "rope_append_tree", "op": "append", "seqs": 12, "new": 26, "context": 1500, "page": 32, "kv_heads": 2,
         "group": 7, "dim": 64, "rot": 32, "norm": False, "pairs": "next", "tree": True, "dtype": "fp16"},
        # prompts of a model with head norms
        {"name": "rope_append_3x2048", "op": "append", "seqs": 3, "new": 2048, "context": 300, "page": 64,
         "kv_heads": 8, "group": 4, "dim": 128, "rot": 128, "norm": True, "pairs": "half", "tree": False,
         "dtype": "bf16"},
        # one sequence's few drafts
        {"name": "mask_1x8", "op": "mask", "seqs": 1, "new": 8, "context": 777},
        # a serving batch of large trees
        {"name": "mask_96x200", "op": "mask", "seqs": 96, "new": 200, "context": 3000},
        # one sequence with a few drafts, where latency is everything
        {"name": "tree_attend_1x8", "op": "attend", "seqs": 1, "new": 8, "context": 777, "page": 16, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "fp16"},
        # a ragged batch, narrow heads, an odd group
        {"name": "tree_attend_16x26", "op": "attend", "seqs": 16, "new": 26, "context": 4096, "page": 32,
         "kv_heads": 4, "group": 7, "dim": 64, "dtype": "bf16"},
        # full trees over long contexts
        {"name": "tree_attend_8x64", "op": "attend", "seqs": 8, "new": 64, "context": 8192, "page": 64, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16"},
        # a tree of one sequence, small vocabulary
        {"name": "verify_1x8", "op": "verify", "seqs": 1, "new": 8, "vocab": 32000, "draft": False},
        # sampled chains of a batch, with the draft's probabilities
        {"name": "verify_64x6", "op": "verify", "seqs": 64, "new": 6, "vocab": 128000, "draft": True},
        # one sequence's accepted drafts, one layer
        {"name": "keep_1x8", "op": "keep", "seqs": 1, "new": 8, "context": 777, "page": 16, "kv_heads": 8, "dim": 128,
         "layers": 1},
        # a batch's, several layers in one call
        {"name": "keep_16x64", "op": "keep", "seqs": 16, "new": 64, "context": 200, "page": 32, "kv_heads": 8,
         "dim": 128, "layers": 8},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "mask", "attend", "attend", "attend", "verify", "keep"])
    if op == "mask":
        return {"op": op, "seqs": _log(rng, 1, 90), "new": _log(rng, 1, 200), "context": _log(rng, 1, 4000)}
    if op == "verify":
        return {"op": op, "seqs": _log(rng, 1, 60), "new": _log(rng, 2, 6), "vocab": _log(rng, 2000, 120000),
                "draft": rng.random() < 0.5}
    page, dim = rng.choice([16, 32, 64, 128]), rng.choice([64, 128])
    heads, dtype = rng.choice([1, 2, 4, 8]), rng.choice(["bf16", "fp16"])
    if op == "keep":
        return {"op": op, "seqs": _log(rng, 1, 16), "new": _log(rng, 4, 64), "context": _log(rng, 1, 200),
                "page": page, "kv_heads": heads, "dim": dim, "layers": rng.choice([1, 2, 4])}
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 64), _log(rng, 65, 250)])
        return {"op": op, "seqs": _log(rng, 1, 48 if new <= 64 else 16), "new": new,
                "context": _log(rng, 1, 2000), "page": page, "kv_heads": heads, "group": rng.choice([1, 3, 4]),
                "dim": dim, "rot": rng.choice([dim, dim // 2, 48]), "norm": rng.random() < 0.5,
                "pairs": rng.choice(["half", "next"]), "tree": rng.random() < 0.5, "dtype": dtype}
    new = rng.choice([1, _log(rng, 2, 12), _log(rng, 13, 64), _log(rng, 65, 150)])
    return {"op": op, "seqs": _log(rng, 1, 12 if new <= 12 else 5), "new": new,
            "context": _log(rng, 1, 5000 if new <= 64 else 2000), "page": page, "kv_heads": heads, "group": group,
            "dim": dim, "dtype": dtype}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """New tokens and total length of every sequence: ragged, the first one the
    longest. They belong to the case (its outputs' shapes follow from them), not
    to the seed."""
    g = torch.Generator().manual_seed(11)
    n = case["seqs"]
    new = torch.full((n,), case["new"])
    if case["new"] > 8 and case["op"] != "verify":
        new = (case["new"] * (0.5 + 0.5 * torch.rand(n, generator=g))).ceil().long()
        new[0] = case["new"]
    old = (case.get("context", 1) * (0.25 + 0.75 * torch.rand(n, generator=g))).ceil().long()
    old[0] = case.get("context", 1)
    return new.tolist(), (new + old).tolist()


def _kept(case):
    """Nodes of each sequence that stay, the root among them: about what trees of that size give."""
    new, _ = _lengths(case)
    g = torch.Generator().manual_seed(12)
    return [1 + int(torch.randint(0, min(max(a // 3, 1), 9), (1,), generator=g)) for a in new]


def _trees(case, seed):
    """Parents [seqs, new] in each sequence's own numbers: node 0 is the root, its
    first children follow it, deeper nodes hang on one of the eight before them or so."""
    g = torch.Generator().manual_seed(seed)
    n, most = case["seqs"], case["new"]
    at = torch.arange(most)
    back = (torch.rand(n, most, generator=g) * torch.minimum(at, torch.tensor(8))).long()
    return torch.where(at == 0, torch.full_like(back, -1), (at - 1 - back).clamp(min=0))


def _ancestors(parents):
    """[seqs, new, new] truth values: column j of row i says that j is i or above it."""
    n, most = parents.shape
    seen = torch.zeros((n, most, most), dtype=torch.bool)
    for j in range(most):
        if j:
            seen[:, j] = seen[torch.arange(n), parents[:, j]]
        seen[:, j, j] = True
    return seen


def _words(bits):
    """[..., n] truth values as [..., ceil(n / 32)] words of 32 bits, the first lowest."""
    n = bits.shape[-1]
    pad = torch.nn.functional.pad(bits.long(), (0, -n % 32)).unflatten(-1, (-1, 32))
    w = (pad << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def _ragged(x, new):
    """The first new[b] rows of every x[b], one behind the other."""
    return torch.cat([x[b, :a] for b, a in enumerate(new)])


def _batch(case, seed, dev):
    """Tables of a pool with more pages than the sequences hold, in no order."""
    new, total = _lengths(case)
    page, n = case["page"], case["seqs"]
    width = (max(total) + page - 1) // page
    used = [(t + page - 1) // page for t in total]
    pool = sum(used) + 5
    order = torch.randperm(pool - 1, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.zeros((n, width), dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    return {"table": table.to(dev), **_rows(new, total, dev)}, pool


def _rows(new, total, dev):
    return {"cu": torch.tensor([0] + new).cumsum(0).int().to(dev), "lens": torch.tensor(total).int().to(dev),
            "max_new": max(new)}


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]
    new, total = _lengths(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    st = {"case": case}
    if op == "mask":
        st.update(_rows(new, total, dev))
        st["parents"] = _ragged(_trees(case, seed), new).int().to(dev)
        return st
    if op == "verify":
        st.update(_rows(new, total, dev))
        parents = _trees(case, seed).to(dev)
        n, most, vocab = case["seqs"], case["new"], case["vocab"]
        logits = 4 * normal(n, most, vocab)
        st["probs"] = torch.softmax(logits, -1).view(n * most, vocab)
        st["uniform"] = torch.rand(n * most, generator=g, device=dev)
        tokens = torch.zeros((n, most), dtype=torch.long, device=dev)
        if case["draft"]:  # a chain, drawn from a distribution close to the target's
            q = torch.softmax(logits.add_(normal(n, most, vocab), alpha=0.7), -1)
            for j in range(1, most):
                tokens[:, j] = torch.multinomial(q[:, j - 1], 1, generator=g)[:, 0]
            st["draft"] = q.view(n * most, vocab)
        else:  # siblings are the likeliest tokens of their parent's row, in order
            top = logits.topk(min(most, vocab), -1).indices
            for j in range(1, most):
                older = (parents[:, :j] == parents[:, j:j + 1])[:, 1:].sum(1)
                tokens[:, j] = top[torch.arange(n, device=dev), parents[:, j], older]
            st["parents"] = parents.int().view(-1)
        st["tokens"] = tokens.int().view(-1)
        return st

    batch, pool = _batch(case, seed, dev)
    st.update(batch)
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    lead = (case["layers"], pool) if op == "keep" else (pool,)

    def codes(*shape):
        return (normal(*lead, *shape) * 90).clamp(-448, 448).to(E4M3)

    def scales():
        return torch.exp2(torch.randint(-8, -5, (*lead, heads), generator=g, device=dev).float())

    st.update(k_cache=codes(heads, page, dim), v_cache=codes(heads, dim, page), k_scales=scales(), v_scales=scales())
    if op == "keep":
        kept = _kept(case)
        path = torch.full((case["seqs"], case["new"]), -1, dtype=torch.int32)
        order = torch.Generator().manual_seed(seed)
        for b, (a, m) in enumerate(zip(new, kept)):  # the root, then nodes behind the kept places
            path[b, 0] = 0
            path[b, 1:m] = (m + torch.randperm(a - m, generator=order)[:m - 1]).sort().values.int()
        st["path"], st["kept"] = path.to(dev), torch.tensor(kept).int().to(dev)
        return st

    dt = st["dt"] = DTYPES[case["dtype"]]
    tokens, q_heads = sum(new), heads * case["group"]
    if op == "attend":
        st["q"] = normal(tokens, q_heads, dim).to(dt)
        st["scale"] = dim ** -0.5
        st["tree"] = _ragged(_words(_ancestors(_trees(case, seed))), new).to(dev)
        return st
    # slices of one projection's output, as a model has them
    qkv = normal(tokens, q_heads + 2 * heads, dim).to(dt)
    st["q"], st["k"], st["v"] = qkv.split([q_heads, heads, heads], 1)
    half = case["rot"] // 2
    angle = torch.arange(max(total), device=dev).double()[:, None] * 1e4 ** -(
        torch.arange(half, device=dev).double() / half)
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    st["qw"] = st["kw"] = st["positions"] = None
    if case["norm"]:
        st["qw"], st["kw"] = ((1 + 0.2 * normal(dim)).to(dt) for _ in "qk")
    if case["tree"]:
        depth = _ancestors(_trees(case, seed)).sum(-1) - 1
        start = torch.tensor([t - a for a, t in zip(new, total)])
        st["positions"] = _ragged(start[:, None] + depth, new).int().to(dev)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _codes(c, at):
    return c.view(torch.uint8)[at].view(E4M3)


def _plain_turn(st, x, w, pos):
    """x [T, heads, D] in 32 bits: normed per head, then rotated."""
    case, x = st["case"], x.float()
    if w is not None:
        mean = x.double().square().mean(-1, keepdim=True)
        x = x * (1.0 / (mean + EPS).sqrt()).float() * w.float()
    rot = case["rot"]
    half = rot // 2
    cs = st["cos_sin"][pos]
    c, s = cs[:, None, :half], cs[:, None, half:]
    out = x.clone()
    if case["pairs"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        out[..., :half], out[..., half:rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return out


def _page_scale(amax):
    """Smallest power of two s with amax <= 448 s, its exponent held in [-100, 120]."""
    mant, expo = torch.frexp(amax)  # amax = mant 2^expo, 448 = 0.875 * 2^9
    expo = torch.where(mant > 0.875, expo - 8, expo - 9).clamp(-100, 120)
    return torch.exp2(torch.where(amax > 0, expo, torch.full_like(expo, -100)).double()).float()


def _plain_append(st):
    case = st["case"]
    page, n = case["page"], case["seqs"]
    cu, lens = st["cu"].long(), st["lens"].long()
    new = cu[1:] - cu[:-1]
    start = lens - new
    if st["positions"] is None:
        row = torch.arange(st["q"].shape[0], device=cu.device)
        seq = torch.searchsorted(cu[1:], row, right=True)
        at = start[seq] + row - cu[seq]
    else:
        at = st["positions"].long()
    q = _plain_turn(st, st["q"], st["qw"], at).to(st["dt"])
    k = _plain_turn(st, st["k"], st["kw"], at)
    # every page that may hold new tokens: sequence i, its pages first .. first + span
    span = (st["max_new"] + page - 2) // page + 1
    slot = (start // page)[:, None] + torch.arange(span, device=cu.device)
    pos = slot[..., None] * page + torch.arange(page, device=cu.device)  # [n, span, page]
    fresh = (pos >= start[:, None, None]) & (pos < lens[:, None, None])
    older = slot * page < start[:, None]
    live = fresh.any(-1)
    ids = st["table"].long().gather(1, slot.clamp(max=st["table"].shape[1] - 1))
    token = (cu[:-1, None, None] + pos - start[:, None, None]).clamp(0, k.shape[0] - 1)
    # pages without new tokens write the last page of the pool, which no table names, its own contents
    ids = torch.where(live, ids, torch.full_like(ids, st["k_cache"].shape[0] - 1)).view(-1)
    fresh, older, live = fresh.view(n * span, 1, page, 1), older.view(-1, 1), live.view(-1, 1)
    for x, cache, scales, axes in ((k, st["k_cache"], st["k_scales"], (0, 1, 2, 3)),
                                   (st["v"].float(), st["v_cache"], st["v_scales"], (0, 1, 3, 2))):
        t = x[token.view(-1)].view(n * span, page, *x.shape[1:]).transpose(1, 2)  # [pages, heads, page, dim]
        s_new = _page_scale(torch.where(fresh, t.abs(), torch.zeros_like(t)).amax((2, 3)))
        s_old = scales[ids]
        s = torch.where(older, torch.maximum(s_old, s_new), s_new)
        s = torch.where(live, s, s_old)
        had = _codes(cache, ids).permute(axes).float()
        grown = live & older & (s > s_old)
        ratio = torch.where(grown, s_old / s, torch.ones_like(s))[..., None, None]
        # tokens of a page that are neither new nor older stay as they are
        before = torch.where(pos.view(n * span, 1, page, 1) < start.repeat_interleave(span).view(-1, 1, 1, 1),
                             had * ratio, had)
        val = torch.where(fresh, (t / s[..., None, None]).clamp(-448, 448), before).to(E4M3)
        cache.view(torch.uint8)[ids] = val.permute(axes).contiguous().view(torch.uint8)
        scales[ids] = s
    return q, st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"]


def _padded(st, x, fill):
    """Rows [T, ...] as [seqs, most, ...], and where they come from [T] twice."""
    cu = st["cu"].long()
    row = torch.arange(x.shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], row, right=True)
    at = row - cu[seq]
    out = torch.full((cu.shape[0] - 1, st["max_new"], *x.shape[1:]), fill, dtype=x.dtype, device=x.device)
    out[seq, at] = x
    return out, seq, at


def _plain_mask(st):
    """Ancestors by doubling: after round r a row knows those up to 2^r above it."""
    parents, seq, at = _padded(st, st["parents"].long(), -1)
    most = parents.shape[1]
    parents = torch.where(parents < torch.arange(most, device=parents.device), parents, torch.full_like(parents, -1))
    seen = torch.eye(most + 1, dtype=torch.bool, device=parents.device).repeat(parents.shape[0], 1, 1)
    up = torch.cat([parents, torch.full_like(parents[:, :1], -1)], 1)
    up = torch.where(up < 0, torch.full_like(up, most), up)  # above a root stands node `most`, its own parent
    for _ in range(max(most - 1, 1).bit_length()):
        seen = seen | seen.gather(1, up[..., None].expand_as(seen))
        up = up.gather(1, up)
    seen = seen[:, :most, :most]
    start = (st["lens"] - st["cu"][1:] + st["cu"][:-1]).long()
    return _words(seen)[seq, at], (start[:, None] + seen.sum(-1) - 1)[seq, at].int()


def _plain_attend(st):
    case = st["case"]
    n, heads, group, dim, page = (case[x] for x in ("seqs", "kv_heads", "group", "dim", "page"))
    lens, table, mq = st["lens"].long(), st["table"].long(), st["max_new"]
    dev = lens.device
    k = _codes(st["k_cache"], table).float() * st["k_scales"][table][..., None, None]
    v = _codes(st["v_cache"], table).float() * st["v_scales"][table][..., None, None]
    length = table.shape[1] * page
    k = k.permute(0, 2, 1, 3, 4).reshape(n, heads, length, dim)
    v = v.permute(0, 2, 1, 4, 3).reshape(n, heads, length, dim)
    q, seq, at = _padded(st, st["q"].float(), 0.0)
    q = q.view(n, mq, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(n, heads, mq * group, dim)
    s = (q @ k.transpose(2, 3).contiguous()) * st["scale"]
    tree = _padded(st, st["tree"], 0)[0].long()  # [n, mq, words]
    bits = ((tree[..., None] >> torch.arange(32, device=dev)) & 1).flatten(2)
    pos = torch.arange(length, device=dev)
    start = (st["lens"] - st["cu"][1:] + st["cu"][:-1]).long()
    j = (pos - start[:, None]).clamp(0, bits.shape[2] - 1)  # [n, length]: which new token
    named = bits.gather(2, j[:, None].expand(n, mq, length)).bool() & (pos < lens[:, None])[:, None]
    seen = torch.where((pos < start[:, None])[:, None], torch.ones_like(named), named)
    s = s.masked_fill(~seen.repeat_interleave(group, 1)[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    live = (pos < lens[:, None])[:, None, :, None]
    o = (p @ torch.where(live, v, torch.zeros_like(v))) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(n, heads, mq, group, dim).permute(0, 2, 1, 3, 4).reshape(n, mq, heads * group, dim)
    return o[seq, at].to(st["dt"])


def _plain_verify(st):
    """One pass over the nodes in order: a node is tested where its parent is the last one taken."""
    case = st["case"]
    n, most, vocab = case["seqs"], case["new"], case["vocab"]
    probs = st["probs"].view(n, most, vocab)
    tokens, uniform = st["tokens"].long().view(n, most), st["uniform"].double().view(n, most)
    dev, seq = probs.device, torch.arange(n, device=probs.device)
    if case["draft"]:
        draft = st["draft"].view(n, most, vocab)
        parents = torch.arange(-1, most - 1, device=dev).expand(n, most)
    else:
        parents = st["parents"].long().view(n, most)
    cur = torch.zeros(n, dtype=torch.long, device=dev)
    kept = torch.ones_like(cur)
    path = torch.full((n, most), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0
    gone = torch.zeros((n, most), dtype=torch.bool, device=dev)  # tested and rejected
    rest = torch.ones(n, dtype=torch.float64, device=dev)
    for j in range(1, most):
        child, x = parents[:, j] == cur, tokens[:, j]
        p = probs[seq, cur, x].double()
        if case["draft"]:
            yes = uniform[:, j] * draft[seq, cur, x].double() < p
        else:
            again = (gone[:, :j] & (parents[:, :j] == cur[:, None]) & (tokens[:, :j] == x[:, None])).any(1)
            p = torch.where(again, torch.zeros_like(p), p)
            yes = uniform[:, j] * rest < p
        yes, no = yes & child, child & ~yes
        gone[:, j] = no
        rest = torch.where(yes, torch.ones_like(rest), torch.where(no, rest - p, rest))
        path[seq, torch.where(yes, kept, torch.zeros_like(kept))] = torch.where(yes, torch.full_like(kept, j), path[:, 0])
        kept = kept + yes.long()
        cur = torch.where(yes, torch.full_like(cur, j), cur)
    own_row = probs[seq, cur].double()
    left = gone & (parents == cur[:, None])
    if case["draft"]:
        r = torch.where(left.any(1)[:, None], (own_row - draft[seq, cur].double()).clamp(min=0), own_row)
    else:
        r = own_row.clone()
        at = torch.where(left, tokens, torch.full_like(tokens, vocab))
        r = torch.nn.functional.pad(r, (0, 1)).scatter_(1, at, 0.0)[:, :vocab]
    r = torch.where(r.sum(1, keepdim=True) > 0, r, own_row)
    cum = r.cumsum(1)
    nxt = (cum > uniform[:, :1] * cum[:, -1:]).int().argmax(1)
    return kept.int(), path.int(), nxt.int()


def _plain_keep(st):
    case = st["case"]
    page, n = case["page"], case["seqs"]
    kept, path, table = st["kept"].long(), st["path"].long(), st["table"].long()
    start = (st["lens"] - st["cu"][1:] + st["cu"][:-1]).long()
    dev = start.device
    span = (path.shape[1] + page - 2) // page + 1
    slot = (start // page)[:, None] + torch.arange(span, device=dev)
    pos = slot[..., None] * page + torch.arange(page, device=dev)  # [n, span, page]
    moved = (pos >= start[:, None, None]) & (pos < (start + kept)[:, None, None])
    live = moved.any(-1).view(-1)
    ids = table.gather(1, slot.clamp(max=table.shape[1] - 1)).view(-1)
    ids = torch.where(live, ids, torch.full_like(ids, st["k_cache"].shape[1] - 1))
    node = path.gather(1, (pos - start[:, None, None]).clamp(0, path.shape[1] - 1).view(n, -1)).clamp(min=0)
    src = start[:, None] + node
    src_page = table.gather(1, (src // page).clamp(max=table.shape[1] - 1)).view(-1)
    src_row = (src % page).view(-1)
    moved = moved.view(1, n * span, 1, page, 1)
    for cache, scales, axes in ((st["k_cache"], st["k_scales"], (0, 1, 2, 3, 4)),
                                (st["v_cache"], st["v_scales"], (0, 1, 2, 4, 3))):
        layers, heads = cache.shape[0], cache.shape[2]
        u8 = cache.view(torch.uint8)
        rows = u8.permute(axes)[:, src_page, :, src_row].view(E4M3).float()  # [rows, layers, heads, dim]
        rows = (rows * scales[:, src_page].transpose(0, 1)[..., None]).view(n * span, page, layers, heads, -1)
        rows = rows.permute(2, 0, 3, 1, 4)  # [layers, pages, heads, page, dim], as real values
        s_old = scales[:, ids]
        s = torch.maximum(s_old, _page_scale(torch.where(moved, rows.abs(), torch.zeros_like(rows)).amax((3, 4))))
        s = torch.where(live[:, None], s, s_old)
        had = u8[:, ids].view(E4M3).permute(axes).float() * (s_old / s)[..., None, None]
        val = torch.where(moved, rows / s[..., None, None], had).to(E4M3)
        u8[:, ids] = val.permute(axes).contiguous().view(torch.uint8)
        scales[:, ids] = s
    return st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"]


PLAIN = {"append": _plain_append, "mask": _plain_mask, "attend": _plain_attend, "verify": _plain_verify,
         "keep": _plain_keep}


def _run_own(st):
    import weight_activation_quantized_amd as mq
    case, op = st["case"], st["case"]["op"]
    if op == "mask":
        return mq.kv8_tree_mask(st["parents"], st["cu"], st["lens"], max_q_len=st["max_new"])
    if op == "verify":
        return mq.draft_verify(st["probs"], st["tokens"], st["uniform"], st["cu"], max_q_len=case["new"],
                               parents=st.get("parents"), draft_probs=st.get("draft"))
    cache = st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], st["table"], st["cu"], st["lens"]
    if op == "keep":
        mq.kv8_tree_keep(*cache, st["path"], st["kept"])
        return cache[:4]
    if op == "attend":
        return mq.kv8_tree_attention(st["q"], st["tree"], *cache, max_q_len=st["max_new"], softmax_scale=st["scale"])
    q = mq.kv8_rope_append(st["q"], st["k"], st["v"], *cache, max_q_len=st["max_new"], cos_sin=st["cos_sin"],
                           positions=st["positions"], q_weight=st["qw"], k_weight=st["kw"], eps=EPS,
                           interleaved=case["pairs"] == "next")
    return (q, *cache[:4])


def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    new, total = _lengths(case)
    if op == "mask":
        words = (max(new) + 31) // 32
        return {"bytes": sum(new) * (4 + 4 + 4 * words) + 8 * case["seqs"], "flops": sum(new) * words}
    if op == "verify":
        rows = case["seqs"] * (2 if case["draft"] else 1)
        return {"bytes": 4 * rows * case["vocab"], "flops": 2 * rows * case["vocab"]}
    heads, dim = case["kv_heads"], case["dim"]
    if op == "keep":
        moved = sum(m - 1 for m in _kept(case)) * case["layers"] * heads * dim * 2
        return {"bytes": 2 * moved + 4 * sum(new), "flops": 2 * moved}
    if op == "append":
        values = sum(new) * heads * dim
        return {"bytes": values * (4 * case["group"] + 6) + 4 * max(new) * case["rot"],
                "flops": values * (6 * case["group"] + 10)}
    rows = sum(new) * heads * case["group"]
    pairs = sum(a * (t - a) + a * (a + 1) // 2 for a, t in zip(new, total)) * heads * case["group"]
    return {"bytes": sum(total) * heads * dim * 2 + rows * dim * 4, "flops": 4 * dim * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_turn(x, w, angle, half_pairs, rot):
    x = x.double()
    if w is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
    cs = angle.double()
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None]
    body = x[..., :rot].reshape(*x.shape[:2], *((2, rot // 2) if half_pairs else (rot // 2, 2)))
    axis = -2 if half_pairs else -1
    z = torch.complex(body.select(axis, 0), body.select(axis, 1)) * turn
    return torch.cat([torch.stack([z.real, z.imag], axis).flatten(-2), x[..., rot:]], -1)


def _scale_64(a):
    return torch.exp2(torch.ceil(torch.log2(a.clamp(min=2.0 ** -140) / 448.0)).clamp(-100, 120))


def _exact_append(st):
    """Codes as the values they approximate: new tokens over their page's scale,
    older ones moved to it; everything else as it was."""
    case = st["case"]
    page = case["page"]
    new, total = _lengths(case)
    at = st["positions"]
    if at is None:
        at = torch.cat([torch.arange(t - a, t) for a, t in zip(new, total)])
    angle = st["cos_sin"][at.long().to(st["q"].device)]
    q, k_new = (_exact_turn(x, w, angle, case["pairs"] == "half", case["rot"])
                for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])))
    table, first = st["table"].tolist(), 0
    k, v = st["k_cache"].double(), st["v_cache"].double()
    ks, vs = st["k_scales"].double(), st["v_scales"].double()
    for i, (a, t) in enumerate(zip(new, total)):
        begin = t - a
        for slot in range(begin // page, (t - 1) // page + 1):
            lo, hi, p = max(begin, slot * page), min(t, (slot + 1) * page), table[i][slot]
            rows = slice(first + lo - begin, first + hi - begin)
            inside = slice(lo - slot * page, hi - slot * page)
            for x, c, s in ((k_new, k, ks), (st["v"], v.transpose(2, 3), vs)):
                x = x[rows].double().transpose(0, 1)
                want = _scale_64(x.abs().amax((1, 2)))
                if lo > slot * page:
                    want = torch.maximum(want, s[p])
                    c[p, :, :lo - slot * page] *= (s[p] / want)[:, None, None]
                c[p, :, inside] = x / want[:, None, None]
                s[p] = want
        first += a
    return q, k, v, ks, vs


def _exact_mask(st):
    """Every node's way up, one step at a time."""
    new, total = _lengths(st["case"])
    parents, most = st["parents"].tolist(), st["max_new"]
    words, depth, first = [], [], 0
    for a, t in zip(new, total):
        for j in range(a):
            bits, at, d = 1 << j, parents[first + j], 0
            while at >= 0:
                bits, at, d = bits | 1 << at, parents[first + at], d + 1
            row = [(bits >> 32 * w) & 0xFFFFFFFF for w in range((most + 31) // 32)]
            words.append([x - 2 ** 32 if x >= 2 ** 31 else x for x in row])
            depth.append(t - a + d)
        first += a
    return torch.tensor(words).int(), torch.tensor(depth).int()


def _exact_attend(st):
    case = st["case"]
    heads, group, dim, page = (case[x] for x in ("kv_heads", "group", "dim", "page"))
    new, total = _lengths(case)
    table, at, res = st["table"].long(), 0, []
    words = st["tree"].cpu()
    for i, (a, t) in enumerate(zip(new, total)):
        ids = table[i, :(t + page - 1) // page]
        k = st["k_cache"].view(torch.uint8)[ids].view(E4M3).double() * st["k_scales"][ids].double()[..., None, None]
        v = st["v_cache"].view(torch.uint8)[ids].view(E4M3).double() * st["v_scales"][ids].double()[..., None, None]
        k = k.transpose(0, 1).reshape(heads, -1, dim)[:, :t]
        v = v.transpose(2, 3).transpose(0, 1).reshape(heads, -1, dim)[:, :t]
        q = st["q"][at:at + a].double().view(a, heads, group, dim).permute(1, 2, 0, 3).reshape(heads, group * a, dim)
        s = torch.bmm(q, k.transpose(1, 2).contiguous()) * st["scale"]
        hidden = torch.zeros((a, t), dtype=torch.bool)
        for j in range(a):
            hidden[:, t - a + j] = (words[at:at + a, j // 32] & (1 << j % 32 if j % 32 < 31 else -2 ** 31)) == 0
        s.view(heads, group, a, t).masked_fill_(hidden.to(s.device), -math.inf)
        o = torch.bmm(torch.softmax(s, -1), v.contiguous())
        res.append(o.view(heads, group, a, dim).permute(2, 0, 1, 3).reshape(a, heads * group, dim))
        at += a
    return torch.cat(res)


def _exact_verify(st):
    """Sequence by sequence on the host, with the rest of the row held as a whole."""
    case = st["case"]
    n, most = case["seqs"], case["new"]
    tokens, uniform = st["tokens"].view(n, most).tolist(), st["uniform"].double().view(n, most).tolist()
    parents = st["parents"].view(n, most).tolist() if not case["draft"] else [list(range(-1, most - 1))] * n
    out = [], [], []
    for b in range(n):
        cur, path, j = 0, [0], 1
        rest, lost = st["probs"][b * most].double(), 0.0
        while j < most:
            if parents[b][j] == cur:
                x = tokens[b][j]
                p = rest[x].item()
                if case["draft"]:
                    q = st["draft"][b * most + cur].double()
                    yes = uniform[b][j] * q[x].item() < p
                    left = torch.relu(rest - q)
                else:
                    yes = uniform[b][j] * (1.0 - lost) < p
                    left = rest.clone()
                    left[x] = 0.0
                if yes:
                    cur, lost = j, 0.0
                    path.append(j)
                    rest = st["probs"][b * most + j].double()
                else:
                    rest, lost = left, lost + p
            j += 1
        if not rest.sum().item() > 0:
            rest = st["probs"][b * most + cur].double()
        cum = rest.cumsum(0)
        out[0].append(len(path))
        out[1].append(path + [-1] * (most - len(path)))
        out[2].append(int(torch.searchsorted(cum, cum[-1] * uniform[b][0], right=True)))
    return tuple(torch.tensor(x).int() for x in out)


def _exact_keep(st):
    case = st["case"]
    page = case["page"]
    new, total = _lengths(case)
    table, path, kept = st["table"].tolist(), st["path"].tolist(), _kept(case)
    k, v = st["k_cache"].double(), st["v_cache"].double()
    ks, vs = st["k_scales"].double(), st["v_scales"].double()
    for i, (a, t) in enumerate(zip(new, total)):
        begin = t - a
        for slot in range(begin // page, (begin + kept[i] - 1) // page + 1):
            lo, hi, p = max(begin, slot * page), min(begin + kept[i], (slot + 1) * page), table[i][slot]
            src = [begin + path[i][x - begin] for x in range(lo, hi)]
            for c, s in ((k, ks), (v.transpose(3, 4), vs)):
                x = torch.stack([c[:, table[i][y // page], :, y % page] * s[:, table[i][y // page], :, None]
                                 for y in src], 2)
                want = torch.maximum(s[:, p], _scale_64(x.abs().amax((2, 3))))
                c[:, p] *= (s[:, p] / want)[..., None, None]
                c[:, p, :, lo - slot * page:hi - slot * page] = x / want[..., None, None]
                s[:, p] = want
    return k, v, ks, vs


EXACT = {"append": _exact_append, "mask": _exact_mask, "attend": _exact_attend, "verify": _exact_verify,
         "keep": _exact_keep}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))

"""Operators of speculative decoding over a paged cache: what is measured and how it is computed in plain form.

A step forwards several new rows of each sequence at once: one token, a chain of drafted tokens, or a tree of them whose
node 0 is the last sampled token. Queries and keys are normed and rotated, and keys and values appended behind the
sequence's slots (`paged_append`); the rows attend over the slots and their own ancestors (`attn_paged`); the target's
probabilities then decide with given random numbers which drafts stay and what token comes next (`verify_drafts`), and
the keys and values of the path that stays move to the slots behind the prefix (`paged_keep`).

The cache, as the framework documents it: k and v are [pages, KV heads, page_size, d]; slot s of sequence b is row
s % page_size of page pages[b, s // page_size]; lens[b] slots are filled. Rows are packed: sequence b's are
cu[b] .. cu[b + 1] - 1, `parents` numbers them within their sequence (-1: no parent), a parent before its children.
"""
import math
import random

import torch

own = False

THETA, EPS = 10000.0, 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token each of 64 sequences (the decode batch of the benchmark), with q/k norms: latency alone
        dict(name="append decode 64", op="append", batch=64, nodes=1, heads=32, kv=8, d=128, dims=128, interleaved=False, norm=True,
             dtype="bf16", page=64, longest=500, lens=1),
        # a ragged prefill batch; half of the head turns, neighbouring channels form the pairs
        dict(name="append prompts", op="append", batch=8, nodes=2048, heads=32, kv=8, d=128, dims=64, interleaved=True, norm=False,
             dtype="bf16", page=16, longest=100, lens=2),
        # the fp32 path, 64-channel heads, chunks of an odd number of rows
        dict(name="append fp32", op="append", batch=3, nodes=333, heads=32, kv=8, d=64, dims=64, interleaved=False, norm=True,
             dtype="f32", page=32, longest=1000, lens=3),
        # one conversation, one token: few rows, a long axis
        dict(name="attn one token", op="attn", kind="chain", batch=1, nodes=1, heads=32, kv=8, page=64, longest=4000, window=0, lens=0),
        # the benchmark's decode batch with ragged lengths up to twice its cache
        dict(name="attn 64 tokens ragged", op="attn", kind="chain", batch=64, nodes=1, heads=32, kv=8, page=64, longest=8192, window=0, lens=4),
        # trees of up to 64 drafted tokens, sequences of up to 4096
        dict(name="attn trees", op="attn", kind="tree", batch=16, nodes=64, heads=32, kv=8, page=64, longest=4096, window=0, lens=5),
        # short chains on the sliding-window layers of a small model, small pages
        dict(name="attn chains window", op="attn", kind="chain", batch=32, nodes=5, heads=8, kv=2, page=16, longest=8192, window=2048, lens=6),
        # a chain of four drafts of one conversation, with the draft model's probabilities
        dict(name="verify one", op="verify", kind="chain", batch=1, nodes=5, vocab=32000, draft=True, lens=0),
        # ... of 64 of them
        dict(name="verify chains", op="verify", kind="chain", batch=64, nodes=6, vocab=32000, draft=True, lens=7),
        # trees of candidates that a draft ranks (no probabilities of theirs), a large vocabulary
        dict(name="verify trees", op="verify", kind="tree", batch=16, nodes=64, vocab=131072, draft=False, lens=8),
        # the layers of one conversation's cache after a tree
        dict(name="keep one", op="keep", batch=1, nodes=24, layers=24, kv=8, page=64, longest=300, lens=9),
        # ... of the decode batch, fewer layers
        dict(name="keep 64", op="keep", batch=64, nodes=40, layers=8, kv=8, page=16, longest=200, lens=10),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 32), (32, 8), (8, 2), (20, 4), (16, 1), (4, 4), (12, 2)]


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "verify", "keep"])
    heads, kv = rng.choice(HEADS)
    lens, page = rng.randrange(1, 1 << 30), rng.choice([16, 32, 64, 128])
    kind = rng.choice(["chain", "tree"])
    if op == "append":
        f32 = rng.random() < 0.25
        d = rng.choice([64, 128]) if f32 else 128
        batch = _between(rng, 1, 64)
        return dict(op=op, batch=batch, nodes=_between(rng, 1, max(1, (4096 if f32 else 8192) // batch)), heads=heads, kv=kv, d=d,
                    dims=rng.choice([d, d // 2, d // 4]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.6,
                    dtype="f32" if f32 else "bf16", page=page, longest=_between(rng, 1, 500), lens=lens)
    if op == "attn":
        batch, nodes = _between(rng, 1, 64), _between(rng, 1, 64)
        # at most as many keys to read and as many scores as the largest listed cases have
        top = min(32768, 64 * 8 * 8192 // (batch * max(kv, 2)), (1 << 27) // (batch * heads * nodes))
        return dict(op=op, kind=kind, batch=batch, nodes=nodes, heads=heads, kv=kv, page=page,
                    longest=_between(rng, 1, top), window=rng.choice([0, 0, 0, 100, 1000, 2048]), lens=lens)
    if op == "verify":
        batch, nodes, draft = _between(rng, 1, 64), _between(rng, 1, 64), rng.random() < 0.5
        if kind == "tree" and draft:
            nodes = min(nodes, 16)  # children drawn from one distribution
        return dict(op=op, kind=kind, batch=batch, nodes=nodes, vocab=_between(rng, 1000, min(131072, (1 << 26) // (batch * nodes))),
                    draft=draft, lens=lens)
    return dict(op=op, batch=_between(rng, 1, 64), nodes=rng.randrange(2, 65), layers=rng.choice([1, 2, 4, 8]), kv=kv, page=page,
                longest=_between(rng, 1, 250), lens=lens)


def _lengths(case):
    """Slots filled before the step: all `longest` where lens is 0, else ragged up to it (the first one has it)."""
    n, top = case["batch"], case["longest"]
    if not case["lens"]:
        return [top] * n
    r = random.Random(case["lens"])
    least = max(1, top // 3)
    return [top] + [_between(r, least, top) for _ in range(n - 1)]


def _rows(case):
    """New rows of each sequence: `nodes`, or ragged up to it (the first one has it)."""
    n, top = case["batch"], case["nodes"]
    if not case["lens"]:
        return [top] * n
    r = random.Random(case["lens"] + 1)
    return [top] + [_between(r, max(1, top // (20 if case["op"] == "append" else 2)), top) for _ in range(n - 1)]


def _parents(case):
    """The parent of each node of each sequence's tree, numbered within it: chains, or trees a few levels deep."""
    r = random.Random(case["lens"] + 2)
    if case.get("kind", "tree") == "chain":
        return [[i - 1 for i in range(n)] for n in _rows(case)]
    return [[-1] + [r.randint(max(0, (i - 1) // 4 - 2), (i - 1) // 2) for i in range(1, n)] for n in _rows(case)]


def _paths(case):
    """A path down each sequence's tree that leaves the nodes right behind the root, as paths down wide trees do."""
    r = random.Random(case["lens"] + 3)
    out = []
    for n in _rows(case):
        kept = r.randint(1, max(1, min(8, n // 2)))
        out.append([0] + sorted(r.sample(range(kept, n), kept - 1)))
    return out


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


# ---------------------------------------------------------------- inputs

def _block(case, max_seq, **kw):
    from llama_family_decoder_gb300 import DecoderBlock

    heads, kv = case.get("heads", case.get("kv", 8)), case.get("kv", 8)
    d, dtype = case.get("d", 128), case.get("dtype", "bf16")
    return DecoderBlock(hidden=heads * d, n_heads=heads, n_kv_heads=kv, head_dim=d, ffn=4 * heads * d, act="relu2", dtype=dtype,
                        rope_theta=THETA, eps=EPS, max_batch=case["batch"], max_seq=max_seq, **kw)


def _cu(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _flat(lists):
    return torch.tensor([x for one in lists for x in one], dtype=torch.int32, device="cuda")


def _page_table(case, g):
    """Pages for the filled slots and the new rows of every sequence, in any order; -1 behind a sequence's own."""
    need = [-(-(n + t) // case["page"]) for n, t in zip(_lengths(case), _rows(case))]
    order = torch.randperm(sum(need), generator=g, device="cuda").tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(need) - n))
        at += n
    return torch.tensor(table, dtype=torch.int32, device="cuda"), sum(need)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    op, b = case["op"], case["batch"]
    rows = _rows(case)
    total = sum(rows)
    s = dict(case=case, total=total, cu=_cu(rows))
    if op == "verify":
        v = case["vocab"]
        parents = _parents(case)
        s["parents"] = _flat(parents)
        logits = 3 * torch.randn(total, v, generator=g, device="cuda")
        s["target"] = torch.softmax(logits, -1)
        logits += torch.randn(total, v, generator=g, device="cuda")  # the draft model is a little off
        first = s["cu"][:-1].long().repeat_interleave((s["cu"][1:] - s["cu"][:-1]).long())
        of = (first + s["parents"]).clamp(min=0)  # the parent's row
        if case["draft"]:  # each candidate drawn from its parent's distribution
            s["draft"] = torch.softmax(logits, -1)
            noise = torch.empty(total, v, device="cuda").exponential_(generator=g)
            s["tokens"] = (s["draft"][of] / noise).argmax(-1).to(torch.int32)
        else:  # the first candidates of its parent's, best ones first
            s["draft"] = None
            rank = []
            for tree in parents:
                rank += [sum(1 for p in tree[:i] if p == tree[i]) for i in range(len(tree))]
            best = logits.topk(max(rank) + 1, -1).indices
            s["tokens"] = best[of, torch.tensor(rank, device="cuda")].to(torch.int32)
        s["u"], s["u_next"] = torch.rand(total, generator=g, device="cuda"), torch.rand(b, generator=g, device="cuda")
        s["blk"] = _block(case, 64) if own else None
        return s
    lens = _lengths(case)
    d, kv = case.get("d", 128), case["kv"]
    pages, n_pages = _page_table(case, g)
    shape = (n_pages, kv, case["page"], d)
    if op == "keep":
        paths = _paths(case)
        s["path"] = _flat([p + [-1] * (n - len(p)) for p, n in zip(paths, rows)])
        s["counts"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        s["starts"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["lens"] = s["starts"].clone()
        s["caches"] = [dict(k=normal(*shape), v=normal(*shape), pages=pages, lens=s["lens"]) for _ in range(case["layers"])]
        s["blk"] = _block(case, 64) if own else None
        return s
    cache = dict(pages=pages, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    s["cache"] = cache
    if op == "append":
        h = case["heads"]
        fused = normal(total, h + 2 * kv, d)  # q, k and v are columns of one projection's rows
        s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + kv], fused[:, h + kv:]
        s["gq"], s["gk"] = (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt), (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt)
        cache["k"], cache["v"] = torch.zeros(*shape, dtype=dt, device="cuda"), torch.zeros(*shape, dtype=dt, device="cuda")
        s["blk"] = _block(case, max(lens) + case["nodes"], qk_norm=case["norm"]) if own else None
        s["table"] = s["blk"].rope_table(case["dims"]) if own and case["dims"] < d else None
        return s
    s["parents"] = _flat(_parents(case)) if case["kind"] == "tree" else None
    s["q"] = normal(total, case["heads"], 128)
    big = 1 + 4 * (torch.rand(kv, 1, 128, generator=g, device="cuda") < 0.04)  # keys have a few large channels, as rotated keys do
    cache["k"], cache["v"] = (torch.randn(*shape, generator=g, device="cuda") * big).bfloat16(), normal(*shape)
    s["blk"] = _block(case, 64, sliding_window=case["window"]) if own else None
    return s


# ---------------------------------------------------------------- plain forms

def _places(cu, total):
    """Each packed row's sequence, and its number within it."""
    r = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous().long(), r, right=True)
    return seq, r - cu.long()[seq]


def _slot_rows(pages, page, seq, slot):
    """Page and row within it of slots."""
    return pages.long()[seq, slot // page], slot % page


def _turn(x, cos, sin, dims, interleaved):
    y = x[..., :dims]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :dims // 2], y[..., dims // 2:])
    turned = [a * cos - b * sin, b * cos + a * sin]
    y = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat([y, x[..., dims:]], -1)


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    dims = case["dims"]
    seq, i = _places(s["cu"], s["total"])
    slot = cache["lens"].long()[seq] + i
    # far positions times frequencies lose their turns in 32 bits: angles in 64
    pair = torch.arange(dims // 2, device="cuda", dtype=torch.float64)
    angle = slot.double()[:, None] * THETA ** (-2.0 * pair / dims)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, gain in ((s["q"], s["gq"]), (s["k"], s["gk"])):
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gain.float()
        out.append(_turn(y, cos, sin, dims, case["interleaved"]).to(x.dtype))
    page, row = _slot_rows(cache["pages"], case["page"], seq, slot)
    cache["k"][page, :, row] = out[1]
    cache["v"][page, :, row] = s["v"]
    return out[0], cache["k"], cache["v"]


def _seen(s):
    """[B, nodes, slots]: which slots each node attends to, with what lies behind a sequence's rows hidden."""
    case, cu = s["case"], s["cu"].long()
    b, t = case["batch"], case["nodes"]
    i = torch.arange(t, device="cuda")
    count = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=s["total"] - 1)
    parent = s["parents"].long()[at] if s["parents"] is not None else (i - 1).expand(b, t)
    kin = torch.eye(t, dtype=torch.bool, device="cuda").repeat(b, 1, 1)  # ancestors and the node itself
    depth = torch.zeros(b, t, dtype=torch.long, device="cuda")
    every = torch.arange(b, device="cuda")
    for n in range(1, t):
        p = parent[:, n].clamp(min=0)
        has = parent[:, n] >= 0
        kin[:, n] |= kin[every, p] & has[:, None]
        depth[:, n] = torch.where(has, depth[every, p] + 1, 0)
    slots = torch.arange(s["cache"]["pages"].shape[1] * case["page"], device="cuda")
    lens = s["cache"]["lens"].long()
    new = slots[None] - lens[:, None]  # a slot's node
    node = new.clamp(0, t - 1)
    own_rows = torch.gather(kin, 2, node[:, None].expand(-1, t, -1)) & ((new >= 0) & (new < count[:, None]))[:, None]
    seen = own_rows | (new < 0)[:, None]
    if case["window"]:
        where = torch.where(new < 0, slots[None], lens[:, None] + torch.gather(depth, 1, node))
        seen = seen & (where[:, None] > (lens[:, None] + depth)[..., None] - case["window"])
    return seen, at, count


def _plain_attn(s):
    case, cache = s["case"], s["cache"]
    b, t, h, kv = case["batch"], case["nodes"], case["heads"], case["kv"]
    seen, at, count = _seen(s)
    pages = cache["pages"].long().clamp(min=0)
    k, v = (cache[x][pages].float().transpose(1, 2).flatten(2, 3) for x in "kv")  # [B, kv, slots, 128]
    q = s["q"].float()[at].unflatten(2, (kv, h // kv)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, kv, G * nodes, 128]
    score = torch.where(seen.repeat(1, h // kv, 1)[:, None], q @ k.transpose(-1, -2) * 128**-0.5, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e38)
    p = torch.exp(score - top)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = o.reshape(b, h, t, 128).transpose(1, 2)
    seq, i = _places(s["cu"], s["total"])
    return o[seq, i].bfloat16()


def _plain_verify(s):
    """All sequences node by node: a node whose parent is the current one is a candidate."""
    case, cu = s["case"], s["cu"].long()
    b, t = case["batch"], case["nodes"]
    count = cu[1:] - cu[:-1]
    first = cu[:-1]
    every = torch.arange(b, device="cuda")
    cur = torch.zeros(b, dtype=torch.long, device="cuda")
    kept = torch.ones(b, dtype=torch.long, device="cuda")
    path = torch.full((b, t), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    # what is left of the target's distribution and its sum, in 64 bits: the answers are whole numbers
    left, scale = s["target"][first].double(), torch.ones(b, dtype=torch.float64, device="cuda")
    for n in range(1, t):
        row = (first + n).clamp(max=s["total"] - 1)
        tried = (s["parents"].long()[row] == cur) & (n < count)
        x = s["tokens"].long()[row]
        here = left[every, x]
        if s["draft"] is not None:
            q = s["draft"][first + cur].double()
            taken = tried & (s["u"].double()[row] * scale * q[every, x] < here)
            rest = (left - scale[:, None] * q).clamp(min=0)
            rest_scale = rest.sum(-1)
        else:
            taken = tried & (s["u"].double()[row] * scale < here) & (here > 0)
            rest = left.clone()
            rest[every, x] = 0
            rest_scale = scale - here
        fresh = s["target"][row].double()
        left = torch.where(taken[:, None], fresh, torch.where(tried[:, None], rest, left))
        scale = torch.where(taken, 1.0, torch.where(tried, rest_scale, scale))
        cur = torch.where(taken, n, cur)
        path.scatter_(1, kept.clamp(max=t - 1)[:, None], torch.where(taken, n, path.gather(1, kept.clamp(max=t - 1)[:, None])[:, 0])[:, None])
        kept = kept + taken
    nothing = left.sum(-1) <= 0
    left = torch.where(nothing[:, None], s["target"][first + cur].double(), left)
    upto = left.cumsum(-1)
    token = (upto <= s["u_next"].double()[:, None] * upto[:, -1:]).sum(-1).clamp(max=case["vocab"] - 1)
    seq, i = _places(s["cu"], s["total"])
    return kept.to(torch.int32), path[seq, i].to(torch.int32), token.to(torch.int32)


def _plain_keep(s):
    case = s["case"]
    seq, i = _places(s["cu"], s["total"])
    moved = (s["path"] >= 0) & (s["path"] != i)
    start = s["starts"].long()[seq]
    pages = s["caches"][0]["pages"]
    page_to, row_to = _slot_rows(pages, case["page"], seq, start + i)
    page_from, row_from = _slot_rows(pages, case["page"], seq, start + s["path"].long().clamp(min=0))
    page_from, row_from = torch.where(moved, page_from, page_to), torch.where(moved, row_from, row_to)
    out = []
    for c in s["caches"]:
        for x in "kv":
            c[x][page_to, :, row_to] = c[x][page_from, :, row_from]
            out.append(c[x])
    s["lens"].copy_(s["starts"] + s["counts"])
    return out, s["lens"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"append": _plain_append, "attn": _plain_attn, "verify": _plain_verify, "keep": _plain_keep}[op](state)
    blk = state["blk"]
    if op == "append":
        c = state["cache"]
        q = blk.paged_append(c, state["q"], state["k"], state["v"], state["cu"], q_gain=state["gq"], k_gain=state["gk"],
                             rope_table=state["table"], interleaved=state["case"]["interleaved"])
        return q, c["k"], c["v"]
    if op == "attn":
        return blk.attn_paged(state["q"], state["cache"], state["cu"], parents=state["parents"])
    if op == "verify":
        return blk.verify_drafts(state["target"], state["tokens"], state["u"], state["u_next"], state["cu"], parents=state["parents"],
                                 draft=state["draft"])
    blk.paged_keep(state["caches"], state["counts"], state["path"], state["cu"], starts=state["starts"])
    return [c[x] for c in state["caches"] for x in "kv"], state["lens"]


# ---------------------------------------------------------------- work

def work(case):
    rows = _rows(case)
    total, b = sum(rows), case["batch"]
    if case["op"] == "append":
        e, d, h, kv = 4 if case["dtype"] == "f32" else 2, case["d"], case["heads"], case["kv"]
        return {"bytes": 2 * total * (h + 2 * kv) * d * e + 2 * d * e, "flops": total * (h + kv) * (4 * d * case["norm"] + 3 * case["dims"])}
    if case["op"] == "attn":
        keys = scores = 0
        for n, tree in zip(_lengths(case), _parents(case)):
            w = case["window"] or n + len(tree)
            depth = _depths(tree)
            # the prefix's slots that any node sees, and the rows themselves
            keys += min(n, max(0, w - 1 - min(depth))) + len(tree)
            scores += sum(min(n, max(0, w - 1 - x)) + min(x + 1, w) for x in depth)
        return {"bytes": 2 * keys * case["kv"] * 256 + 2 * total * case["heads"] * 256, "flops": 512 * case["heads"] * scores}
    if case["op"] == "verify":  # the row that each walk stops at, and the numbers that decide it
        each = 2 if case["draft"] else 1
        return {"bytes": b * case["vocab"] * 4 * each + total * (12 + 4 * each) + b * 8, "flops": b * case["vocab"] * 2 * each}
    moved = sum(sum(1 for j, n in enumerate(p) if n != j) for p in _paths(case))
    return {"bytes": 2 * moved * case["layers"] * 2 * case["kv"] * 256 + total * 4, "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](case, s)


def _exact_append(case, s):
    dims, half = case["dims"], case["dims"] // 2
    cu, lens, table = s["cu"].tolist(), s["cache"]["lens"].tolist(), s["cache"]["pages"].tolist()
    q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    k_out, v_out = (s["cache"][x].double() for x in "kv")
    freq = torch.tensor([THETA ** (-2.0 * i / dims) for i in range(half)], dtype=torch.float64, device="cuda")
    low = list(range(0, dims, 2)) if case["interleaved"] else list(range(half))
    high = [c + 1 for c in low] if case["interleaved"] else [c + half for c in low]
    for b in range(case["batch"]):
        rows = slice(cu[b], cu[b + 1])
        pos = torch.arange(lens[b], lens[b] + cu[b + 1] - cu[b], device="cuda")
        turn = torch.polar(torch.ones(len(pos), half, dtype=torch.float64, device="cuda"), pos.double()[:, None] * freq)[:, None]
        got = []
        for x, gain in ((s["q"][rows], s["gq"]), (s["k"][rows], s["gk"])):
            y = x.double()
            if case["norm"]:
                y = y / (y.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * gain.double()
            z = torch.complex(y[..., low], y[..., high]) * turn
            y = y.clone()
            y[..., low], y[..., high] = z.real, z.imag
            got.append(y)
        q_out[rows] = got[0]
        for lo in range(0, len(pos)):  # page by page
            slot = lens[b] + lo
            if lo and slot % case["page"]:
                continue
            n = min(case["page"] - slot % case["page"], len(pos) - lo)
            page, row = table[b][slot // case["page"]], slot % case["page"]
            k_out[page, :, row:row + n] = got[1][lo:lo + n].transpose(0, 1)
            v_out[page, :, row:row + n] = s["v"][rows][lo:lo + n].double().transpose(0, 1)
    return q_out, k_out, v_out


def _exact_attn(case, s):
    out = torch.zeros(s["total"], case["heads"], 128, dtype=torch.float64, device="cuda")
    cu, lens, table = s["cu"].tolist(), s["cache"]["lens"].tolist(), s["cache"]["pages"].tolist()
    per = case["heads"] // case["kv"]
    for b, tree in enumerate(_parents(case)):
        n, t = lens[b], len(tree)
        depth = _depths(tree)
        pages = table[b][:-(-(n + t) // case["page"])]
        k, v = (torch.cat([s["cache"][x][p] for p in pages], 1)[:, :n + t].double() for x in "kv")
        seen = torch.zeros(t, n + t, dtype=torch.bool)
        for i in range(t):
            seen[i, :n] = True
            j = i
            while j >= 0:
                seen[i, n + j] = True
                j = tree[j]
            if case["window"]:
                place = torch.tensor(list(range(n)) + [n + x for x in depth])
                seen[i] &= n + depth[i] - place < case["window"]
        seen = seen.cuda()
        for j in range(case["kv"]):
            q = s["q"][cu[b]:cu[b + 1], j * per:(j + 1) * per].double()
            score = torch.einsum("tgd,nd->tgn", q, k[j]) / math.sqrt(128)
            weight = torch.softmax(score.masked_fill(~seen[:, None], -math.inf), -1)
            out[cu[b]:cu[b + 1], j * per:(j + 1) * per] = torch.einsum("tgn,nd->tgd", weight, v[j])
    return out


def _exact_verify(case, s):
    """One sequence after the other, down its tree."""
    cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
    u, u_next = s["u"].double().tolist(), s["u_next"].double().tolist()
    counts, path, token = [], [], []
    for b, tree in enumerate(_parents(case)):
        cur, walk = 0, [0]
        while True:
            p = s["target"][cu[b] + cur].double().cpu()
            q = s["draft"][cu[b] + cur].double().cpu() if s["draft"] is not None else None
            left, total, after = p.clone(), 1.0, None
            for child in [i for i in range(len(tree)) if tree[i] == cur]:
                x = tokens[cu[b] + child]
                of = 1.0 if q is None else float(q[x])
                if left[x] > 0 and u[cu[b] + child] * total * of < float(left[x]):
                    after = child
                    break
                if q is None:
                    total -= float(left[x])
                    left[x] = 0.0
                else:
                    left = torch.clamp(left - total * q, min=0.0)
                    total = float(left.sum())
            if after is None:
                break
            walk.append(after)
            cur = after
        if float(left.sum()) <= 0:
            left = p
        upto = torch.cumsum(left, 0)
        token.append(min(int(torch.searchsorted(upto, u_next[b] * float(upto[-1]), right=True)), case["vocab"] - 1))
        counts.append(len(walk))
        path += walk + [-1] * (len(tree) - len(walk))
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (counts, path, token))


def _exact_keep(case, s):
    cu, path, starts, table = s["cu"].tolist(), s["path"].tolist(), s["starts"].tolist(), s["caches"][0]["pages"].tolist()
    out = []
    for c in s["caches"]:
        for x in "kv":
            was, now = c[x], c[x].clone()
            for b, n in enumerate(s["counts"].tolist()):
                for j in range(n):
                    to, of = starts[b] + j, starts[b] + path[cu[b] + j]
                    now[table[b][to // case["page"]], :, to % case["page"]] = was[table[b][of // case["page"]], :, of % case["page"]]
            out.append(now.double())
    return out, s["starts"] + s["counts"]

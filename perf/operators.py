"""Operators of a packed, mixed-length serving path: what is measured and how it is computed in plain form.

A batch of prompts of different lengths is packed into one run of token rows (`cu_seqlens`). Its queries and keys are
normed per head and rotated (`qk_norm_rope`), attend causally within their own sequence (`attn_packed`), its keys and
values go into a cache held in 4 bits (`kv4_store`), and later single tokens attend over that cache (`attn_decode_kv4`).

The 4-bit cache, as the framework documents it: a row is one key or value of one head, 128 channels in four groups of
32. A group with least value `lo` and greatest `hi` keeps the bf16 numbers scale = (hi - lo) / 15 and offset = lo and
the codes clamp(rint((x - offset) / scale), 0, 15); a code stands for offset + scale * code. A row's 64 code bytes:
byte 16 t + 4 j + 2 u + e holds channel 16 (2 j + e) + 2 t + u in its low and the channel 8 further in its high nibble;
its 8 bf16 numbers are the four scales, then the four offsets.
"""
import math
import random

import torch

own = False

D = 128  # channels of a head in the bf16 cases
GROUP = 32
THETA, EPS = 10000.0, 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token each of 64 sequences (the decode batch of the benchmark), norms and plain rotary: latency alone
        dict(name="rope decode 64", op="rope", tokens=64, heads=32, kv=8, d=128, dtype="bf16", axes=1, mix=False, norm=True, layout="rows"),
        # a packed prompt with image patches: three position axes in sections, an odd number of rows
        dict(name="rope prompt 3 axes", op="rope", tokens=8191, heads=32, kv=8, d=128, dtype="bf16", axes=3, mix=False, norm=True, layout="rows"),
        # head-major projections without norms, interleaved axes, more rows
        dict(name="rope heads interleaved", op="rope", tokens=16384, heads=32, kv=32, d=128, dtype="bf16", axes=3, mix=True, norm=False, layout="heads"),
        # the fp32 path, 64-channel heads
        dict(name="rope fp32", op="rope", tokens=2000, heads=32, kv=8, d=64, dtype="f32", axes=1, mix=False, norm=True, layout="rows"),
        # many short chat turns at once
        dict(name="attn short turns", op="attn", batch=48, longest=200, heads=32, kv=8, window=0, lens=1),
        # a ragged prefill batch
        dict(name="attn ragged", op="attn", batch=8, longest=2048, heads=32, kv=8, window=0, lens=2),
        # one long document, every query head with its own key head
        dict(name="attn long", op="attn", batch=1, longest=8190, heads=32, kv=32, window=0, lens=3),
        # sliding-window layers of a small model
        dict(name="attn window", op="attn", batch=6, longest=4096, heads=8, kv=2, window=2048, lens=4),
        # the step's new keys and values of 64 sequences
        dict(name="store decode 64", op="store", batch=64, longest=1, kv=8, lens=0),
        # the keys and values of a ragged prefill batch
        dict(name="store prompts", op="store", batch=8, longest=2048, kv=8, lens=5),
        # one conversation: few rows, a long axis
        dict(name="decode one", op="decode", batch=1, longest=4000, heads=32, kv=8, window=0, lens=0),
        # the benchmark's decode batch with ragged lengths up to twice its cache
        dict(name="decode 64 ragged", op="decode", batch=64, longest=8192, heads=32, kv=8, window=0, lens=6),
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 32), (32, 8), (8, 2), (20, 4), (16, 1), (4, 4), (12, 2)]


def draw(rng):
    op = rng.choice(["rope", "attn", "store", "decode"])
    heads, kv = rng.choice(HEADS)
    lens = rng.randrange(1, 1 << 30)
    if op == "rope":
        f32 = rng.random() < 0.25
        return dict(op=op, tokens=_between(rng, 1, 16384 if not f32 else 8192), heads=heads, kv=kv, d=rng.choice([64, 128]) if f32 else 128,
                    dtype="f32" if f32 else "bf16", axes=rng.choice([1, 2, 3]), mix=rng.random() < 0.5, norm=rng.random() < 0.7,
                    layout=rng.choice(["rows", "heads"]))
    if op == "attn":
        batch = _between(rng, 1, 64)
        # the plain form pads to the longest sequence: batch * heads * longest^2 scores at most 2^31
        top = int(min(8192, math.sqrt(2.0**31 / (batch * heads)), 65536 / batch))
        return dict(op=op, batch=batch, longest=_between(rng, 1, top), heads=heads, kv=kv, window=rng.choice([0, 0, 64, 500, 2048]), lens=lens)
    if op == "store":
        batch = _between(rng, 1, 128)
        return dict(op=op, batch=batch, longest=_between(rng, 1, max(1, min(8192, 24000 // batch))), kv=kv, lens=lens)
    batch = _between(rng, 1, 128)
    top = min(65536, 64 * 8 * 8192 // (batch * max(kv, 2)))
    return dict(op=op, batch=batch, longest=_between(rng, 16, top), heads=heads, kv=kv, window=rng.choice([0, 0, 0, 1000, 2048]), lens=lens)


def _lengths(case):
    """The sequences' lengths: all `longest` where lens is 0, else ragged up to it (the first one has it)."""
    n, top = case["batch"], case["longest"]
    if not case["lens"]:
        return [top] * n
    r = random.Random(case["lens"])
    least = max(1, top // (3 if case["op"] == "decode" else 20))
    return [top] + [_between(r, least, top) for _ in range(n - 1)]


def _sections(case):
    """Rotary pairs of each position axis; time keeps the smaller share, as in image and video models."""
    half = case["d"] // 2
    if case["axes"] == 1:
        return [half]
    if case["axes"] == 2:
        return [half // 2, half - half // 2]
    side = 3 * half // 8 if not case["mix"] else half // 3
    return [half - 2 * side, side, side]


# ---------------------------------------------------------------- inputs

def _block(case, max_seq, **kw):
    from llama_family_decoder_gb300 import DecoderBlock

    heads = case.get("heads", case["kv"])
    d, dtype = case.get("d", D), case.get("dtype", "bf16")
    return DecoderBlock(hidden=heads * d, n_heads=heads, n_kv_heads=case["kv"], head_dim=d, ffn=4 * heads * d, act="relu2", dtype=dtype,
                        rope_theta=THETA, eps=EPS, max_batch=max(1, case.get("batch", 1)), max_seq=max_seq, **kw)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    s = dict(case=case)
    if case["op"] == "rope":
        n, h, kv, d = case["tokens"], case["heads"], case["kv"], case["d"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        if case["layout"] == "rows":  # q and k are columns of one projection's rows
            fused = normal(n, h + 2 * kv, d, dtype=dt)
            s["q"], s["k"] = fused[:, :h], fused[:, h:h + kv]
        else:  # head-major projections
            s["q"], s["k"] = normal(h, n, d, dtype=dt).transpose(0, 1), normal(kv, n, d, dtype=dt).transpose(0, 1)
        s["gq"], s["gk"] = (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt), (1 + 0.1 * normal(d, dtype=torch.float32)).to(dt)
        if n <= 256:  # single tokens of sequences at positions of their own
            pos = torch.randint(0, 8192, (case["axes"], n), generator=g, device="cuda")
        else:  # text positions, or patches of 32 x 32 in time order
            r = torch.arange(n, device="cuda")
            pos = torch.stack([r, r, r] if case["axes"] == 1 else [r // 1024, r // 32 % 32, r % 32])[:case["axes"]]
            pos = pos + torch.randint(0, 64, (1, 1), generator=g, device="cuda")
        s["pos"] = pos.to(torch.int32).contiguous()
        s["sections"] = _sections(case)
        s["blk"] = _block(case, 16384 + 64, qk_norm=case["norm"]) if own else None
        return s
    lens = _lengths(case)
    s["lens"], s["total"] = lens, sum(lens)
    if case["op"] in ("attn", "store"):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "attn":
        # heads as rows of a normed and rotated projection: about N(0, 1) per channel
        s["q"], s["k"], s["v"] = (normal(s["total"], n, D) for n in (case["heads"], case["kv"], case["kv"]))
        s["blk"] = _block(case, 64, sliding_window=case["window"]) if own else None
        return s
    # keys have a few large channels, as rotated keys do
    big = 1 + 4 * (torch.rand(case["kv"], D, generator=g, device="cuda") < 0.04)
    if case["op"] == "store":
        s["k"], s["v"] = (normal(s["total"], case["kv"], D, dtype=torch.float32) * big).bfloat16(), normal(s["total"], case["kv"], D)
        s["starts"] = torch.randint(0, 100, (case["batch"],), generator=g, device="cuda").to(torch.int32)
        s["blk"] = _block(case, 64) if own else None
        s["cache"] = s["blk"].kv4_cache(case["batch"], case["longest"] + 100) if own else None
        return s
    shape = (case["batch"], case["kv"], case["longest"])
    s["q"] = normal(case["batch"], case["heads"], D)
    s["cache"] = {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for name, by in (("k", big[:, None]), ("v", 1.0)):
        codes, scale, offset = _quantise(torch.randn(*shape, D, generator=g, device="cuda") * by)
        s["cache"][name], s["cache"][name + "_scale"] = _pack(codes), torch.cat([scale, offset], -1).bfloat16()
    s["blk"] = _block(case, 64, sliding_window=case["window"]) if own else None
    return s


# ---------------------------------------------------------------- plain forms

def _byte_channels(device):
    """The channel in the low nibble of each of a row's 64 code bytes."""
    p = torch.arange(64, device=device)
    t, j, u, e = p // 16, p // 4 % 4, p // 2 % 2, p % 2
    return 16 * (2 * j + e) + 2 * t + u


def _quantise(x):
    """Codes [..., 128] and the bf16 scale and offset [..., 4], as fp32, of rows x [..., 128]."""
    g = x.unflatten(-1, (D // GROUP, GROUP)).float()
    lo, hi = g.amin(-1), g.amax(-1)
    scale, offset = ((hi - lo) / 15).bfloat16().float(), lo.bfloat16().float()
    code = torch.where(scale[..., None] > 0, (g - offset[..., None]) / scale[..., None], 0.0).round().clamp(0, 15)
    return code.flatten(-2), scale, offset


def _pack(codes):
    low = _byte_channels(codes.device)
    c = codes.to(torch.uint8)
    return c[..., low] | (c[..., low + 8] << 4)


def _values(packed, scales):
    """The fp32 values [..., 128] that a cache's code bytes and scales stand for."""
    low = _byte_channels(packed.device)
    order = torch.argsort(torch.cat([low, low + 8]))
    codes = torch.cat([packed & 15, packed >> 4], -1)[..., order].float().unflatten(-1, (D // GROUP, GROUP))
    scales = scales.float()
    return (scales[..., 4:, None] + scales[..., :4, None] * codes).flatten(-2)


def _axis_of_pair(case, device):
    """Which position axis turns each rotary pair: sections one after the other, or dealt out in turn."""
    sec, i = _sections(case), torch.arange(case["d"] // 2, device=device)
    if not case["mix"]:
        return torch.searchsorted(torch.tensor(sec, device=device).cumsum(0), i, right=True)
    n = len(sec)
    a = i % n
    return torch.where(i < n * torch.tensor(sec, device=device)[a], a, 0)


def _plain_rope(s):
    case = s["case"]
    half = case["d"] // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    # far positions times frequencies lose their turns in 32 bits: angles in 64
    angle = s["pos"][_axis_of_pair(case, "cuda")].T.double() * THETA ** (-2.0 * i / case["d"])
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, gain in ((s["q"], s["gq"]), (s["k"], s["gk"])):
        y = x.float()
        if case["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * gain.float()
        a, b = y[..., :half], y[..., half:]
        out.append(torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype))
    return out


def _masked_attention(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v over the keys that `seen` shows; zero where it shows none. q [B, Hkv, G * Tq, d]."""
    score = torch.where(seen, q @ k.transpose(-1, -2) * D**-0.5, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e38)
    p = torch.exp(score - top)
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_attn(s):
    case = s["case"]
    b, n, h, kv = case["batch"], case["longest"], case["heads"], case["kv"]
    cu = s["cu"].long()
    i = torch.arange(n, device="cuda")
    rows = (cu[:-1, None] + i).clamp(max=s["total"] - 1)  # padded to the longest sequence
    length = cu[1:] - cu[:-1]
    seen = (i[None, :] <= i[:, None]) & (i[None, :] < length[:, None, None])
    if case["window"]:
        seen = seen & (i[None, :] > i[:, None] - case["window"])
    q = s["q"].float()[rows].unflatten(2, (kv, h // kv)).permute(0, 2, 3, 1, 4).reshape(b, kv, h // kv * n, D)
    k, v = (s[x].float()[rows].transpose(1, 2) for x in "kv")
    o = _masked_attention(q, k, v, seen[:, None, None].expand(b, 1, h // kv, n, n).reshape(b, 1, h // kv * n, n))
    o = o.reshape(b, h, n, D)
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), length, output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - cu[seq]
    return o[seq, :, at].bfloat16()


def _plain_store(s):
    cu = s["cu"]
    out = []
    for x in (s["k"], s["v"]):
        codes, scale, offset = _quantise(x)
        out.append((offset[..., None] + scale[..., None] * codes.unflatten(-1, (D // GROUP, GROUP))).flatten(-2).bfloat16())
    return out[0], out[1], s["starts"] + (cu[1:] - cu[:-1])


def _plain_decode(s):
    case, c = s["case"], s["cache"]
    b, h, kv = case["batch"], case["heads"], case["kv"]
    i = torch.arange(case["longest"], device="cuda")
    length = c["lens"].long()[:, None, None, None]
    seen = i < length
    if case["window"]:
        seen = seen & (i >= length - case["window"])
    k, v = _values(c["k"], c["k_scale"]), _values(c["v"], c["v_scale"])
    return _masked_attention(s["q"].float().reshape(b, kv, h // kv, D), k, v, seen).reshape(b, h, D).bfloat16()


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "attn": _plain_attn, "store": _plain_store, "decode": _plain_decode}[op](state)
    blk = state["blk"]
    if op == "rope":
        return list(blk.qk_norm_rope(state["q"], state["k"], state["pos"], state["gq"], state["gk"], sections=state["sections"],
                                     interleaved=state["case"]["mix"]))
    if op == "attn":
        return blk.attn_packed(state["q"], state["k"], state["v"], state["cu"])
    if op == "store":
        blk.kv4_store(state["cache"], state["k"], state["v"], state["cu"], starts=state["starts"])
        k, v = blk.kv4_load(state["cache"], state["cu"], state["total"], starts=state["starts"])
        return k, v, state["cache"]["lens"]
    return blk.attn_decode_kv4(state["q"], state["cache"])


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "rope":
        n, d, e = case["tokens"], case["d"], 4 if case["dtype"] == "f32" else 2
        values = n * (case["heads"] + case["kv"]) * d
        return {"bytes": 2 * values * e + n * case["axes"] * 4 + 2 * d * e, "flops": values * (3 + 4 * case["norm"])}
    lens = _lengths(case)
    if case["op"] == "attn":
        w = case["window"]
        pairs = sum(n * (n + 1) // 2 if not w or n <= w else w * (w + 1) // 2 + (n - w) * w for n in lens)
        return {"bytes": sum(lens) * (2 * case["heads"] + 2 * case["kv"]) * D * 2, "flops": 4 * D * case["heads"] * pairs}
    row = 64 + 16  # codes and scales of one key or value
    if case["op"] == "store":  # stored, and read back as the values they stand for
        rows = 2 * sum(lens) * case["kv"]
        return {"bytes": rows * (2 * D * 2 + 2 * row), "flops": rows * D * 6}
    keys = sum(min(n, case["window"] or n) for n in lens)
    return {"bytes": 2 * keys * case["kv"] * row + 2 * case["batch"] * case["heads"] * D * 2, "flops": 4 * D * case["heads"] * keys}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_exact_rope(case, s, *x) for x in ((s["q"], s["gq"]), (s["k"], s["gk"]))]
    if case["op"] == "attn":
        out, at = torch.zeros(s["total"], case["heads"], D, dtype=torch.float64, device="cuda"), 0
        for n in s["lens"]:
            rows = slice(at, at + n)
            keys = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
            if case["window"]:
                keys = keys & ~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(-case["window"])
            for h in range(case["heads"]):
                j = h // (case["heads"] // case["kv"])
                score = (s["q"][rows, h].double() @ s["k"][rows, j].double().T) / math.sqrt(D)
                out[rows, h] = torch.softmax(score.masked_fill(~keys, -math.inf), -1) @ s["v"][rows, j].double()
            at += n
        return out
    if case["op"] == "store":
        return _exact_stored(s["k"]), _exact_stored(s["v"]), None
    out = torch.zeros(case["batch"], case["heads"], D, dtype=torch.float64, device="cuda")
    c, per = s["cache"], case["heads"] // case["kv"]
    for b, n in enumerate(s["lens"]):
        first = max(0, n - case["window"]) if case["window"] else 0
        k, v = (_exact_values(c[x][b, :, first:n], c[x + "_scale"][b, :, first:n]) for x in "kv")
        score = torch.einsum("jgd,jnd->jgn", s["q"][b].double().reshape(case["kv"], per, D), k) / math.sqrt(D)
        out[b] = torch.einsum("jgn,jnd->jgd", torch.softmax(score, -1), v).reshape(case["heads"], D)
    return out


def _exact_rope(case, s, x, gain):
    """Each pair as a complex number, turned by its axis's position times its frequency."""
    half, sec = case["d"] // 2, _sections(case)
    axis = [0] * half
    if case["mix"]:
        for a in range(1, len(sec)):
            for i in range(a, min(half, len(sec) * sec[a]), len(sec)):
                axis[i] = a
    else:
        axis = [a for a, n in enumerate(sec) for _ in range(n)]
    y = x.double()
    if case["norm"]:
        y = y / (y.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt() * gain.double()
    freq = torch.tensor([THETA ** (-2.0 * i / case["d"]) for i in range(half)], dtype=torch.float64, device="cuda")
    angle = torch.stack([s["pos"][a].double() for a in axis], 1) * freq
    z = torch.complex(y[..., :half], y[..., half:]) * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.cat([z.real, z.imag], -1)


def _exact_stored(x):
    """What 16 evenly spaced steps from a group's least to its greatest value keep of it, steps and least value in bf16."""
    g = x.double().reshape(*x.shape[:-1], D // GROUP, GROUP)
    least = g.min(-1, keepdim=True).values
    step = ((g.max(-1, keepdim=True).values - least) / 15).bfloat16().double()
    least = least.bfloat16().double()
    n = torch.clamp(torch.round((g - least) / torch.where(step > 0, step, 1.0)), 0, 15)
    return (least + step * n).reshape(x.shape)


def _exact_values(packed, scales):
    out = torch.zeros(*packed.shape[:-1], D, dtype=torch.float64, device=packed.device)
    for p in range(64):
        t, j, u, e = p // 16, p // 4 % 4, p // 2 % 2, p % 2
        c = 16 * (2 * j + e) + 2 * t + u
        for channel, code in ((c, packed[..., p] % 16), (c + 8, packed[..., p] // 16)):
            out[..., channel] = scales[..., 4 + channel // 32].double() + scales[..., channel // 32].double() * code.double()
    return out

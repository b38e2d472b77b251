"""Speculative decoding over a paged cache: the append with norm and rotary (blk_paged_append), attention of
chains and trees of new rows (blk_attn_paged), the verification of drafts (blk_verify_drafts), the
move of what is kept (blk_paged_keep) and the model that calls them (blk_model_forward_paged), against fp64 references.

Bounds count roundings. bf16 rounds by at most u = 2^-8 of the value (half a step), fp32 by 2^-24:
 - append: the fp32 chain of norm and rotary stays under 20 * 2^-24 * 1.5 (|a| + |b|) of a pair (a, b), a
   bf16 result adds u |out|. Channels outside the rotary have the norm's roundings alone. Values are copies.
 - attention: p is rounded to bf16 before the product with v (its sum is not), the output once:
   u sum(p |v|) + u |o|. Scores are sums of 128 exact products in fp32, off by at most
   128 * 2^-23 sum|q k| / sqrt(128); exp adds 2^-22. Both under 2e-4 of sum(p |v|) at these inputs.
 - verification: whole numbers, equal to those of the definition in fp64.
"""
import numpy as np
import pytest
import torch

import oracle
from llama_family_decoder_gb300 import BlkError, DecoderBlock
from llama_family_decoder_gb300.binding import lib, set_wait_timeout_ns
from llama_family_decoder_gb300.synth import Workload, make_model
from tests.helpers import TOL, cfg_of, np64, rel_err, to_dev, weights_np

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -8
D = 128


def block(H=8, Hkv=2, dtype="bf16", d=128, max_seq=4096, **kw):
    return DecoderBlock(hidden=H * d if H * d % 8 == 0 else 256, n_heads=H, n_kv_heads=Hkv, head_dim=d, ffn=256,
                        act="relu2", dtype=dtype, max_batch=4, max_seq=max_seq, **kw)


def randn(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cu_of(rows, first=0):
    return ints(np.concatenate([[first], first + np.cumsum(rows)]).tolist())


def cache_of(blk, lens, rows, page, seed=0, spare=1):
    """A paged cache with pages dealt out in any order, those not needed -1, and lens set."""
    r = np.random.default_rng(seed)
    need = [-(-(n + t) // page) for n, t in zip(lens, rows)]
    total = sum(need) + spare
    order = r.permutation(total)
    c = blk.paged_cache(len(lens), max(need + [1]) * page, page, n_pages=total)
    table = np.full(c["pages"].shape, -1)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    c["pages"].copy_(torch.from_numpy(table))
    c["lens"].copy_(ints(lens))
    return c


def slots_of(c, x, b, n):
    """The first n slots of sequence b, [n, Hkv, d]."""
    t = c[x]
    page = t.shape[2]
    pages = c["pages"][b, :-(-n // page)].long()
    return t[pages].transpose(1, 2).flatten(0, 1)[:n]


def fill(c, seed, lens):
    """Random keys and values in the slots below lens, as a prompt's."""
    for i, x in enumerate(("k", "v")):
        c[x].copy_(randn(seed + i, *c[x].shape, dtype=c[x].dtype))


def chain(n):
    return [i - 1 for i in range(n)]


def tree_of(n, seed):
    r = np.random.default_rng(seed)
    return [-1] + [int(r.integers(max(0, (i - 1) // 4 - 2), (i - 1) // 2 + 1)) for i in range(1, n)]


def kin_of(parents):
    n = len(parents)
    kin, depth = np.eye(n, dtype=bool), np.zeros(n, int)
    for i, p in enumerate(parents):
        if p >= 0:
            kin[i] |= kin[p]
            depth[i] = depth[p] + 1
    return kin, depth


# ------------------------------------------------------------------ append

def rope_ref(x, pos, gain, dims, interleaved, theta=10000.0, scaling=None):
    """x [n, heads, d] at positions pos -> (rotated, |a| + |b| of each pair, per element)."""
    y = np64(x)
    if gain is not None:
        y = oracle.rms_norm(y, np64(gain), 1e-5)
    half = dims // 2
    a_at = np.arange(0, dims, 2) if interleaved else np.arange(half)
    b_at = a_at + 1 if interleaved else a_at + half
    ang = np.asarray(pos, np.float64)[:, None] * oracle.rope_inv_freq(dims, theta, scaling)
    m = oracle.rope_attention_factor(scaling)
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    out, size = y.copy(), np.abs(y)
    a, b = y[..., a_at], y[..., b_at]
    out[..., a_at], out[..., b_at] = a * c - b * s, b * c + a * s
    size[..., a_at] = size[..., b_at] = np.abs(a) + np.abs(b)
    return out, size


def check_rope(got, x, pos, gain, dims, interleaved, **kw):
    ref, size = rope_ref(x, pos, gain, dims, interleaved, **kw)
    bound = 20 * 2.0 ** -24 * 1.5 * size + (U * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(np64(got) - ref) <= bound)


@pytest.mark.parametrize("lens,rows", [([0], [1]), ([37, 0, 200], [1, 1, 1]), ([5, 100, 0, 31], [3, 0, 700, 17]),
                                       ([63, 64, 65] * 30, [1, 2, 5] * 30)])
@pytest.mark.parametrize("H,Hkv,dtype,d,norm,dims,interleaved,page", [
    (32, 8, "bf16", 128, True, 128, False, 64), (8, 2, "bf16", 128, False, 64, True, 16),
    (5, 1, "bf16", 128, True, 128, True, 256), (3, 3, "bf16", 128, True, 48, False, 32),
    (4, 2, "f32", 64, True, 64, False, 16), (3, 1, "f32", 80, True, 40, True, 32), (2, 1, "f32", 256, False, 256, True, 128),
    (6, 2, "f32", 8, False, 8, False, 16)])
def test_paged_append(lens, rows, H, Hkv, dtype, d, norm, dims, interleaved, page):
    blk = block(H, Hkv, dtype, d, qk_norm=norm)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = sum(rows)
    c = cache_of(blk, lens, rows, page)
    fill(c, 50, lens)
    before = {x: c[x].clone() for x in "kv"}
    q, k, v = randn(1, n, H, d, dtype=dt), randn(2, n, Hkv, d, dtype=dt), randn(3, n, Hkv, d, dtype=dt)
    q[0] *= 1e4
    gq, gk = 1 + 0.2 * randn(4, d, dtype=dt), 1 + 0.2 * randn(5, d, dtype=dt)
    table = blk.rope_table(dims, 1000) if dims < d else None
    depths = [[i // 2 for i in range(t)] for t in rows]
    cu = cu_of(rows) if rows != [1] * len(rows) else None
    got = blk.paged_append(c, q, k, v, cu, ints(sum(depths, [])), gq, gk, rope_table=table, interleaved=interleaved)
    assert blk.last_status() == 0
    assert c["lens"].tolist() == lens
    pos = np.array([n0 + x for n0, dep in zip(lens, depths) for x in dep])
    check_rope(got, q, pos, gq if norm else None, dims, interleaved)
    at = 0
    for b, (n0, t) in enumerate(zip(lens, rows)):
        if t:
            check_rope(slots_of(c, "k", b, n0 + t)[n0:], k[at:at + t], pos[at:at + t], gk if norm else None, dims, interleaved)
            assert torch.equal(slots_of(c, "v", b, n0 + t)[n0:], v[at:at + t])
        for x in "kv":  # the slots before are as they were
            assert torch.equal(slots_of(c, x, b, n0), slots_of(dict(c, **before), x, b, n0))
        at += t
    # ... and the values outside every sequence's rows
    mine = torch.zeros(c["k"].shape[0], page, dtype=torch.bool, device=DEV)
    for b, (n0, t) in enumerate(zip(lens, rows)):
        for s in range(n0, n0 + t):
            mine[c["pages"][b, s // page].long(), s % page] = True
    for x in "kv":
        assert torch.equal(c[x].transpose(1, 2)[~mine], before[x].transpose(1, 2)[~mine])


@pytest.mark.parametrize("scaling", [("yarn", 20.0, 4096, 1.0, 32.0), ("llama3", 8.0, 8192, 1.0, 4.0)])
@pytest.mark.parametrize("dims", [128, 64])
def test_paged_append_stretched(scaling, dims):
    blk = block(4, 2, max_seq=9000, rope_scaling=scaling, rope_theta=5e5)
    lens, rows = [0, 8000, 4000], [40, 30, 30]
    c = cache_of(blk, lens, rows, 128)
    q, k, v = randn(1, 100, 4, D), randn(2, 100, 2, D), randn(3, 100, 2, D)
    got = blk.paged_append(c, q, k, v, cu_of(rows), rope_table=blk.rope_table(dims) if dims < 128 else None)
    pos = np.concatenate([n + np.arange(t) for n, t in zip(lens, rows)])
    check_rope(got, q, pos, None, dims, False, theta=5e5, scaling=oracle.RopeScaling(*scaling))
    check_rope(slots_of(c, "k", 1, 8030)[8000:], k[40:70], pos[40:70], None, dims, False, theta=5e5,
               scaling=oracle.RopeScaling(*scaling))
    assert blk.last_status() == 0


def test_the_handles_table_is_the_one_made():
    blk = block(4, 2, max_seq=300, rope_theta=1e6)
    rows = [17, 9]
    q, k, v = randn(1, 26, 4, D), randn(2, 26, 2, D), randn(3, 26, 2, D)
    outs = []
    for table in (None, blk.rope_table(), blk.rope_table(128, 300)):
        c = cache_of(blk, [5, 270], rows, 16)
        outs.append((blk.paged_append(c, q, k, v, cu_of(rows), rope_table=table), c["k"]))
    for o, kk in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(kk, outs[0][1])
    # without a cache in between, the packed stage turns the same
    pos = ints([5 + i for i in range(17)] + [270 + i for i in range(9)])
    qo, ko = blk.qk_norm_rope(q, k, pos)
    assert torch.equal(qo, outs[0][0])
    assert torch.equal(torch.cat([slots_of(c, "k", 0, 22)[5:], slots_of(c, "k", 1, 279)[270:]]), ko)


def test_paged_append_layouts_and_in_place():
    H, Hkv, n = 6, 2, 77
    blk = block(H, Hkv, qk_norm=True)
    g = 1 + 0.1 * randn(3, D)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(4, n, Hkv, D)
    cu = ints([3, 40, 70])  # rows 0 .. 2 and 70 .. of no sequence

    def run(q, k, v, **kw):
        c = cache_of(blk, [9, 0], [37, 30], 32)
        return blk.paged_append(c, q, k, v, cu, None, g, g, **kw), c

    want, c0 = run(q, k, v, q_out=torch.full_like(q, 7.0))
    assert torch.all(want[:3] == 7) and torch.all(want[70:] == 7)
    fused = torch.cat([q, k, v], 1).contiguous()
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    out = torch.full((H, n, D), 7.0, dtype=torch.bfloat16, device=DEV)
    a, c1 = run(fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:], q_out=out.transpose(0, 1))
    b, c2 = run(*hm, q_out=torch.full_like(q, 7.0))
    for o, c in ((a, c1), (b, c2)):
        assert torch.equal(o, want) and torch.equal(c["k"], c0["k"]) and torch.equal(c["v"], c0["v"])
    q2 = q.clone()
    run(q2, k, v, q_out=q2)
    assert torch.equal(q2[3:70], want[3:70]) and torch.equal(q2[:3], q[:3])
    _, c3 = run(q, k[:, :1].expand(n, Hkv, D), v)  # one head's keys for both
    assert torch.equal(c3["k"][:, 0], c0["k"][:, 0]) and torch.equal(c3["k"][:, 1], c0["k"][:, 0])
    assert blk.last_status() == 0


def test_paged_append_without_room_or_page():
    blk = block(4, 2, max_seq=64)
    q, k, v = randn(1, 6, 4, D), randn(2, 6, 2, D), randn(3, 6, 2, D)
    c = blk.paged_cache(2, 32, 16)
    c["lens"].copy_(ints([30, 4]))
    before = c["k"].clone()
    out = blk.paged_append(c, q, k, v, ints([0, 4, 6]))
    assert blk.last_status() == 4  # two of four rows fit
    check_rope(out, q, np.array([30, 31, 32, 33, 4, 5]), None, D, False)
    assert torch.equal(slots_of(c, "v", 0, 32)[30:], v[:2]) and torch.equal(slots_of(c, "v", 1, 6)[4:], v[4:])
    for page in (-1, 4, 2**31 - 1):
        c["k"].copy_(before)
        c["pages"][1, 0] = page
        blk.paged_append(c, q, k, v, ints([0, 1, 6]))
        assert blk.last_status() == 1
        assert torch.equal(slots_of(c, "k", 0, 30), torch.zeros_like(k[:1]).expand(30, 2, D))
        assert torch.count_nonzero(c["k"]) <= 2 * D  # row 0 of sequence 0 alone
    c["pages"][1, 0] = 2
    with pytest.raises(BlkError, match="CACHE_FULL"):
        blk.paged_append(c, q, k, v, ints([0, 4, 6]), host_lens_max=34)
    c["lens"].copy_(ints([-3, 0]))
    blk.paged_append(c, q, k, v, ints([0, 4, 6]))
    assert blk.last_status() == 1
    # positions outside the table are clamped
    c["lens"].copy_(ints([0, 0]))
    out = blk.paged_append(c, q[:2], k[:2], v[:2], depths=ints([64, -1]))
    assert blk.last_status() == 1
    check_rope(out, q[:2], np.array([63, 0]), None, D, False)
    # a list that falls or leaves the rows stays in bounds
    for cu in ([0, 60, 2], [5, 2, 6], [-7, 3, 6], [0, 3, 99]):
        blk.paged_append(c, q, k, v, ints(cu))
        assert blk.last_status() == 1
    blk.paged_append(c, q[:0], k[:0], v[:0], ints([0, 0, 0]))
    assert blk.last_status() == 0


def test_paged_append_far_rows():
    """Slots whose bytes lie behind 2^32, and rows 2^31 elements apart."""
    blk = block(1, 1)
    n_pages = 300000
    c = blk.paged_cache(1, 64, 64, n_pages=n_pages)  # 64 * 256 bytes a page: 4.9 GB each of k and v
    c["pages"][0, 0] = n_pages - 1
    far = torch.empty(2**31 + 2 * D, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(far, (2, 1, D), (2**31, D, 1))
    x.copy_(randn(1, 2, 1, D))
    blk.paged_append(c, x, x, x, ints([0, 2]))
    assert torch.equal(c["v"][-1, :, :2], x.transpose(0, 1))
    c["lens"].fill_(2)
    q = randn(2, 1, 1, D)
    blk.paged_append(c, q, q, q)
    c["lens"].fill_(2)
    o = blk.attn_paged(q, c)
    k, v = slots_of(c, "k", 0, 3), slots_of(c, "v", 0, 3)
    check_attn(o, q, [k], [v], [chain(1)], [2])
    assert blk.last_status() == 0


# ------------------------------------------------------------------ attention

def attn_ref(q, k, v, parents, n, window):
    """Rows q [t, H, d] over k, v [n + t, Hkv, d], all fp64 -> (o, sum p |v|)."""
    t, H, d = q.shape
    per = H // k.shape[1]
    kin, depth = kin_of(parents)
    seen = np.concatenate([np.ones((t, n), bool), kin], 1)
    if window:
        place = np.concatenate([np.arange(n), n + depth])
        seen &= place[None] > (n + depth)[:, None] - window
    o, mag = np.empty_like(q), np.empty_like(q)
    for h in range(H):
        s = np.where(seen, q[:, h] @ k[:, h // per].T / np.sqrt(d), -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o[:, h], mag[:, h] = p @ v[:, h // per], p @ np.abs(v[:, h // per])
    return o, mag


def check_attn(out, q, ks, vs, trees, lens, window=0, first=0):
    at = first
    for k, v, parents, n in zip(ks, vs, trees, lens):
        t = len(parents)
        if t:
            ref, mag = attn_ref(np64(q[at:at + t]), np64(k), np64(v), parents, n, window)
            err = np.abs(np64(out[at:at + t]) - ref)
            assert np.all(err <= (U + 2e-4) * mag + U * np.abs(ref)), (n, t, float((err / mag).max()))
        at += t


def attn_case(H, Hkv, lens, trees, page, window=0, seed=0, **kw):
    blk = block(H, Hkv, sliding_window=window)
    rows = [len(t) for t in trees]
    c = cache_of(blk, lens, rows, page, seed)
    fill(c, 60 + seed, lens)
    q = randn(70 + seed, sum(rows), H, D)
    ks, vs = ([slots_of(c, x, b, n + t).clone() for b, (n, t) in enumerate(zip(lens, rows))] for x in "kv")
    return blk, c, q, ks, vs, cu_of(rows), ints([p for t in trees for p in t])


LENS = [([0], [1]), ([1], [1]), ([63], [2]), ([64], [1]), ([65], [64]), ([300], [33]), ([0, 5, 0, 700], [64, 0, 7, 20]),
        ([127, 128, 129, 1, 2], [1, 1, 1, 1, 1]), ([2000, 17], [8, 64]), ([10] * 40, [3] * 40), ([5000], [1])]


@pytest.mark.parametrize("lens,rows", LENS)
@pytest.mark.parametrize("H,Hkv,page", [(8, 2, 64), (3, 3, 16), (5, 1, 32), (16, 1, 128), (2, 2, 256), (12, 4, 16)])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged(lens, rows, H, Hkv, page, kind):
    trees = [chain(t) if kind == "chain" else tree_of(t, 7 + b) if t else [] for b, t in enumerate(rows)]
    blk, c, q, ks, vs, cu, parents = attn_case(H, Hkv, lens, trees, page)
    one_each = rows == [1] * len(rows)
    out = blk.attn_paged(q, c, None if one_each else cu, parents if kind == "tree" else None)
    assert blk.last_status() == 0
    check_attn(out, q, ks, vs, trees, lens)


@pytest.mark.parametrize("window", [1, 2, 5, 64, 100, 1000])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged_window(window, kind):
    lens, rows = [0, 3, 64, 500, 1500], [5, 64, 1, 40, 12]
    trees = [chain(t) if kind == "chain" else tree_of(t, b) for b, t in enumerate(rows)]
    blk, c, q, ks, vs, cu, parents = attn_case(6, 2, lens, trees, 32, window)
    # pages wholly before every row's window are not looked at
    for b, n in enumerate(lens):
        c["pages"][b, :max(0, n - window + 1) // 32] = -1 if b % 2 else 2**30
    out = blk.attn_paged(q, c, cu, parents if kind == "tree" else None)
    assert blk.last_status() == 0
    check_attn(out, q, ks, vs, trees, lens, window)


@pytest.mark.parametrize("H,Hkv,lens,rows", [(8, 2, [0], [700]), (4, 4, [130, 3], [257, 300]), (16, 1, [77], [100]),
                                             (5, 1, [0, 64], [129, 65]), (32, 8, [1000, 20], [90, 400])])
@pytest.mark.parametrize("window", [0, 50])
def test_attn_paged_long_chains(H, Hkv, lens, rows, window):
    trees = [chain(t) for t in rows]
    blk, c, q, ks, vs, cu, _ = attn_case(H, Hkv, lens, trees, 64, window)
    out = blk.attn_paged(q, c, cu)
    assert blk.last_status() == 0
    check_attn(out, q, ks, vs, trees, lens, window)


@pytest.mark.parametrize("lens", [[8000], [3000, 10, 0, 4100, 777, 2222, 64, 1], [200] * 100, [20000, 1], [700, 0, 64, 1500] * 10])
@pytest.mark.parametrize("H,Hkv,rows", [(32, 8, 1), (8, 2, 5), (8, 8, 20), (16, 2, 64)])
def test_attn_paged_split_keys(lens, H, Hkv, rows):
    """Work that many CTAs share, whole and in parts."""
    trees = [tree_of(rows, b) for b in range(len(lens))]
    blk, c, q, ks, vs, cu, parents = attn_case(H, Hkv, lens, trees, 64)
    out = blk.attn_paged(q, c, cu, parents)
    assert blk.last_status() == 0
    some = [0, len(lens) - 1] if len(lens) > 10 else range(len(lens))
    for b in some:
        check_attn(out, q, [ks[b]], [vs[b]], [trees[b]], [lens[b]], first=b * rows)
    assert torch.equal(out, blk.attn_paged(q, c, cu, parents))  # the same sums in the same order


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged_many_ragged_sequences(kind, window):
    """More units than CTAs, from none to 64 rows over none to 6000 slots: stretches that end anywhere in them."""
    r = np.random.default_rng(4)
    rows = [int(t) for t in r.choice([0, 1, 1, 2, 16, 17, 33, 64], 90)]
    lens = [int(n) for n in r.choice([0, 1, 50, 64, 333, 1000], 90)]
    lens[7], rows[7], lens[50], rows[50] = 6000, 64, 4100, 1
    trees = [chain(t) if kind == "chain" else tree_of(t, b) if t else [] for b, t in enumerate(rows)]
    blk, c, q, ks, vs, cu, parents = attn_case(8, 2, lens, trees, 32, window)
    out = blk.attn_paged(q, c, cu, parents if kind == "tree" else None)
    assert blk.last_status() == 0
    check_attn(out, q, ks, vs, trees, lens, window)


def test_attn_paged_chain_is_a_tree_of_one_branch():
    trees = [chain(t) for t in (64, 5, 1)]
    blk, c, q, ks, vs, cu, parents = attn_case(8, 2, [90, 0, 400], trees, 16)
    for up in (None, parents):  # the keys may be shared out differently
        check_attn(blk.attn_paged(q, c, cu, up), q, ks, vs, trees, [90, 0, 400])


@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged_what_nobody_sees(kind):
    """Unused slots and pages, rows of no sequence and other sequences may hold anything."""
    lens, rows = [100, 37, 0, 260], [20, 1, 0, 50]
    trees = [chain(t) if kind == "chain" else tree_of(t, b) if t else [] for b, t in enumerate(rows)]
    blk, c, q, ks, vs, _, parents = attn_case(4, 2, lens, trees, 64)
    n, first = sum(rows), 6
    pad = lambda x, v: torch.cat([torch.full_like(x[:first], v), x, torch.full_like(x[:first], v)])
    cu = cu_of(rows, first)
    up = pad(parents, 5) if kind == "tree" else None
    clean = blk.attn_paged(pad(q, 0.0), c, cu, up)
    used = torch.zeros(c["k"].shape[0], 64, dtype=torch.bool, device=DEV)
    for b, (m, t) in enumerate(zip(lens, rows)):
        for s in range(m + t if t else 0):
            used[c["pages"][b, s // 64].long(), s % 64] = True
    for x, bad in (("k", float("nan")), ("v", float("inf"))):
        c[x].transpose(1, 2)[~used] = bad
    out = torch.full((n + 2 * first, 4, D), 3.0, dtype=torch.bfloat16, device=DEV)
    blk.attn_paged(pad(q, float("nan")), c, cu, up, out=out)
    mine = slice(first, first + n)
    assert torch.equal(out[mine], clean[mine])
    assert torch.all(out[:first] == 3) and torch.all(out[mine.stop:] == 3)
    check_attn(out, pad(q, 0.0), ks, vs, trees, lens, first=first)
    assert blk.last_status() == 0
    # a whole sequence of NaN between two others
    for x in "kv":
        pages = c["pages"][1, :1].long()
        c[x][pages] = float("nan")
    again = blk.attn_paged(pad(q, float("nan")), c, cu, up)
    assert torch.equal(again[first:first + 20], clean[first:first + 20])
    assert torch.equal(again[first + 21:first + n], clean[first + 21:first + n])
    assert torch.isnan(again[first + 20]).all()


def test_attn_paged_scores_that_are_no_numbers():
    blk, c, q, ks, vs, cu, _ = attn_case(4, 2, [70], [chain(3)], 64)
    want = blk.attn_paged(q, c, cu)
    page, row = c["pages"][0, 1].long(), 71 % 64  # row 1's own key, head 0: rows 1 and 2 see it
    c["k"][page, 0, row, 5] = float("nan")
    out = blk.attn_paged(q, c, cu)
    assert torch.equal(out[0], want[0]) and torch.equal(out[:, 2:], want[:, 2:])
    assert torch.isnan(out[1:, :2]).all()
    # all scores -inf: 0 / 0
    c["k"].fill_(0)
    c["k"][..., 0] = float("-inf")
    q[:] = 0
    q[..., 0] = 1
    assert torch.isnan(blk.attn_paged(q, c, cu)).all()


def test_attn_paged_large_scores():
    """Scores in the thousands, growing and falling along the keys: the reference of the exponentials moves."""
    for sign in (1, -1):
        blk, c, q, ks, vs, cu, _ = attn_case(2, 1, [1000], [chain(4)], 64)
        q[:] = 0
        q[..., 0] = 64.0
        grow = (torch.arange(1004, device=DEV) // 8 * 8).float() * sign  # exact in bf16; scores 64 s / sqrt(128)
        for s in range(1004):
            c["k"][c["pages"][0, s // 64].long(), :, s % 64] = 0
            c["k"][c["pages"][0, s // 64].long(), :, s % 64, 0] = grow[s]
        k = slots_of(c, "k", 0, 1004)
        check_attn(blk.attn_paged(q, c, cu), q, [k], [vs[0]], [chain(4)], [1000])


def test_attn_paged_layouts():
    trees = [tree_of(30, 1), tree_of(7, 2)]
    blk, c, q, ks, vs, cu, parents = attn_case(6, 2, [100, 9], trees, 16)
    want = blk.attn_paged(q, c, cu, parents)
    wide = torch.randn(37, 10, D, device=DEV).bfloat16()
    wide[:, 2:8] = q
    out = torch.zeros(6, 37, D, dtype=torch.bfloat16, device=DEV)
    got = blk.attn_paged(wide[:, 2:8], c, cu, parents, out=out.transpose(0, 1))
    assert torch.equal(got, want) and torch.equal(out.transpose(0, 1), want)
    with pytest.raises(BlkError, match="broadcast"):
        blk.attn_paged(q[:, :1].expand(37, 6, D), c, cu, parents)


def test_attn_paged_shared_pages():
    """Two sequences over the same prompt's pages."""
    blk, c, q, ks, vs, cu, _ = attn_case(4, 2, [128, 128], [chain(3), chain(5)], 64)
    c["pages"][1, :2] = c["pages"][0, :2]
    ks, vs = ([slots_of(c, x, b, 128 + t) for b, t in ((0, 3), (1, 5))] for x in "kv")
    check_attn(blk.attn_paged(q, c, cu), q, ks, vs, [chain(3), chain(5)], [128, 128])


def test_attn_paged_bad_lists_stay_in_bounds():
    trees = [tree_of(64, 1), tree_of(20, 2)]
    blk, c, q, ks, vs, cu, parents = attn_case(4, 2, [100, 9], trees, 32)
    want = blk.attn_paged(q, c, cu, parents)
    blk.last_status()
    for bad in ([0, 200, 84], [64, 0, 84], [-5, 64, 84], [0, 64, 2**31 - 1]):
        blk.attn_paged(q, c, ints(bad), parents)
        assert blk.last_status() == 1
    blk.attn_paged(q, c, ints([0, 0, 84]), parents)  # more than 64 rows of a tree
    assert blk.last_status() == 1
    for at, up in ((5, 5), (5, 63), (70, 2**31 - 1)):
        p = parents.clone()
        p[at] = up
        out = blk.attn_paged(q, c, cu, p)
        assert blk.last_status() == 1
        p[at] = -1
        assert torch.equal(out, blk.attn_paged(q, c, cu, p))  # read as none
        assert blk.last_status() == 0
    for page in (-1, c["k"].shape[0], 2**31 - 1):
        t = c["pages"].clone()
        t[1, 0] = page
        out = blk.attn_paged(q, dict(c, pages=t), cu, parents)
        assert blk.last_status() == 1
        assert torch.equal(out[:64], want[:64])  # the other sequence's rows
    for lens, code in (([-1, 9], 1), ([2**31 - 1, 9], 4), ([161, 9], 4)):
        out = torch.full_like(q, 5.0)
        blk.attn_paged(q, dict(c, lens=ints(lens)), cu, parents, out=out)
        assert blk.last_status() == code
        assert torch.all(out[:64] == 5) and torch.equal(out[64:], want[64:])
    assert blk.attn_paged(q[:0], c, ints([0, 0, 0])).shape == (0, 4, D)
    assert blk.last_status() == 0


@pytest.mark.parametrize("H,Hkv,lens,rows", [(4, 2, [100, 9], [60, 20]),               # clusters
                                             (32, 8, [300] * 40, [1, 5] * 20)])         # the line and its join
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged_a_list_that_falls(H, Hkv, lens, rows, kind):
    """Its sequences claim rows twice: none gets an output, and the next call is right."""
    trees = [chain(t) if kind == "chain" else tree_of(t, b) for b, t in enumerate(rows)]
    blk, c, q, ks, vs, cu, parents = attn_case(H, Hkv, lens, trees, 32)
    up = parents if kind == "tree" else None
    n = cu[-1].item()
    for at, entry in ((0, n), (1, 0), (1, n), (len(rows) - 1, n), (len(rows), 0), (len(rows), -5)):
        bad = cu.clone()
        bad[at] = entry
        falls = bool((bad[1:] < bad[:-1]).any())
        out = blk.attn_paged(q, c, bad, up, out=torch.full_like(q, 5.0))
        status = blk.last_status()
        if falls:
            assert status == 1 and torch.all(out == 5), (at, entry)
        check_attn(blk.attn_paged(q, c, cu, up), q, ks[:1], vs[:1], trees[:1], lens[:1])
    assert blk.last_status() == 0


def test_attn_paged_a_list_that_falls_past_32_bits():
    """Eleven of its sequences claim all rows over 2^28 slots each: more than 2^32 tiles of keys."""
    blk, rows, B = block(1, 1), 25600, 22
    c = blk.paged_cache(1, 64, 64)
    c["pages"] = torch.zeros(B, 2**22, dtype=torch.int32, device=DEV)
    c["lens"] = torch.full((B,), 2**28 - rows, dtype=torch.int32, device=DEV)
    q = randn(1, rows, 1, D)
    out = blk.attn_paged(q, c, ints([0, rows] * (B // 2) + [0]), out=torch.full_like(q, 5.0))
    assert blk.last_status() == 1 and torch.all(out == 5)


def test_attn_paged_at_the_last_slots():
    """A page list of 2^31 slots, all of them one page; a window leaves the last ones of it."""
    blk = block(2, 1, sliding_window=100)
    c = blk.paged_cache(1, 64, 64)
    c["pages"] = torch.zeros(1, 2**25, dtype=torch.int32, device=DEV)
    for x in "kv":
        c[x].copy_(randn(5 + ord(x), 1, 1, 64, D))
    q, end = randn(1, 3, 2, D), 2**31 - 2**16
    c["lens"].fill_(end - 3)
    out = blk.attn_paged(q, c, ints([0, 3]))
    assert blk.last_status() == 0
    k, v = ([c[x][0].transpose(0, 1)[(torch.arange(end - 110, end) % 64).to(DEV)]] for x in "kv")
    check_attn(out, q, k, v, [chain(3)], [107], 100)
    for n in (end - 2, 2**31 - 4, 2**31 - 1):
        c["lens"].fill_(n)
        kept = blk.attn_paged(q, c, ints([0, 3]), out=torch.full_like(q, 2.0))
        assert blk.last_status() == 4 and torch.all(kept == 2)


@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_attn_paged_thousands_of_sequences(kind):
    """More of them than a warp looks up at once, most without rows."""
    rows, lens = [0] * 3001, [3] * 3001
    for b in (0, 31, 127, 128, 129, 1000, 2999, 3000):
        rows[b], lens[b] = 1 + b % 40, b
    trees = [chain(t) if kind == "chain" else tree_of(t, b) if t else [] for b, t in enumerate(rows)]
    blk, c, q, ks, vs, cu, parents = attn_case(8, 2, lens, trees, 64)
    out = blk.attn_paged(q, c, cu, parents if kind == "tree" else None)
    assert blk.last_status() == 0
    check_attn(out, q, ks, vs, trees, lens)
    one = randn(3, 3001, 8, D)
    out = blk.attn_paged(one, c)
    for b in (0, 31, 128, 1000, 1001, 2999, 3000):
        check_attn(out[b:b + 1], one[b:b + 1], [slots_of(c, "k", b, lens[b] + 1)], [slots_of(c, "v", b, lens[b] + 1)],
                   [chain(1)], [lens[b]])
    assert blk.last_status() == 0


def test_attn_paged_is_the_decode_stage():
    """One token a sequence: the same as decode attention over a contiguous cache, to both roundings."""
    H, Hkv, lens = 8, 2, [5, 700, 64]
    blk, c, q, ks, vs, _, _ = attn_case(H, Hkv, lens, [chain(1)] * 3, 64)
    k, v = (torch.zeros(3, Hkv, 704, D, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    for b, n in enumerate(lens):
        k[b, :, :n + 1], v[b, :, :n + 1] = ks[b].transpose(0, 1), vs[b].transpose(0, 1)
    o = torch.empty(3, 1, H, D, dtype=torch.bfloat16, device=DEV)
    blk.attn_gqa(q[:, :, None], k, v, o, kv_lens=ints([n + 1 for n in lens]))
    got = blk.attn_paged(q, c)
    for b, n in enumerate(lens):
        _, mag = attn_ref(np64(q[b:b + 1]), np64(ks[b]), np64(vs[b]), chain(1), n, 0)
        assert np.all(np.abs(np64(got[b]) - np64(o[b, 0])) <= 2 * ((U + 2e-4) * mag[0] + U * mag[0]))


def test_streams_and_graphs():
    """A captured step replayed with other contents, beside an eager one on another stream."""
    trees = [tree_of(33, 1), tree_of(64, 2), tree_of(3, 3)]
    lens = [300, 0, 1500]
    blk, c, q, ks, vs, cu, parents = attn_case(8, 2, lens, trees, 64)
    other = {x: c[x].clone() for x in "kv"}
    n = q.shape[0]
    k, v = randn(80, n, 2, D), randn(81, n, 2, D)
    target = torch.softmax(3 * randn(82, n, 1000, dtype=torch.float32), -1)
    tokens = torch.randint(0, 1000, (n,), device=DEV, dtype=torch.int32)
    u, u_next = torch.rand(n, device=DEV), torch.rand(3, device=DEV)
    starts = ints(lens)

    def step(cache, q, k, v):
        cache["lens"].copy_(starts)
        qr = blk.paged_append(cache, q, k, v, cu)
        o = blk.attn_paged(qr, cache, cu, parents)
        counts, path, nxt = blk.verify_drafts(target, tokens, u, u_next, cu, parents)
        blk.paged_keep([cache], counts, path, cu)
        return o, counts, path, nxt

    fresh = dict(c, k=other["k"].clone(), v=other["v"].clone(), lens=c["lens"].clone())
    want = step(fresh, q, k, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(dict(c, k=other["k"].clone(), v=other["v"].clone(), lens=c["lens"].clone()), q, k, v)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    q2, k2 = q.clone(), k.clone()
    graphed = dict(c, k=other["k"].clone(), v=other["v"].clone(), lens=c["lens"].clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(graphed, q2, k2, v)
    for _ in range(3):
        q2.zero_()
        k2.zero_()
        graphed["k"].copy_(other["k"])
        graphed["v"].copy_(other["v"])
        eager = dict(c, k=other["k"].clone(), v=other["v"].clone(), lens=c["lens"].clone())
        s.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(s):  # two at once
            again = step(eager, q, k, v)
        torch.cuda.synchronize()
        q2.copy_(q)
        k2.copy_(k)
        graphed["k"].copy_(other["k"])
        graphed["v"].copy_(other["v"])
        g.replay()
        torch.cuda.synchronize()
        for a, b, w in zip(outs, again, want):
            assert torch.equal(a, w) and torch.equal(b, w)
        for x in ("k", "v", "lens"):
            assert torch.equal(graphed[x], fresh[x]) and torch.equal(eager[x], fresh[x])
    # a stream given by the caller
    with_stream = dict(c, k=other["k"].clone(), v=other["v"].clone(), lens=starts.clone())
    qr = blk.paged_append(with_stream, q, k, v, cu, stream=s)
    o = blk.attn_paged(qr, with_stream, cu, parents, stream=s)
    r = blk.verify_drafts(target, tokens, u, u_next, cu, parents, stream=s)
    blk.paged_keep([with_stream], r[0], r[1], cu, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(r[2], want[3]) and torch.equal(with_stream["lens"], fresh["lens"])
    assert blk.last_status() == 0


@pytest.mark.parametrize("H,Hkv,lens,rows", [(8, 2, [3000], 1),        # clusters, slots of the same rows
                                             (8, 2, [3000], 60),       # clusters, two slots of rows
                                             (8, 2, [200] * 16, 1),    # a CTA a unit
                                             (32, 8, [3000] * 40, 1),  # the line, slots that take units in turn
                                             (32, 8, [900] * 24, 60)])  # the line, two slots of a unit
@pytest.mark.parametrize("limit", [100, 2000])
def test_attn_paged_waits_that_run_out(H, Hkv, lens, rows, limit):
    """A limit below the time of a first tile: waits give up, the status says so, the CTAs' copies and products end, and
    the next call is right."""
    trees = [tree_of(rows, b) for b in range(len(lens))]
    blk, c, q, ks, vs, cu, parents = attn_case(H, Hkv, lens, trees, 64)
    want = blk.attn_paged(q, c, cu, parents)
    assert blk.last_status() == 0
    for _ in range(3):
        set_wait_timeout_ns(limit)
        try:
            blk.attn_paged(q, c, cu, parents)
            torch.cuda.synchronize()
        finally:
            set_wait_timeout_ns(0)
        status = blk.last_status()
        assert status == 6 if limit == 100 else status in (0, 6)
        assert torch.equal(blk.attn_paged(q, c, cu, parents), want)
        assert blk.last_status() == 0
    check_attn(want, q, ks[:1], vs[:1], trees[:1], lens[:1])


# ------------------------------------------------------------------ verification

def verify_ref(target, draft, tokens, parents, u, u_next):
    """One sequence by the definition, all fp64 -> (path, next)."""
    cur, path = 0, [0]
    while True:
        left, c, taken = target[cur].copy(), 1.0, None
        for x in range(1, len(parents)):
            if parents[x] != cur:
                continue
            t = tokens[x]
            if u[x] * c * (1.0 if draft is None else draft[cur][t]) < left[t] and left[t] > 0:
                taken = x
                break
            if draft is None:
                c -= left[t]
                left[t] = 0
            else:
                left = np.maximum(0, left - c * draft[cur])
                c = left.sum()
        if taken is None:
            break
        path.append(taken)
        cur = taken
    if not left.sum() > 0:
        left = target[cur]
    upto = np.cumsum(left)
    return path, min(int(np.searchsorted(upto, u_next * upto[-1], side="right")), len(left) - 1)


def check_verify(blk, trees, vocab, with_draft, seed, sharp=3.0, near=0.7, cu=None, shared_tokens=False):
    rows = [len(t) for t in trees]
    n, B = sum(rows), len(trees)
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = sharp * torch.randn(n, vocab, generator=g, device=DEV)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + near * torch.randn(n, vocab, generator=g, device=DEV), -1)
    first = np.concatenate([[0], np.cumsum(rows)])
    of = torch.tensor([first[b] + max(p, 0) for b, t in enumerate(trees) for p in t], dtype=torch.long, device=DEV)
    noise = torch.empty(n, vocab, device=DEV).exponential_(generator=g)
    if shared_tokens:
        noise = noise[:1]
    tokens = (draft[of] / noise).argmax(-1).to(torch.int32)
    u, u_next = torch.rand(n, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
    parents = ints([p for t in trees for p in t])
    counts, path, nxt = blk.verify_drafts(target, tokens, u, u_next, cu_of(rows), parents, draft if with_draft else None)
    assert blk.last_status() == 0
    counts, path, nxt, tok = counts.tolist(), path.tolist(), nxt.tolist(), tokens.tolist()
    T, G, uu, un = np64(target), np64(draft), np64(u), np64(u_next)
    for b, t in enumerate(trees):
        lo, hi = first[b], first[b + 1]
        if lo == hi:
            assert counts[b] == 0 and nxt[b] == -1
            continue
        want, token = verify_ref(T[lo:hi], G[lo:hi] if with_draft else None, tok[lo:hi], t, uu[lo:hi], un[b])
        assert path[lo:hi] == want + [-1] * (len(t) - len(want)), b
        assert counts[b] == len(want) and nxt[b] == token, b
    return counts


@pytest.mark.parametrize("vocab", [1, 2, 15, 17, 511, 512, 513, 4099, 32000, 50257])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_drafts(vocab, with_draft):
    blk = block()
    trees = [chain(5), chain(1), [], tree_of(20, 1), tree_of(64, 2), chain(64), tree_of(9, 3), [-1, 0, 0, 0, 0, -1, 5]]
    for seed in range(2):
        check_verify(blk, trees, vocab, with_draft, seed)
        check_verify(blk, trees, vocab, with_draft, 10 + seed, sharp=0.3, near=0.1)  # long walks
        check_verify(blk, trees, vocab, with_draft, 20 + seed, near=3.0, shared_tokens=True)  # many rejections, a token twice


@pytest.mark.parametrize("B,vocab", [(300, 1000), (1000, 64), (40, 131072)])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_many_sequences(B, vocab, with_draft):
    counts = check_verify(block(), [tree_of(4 + b % 3, b) if b % 2 else chain(4) for b in range(B)], vocab, with_draft, B)
    assert min(counts) == 1 and max(counts) > 1


def test_verify_unaligned_rows():
    """Rows of odd strides that begin anywhere."""
    blk, vocab, n = block(), 1001, 6
    wide = torch.rand(n, vocab + 6, device=DEV)
    t = wide[:, 3:3 + vocab]
    t /= t.sum(-1, keepdim=True)
    d = torch.softmax(torch.randn(n, vocab + 2, device=DEV), -1)[:, 1:1 + vocab]
    tokens, u, un = torch.randint(0, vocab, (n,), device=DEV, dtype=torch.int32), torch.rand(n, device=DEV), torch.rand(1, device=DEV)
    for draft in (None, d):
        got = blk.verify_drafts(t, tokens, u, un, ints([0, n]), None, draft)
        want = blk.verify_drafts(t.contiguous(), tokens, u, un, ints([0, n]), None, None if draft is None else d.contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        path, nxt = verify_ref(np64(t), None if draft is None else np64(d), tokens.tolist(), chain(n), np64(u), float(un))
        assert got[0].item() == len(path) and got[2].item() == nxt


def test_verify_edges():
    blk, V = block(), 700
    one = torch.zeros(3, V, device=DEV)
    one[0, 5] = one[1, 699] = one[2, 3] = 1.0
    cu, zero = ints([0, 3]), torch.zeros(1, device=DEV)
    top = torch.tensor([1 - 2.0 ** -24], device=DEV)
    for un, u in ((zero, torch.zeros(3, device=DEV)), (top, top.expand(3).contiguous())):
        # a target of one token each: exactly that chain is accepted, whatever the numbers
        got = blk.verify_drafts(one, ints([9, 5, 699]), u, un, cu)
        assert [x.tolist() for x in got] == [[3], [0, 1, 2], [3]]
        got = blk.verify_drafts(one, ints([9, 5, 698]), u, un, cu)
        assert [x.tolist() for x in got] == [[2], [0, 1, -1], [699]]
        # a draft equal to the target is always accepted; a token that neither has leaves nothing: the target's own
        got = blk.verify_drafts(one, ints([9, 5, 4]), u, un, cu, None, one)
        assert [x.tolist() for x in got] == [[2], [0, 1, -1], [699]]
    # first values and last values of a flat distribution
    flat = torch.full((1, V), 1.0 / V, device=DEV)
    assert blk.verify_drafts(flat, ints([0]), zero, zero)[2].item() == 0
    assert blk.verify_drafts(flat, ints([0]), zero, top)[2].item() == V - 1
    tail = flat.clone()
    tail[0, 300:] = 0  # zeros behind are never drawn
    assert blk.verify_drafts(tail, ints([0]), zero, top)[2].item() == 299
    assert blk.last_status() == 0
    # bad tokens, parents and lists
    for tokens, parents in (([9, 5, V], [-1, 0, 1]), ([9, 5, -1], [-1, 0, 1]), ([9, 5, 699], [-1, 0, 2]), ([9, 5, 699], [-1, 0, 99])):
        got = blk.verify_drafts(one, ints(tokens), torch.zeros(3, device=DEV), zero, cu, ints(parents))
        assert blk.last_status() == 1 and [x.tolist() for x in got] == [[2], [0, 1, -1], [699]]
    for bad in ([0, 99], [2, 1], [-1, 3]):
        blk.verify_drafts(one, ints([9, 5, 699]), torch.zeros(3, device=DEV), zero, ints(bad))
        assert blk.last_status() == 1
    big = torch.full((65, 8), 0.125, device=DEV)
    got = blk.verify_drafts(big, torch.zeros(65, dtype=torch.int32, device=DEV), torch.zeros(65, device=DEV), zero, ints([0, 65]))
    assert blk.last_status() == 1 and got[0].tolist() == [0] and got[2].tolist() == [-1] and set(got[1].tolist()) == {-1}
    # probabilities that are no numbers: some token of the vocabulary, no fault
    nan = torch.full((3, V), float("nan"), device=DEV)
    got = blk.verify_drafts(nan, ints([9, 5, 699]), torch.zeros(3, device=DEV), zero, cu, None, nan)
    assert got[0].tolist() == [1] and 0 <= got[2].item() < V


def test_verified_tokens_are_the_targets():
    """The first token after the root is distributed as the target's row: counts of 65536 draws of 6 tokens are
    within 6 standard deviations, with and without the draft's probabilities, two candidates each."""
    B, V = 65536, 6
    g = torch.Generator(device=DEV).manual_seed(5)
    p = torch.tensor([0.4, 0.05, 0.25, 0.1, 0.0, 0.2], device=DEV)
    q = torch.tensor([0.1, 0.3, 0.25, 0.05, 0.2, 0.1], device=DEV)
    blk = block()
    target, draft = p.expand(3 * B, V).contiguous(), q.expand(3 * B, V).contiguous()
    cu, parents = ints(list(range(0, 3 * B + 1, 3))), ints([-1, 0, 0] * B)
    for given in (draft, None):
        if given is not None:
            tokens = torch.multinomial(q, 3 * B, replacement=True, generator=g).to(torch.int32)
        else:
            tokens = ints([0, 1, 2] * B)
        counts, path, nxt = blk.verify_drafts(target, tokens, torch.rand(3 * B, generator=g, device=DEV),
                                              torch.rand(B, generator=g, device=DEV), cu, parents, given)
        at = 3 * torch.arange(B, device=DEV) + path.view(B, 3)[:, 1].clamp(min=0)
        first = torch.where(counts > 1, tokens[at], nxt)
        seen = torch.bincount(first.long(), minlength=V).double().cpu()
        want = B * p.double().cpu()
        assert torch.all((seen - want).abs() <= 6 * (want * (1 - p.double().cpu())).sqrt()), (seen, want)


# ------------------------------------------------------------------ keep

@pytest.mark.parametrize("dtype,d,Hkv,page,layers", [("bf16", 128, 2, 16, 1), ("bf16", 128, 8, 64, 3), ("f32", 80, 3, 32, 2),
                                                    ("f32", 8, 1, 16, 2), ("bf16", 128, 1, 256, 70)])
def test_paged_keep(dtype, d, Hkv, page, layers):
    lens = [0, 15, 16, 100, 33, 7]
    rows = [64, 1, 40, 0, 64, 30]
    paths = [[0, 1, 2, 3, 40, 41, 63], [0], [0, 39], [], list(range(64)), [3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 28, 29]]
    blk = block(Hkv, Hkv, dtype, d)
    c = cache_of(blk, lens, rows, page)
    caches = [c] + [blk.paged_cache(0, 0, shared=c) for _ in range(layers - 1)]
    for i, x in enumerate(caches):
        fill(x, 100 + 2 * i, lens)
    before = [{x: t[x].clone() for x in "kv"} for t in caches]
    path = ints([y for p, t in zip(paths, rows) for y in p + [-1] * (t - len(p))])
    blk.paged_keep(caches, ints([len(p) for p in paths]), path, cu_of(rows))
    assert blk.last_status() == 0
    assert c["lens"].tolist() == [n + len(p) for n, p in zip(lens, paths)]
    for t, was in zip(caches, before):
        for x in "kv":
            want = dict(t, **{x: was[x].clone()})
            for b, (n, p) in enumerate(zip(lens, paths)):
                src = slots_of(dict(t, **was), x, b, n + rows[b])
                for j, y in enumerate(p):
                    s = n + j
                    want[x][c["pages"][b, s // page].long(), :, s % page] = src[n + y]
            assert torch.equal(t[x], want[x])


def test_paged_keep_lens_alone_and_refusals():
    blk = block(2, 2)
    c = cache_of(blk, [5, 10, 0], [20, 20, 20], 16)
    cap = c["pages"].shape[1] * 16
    fill(c, 1, None)
    k = c["k"].clone()
    blk.paged_keep([c], ints([3, 0, 7]))
    assert c["lens"].tolist() == [8, 10, 7] and blk.last_status() == 0
    blk.paged_keep([c], ints([2, 1, 1]), starts=ints([0, 4, 6]))
    assert c["lens"].tolist() == [2, 5, 7] and blk.last_status() == 0
    blk.paged_keep([c], ints([1, 1, 1]), starts=c["lens"])
    assert c["lens"].tolist() == [3, 6, 8]
    # what is not valid leaves its sequence as it was, the others go on
    for counts, code in (([-1, 1, 1], 1), ([cap, 1, 1], 4)):
        c["lens"].copy_(ints([3, 6, 8]))
        blk.paged_keep([c], ints(counts))
        assert blk.last_status() == code and c["lens"].tolist() == [3, 7, 9]
    cu = ints([0, 4, 8, 12])
    good = [0, 1, 2, 3]
    for path in ([0, 2, 1, 3], [0, 0, 1, 3], [1, 0, 2, 3], [0, 1, 4, 5], [-1, 1, 2, 3], [0, 1, 2, 2**31 - 1]):
        c["lens"].copy_(ints([3, 6, 8]))
        blk.paged_keep([c], ints([4, 4, 4]), ints(path + good + good), cu)
        assert blk.last_status() == 1 and c["lens"].tolist() == [3, 10, 12] and torch.equal(c["k"], k)
    c["lens"].copy_(ints([3, 6, 8]))
    blk.paged_keep([c], ints([5, 4, 4]), ints(good * 3), cu)  # more than its rows
    assert blk.last_status() == 1 and c["lens"].tolist() == [3, 10, 12]
    c["lens"].copy_(ints([3, 6, 8]))
    blk.paged_keep([c], ints([2, 2, 2]), ints(good * 3), ints([0, 4, 2, 12]))  # a list that falls
    assert blk.last_status() == 1 and c["lens"].tolist() == [5, 6, 10]
    # a page that is none: rows to or from it stay
    c["lens"].copy_(ints([3, 6, 8]))
    c["pages"][0, 0] = 10**6
    k = c["k"].clone()
    blk.paged_keep([c], ints([2, 2, 2]), ints([1, 3, -1, -1] + good + good), cu)
    assert blk.last_status() == 1 and torch.equal(c["k"], k)
    for bad in (dict(counts=c["lens"]), dict(counts=ints([1, 1, 1]), starts=c["lens"].repeat(2)[:3].clone(), path=c["lens"], cu_seqlens=ints([0, 1, 2, 3]))):
        with pytest.raises(BlkError, match="INVALID_ARG"):
            blk.paged_keep([c], **bad)
    with pytest.raises(BlkError, match="same k or v"):
        blk.paged_keep([c, dict(c)], ints([1, 1, 1]))
    with pytest.raises(BlkError, match="share"):
        blk.paged_keep([c, dict(blk.paged_cache(0, 0, shared=c), lens=c["lens"].clone())], ints([1, 1, 1]))


@pytest.mark.parametrize("layers", [1, 70])
def test_paged_keep_of_rows_that_pass_the_page_list(layers):
    """A sequence some of whose rows have no slot is left alone, whatever was kept of it: attention saw none of them."""
    blk = block(2, 2)
    c = blk.paged_cache(3, 32, 16)
    caches = [c] + [blk.paged_cache(0, 0, shared=c) for _ in range(layers - 1)]
    cu, rows = ints([0, 6, 12, 18]), [0, 3, 5, -1, -1, -1]
    for lens, path, count, code in ((27, rows, 2, 4), (27, rows, 3, 4), (30, rows, 1, 4), (31, rows, 0, 4), (27, rows, 7, 1),
                                    (26, rows, 3, 0)):
        for i, x in enumerate(caches):
            fill(x, 7 + 2 * i, None)
        c["lens"].copy_(ints([1, lens, 2]))
        before = [{x: t[x].clone() for x in "kv"} for t in caches]
        blk.paged_keep(caches, ints([3, count, 2]), ints(rows + path + rows), cu)
        assert blk.last_status() == code and c["lens"].tolist() == [4, lens + (count if code == 0 else 0), 4]
        for t, was in zip(caches, before):
            for x in "kv":
                same = torch.equal(slots_of(t, x, 1, 32), slots_of(dict(t, **was), x, 1, 32))
                assert same == (code != 0)
                assert torch.equal(slots_of(t, x, 0, 4)[1:], slots_of(dict(t, **was), x, 0, 7)[[1, 4, 6]])
                assert torch.equal(slots_of(t, x, 2, 4)[2:], slots_of(dict(t, **was), x, 2, 8)[[2, 5]])


@pytest.mark.parametrize("page", [-1, 10**6, 2**31 - 1])
def test_paged_keep_of_rows_whose_page_is_none(page):
    """Neither the rows nor lens of a sequence move if one of its kept rows comes from or goes to no page."""
    blk = block(2, 2)
    c = cache_of(blk, [14, 3, 20], [40, 20, 300], 16)
    cu = cu_of([40, 20, 300])
    whole = c["pages"].clone()
    long = [i + i // 2 for i in range(200)]  # more rows than are looked up at a time
    for b, at, path in ((0, 0, [0, 3, 9]),      # goes to
                        (0, 2, [0, 3, 9, 30]),  # comes from
                        (0, 1, [0, 1, 2, 3]),   # stays there
                        (2, 19, long), (2, 13, long)):
        paths = [[0, 1], [0, 2], [0, 4]]
        paths[b] = path
        fill(c, 5, None)
        c["lens"].copy_(ints([14, 3, 20]))
        c["pages"].copy_(whole)
        c["pages"][b, at] = page
        before = {x: c[x].clone() for x in "kv"}
        flat = [y for p, n in zip(paths, (40, 20, 300)) for y in p + [-1] * (n - len(p))]
        blk.paged_keep([c], ints([len(p) for p in paths]), ints(flat), cu)
        assert blk.last_status() == 1
        c["pages"].copy_(whole)
        for s, (n, t) in enumerate(zip((14, 3, 20), (40, 20, 300))):
            assert c["lens"][s].item() == (n if s == b else n + 2)
            for x in "kv":
                now, was = slots_of(c, x, s, n + t), slots_of(dict(c, **before), x, s, n + t)
                want = was.clone()
                if s != b:
                    want[n:n + 2] = was[[n + y for y in paths[s]]]
                assert torch.equal(now, want)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("page", [16, 64])
def test_a_run_of_steps_is_plain_decoding(page):
    """Prompts, then steps of drafted trees whose accepted path is kept: the slots are those of the same tokens
    appended one after the other (copies of rows that turned by the same positions), and so is a last query's
    attention."""
    H, Hkv, V = 8, 2, 50
    blk = block(H, Hkv, qk_norm=True)
    g = 1 + 0.1 * randn(1, D)
    # a token's q, k and v depend on the token alone here, as if the model were one layer without a residual
    qt, kt, vt = randn(2, V, H, D), randn(3, V, Hkv, D), randn(4, V, Hkv, D)
    prompts = [[7, 3, 9, 40, 2], [11], list(range(30))]
    cap = 128
    c = blk.paged_cache(3, cap, page)
    c["pages"].copy_(c["pages"][torch.arange(3, device=DEV).flip(0)])

    def append(cache, lists, depths=None, cu=None):
        t = torch.tensor([x for one in lists for x in one], device=DEV)
        return blk.paged_append(cache, qt[t], kt[t], vt[t], cu_of([len(x) for x in lists]), depths, g, g)

    append(c, prompts)
    blk.paged_keep([c], ints([len(x) for x in prompts]))
    history = [list(x) for x in prompts]
    r = np.random.default_rng(3)
    last = [1, 2, 3]
    gen = torch.Generator(device=DEV).manual_seed(9)
    for step in range(6):
        trees = [tree_of(int(r.integers(2, 12)), 10 * step + b) for b in range(3)]
        drafts = [[last[b]] + r.integers(0, V, len(t) - 1).tolist() for b, t in enumerate(trees)]
        rows = [len(t) for t in trees]
        n = sum(rows)
        cu, parents = cu_of(rows), ints([p for t in trees for p in t])
        qr = append(c, drafts, ints([int(x) for t in trees for x in kin_of(t)[1]]))
        lens = c["lens"].tolist()
        o = blk.attn_paged(qr, c, cu, parents)
        ks, vs = ([slots_of(c, x, b, lens[b] + rows[b]) for b in range(3)] for x in "kv")
        check_attn(o, qr, ks, vs, trees, lens)
        # many drafts are likely
        target = torch.full((n, V), 0.1 / V, device=DEV)
        at = 0
        for t, d in zip(trees, drafts):
            for x, p in enumerate(t):
                if p >= 0:
                    target[at + p, d[x]] += 0.5
            at += len(t)
        target /= target.sum(-1, keepdim=True)
        tokens = ints([x for d in drafts for x in d])
        u, un = torch.rand(n, generator=gen, device=DEV), torch.rand(3, generator=gen, device=DEV)
        counts, path, nxt = blk.verify_drafts(target, tokens, u, un, cu, parents)
        blk.paged_keep([c], counts, path, cu)
        at = 0
        for b in range(3):
            kept = path[at:at + counts[b]].tolist()
            history[b] += [drafts[b][x] for x in kept]
            last[b] = int(nxt[b])
            at += rows[b]
        assert c["lens"].tolist() == [len(x) for x in history]
    assert max(len(h) - len(p) for h, p in zip(history, prompts)) > 8
    plain = blk.paged_cache(3, cap, page)
    for i in range(max(map(len, history))):  # token by token
        lists = [[h[i]] if i < len(h) else [] for h in history]
        append(plain, lists)
        blk.paged_keep([plain], ints([len(x) for x in lists]))
    for b, h in enumerate(history):
        for x in "kv":
            assert torch.equal(slots_of(c, x, b, len(h)), slots_of(plain, x, b, len(h)))
    outs = [blk.attn_paged(append(x, [[t] for t in last]), x) for x in (c, plain)]
    assert torch.equal(*outs)
    assert blk.last_status() == 0


# ------------------------------------------------------------------ the model

# The bar of a bf16 block (max|err| / RMS <= 2e-2) over two layers whose errors are independent
TOL_MODEL_2 = TOL["bf16"] * np.sqrt(2)


def model_of(act="silu", qk_norm=False, vocab=1024, seed=31, max_seq=256, **kw):
    wl = Workload("paged_model", "bf16", 2, 8, 512, 8, 2, 128, 1000, act, qk_norm=qk_norm, seed=seed)
    layers, embed, norm_g, lm_head, _ = make_model(wl, n_layers=2, vocab=vocab)
    blk = DecoderBlock.from_workload(wl, max_seq=max_seq)
    dev = [to_dev(w) for w in layers], embed.to(DEV), norm_g.to(DEV), lm_head.to(DEV)

    def exact(tokens):
        return oracle.model_forward(cfg_of(wl), [weights_np(w) for w in layers], np64(embed), np64(norm_g), np64(lm_head),
                                    np.asarray([tokens]))[0]

    return blk, dev, exact


@pytest.mark.parametrize("act,qk_norm,page", [("silu", False, 64), ("xielu", True, 16)])
def test_model_over_a_paged_cache(act, qk_norm, page):
    blk, dev, exact = model_of(act, qk_norm)
    r = np.random.default_rng(1)
    prompts = [r.integers(0, 1024, n).tolist() for n in (5, 40)]
    c = cache_of(blk, [0, 0], [80, 80], page)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    got = blk.model_forward_paged(ints(sum(prompts, [])), *dev, caches, cu_of([5, 40]))
    assert rel_err(got, np.concatenate([exact(x) for x in prompts])) <= TOL_MODEL_2
    blk.paged_keep(caches, ints([5, 40]))
    trees = [tree_of(11, 1), tree_of(7, 2)]
    new = [r.integers(0, 1024, len(t)).tolist() for t in trees]
    cu, parents = cu_of([11, 7]), ints(sum(trees, []))
    depths = ints([int(x) for t in trees for x in kin_of(t)[1]])
    args = (ints(sum(new, [])), *dev, caches, cu, depths, parents)
    got = blk.model_forward_paged(*args)
    want = []
    for prompt, t, x in zip(prompts, trees, new):
        for i, kin in enumerate(kin_of(t)[0]):
            want.append(exact(prompt + [x[j] for j in np.nonzero(kin)[0]])[-1])
    assert rel_err(got, np.stack(want)) <= TOL_MODEL_2
    assert c["lens"].tolist() == [5, 40] and blk.last_status() == 0
    # a token each, without lists
    one = blk.model_forward_paged(ints([x[0] for x in new]), *dev, caches)
    assert rel_err(one, np.stack([exact(p + x[:1])[-1] for p, x in zip(prompts, new)])) <= TOL_MODEL_2
    # probabilities: the logits' softmax. Each exponent is off by at most (|x| + max|x|) / T of fp32's half steps
    # twice, the exponentials and their sum by a few more
    x = np64(got)
    for temperature in (1.0, 0.5, 3.0):
        p = np64(blk.model_forward_paged(*args, temperature=temperature))
        e = np.exp((x - x.max(-1, keepdims=True)) / temperature)
        bound = 2.0 ** -24 * (4 * np.abs(x).max() / temperature + 40)
        assert np.all(np.abs(p - e / e.sum(-1, keepdims=True)) <= bound * p)
    hot = blk.model_forward_paged(*args, temperature=0)
    assert torch.equal(hot.argmax(-1), got.float().argmax(-1)) and torch.equal(hot.sum(-1), torch.ones(18, device=DEV))
    assert torch.all((hot == 0) | (hot == 1)) and blk.last_status() == 0


@pytest.mark.parametrize("hidden,heads,kv,ffn,kw", [(384, 3, 3, 640, {}), (512, 8, 2, 1000, dict(sliding_window=33)),
                                                    (512, 4, 1, 1544, dict(use_rope=False)),
                                                    (640, 5, 1, 512, dict(rope_scaling=("yarn", 4.0, 256, 1.0, 32.0)))])
@pytest.mark.parametrize("chunks", [[1, 64, 65], [700], [129, 1, 300]])
def test_model_over_a_paged_cache_in_chunks(hidden, heads, kv, ffn, kw, chunks):
    """A prompt in chunks of one row to hundreds: the whole sequence's logits, whatever the block's options."""
    wl = Workload("paged_chunks", "bf16", 1, 8, hidden, heads, kv, 128, ffn, "relu2", seed=9, **kw)
    layers, embed, norm_g, lm_head, _ = make_model(wl, n_layers=2, vocab=512)
    blk = DecoderBlock.from_workload(wl, max_seq=1024)
    dev = [to_dev(w) for w in layers], embed.to(DEV), norm_g.to(DEV), lm_head.to(DEV)
    tokens = np.random.default_rng(3).integers(0, 512, sum(chunks))
    c = cache_of(blk, [0], [sum(chunks)], 32)
    caches, got = [c, blk.paged_cache(0, 0, shared=c)], []
    for n in chunks:
        at = int(c["lens"].item())
        got.append(blk.model_forward_paged(ints(tokens[at:at + n].tolist()), *dev, caches, cu_of([n])))
        blk.paged_keep(caches, ints([n]))
    assert blk.last_status() == 0 and c["lens"].item() == sum(chunks)
    want = oracle.model_forward(cfg_of(wl), [weights_np(w) for w in layers], np64(embed), np64(norm_g), np64(lm_head), tokens[None])[0]
    assert rel_err(torch.cat(got), want) <= TOL_MODEL_2


def test_probabilities_of_rows_with_ties_and_infinities():
    """One layer whose lm_head repeats rows: the first of equal logits; NaN rows stay NaN."""
    blk, (layers, embed, norm_g, lm_head), _ = model_of(vocab=64, seed=3)
    lm_head[32:] = lm_head[:32]
    c = cache_of(blk, [0, 0], [8, 8], 16)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    logits = blk.model_forward_paged(ints([1, 2, 3]), layers, embed, norm_g, lm_head, caches, ints([0, 1, 3]))
    hot = blk.model_forward_paged(ints([1, 2, 3]), layers, embed, norm_g, lm_head, caches, ints([0, 1, 3]), temperature=0)
    assert torch.equal(logits[:, :32], logits[:, 32:])
    assert hot.argmax(-1).tolist() == logits[:, :32].float().argmax(-1).tolist() and hot.sum().item() == 3
    # temperatures whose reciprocal is no fp32 number: the limits
    top = logits == logits.amax(-1, keepdim=True)
    cold = blk.model_forward_paged(ints([1, 2, 3]), layers, embed, norm_g, lm_head, caches, ints([0, 1, 3]), temperature=1e-40)
    assert torch.equal(cold, top.float() / top.sum(-1, keepdim=True))
    warm = blk.model_forward_paged(ints([1, 2, 3]), layers, embed, norm_g, lm_head, caches, ints([0, 1, 3]), temperature=float("inf"))
    assert torch.equal(warm, torch.full_like(warm, 1 / 64))
    embed[2] = float("nan")
    p = blk.model_forward_paged(ints([1, 2, 3]), layers, embed, norm_g, lm_head, caches, ints([0, 1, 3]), temperature=1)
    assert torch.isfinite(p[0]).all() and torch.isnan(p[1:]).all()  # the third row sees the second


def logits_of(values, seed=3):
    """A model whose logits in a row are c * values (bf16, as it gives them itself), c > 0 another one in each row: all rows
    of lm_head are multiples of one vector. Returns a call of it for n tokens and a temperature."""
    blk, (layers, _, norm_g, _), _ = model_of(vocab=64, seed=seed, max_seq=512)
    embed = randn(seed, len(values), norm_g.numel())
    lm_head = torch.zeros(len(values), embed.shape[1], dtype=torch.bfloat16, device=DEV)
    lm_head[:, 0] = values.to(DEV).bfloat16()  # 0 * y is 0 for all finite y

    def call(n, temperature):
        c = blk.paged_cache(1, n + 1, 256)
        caches = [c, blk.paged_cache(0, 0, shared=c)]
        return blk.model_forward_paged(1 + torch.arange(n, device=DEV, dtype=torch.int32) % (len(values) - 1), layers, embed, norm_g,
                                       lm_head, caches, ints([0, n]), temperature=temperature)

    return call, blk


def softmax_case(kind, vocab, seed):
    """What stands in lm_head's one column: the logits are multiples of it, of either sign."""
    g = torch.Generator().manual_seed(seed)
    if kind == "rising":  # the maximum moves in every chunk, or never
        return torch.linspace(-8, 8, vocab)
    x = torch.randn(vocab, generator=g)
    if kind == "equal":  # the largest many times in every stretch of a row
        x = x.clamp(-1, 1)
    elif kind == "minus inf":
        x[torch.rand(vocab, generator=g) < 0.5] = float("-inf")
    elif kind == "plus inf":
        x[vocab - 5] = float("inf")
    elif kind == "nan":
        x[vocab // 3] = float("nan")
    elif kind == "last":  # far above or below the others
        x[-1] = 30.0
    return x


@pytest.mark.parametrize("kind", ["normal", "rising", "equal", "minus inf", "plus inf", "nan", "last"])
@pytest.mark.parametrize("vocab,rows", [(4096, 1), (4104, 3), (8192, 1), (8200, 7), (12296, 40), (32000, 1), (32000, 64), (32000, 400),
                                        (50264, 100), (128256, 1), (128256, 64), (128256, 160)])
def test_probabilities_of_long_rows(kind, vocab, rows):
    """Rows of one to eight CTAs, with uneven ends and more chunks than are under way at a time, against fp64 on the same
    logits. u = 2^-24 (half a step of fp32), gap = (max - x) / T:
     - an exponent takes the roundings of the difference, of 1 / T log2(e) (two) and of the product: 4 u gap. Moving a
       sum to new maxima adds those of the parts that the gap is made of: 4 u gap of each term again, in the weighted mean;
     - ex2 is within 2 units in the last place, 4 u; a sum is moved at most once a chunk and in 16 joins, by an ex2 and a
       product, 5 u each; it has 8 additions a chunk and 16 joins, u each;
     - the result takes an ex2, a division and a product: 6 u."""
    call, blk = logits_of(softmax_case(kind, vocab, rows))
    x = call(rows, None).double()
    top = x.amax(-1, keepdim=True)  # NaN where one is
    u, chunks = 2.0 ** -24, -(-vocab // 8 // 512)  # a thread's, in a row of one CTA
    fine = top[:, 0].isfinite()
    assert kind in ("nan", "plus inf", "minus inf") or fine.all()
    for temperature in (1.0, 0.3):
        p = call(rows, temperature).double()
        assert p[~fine].isnan().all()
        gap = (top - x)[fine] / float(np.float32(temperature))
        e = torch.exp(-gap)
        want = e / e.sum(-1, keepdim=True)
        gap = torch.where(gap.isinf(), 0.0, gap)
        bound = u * (4 * gap + 4 * (want * gap).sum(-1, keepdim=True) + 5 * (chunks + 16) + 8 * chunks + 16 + 6)
        assert torch.all((p[fine] - want).abs() <= 1.01 * bound * want + 2.0 ** -140)
    best = torch.where(x.isnan(), -float("inf"), x)
    first = (best == best.amax(-1, keepdim=True)).to(torch.uint8).argmax(-1, keepdim=True)
    assert torch.all(torch.gather((best == best.amax(-1, keepdim=True)).to(torch.uint8).cumsum(-1), 1, first) == 1)  # the first
    assert torch.equal(call(rows, 0.0), torch.zeros(rows, vocab, device=DEV).scatter_(1, first, 1.0))
    assert blk.last_status() == 0


@pytest.mark.parametrize("vocab", [8, 1024, 4104, 32000])
def test_greedy_rows_without_a_number_above_minus_infinity(vocab):
    inf, nan = float("inf"), float("nan")
    call, _ = logits_of(torch.full((vocab,), inf))
    logits, hot = call(64, None), call(64, 0.0)
    low = (logits == -inf).all(-1)
    assert 0 < low.sum() < 64 and ((logits == inf).all(-1) == ~low).all()  # all of one sign in each row
    assert torch.equal(hot, torch.eye(vocab, device=DEV)[0].expand(64, vocab))  # the first of equal ones
    for at in (0, vocab // 2, vocab - 1):
        values = torch.full((vocab,), inf)
        values[at] = nan
        hot = logits_of(values)[0](64, 0.0)
        assert torch.isnan(hot[low]).all()
        first = 1 if at == 0 else 0
        assert torch.equal(hot[~low], torch.eye(vocab, device=DEV)[first].expand(int((~low).sum()), vocab))
    assert torch.isnan(logits_of(torch.full((vocab,), nan))[0](3, 0.0)).all()


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_model_steps_of_drafts(temperature):
    """Prompts, then steps of model_verify. Without a temperature every new token is the target's largest, to the
    error of its logits; with one it has a probability. The cache is that of the tokens that were kept."""
    blk, dev, exact = model_of(seed=5)
    r = np.random.default_rng(2)
    history = [r.integers(0, 1024, n).tolist() for n in (9, 33)]
    c = cache_of(blk, [0, 0], [120, 120], 16)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    p = blk.model_forward_paged(ints(sum(history, [])), *dev, caches, cu_of([9, 33]), temperature=temperature)
    blk.paged_keep(caches, ints([9, 33]))
    last = p[[8, 41]].argmax(-1).tolist()
    start = [len(h) for h in history]
    gen, kept = torch.Generator(device=DEV).manual_seed(1), 0
    for step in range(5):
        # drafts: a chain of the oracle's own greedy tokens, beside others
        drafts, trees = [], []
        for h, x in zip(history, last):
            chain_tokens, seq = [x], h + [x]
            for _ in range(3):
                chain_tokens.append(int(exact(seq)[-1].argmax()))
                seq = seq + chain_tokens[-1:]
            drafts.append([chain_tokens[0], 17, chain_tokens[1], chain_tokens[2], 4, chain_tokens[3]])
            trees.append([-1, 0, 0, 2, 2, 3])
        cu = cu_of([6, 6])
        depths = ints([int(x) for t in trees for x in kin_of(t)[1]])
        counts, path, nxt = blk.model_verify(ints(sum(drafts, [])), *dev, caches, torch.rand(12, generator=gen, device=DEV),
                                             torch.rand(2, generator=gen, device=DEV), cu, depths, ints(sum(trees, [])),
                                             temperature=temperature)
        for b in range(2):
            n = int(counts[b])
            history[b] += [drafts[b][x] for x in path[6 * b:6 * b + n].tolist()]
            kept += n
            last[b] = int(nxt[b])
        assert c["lens"].tolist() == [len(h) for h in history]
    assert blk.last_status() == 0
    if temperature == 0:
        assert kept > 2 * 5 + 10  # most drafts stay
        for h, x, n in zip(history, last, start):
            logits = exact(h + [x])
            rms = np.sqrt(np.mean(logits ** 2))
            for i in range(n, len(h)):
                assert logits[i - 1].max() - logits[i - 1][h[i]] <= 2 * TOL_MODEL_2 * rms
    # the next row over the cache of the steps is that of the whole sequence
    got = blk.model_forward_paged(ints(last), *dev, caches)
    assert rel_err(got, np.stack([exact(h + [x])[-1] for h, x in zip(history, last)])) <= TOL_MODEL_2


def test_model_steps_captured():
    """A whole step in a graph, replayed from other lengths and tokens than it was captured with, beside an eager one."""
    blk, dev, _ = model_of(seed=6)
    r = np.random.default_rng(5)
    c = cache_of(blk, [0, 0], [200, 200], 16)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    blk.model_forward_paged(ints(r.integers(0, 1024, 97).tolist()), *dev, caches, cu_of([40, 57]))
    blk.paged_keep(caches, ints([40, 57]))
    start = [{k: v.clone() for k, v in x.items()} for x in caches]
    trees = [tree_of(9, 3), tree_of(5, 4)]
    cu, parents = cu_of([9, 5]), ints(sum(trees, []))
    depths = ints([int(x) for t in trees for x in kin_of(t)[1]])
    steps = [(ints(r.integers(0, 1024, 14).tolist()), torch.rand(14, device=DEV) * 0.02, torch.rand(2, device=DEV)) for _ in range(3)]

    def eager():
        mine = [dict(start[0], k=start[0]["k"].clone(), v=start[0]["v"].clone(), lens=start[0]["lens"].clone())]
        mine.append(dict(mine[0], k=start[1]["k"].clone(), v=start[1]["v"].clone()))
        return [[x.clone() for x in blk.model_verify(t, *dev, mine, u, un, cu, depths, parents, temperature=0.7)] for t, u, un in steps], mine

    want, kept = eager()
    tok, u, un = (x.clone() for x in steps[0])
    blk.model_verify(tok, *dev, caches, u, un, cu, depths, parents, temperature=0.7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = blk.model_verify(tok, *dev, caches, u, un, cu, depths, parents, temperature=0.7)
    for x, y in zip(caches, start):
        x["k"].copy_(y["k"])
        x["v"].copy_(y["v"])
    c["lens"].copy_(start[0]["lens"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        beside, _ = eager()
    for step, w in zip(steps, want):
        for x, y in zip((tok, u, un), step):
            x.copy_(y)
        g.replay()
        for x, y in zip(out, w):
            assert torch.equal(x, y)
    torch.cuda.synchronize()
    for a, b in zip(beside, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for x, y in zip(caches, kept):
        assert all(torch.equal(x[k], y[k]) for k in ("k", "v", "lens"))
    assert blk.last_status() == 0


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("room", [2, 5])
def test_model_verify_at_the_end_of_a_page_list(kind, room):
    """One of three sequences has no room for all of its rows: it is left as it is, the others' steps are those of a
    cache where it fits, and what memory held before reaches nothing."""
    blk, dev, _ = model_of(seed=12)
    r = np.random.default_rng(8)
    tree = chain(6) if kind == "chain" else [-1, 0, 0, 1, 1, 2]
    tokens, new = r.integers(0, 1024, 120).tolist(), ints(r.integers(0, 1024, 18).tolist())
    cu, parents = cu_of([6] * 3), ints(tree * 3) if kind == "tree" else None
    depths = ints(kin_of(tree)[1].tolist() * 3) if kind == "tree" else None
    u, un = torch.zeros(18, device=DEV), torch.tensor([0.1, 0.5, 0.9], device=DEV)  # drafts are accepted

    def step(cap, left, garbage):
        c = blk.paged_cache(3, cap, 16)
        caches = [c, blk.paged_cache(0, 0, shared=c)]
        blk.model_forward_paged(ints(tokens), *dev, caches, cu_of([40] * 3))
        blk.paged_keep(caches, ints([40] * 3))
        c["lens"][1] = cap - left if left else 40
        n = blk.model_verify(new, *dev, caches, u, un, cu, depths, parents, temperature=0.7)[0].numel()
        assert blk.last_status() == (4 if left else 0) and n == 3
        # ... and again in memory that holds something else
        for x in caches:
            x["lens"].copy_(ints([40, cap - left if left else 40, 40]))
        nbytes = lib().blk_model_paged_workspace_bytes(blk.handle, 18, 1, parents is not None, 3, blk._paged(c)[0], 1024, 1)
        junk = [torch.full((nbytes // 4,), garbage, device=DEV) for _ in range(8)]
        del junk  # the model's workspace is one of these
        p = blk.model_forward_paged(new, *dev, caches, cu, depths, parents, temperature=0.7)
        out = blk.model_verify(new, *dev, caches, u, un, cu, depths, parents, temperature=0.7)
        assert blk.last_status() == (4 if left else 0)
        return caches, p, out

    whole, p0, (n0, path0, t0) = step(64, 0, 1.0)
    first = None
    for garbage in (3e38, float("nan"), -1.0):
        caches, p, (n, path, t) = step(64, room, garbage)
        assert torch.isfinite(p).all()
        if first is None:
            first = p
        assert torch.equal(p, first)
        for b in (0, 2):
            rows = slice(6 * b, 6 * b + 6)
            assert torch.equal(p[rows], p0[rows]) and torch.equal(path[rows], path0[rows])
            assert n[b] == n0[b] and t[b] == t0[b]
            for x, y in zip(caches, whole):
                for z in "kv":
                    m = 40 + int(n[b])
                    assert torch.equal(slots_of(x, z, b, m), slots_of(y, z, b, m))
        assert caches[0]["lens"].tolist() == [40 + int(n[0]), 64 - room, 40 + int(n[2])]


@pytest.mark.parametrize("vocab", [1024, 4104])
@pytest.mark.parametrize("temperature", [None, 0.0, 1.0])
def test_model_rows_of_no_sequence(vocab, temperature):
    """A padded batch: out is left as it was before the first and behind the last sequence, whatever stands there for
    tokens, and the status word says nothing of them."""
    blk, dev, _ = model_of(vocab=vocab, seed=14)
    r = np.random.default_rng(2)
    rows, first, behind = [3, 0, 5, 130], 4, 150
    n = first + sum(rows) + behind
    tokens = r.integers(0, vocab, sum(rows)).tolist()
    c = blk.paged_cache(4, 160, 16)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    dtype = torch.bfloat16 if temperature is None else torch.float32
    plain = blk.model_forward_paged(ints(tokens), *dev, caches, cu_of(rows), temperature=temperature)
    want = blk.model_forward_paged(ints([0] * first + tokens + [0] * behind), *dev, caches, cu_of(rows, first), temperature=temperature)
    want = want[first:n - behind]
    if temperature is None:  # keys may be cut elsewhere for another number of rows
        assert rel_err(want, np64(plain)) <= 2 * TOL_MODEL_2
    out = torch.full((n, vocab), 7.0, dtype=dtype, device=DEV)
    padded = ints([-1] * first + tokens + [2**31 - 1, -1, 5] * (behind // 3))
    got = blk.model_forward_paged(padded, *dev, caches, cu_of(rows, first), temperature=temperature, out=out)
    assert blk.last_status() == 0 and got is out
    assert torch.equal(out[first:n - behind], want)
    assert torch.all(out[:first] == 7) and torch.all(out[n - behind:] == 7)
    # a token of a sequence that is none is still said
    padded[first] = -1
    blk.model_forward_paged(padded, *dev, caches, cu_of(rows, first), temperature=temperature, out=out)
    assert blk.last_status() == 1


def test_model_over_a_paged_cache_refusals():
    blk, dev, _ = model_of()
    c = blk.paged_cache(2, 32, 16)
    caches = [c, blk.paged_cache(0, 0, shared=c)]
    tok = ints([1, 2])
    blk.model_forward_paged(tok, *dev, caches)
    for kw, match in ((dict(caches=caches[:1]), "each layer"), (dict(caches=[c, blk.paged_cache(2, 32, 16)]), "share"),
                      (dict(caches=[c, c]), "same k or v"),
                      (dict(parents=ints([-1, -1])), "depths"), (dict(temperature=-1.0), "temperature"),
                      (dict(temperature=float("nan")), "temperature"), (dict(tokens=tok.long()), "tokens"),
                      (dict(tokens=tok[:1]), "row per sequence"), (dict(host_lens_max=33), "CACHE_FULL"),
                      (dict(out=torch.empty(2, 1024, device=DEV)), "out")):
        with pytest.raises((BlkError, ValueError), match=match):
            blk.model_forward_paged(**{**dict(tokens=tok, layers=dev[0], embed=dev[1], norm_g=dev[2], lm_head=dev[3], caches=caches), **kw})
    for kw in (dict(attn_gate=True), dict(dtype="f32", d=64)):
        other = block(4, 2, **kw)
        cc = other.paged_cache(1, 32, 16)
        w = torch.zeros(8, other.desc.hidden, dtype=cc["k"].dtype, device=DEV)
        with pytest.raises(BlkError, match="UNSUPPORTED"):
            other.model_forward_paged(ints([1]), [dict()], w, w[0].contiguous(), w, [cc])
    assert blk.last_status() == 0
    blk.model_forward_paged(ints([1, 5000]), *dev, caches)
    assert blk.last_status() == 1
    assert torch.isfinite(blk.model_forward_paged(tok, *dev, caches)).all()


# ------------------------------------------------------------------ refusals

def test_refusals():
    blk, f32 = block(4, 2, qk_norm=True), block(4, 2, "f32", 64)
    c = blk.paged_cache(2, 64, 16)
    q, k, v, g = randn(1, 2, 4, D), randn(2, 2, 2, D), randn(3, 2, 2, D), randn(4, D)
    ok = dict(cache=c, q=q, k=k, v=v, q_gain=g, k_gain=g)
    blk.paged_append(**ok)

    def refused(match, error=ValueError, **kw):
        with pytest.raises(error, match=match):
            blk.paged_append(**{**ok, **kw})

    refused("q_gain", q_gain=None)
    refused("bfloat16", q=q.float())
    refused("bfloat16", v=v[:1])
    refused("int32", depths=ints([1, 2, 3]))
    refused("int32", cu_seqlens=torch.tensor([0, 1, 2], device=DEV))
    refused("contiguous", q=randn(1, 2, 4, 2 * D)[..., ::2])
    refused("cache lens", cache=dict(c, lens=ints([0])))
    refused("cache v", cache=dict(c, v=c["v"][:-1]))
    refused("rope_table", rope_table=torch.zeros(4, 64, device=DEV))
    refused("row per sequence", BlkError, q=q[:1], k=k[:1], v=v[:1])
    refused("INVALID_ARG", BlkError, rope_table=torch.zeros(8, 65, 2, device=DEV))  # 130 channels
    refused("UNSUPPORTED", BlkError, rope_table=torch.zeros(8, 12, 2, device=DEV))  # 24 channels: not 16-byte chunks
    refused("INVALID_ARG", BlkError, q_out=q[:1].expand(2, 4, D))  # rows that overlap
    refused("page_size", BlkError, cache=blk.paged_cache(2, 64, 8))
    refused("page_size", BlkError, cache=blk.paged_cache(2, 96, 48))
    refused("ALIGNMENT", BlkError, q=randn(1, 2 * 4 * D + 4)[4:].view(2, 4, D))
    kk = c["k"].view(-1, 2, D)[:2]
    refused("INVALID_ARG", BlkError, k=kk)  # the cache itself
    refused("INVALID_ARG", BlkError, cache=dict(c, v=c["k"]))
    with pytest.raises(BlkError, match="UNSUPPORTED"):
        f32.attn_paged(randn(1, 2, 4, 64, dtype=torch.float32), f32.paged_cache(2, 64, 16))
    with pytest.raises(BlkError, match="UNSUPPORTED"):
        block(4, 2, use_rope=False).rope_table()
    for dims in (0, 63, 130):
        with pytest.raises((BlkError, ValueError)):
            blk.rope_table(dims)
    out = torch.empty_like(q)
    blk.attn_paged(q, c, out=out)
    for kw, match in ((dict(out=q), "INVALID_ARG"), (dict(q=q[:1]), "row per sequence"), (dict(q=q.float()), "bfloat16"),
                      (dict(parents=ints([0])), "parents"), (dict(cu_seqlens=ints([0, 2])), "cu_seqlens")):
        with pytest.raises((BlkError, ValueError), match=match):
            blk.attn_paged(**{**dict(q=q, cache=c), **kw})
    t, tok, u = torch.full((2, 10), 0.1, device=DEV), ints([1, 2]), torch.rand(2, device=DEV)
    args = dict(target=t, tokens=tok, u=u, u_next=u)
    blk.verify_drafts(**args)
    for kw, match in ((dict(target=t.bfloat16()), "target"), (dict(draft=t[:, :9]), "draft"), (dict(tokens=None), "tokens"),
                      (dict(tokens=tok.long()), "tokens"), (dict(u_next=u[:1]), "row per sequence"), (dict(u=u[:1]), "u:"),
                      (dict(target=t.t().contiguous().t()), "contiguous"), (dict(parents=ints([0, 0, 0])), "parents"),
                      (dict(target=t[:, :0]), "vocab"), (dict(target=t[:1].expand(2, 10)), "strides")):
        with pytest.raises((BlkError, ValueError), match=match):
            blk.verify_drafts(**{**args, **kw})
    for kw, match in ((dict(counts=ints([1])), "counts"), (dict(counts=None), "counts"), (dict(caches=[]), "one at least"),
                      (dict(path=ints([0, 0]), cu_seqlens=ints([0, 2])), "cu_seqlens"), (dict(path=ints([0, 0, 0])), "row per sequence")):
        with pytest.raises((BlkError, ValueError), match=match):
            blk.paged_keep(**{**dict(caches=[c], counts=ints([1, 1])), **kw})
    assert blk.last_status() == 0

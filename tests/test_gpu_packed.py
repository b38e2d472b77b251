"""Packed, mixed-length batches: per-head q/k norm with the rotary of several position
axes (blk_qk_norm_rope), causal attention over packed prompts (blk_attn_packed), the
4-bit KV cache (blk_kv4_store, blk_kv4_load) and decode attention over it
(blk_attn_decode_kv4), against fp64 references.

Bounds count roundings. bf16 rounds by at most u = 2^-8 of the value (half a step), fp32 by
2^-24:
 - rotary: the fp32 chain (a sum of up to 256 squares over lanes, rsqrt to 2 ulp, two gain
   products, the rotation's two products and sum, cos and sin rounded to fp32) stays under
   20 * 2^-24 (|a| + |b|) of a pair (a, b); a bf16 result adds u |out|.
 - packed attention: p is rounded to bf16 before the product with v (its sum is not), the
   output once: u sum(p |v|) + u |o|. Scores are sums of 128 exact products in fp32, off by at
   most 128 * 2^-23 sum|q k| / sqrt(128); exp adds 2^-22. Both under 2e-4 of sum(p |v|) at
   these inputs.
 - decode over 4 bits: p is rounded to bf16 for all terms of a value (u |value|), p * scale goes
   in as two bf16 numbers (u^2 scale |code - 8|), the output is rounded once; a score is a sum of exact products
   (of a group's sum of q in 24 bits with its offset) in fp32, off by at most
   2^-21 sum|q| (15 scale + |offset|) / sqrt(128).
"""
import numpy as np
import pytest
import torch

import oracle
from llama_family_decoder_gb300 import BlkError, DecoderBlock
from tests.helpers import np64

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


def cu_of(lens, first=0):
    return ints(np.concatenate([[first], first + np.cumsum(lens)]).tolist())


# ------------------------------------------------------------------ norm and rotary

def axis_of_pair(half, sections, interleaved):
    if sections is None:
        return np.zeros(half, int)
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    return np.array([i % n if i < n * sections[i % n] else 0 for i in range(half)])


def rope_ref(x, pos, gain, eps, theta, sections, interleaved, scaling=None):
    """x [N, heads, d], pos [axes, N] -> (rotated, |a| + |b| of each pair, per element)."""
    y = np64(x)
    if gain is not None:
        y = oracle.rms_norm(y, np64(gain), eps)
    d = y.shape[-1]
    half = d // 2
    freq = oracle.rope_inv_freq(d, theta, scaling)
    ang = np.asarray(pos, np.float64)[axis_of_pair(half, sections, interleaved)].T * freq  # [N, half]
    m = oracle.rope_attention_factor(scaling)
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    a, b = y[..., :half], y[..., half:]
    size = np.abs(a) + np.abs(b)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), np.concatenate([size, size], -1)


def check_rope(got, x, pos, gain, sections=None, interleaved=False, theta=10000.0, scaling=None):
    ref, size = rope_ref(x, pos, gain, 1e-5, theta, sections, interleaved, scaling)
    bound = 20 * 2.0 ** -24 * 1.5 * size + (U * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(np64(got) - ref) <= bound)


@pytest.mark.parametrize("n", [1, 3, 64, 257, 2000])
@pytest.mark.parametrize("H,Hkv,dtype,d,norm", [(32, 8, "bf16", 128, True), (5, 1, "bf16", 128, False),
                                               (4, 2, "f32", 64, True), (3, 3, "f32", 80, True),
                                               (6, 2, "f32", 8, False), (2, 1, "f32", 256, True)])
@pytest.mark.parametrize("sections,interleaved", [(None, False), ("thirds", False), ("thirds", True), ("four", True),
                                                  ("empty", False)])
def test_qk_norm_rope(n, H, Hkv, dtype, d, norm, sections, interleaved):
    half = d // 2
    side = half // 3
    sections = {None: None, "thirds": [half - 2 * side, side, side], "empty": [0, half, 0],
                "four": [half - 3 * (half // 4), half // 4, half // 4, half // 4]}[sections]
    blk = block(H, Hkv, dtype, d, qk_norm=norm)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q, k = randn(1, n, H, d, dtype=dt), randn(2, n, Hkv, d, dtype=dt)
    q[0] *= 1e4
    k[0] *= 1e-4
    gq, gk = 1 + 0.2 * randn(3, d, dtype=dt), 1 + 0.2 * randn(4, d, dtype=dt)
    axes = len(sections) if sections else 1
    pos = torch.randint(0, 4096, (axes, n), device=DEV, dtype=torch.int32)
    pos[:, -1] = 4095
    qo, ko = blk.qk_norm_rope(q, k, pos if sections else pos[0], gq, gk, sections=sections, interleaved=interleaved)
    p = pos.cpu().numpy()
    check_rope(qo, q, p, gq if norm else None, sections, interleaved)
    check_rope(ko, k, p, gk if norm else None, sections, interleaved)
    assert blk.last_status() == 0


@pytest.mark.parametrize("scaling", [("yarn", 20.0, 4096, 1.0, 32.0), ("llama3", 8.0, 8192, 1.0, 4.0)])
def test_qk_norm_rope_stretched(scaling):
    blk = block(4, 2, max_seq=9000, rope_scaling=scaling, rope_theta=5e5)
    q, k = randn(1, 100, 4, D), randn(2, 100, 2, D)
    pos = torch.randint(0, 9000, (100,), device=DEV, dtype=torch.int32)
    qo, ko = blk.qk_norm_rope(q, k, pos)
    sc = oracle.RopeScaling(*scaling)
    check_rope(qo, q, pos[None].cpu().numpy(), None, theta=5e5, scaling=sc)
    check_rope(ko, k, pos[None].cpu().numpy(), None, theta=5e5, scaling=sc)


def test_qk_norm_rope_layouts_and_in_place():
    H, Hkv, n = 6, 2, 77
    blk = block(H, Hkv, qk_norm=True)
    g = 1 + 0.1 * randn(3, D)
    pos = torch.randint(0, 4096, (n,), device=DEV, dtype=torch.int32)
    q, k = randn(1, n, H, D), randn(2, n, Hkv, D)
    want = blk.qk_norm_rope(q, k, pos, g, g)
    # columns of fused rows, head-major rows, a row broadcast over the heads; outputs into strided views
    fused = torch.cat([q, k, k], 1).reshape(n, -1).contiguous().view(n, H + 2 * Hkv, D)
    hm = q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((H + Hkv, n, D), 7.0, dtype=torch.bfloat16, device=DEV)
    a = blk.qk_norm_rope(fused[:, :H], fused[:, H:H + Hkv], pos, g, g, q_out=out[:H].transpose(0, 1),
                         k_out=out[H:].transpose(0, 1))
    b = blk.qk_norm_rope(hm, k, pos, g, g)
    c = blk.qk_norm_rope(q, q[:, :1].expand(n, Hkv, D), pos, g, g)
    for x in (a, b):
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    assert torch.equal(c[1][:, 0], want[0][:, 0]) and torch.equal(c[1][:, 1], want[0][:, 0])
    q2, k2 = fused[:, :H], fused[:, H:H + Hkv]
    blk.qk_norm_rope(q2, k2, pos, g, g, q_out=q2, k_out=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(fused[:, H + Hkv:], k)  # the values beside them are untouched


def test_qk_norm_rope_matches_the_projection_stage():
    """One sequence: the same numbers as the rotary fused into the Q/K/V projections, from plain
    projections of the same rows (blk_qkv_rope of a no_rope handle) - up to the bf16 rounding
    of those projections: u |x| in, u |out| out, against one rounding of the fused stage."""
    from llama_family_decoder_gb300.synth import Workload, make_weights
    wl = Workload("t", "bf16", 1, 200, 1024, 8, 2, 128, 256, "relu2", seed=3)
    w = {k: v.to(DEV) for k, v in make_weights(wl).items()}
    y = randn(5, 200, 1024)
    outs = []
    for kw in (dict(), dict(use_rope=False)):
        b = DecoderBlock.from_workload(wl.scaled(**kw))
        q, k, v = (torch.empty(1, n, 200, D, dtype=torch.bfloat16, device=DEV) for n in (8, 2, 2))
        b.qkv_rope(y, w, 1, 200, q, k, v)
        outs.append((q[0].transpose(0, 1), k[0].transpose(0, 1)))
    b = DecoderBlock.from_workload(wl)
    got = b.qk_norm_rope(*outs[1], ints(list(range(200))))
    for g, fused, plain in zip(got, outs[0], outs[1]):
        size = np.abs(np64(plain))
        size = np.concatenate([size[..., :64] + size[..., 64:]] * 2, -1)
        assert np.all(np.abs(np64(g) - np64(fused)) <= 3.2 * U * size)


def test_qk_norm_rope_positions_outside_the_table():
    blk = block(4, 2, max_seq=64)
    q, k = randn(1, 3, 4, D), randn(2, 3, 2, D)
    qo, _ = blk.qk_norm_rope(q, k, ints([5, 64, -1]))
    assert blk.last_status() == 1
    check_rope(qo, q, np.array([[5, 63, 0]]), None)  # clamped
    assert blk.last_status() == 0
    blk.qk_norm_rope(q[:0], k[:0], ints([]))
    assert blk.last_status() == 0


def test_norm_without_rotary():
    blk = block(4, 2, qk_norm=True, use_rope=False)
    q, k, g = randn(1, 9, 4, D), randn(2, 9, 2, D), 1 + 0.1 * randn(3, D)
    qo, ko = blk.qk_norm_rope(q, k, None, g, g)
    check_rope(qo, q, np.zeros((1, 9)), g)
    check_rope(ko, k, np.zeros((1, 9)), g)


# ------------------------------------------------------------------ packed attention

def attn_ref(q, k, v, window=0):
    """One sequence: q [n, H, d], k, v [n, Hkv, d] in fp64 -> (o, sum p |v|)."""
    n, H, d = q.shape
    per = H // k.shape[1]
    i = np.arange(n)
    seen = i[None, :] <= i[:, None]
    if window:
        seen &= i[None, :] > i[:, None] - window
    o, mag = np.empty_like(q), np.empty_like(q)
    for h in range(H):
        s = q[:, h] @ k[:, h // per].T / np.sqrt(d)
        s = np.where(seen, s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        o[:, h], mag[:, h] = p @ v[:, h // per], p @ np.abs(v[:, h // per])
    return o, mag


def check_packed(out, q, k, v, lens, first=0, window=0):
    at = first
    for n in lens:
        if n:
            sl = slice(at, at + n)
            ref, mag = attn_ref(np64(q[sl]), np64(k[sl]), np64(v[sl]), window)
            err = np.abs(np64(out[sl]) - ref)
            assert np.all(err <= (U + 2e-4) * mag + U * np.abs(ref)), (n, float((err / mag).max()))
        at += n


LENS = [[1], [2], [127], [128], [129], [255, 1, 0, 257, 3], [0, 0, 5], [1] * 40, [64] * 9 + [300], [700, 30, 513]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,Hkv", [(8, 2), (3, 3), (3, 1), (16, 1), (2, 2)])
def test_attn_packed(lens, H, Hkv):
    n = sum(lens)
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    out = blk.attn_packed(q, k, v, cu_of(lens))
    assert blk.last_status() == 0
    check_packed(out, q, k, v, lens)


@pytest.mark.parametrize("lens", [[1] * 3000, [0] * 2500 + [300, 5] + [0] * 10, [3] * 700 + [140] * 20, [600] * 40,
                                  [1] * 9000, [0] * 8180 + [300, 5, 64, 1] + [0] * 8, [0] * 8180 + [300, 5, 64, 1] + [0] * 9])
def test_attn_packed_many_sequences(lens):
    """Batches whose work list a kernel of its own makes, and some near that border."""
    n, H, Hkv = sum(lens), 4, 1
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    out = blk.attn_packed(q, k, v, cu_of(lens))
    assert blk.last_status() == 0
    check_packed(out, q, k, v, lens)


@pytest.mark.parametrize("window", [1, 5, 128, 200, 5000])
def test_attn_packed_window(window):
    lens = [300, 1, 129, 520]
    blk = block(6, 2, sliding_window=window)
    q, k, v = randn(1, sum(lens), 6, D), randn(2, sum(lens), 2, D), randn(3, sum(lens), 2, D)
    check_packed(blk.attn_packed(q, k, v, cu_of(lens)), q, k, v, lens, window=window)


def test_attn_packed_other_rows_neither_read_nor_written():
    """Rows before the first, behind the last and of other sequences may hold anything."""
    lens, first, n = [100, 37, 260], 70, 900
    blk = block(4, 2)
    q, k, v = randn(1, n, 4, D), randn(2, n, 2, D), randn(3, n, 2, D)
    clean = blk.attn_packed(q, k, v, cu_of(lens, first))
    out = torch.full((n, 4, D), 3.0, dtype=torch.bfloat16, device=DEV)
    for x in (q, k, v):
        x[:first] = float("nan")
        x[first + sum(lens):] = float("inf")
    blk.attn_packed(q, k, v, cu_of(lens, first), out=out)
    mine = slice(first, first + sum(lens))
    assert torch.equal(out[mine], clean[mine])
    assert torch.all(out[:first] == 3) and torch.all(out[mine.stop:] == 3)
    check_packed(out, q, k, v, lens, first)
    # a whole sequence of NaN between two others
    k[170:207] = float("nan")
    v[170:207] = float("nan")
    q[170:207] = float("-inf")
    again = blk.attn_packed(q, k, v, cu_of(lens, first))
    assert torch.equal(again[70:170], clean[70:170]) and torch.equal(again[207:467], clean[207:467])


def test_attn_packed_layouts():
    lens, H, Hkv = [140, 9, 300], 4, 2
    n = sum(lens)
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    want = blk.attn_packed(q, k, v, cu_of(lens))
    fused = torch.cat([q, k, v], 1).contiguous()
    out = torch.zeros(H, n, D, dtype=torch.bfloat16, device=DEV)
    hm = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    a = blk.attn_packed(fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:], cu_of(lens), out=out.transpose(0, 1))
    b = blk.attn_packed(*hm, cu_of(lens))
    assert torch.equal(a, want) and torch.equal(b, want)


def test_attn_packed_one_sequence_is_the_prefill_stage():
    """With enough query tiles to fill the GPU the keys of a tile are not split, and every row
    goes through the same products in the same order as in the prefill stage."""
    n, H, Hkv = 4000, 32, 8
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    o = torch.empty(1, n, H, D, dtype=torch.bfloat16, device=DEV)
    blk.attn_gqa(*[x.transpose(0, 1).contiguous()[None] for x in (q, k, v)], o)
    assert torch.equal(blk.attn_packed(q, k, v, ints([0, n])), o[0])


@pytest.mark.parametrize("H,Hkv,window", [(32, 8, 0), (16, 16, 0), (12, 2, 0), (32, 2, 300), (20, 4, 0), (16, 1, 0)])
def test_attn_packed_many_tiles(H, Hkv, window):
    """Batches large enough for two query tiles an item (keys not split), ragged and with single tokens."""
    lens = [1400, 1, 700, 0, 129, 2, 1, 900, 333, 1, 64]
    n = sum(lens)
    blk = block(H, Hkv, sliding_window=window)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    check_packed(blk.attn_packed(q, k, v, cu_of(lens)), q, k, v, lens, window=window)
    assert blk.last_status() == 0


def test_attn_packed_bad_sequences_are_clamped():
    n = 200
    blk = block(4, 2)
    q, k, v = randn(1, n, 4, D), randn(2, n, 2, D), randn(3, n, 2, D)
    out = blk.attn_packed(q, k, v, ints([0, 60, 500]))
    assert blk.last_status() == 1
    check_packed(out, q, k, v, [60, 140])
    out = torch.zeros(n, 4, D, dtype=torch.bfloat16, device=DEV)
    blk.attn_packed(q, k, v, ints([0, 200, 0, 200, 0, 200, 0, 200]), out=out)  # more work than the rows give room for
    assert blk.last_status() == 1
    blk.attn_packed(q, k, v, ints([-5, -1, 50]), out=out)
    assert blk.last_status() == 1
    assert blk.attn_packed(q[:0], k[:0], v[:0], ints([0, 0])).shape == (0, 4, D)


def test_attn_packed_overlapping_sequences_stay_in_bounds():
    """Sequences that claim the same rows many times over have more work than any valid batch."""
    n = 6000
    blk = block(16, 2)
    q, k, v = randn(1, n, 16, D), randn(2, n, 2, D), randn(3, n, 2, D)
    out = torch.full((n + 64, 16, D), 3.0, dtype=torch.bfloat16, device=DEV)
    for pairs in (5, 60, 1500):
        blk.attn_packed(q, k, v, ints([0, n] * pairs + [0]), out=out[:n])
        assert blk.last_status() == 1
        assert torch.isfinite(out[:n]).all() and torch.all(out[n:] == 3)
    lens = [n]
    check_packed(blk.attn_packed(q, k, v, ints([0, n])), q, k, v, lens)


@pytest.mark.parametrize("H,Hkv,lens", [(4, 2, [300, 200]), (32, 8, [2000, 50, 1500])])  # split and not
def test_attn_packed_wait_runs_out_then_recovers(H, Hkv, lens):
    """A wait limit far below a copy's latency: the kernel stops, says so and leaves everything usable."""
    from llama_family_decoder_gb300.binding import set_wait_timeout_ns
    n = sum(lens)
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    set_wait_timeout_ns(100)
    try:
        blk.attn_packed(q, k, v, cu_of(lens))
        assert blk.last_status() == 6 and blk.last_status() == 0
    finally:
        set_wait_timeout_ns(0)
    for _ in range(2):
        check_packed(blk.attn_packed(q, k, v, cu_of(lens)), q, k, v, lens)
        assert blk.last_status() == 0


def test_attn_packed_large_scores():
    """One key takes all the weight, scores in the thousands."""
    lens = [200, 130]
    blk = block(4, 2)
    q, k, v = randn(1, 330, 4, D, scale=30), randn(2, 330, 2, D, scale=30), randn(3, 330, 2, D)
    out = blk.attn_packed(q, k, v, cu_of(lens))
    assert torch.isfinite(out).all()
    at = 0
    for n in lens:
        sl = slice(at, at + n)
        ref, mag = attn_ref(np64(q[sl]), np64(k[sl]), np64(v[sl]))
        # scores off by 128 * 2^-23 sum|q k| / sqrt(128) <= 128 * 2^-23 * 128 * 30^2 / 11.3 ~ 0.16 at the
        # worst; typical rounding is far below, and where one key leads by more nothing moves: 0.35 = e^(2 * 0.15) - 1
        assert np.all(np.abs(np64(out[sl]) - ref) <= (U + 0.35) * mag + U * np.abs(ref))
        at += n


# ------------------------------------------------------------------ 4-bit cache

def quantise(x):
    """The documented format, in fp32 on the CPU: (codes [..., 128], scale [..., 4], offset [..., 4])."""
    g = x.detach().cpu().float().unflatten(-1, (4, 32))
    lo, hi = g.amin(-1), g.amax(-1)
    span = hi - lo
    ok = torch.isfinite(span) & torch.isfinite(g).all(-1)
    scale = torch.where(ok, span / 15, 0.0).bfloat16().float()
    offset = torch.where(ok, lo, float("nan"))
    code = torch.where(scale[..., None] > 0, (g - offset[..., None]) / scale[..., None], torch.zeros(()))
    return torch.nan_to_num(torch.round(code)).clamp(0, 15).flatten(-2), scale, offset


def pack(codes):
    p = torch.arange(64)
    low = 16 * (2 * (p // 4 % 4) + p % 2) + 2 * (p // 16) + p // 2 % 2
    c = codes.to(torch.uint8)
    return c[..., low] | (c[..., low + 8] << 4)


def values(x):
    codes, scale, offset = quantise(x)
    return (offset[..., None] + scale[..., None] * codes.unflatten(-1, (4, 32))).flatten(-2)


def rows_with_corners(seed, n, heads):
    x = randn(seed, n, heads, D)
    x[0] = 2.5                                # no span: codes 0
    if n > 1:
        x[1] *= 1e30
    if n > 2:
        x[2, 0, :32] = torch.linspace(-1, 1, 32, device=DEV)
        x[2, 0, 32:64] = 1000 + x[2, 0, 32:64]  # a large offset
        x[2, 0, 64:96] = 1e-39 * x[2, 0, 64:96]  # subnormal
        x[2, 0, 96:] = torch.arange(32, device=DEV) * 0.5  # ties
    if n > 3:
        x[3, 0, 5] = float("nan")
        x[3, 0, 40] = float("inf")
        x[3, 0, 70] = 3.3e38
        x[3, 0, 71] = -3.3e38                  # a span past fp32
    return x


@pytest.mark.parametrize("Hkv", [1, 2, 3, 8, 20])
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([5, 0, 17, 1], [3, 9, 0, 40]), ([33] * 40, list(range(40)))])
def test_kv4_store_and_load(Hkv, lens, starts):
    B, n, cap = len(lens), sum(lens), 77
    blk = block(Hkv, Hkv)
    k, v = rows_with_corners(1, n, Hkv), randn(2, n, Hkv, D)
    c = blk.kv4_cache(B, cap)
    for x in ("k", "v", "k_scale", "v_scale"):
        c[x].view(torch.uint8).fill_(0xA5)
    before = {x: t.clone() for x, t in c.items()}
    blk.kv4_store(c, k, v, cu_of(lens), starts=ints(starts))
    assert blk.last_status() == 0
    assert c["lens"].tolist() == [a + m for a, m in zip(starts, lens)]
    at, mine = 0, torch.zeros(B, cap, dtype=torch.bool, device=DEV)
    for b, m in enumerate(lens):
        mine[b, starts[b]:starts[b] + m] = True
        for name, x in (("k", k), ("v", v)):
            codes, scale, offset = quantise(x[at:at + m])
            got = c[name][b, :, starts[b]:starts[b] + m].transpose(0, 1).cpu()
            assert torch.equal(got, pack(codes))
            sc = c[name + "_scale"][b, :, starts[b]:starts[b] + m].transpose(0, 1).float().cpu()
            assert torch.equal(sc[..., :4], scale)
            assert torch.equal(torch.isnan(sc[..., 4:]), torch.isnan(offset))
            assert torch.equal(torch.nan_to_num(sc[..., 4:]), torch.nan_to_num(offset))
        at += m
    for x in ("k", "v", "k_scale", "v_scale"):  # every other slot is as it was
        keep = ~mine[:, None].expand(B, Hkv, cap)
        assert torch.equal(c[x][keep].view(torch.uint8), before[x][keep].view(torch.uint8))
    ko, vo = blk.kv4_load(c, cu_of(lens), n, starts=ints(starts))
    for got, x in ((ko, k), (vo, v)):
        want = values(x).bfloat16()
        assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got).cpu(), torch.nan_to_num(want))
        # what the format may lose: half a step, and a step's own rounding over 15 of them
        step = quantise(x)[1].repeat_interleave(32, -1).double()
        off = (want.double() - x.cpu().double()).abs()
        bound = step * (0.5 + 15 * U * 1.01) + U * want.double().abs() + 2.0 ** -133 * 16
        assert torch.all((off <= bound) | torch.isnan(want) | ~torch.isfinite(x.cpu()))


def test_kv4_append_rows_and_single_tokens():
    Hkv, cap = 3, 20
    blk = block(Hkv, Hkv)
    lens = [4, 0, 9]
    k, v = randn(1, 13, Hkv, D), randn(2, 13, Hkv, D)
    c = blk.kv4_cache(3, cap)
    blk.kv4_store(c, k, v, cu_of(lens))
    assert c["lens"].tolist() == lens
    blk.kv4_store(c, k[:4], v[:4], cu_of([2, 1, 1]))
    assert c["lens"].tolist() == [6, 1, 10]
    for i in range(3):
        blk.kv4_store(c, k[i:i + 3], v[i:i + 3])
    assert c["lens"].tolist() == [9, 4, 13]
    order = [[0, 1, 2, 3, 0, 1, 0, 1, 2], [2, 1, 2, 3], [4, 5, 6, 7, 8, 9, 10, 11, 12, 3, 2, 3, 4]]
    ko, vo = blk.kv4_load(c, cu_of([9, 4, 13]), 26)
    at = sum(order, [])
    assert torch.equal(ko.cpu(), values(k[at]).bfloat16()) and torch.equal(vo.cpu(), values(v[at]).bfloat16())
    # single rows at given slots, read back the same way
    blk.kv4_store(c, k[:3], v[:3], starts=ints([0, 2, 19]))
    assert c["lens"].tolist() == [1, 3, 20]
    ko, _ = blk.kv4_load(c, starts=ints([0, 2, 19]))
    assert torch.equal(ko.cpu(), values(k[:3]).bfloat16())


def test_kv4_full_cache():
    blk = block(2, 2)
    k, v = randn(1, 12, 2, D), randn(2, 12, 2, D)
    c = blk.kv4_cache(2, 8)
    blk.kv4_store(c, k, v, cu_of([2, 10]))
    assert blk.last_status() == 4 and c["lens"].tolist() == [2, 8]
    ko, _ = blk.kv4_load(c, cu_of([2, 8]), 10)
    assert torch.equal(ko.cpu(), values(k[:10]).bfloat16())
    blk.kv4_store(c, k[:2], v[:2])  # one fits, one does not
    assert blk.last_status() == 4 and c["lens"].tolist() == [3, 8]
    blk.kv4_store(c, k[:2], v[:2], starts=ints([-1, 100]))
    assert blk.last_status() == 4 and c["lens"].tolist() == [0, 8]
    with pytest.raises(BlkError) as e:
        blk.kv4_store(c, k[:2], v[:2], host_lens_max=9)
    assert e.value.status == 4
    ko, _ = blk.kv4_load(c, starts=ints([7, 8]))
    assert blk.last_status() == 1 and torch.all(ko[1] == 0)


def test_kv4_rows_of_no_sequence():
    blk = block(2, 2)
    k, v = randn(1, 10, 2, D), randn(2, 10, 2, D)
    c = blk.kv4_cache(2, 8)
    blk.kv4_store(c, k, v, ints([3, 4, 6]))
    assert c["lens"].tolist() == [1, 2] and blk.last_status() == 0
    out = torch.full((10, 2, D), 3.0, dtype=torch.bfloat16, device=DEV)
    out2 = out.clone()
    blk.kv4_load(c, ints([3, 4, 6]), 10, k_out=out, v_out=out2)
    assert torch.equal(out[3:6].cpu(), values(k[3:6]).bfloat16())
    assert torch.all(out[:3] == 3) and torch.all(out2[6:] == 3)
    # strided rows in and out
    f = torch.cat([k, v], 1).contiguous()
    c2 = blk.kv4_cache(2, 8)
    blk.kv4_store(c2, f[:, :2], f[:, 2:], ints([3, 4, 6]))
    assert torch.equal(c2["k"], c["k"]) and torch.equal(c2["v_scale"], c["v_scale"])


# ------------------------------------------------------------------ decode over 4 bits

def filled_cache(blk, seed, Hkv, cap, lens, k_scale=1.0, v_scale=1.0):
    """A cache with lens[b] rows each; unused slots hold 0xFF bytes (scales NaN)."""
    B = len(lens)
    k, v = randn(seed, sum(lens), Hkv, D, scale=k_scale), randn(seed + 1, sum(lens), Hkv, D, scale=v_scale)
    k[..., 7] *= 6  # a large channel
    c = blk.kv4_cache(B, cap)
    for x in ("k", "v", "k_scale", "v_scale"):
        c[x].view(torch.uint8).fill_(0xFF)
    blk.kv4_store(c, k, v, cu_of(lens))
    return c, k, v


def check_decode(out, q, k, v, lens, window=0):
    H, Hkv = q.shape[1], k.shape[1]
    per, at = H // Hkv, 0
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(out[b] == 0)
            continue
        f = max(0, n - window) if window else 0
        kk, vv = k[at + f:at + n], v[at + f:at + n]
        K, V = values(kk).double().numpy(), values(vv).double().numpy()
        _, ks, kz = (x.double().numpy() for x in quantise(kk))
        vc, vs, vz = (x.double().numpy() for x in quantise(vv))
        code = np.repeat(vs, 32, -1) * np.abs(vc - 8)
        parts = code + np.abs(np.repeat(vz, 32, -1)) + 8 * np.repeat(vs, 32, -1)  # what fp32 adds up
        for h in range(H):
            j = h // per
            qh = np64(q[b, h])
            s = K[:, j] @ qh / np.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            qa = np.abs(qh).reshape(4, 32).sum(-1)
            delta = 2.0 ** -21 * ((15 * ks[:, j] + np.abs(kz[:, j])) @ qa).max() / np.sqrt(D) + 1e-6
            ref = p @ V[:, j]
            bound = U * (p @ np.abs(V[:, j])) + U * U * (1 + U) * (p @ code[:, j]) + U * np.abs(ref) + \
                np.expm1(2 * delta) * (p @ np.abs(V[:, j])) + 2.0 ** -18 * (p @ parts[:, j])
            err = np.abs(np64(out[b, h]) - ref)
            assert np.all(err <= bound), (b, h, float((err / bound).max()))
        at += n


@pytest.mark.parametrize("H,Hkv", [(8, 2), (4, 4), (16, 1), (9, 1), (6, 2), (32, 8)])
@pytest.mark.parametrize("cap,lens", [(1, [1]), (64, [64, 0, 1, 63]), (1000, [1000, 3, 0, 517, 65, 999]), (130, [129] * 33)])
def test_attn_decode_kv4(H, Hkv, cap, lens):
    blk = block(H, Hkv)
    c, k, v = filled_cache(blk, 1, Hkv, cap, lens)
    q = randn(9, len(lens), H, D)
    out = blk.attn_decode_kv4(q, c)
    assert blk.last_status() == 0
    check_decode(out, q, k, v, lens)
    assert torch.equal(out, blk.attn_decode_kv4(q, c))  # the same to the bit


@pytest.mark.parametrize("cap", [5000, 40000])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (16, 1), (9, 1), (32, 8), (8, 8)])
def test_attn_decode_kv4_few_sequences(H, Hkv, cap):
    """A few sequences over long caches: a cluster of CTAs for each KV head, or stretches of all
    their tiles."""
    lens = [5000, 0, 1, 2177]
    blk = block(H, Hkv)
    c, k, v = filled_cache(blk, 1, Hkv, cap, lens)
    q = randn(9, len(lens), H, D)
    out = blk.attn_decode_kv4(q, c)
    check_decode(out, q, k, v, lens)
    assert torch.equal(out, blk.attn_decode_kv4(q, c))


def test_attn_decode_kv4_long():
    """Thousands of keys: a sequence's keys are split over many CTAs and joined."""
    lens = [20000, 1, 7000, 0, 12345]
    blk = block(8, 2)
    c, k, v = filled_cache(blk, 3, 2, 20001, lens)
    q = randn(9, 5, 8, D)
    check_decode(blk.attn_decode_kv4(q, c), q, k, v, lens)


@pytest.mark.parametrize("window", [1, 63, 64, 300, 4000])
def test_attn_decode_kv4_window(window):
    lens = [700, 64, 0, 1, 301]
    blk = block(4, 2, sliding_window=window)
    c, k, v = filled_cache(blk, 5, 2, 701, lens)
    q = randn(9, 5, 4, D)
    check_decode(blk.attn_decode_kv4(q, c), q, k, v, lens, window)


@pytest.mark.parametrize("ks,vs", [(30.0, 1.0), (1.0, 1e20), (1e-3, 1e-30), (0.0, 1.0)])
def test_attn_decode_kv4_ranges(ks, vs):
    lens = [300, 77]
    blk = block(4, 1)
    c, k, v = filled_cache(blk, 7, 1, 300, lens, ks, vs)
    q = randn(9, 2, 4, D)
    check_decode(blk.attn_decode_kv4(q, c), q, k, v, lens)


def test_attn_decode_kv4_nan_stays_in_its_sequence():
    lens = [200, 100, 50]
    blk = block(4, 2)
    c, k, v = filled_cache(blk, 1, 2, 200, lens)
    q = randn(9, 3, 4, D)
    clean = blk.attn_decode_kv4(q, c)
    k2 = k.clone()
    k2[250, 1, 3] = float("nan")  # sequence 1, KV head 1
    c2 = blk.kv4_cache(3, 200)
    blk.kv4_store(c2, k2, v, cu_of(lens))
    out = blk.attn_decode_kv4(q, c2)
    assert torch.equal(out[[0, 2]], clean[[0, 2]]) and torch.equal(out[1, :2], clean[1, :2])
    assert torch.isnan(out[1, 2:]).all()


def test_attn_decode_kv4_far_offsets():
    """Rows whose byte offset passes 32 bits: only the last keys are looked at (a window)."""
    cap, Hkv = 4_400_000, 8
    blk = block(8, Hkv, sliding_window=100)
    c = blk.kv4_cache(2, cap)  # 4.5 GB of codes each
    k, v = randn(1, 200, Hkv, D), randn(2, 200, Hkv, D)
    blk.kv4_store(c, k, v, cu_of([100, 100]), starts=ints([cap - 100, cap - 100]))
    q = randn(9, 2, 8, D)
    check_decode(blk.attn_decode_kv4(q, c), q, k, v, [100, 100])
    ko, _ = blk.kv4_load(c, cu_of([100, 100]), 200, starts=ints([cap - 100, cap - 100]))
    assert torch.equal(ko.cpu(), values(k).bfloat16())


def test_attn_decode_kv4_strided_rows():
    lens = [90, 33]
    blk = block(4, 2)
    c, k, v = filled_cache(blk, 1, 2, 90, lens)
    q = randn(9, 2, 8, D)
    out = torch.full((4, 2, D), 3.0, dtype=torch.bfloat16, device=DEV)
    blk.attn_decode_kv4(q[:, 2:6], c, out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), blk.attn_decode_kv4(q[:, 2:6].contiguous(), c))


# ------------------------------------------------------------------ together

def test_prompts_then_tokens():
    """A packed prefill and decode steps over the 4-bit cache, from the same projections, as a
    serving loop runs them; every attention output against fp64 on the values it saw."""
    H, Hkv, lens, steps = 8, 2, [150, 1, 0, 333], 3
    B, n = len(lens), sum(lens)
    blk = block(H, Hkv, qk_norm=True)
    gq, gk = 1 + 0.1 * randn(1, D), 1 + 0.1 * randn(2, D)
    fused = randn(3, n, H + 2 * Hkv, D)
    pos = ints([i for m in lens for i in range(m)])
    q, k = blk.qk_norm_rope(fused[:, :H], fused[:, H:H + Hkv], pos, gq, gk)
    v = fused[:, H + Hkv:]
    cu = cu_of(lens)
    out = blk.attn_packed(q, k, v, cu)
    check_packed(out, q, k, v, lens)
    cache = blk.kv4_cache(B, 340)
    blk.kv4_store(cache, k, v, cu)
    ks = [list(x) for x in torch.split(k, lens)]
    vs = [list(x) for x in torch.split(v, lens)]
    for t in range(steps):
        new = randn(10 + t, B, H + 2 * Hkv, D)
        q1, k1 = blk.qk_norm_rope(new[:, :H], new[:, H:H + Hkv], cache["lens"], gq, gk)
        blk.kv4_store(cache, k1, new[:, H + Hkv:])
        o1 = blk.attn_decode_kv4(q1, cache)
        for b in range(B):
            ks[b].append(k1[b])
            vs[b].append(new[b, H + Hkv:])
        now = [len(x) for x in ks]
        assert cache["lens"].tolist() == now
        check_decode(o1, q1, torch.stack(sum(ks, [])), torch.stack(sum(vs, [])), now)
    assert blk.last_status() == 0


def test_streams_and_captured_graphs():
    """Two captured chains replayed at the same time on two streams, and eager calls on a third,
    give what the calls alone give; a graph sees refreshed inputs."""
    H, Hkv, lens = 8, 2, [200, 31, 129]
    n = sum(lens)
    blk = block(H, Hkv)
    cu = cu_of(lens)
    pos = ints([i for m in lens for i in range(m)])

    def chain(fused, q1):
        q, k = blk.qk_norm_rope(fused[:, :H], fused[:, H:H + Hkv], pos)
        o = blk.attn_packed(q, k, fused[:, H + Hkv:], cu)
        c = blk.kv4_cache(3, 200)
        blk.kv4_store(c, k, fused[:, H + Hkv:], cu, starts=zero)
        return o, blk.attn_decode_kv4(q1, c)

    zero = ints([0, 0, 0])
    ins = [(randn(s, n, H + 2 * Hkv, D), randn(s + 50, 3, H, D)) for s in range(3)]
    alone = [chain(*i) for i in ins]
    torch.cuda.synchronize()
    bufs = [(torch.zeros_like(ins[0][0]), torch.zeros_like(ins[0][1])) for _ in range(2)]
    graphs = []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain(*b)
        graphs.append((g, outs))
    for r in range(3):
        for j in range(2):
            for x, y in zip(bufs[j], ins[(r + j) % 3]):
                x.copy_(y)
        torch.cuda.synchronize()
        ss = [torch.cuda.Stream() for _ in range(3)]
        for _ in range(3):
            for j in range(2):
                with torch.cuda.stream(ss[j]):
                    graphs[j][0].replay()
            with torch.cuda.stream(ss[2]):
                eager = chain(*ins[r])
        torch.cuda.synchronize()
        for j in range(2):
            for x, y in zip(graphs[j][1], alone[(r + j) % 3]):
                assert torch.equal(x, y)
        for x, y in zip(eager, alone[r]):
            assert torch.equal(x, y)
    # a stream passed by hand
    s = torch.cuda.Stream()
    out = blk.attn_packed(*[ins[0][0][:, a:b] for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv))], cu, stream=s)
    s.synchronize()
    check_packed(out, ins[0][0][:, :H], ins[0][0][:, H:H + Hkv], ins[0][0][:, H + Hkv:], lens)


def test_refusals():
    blk = block(4, 2, qk_norm=True)
    q, k, g = randn(1, 8, 4, D), randn(2, 8, 2, D), randn(3, D)
    pos = ints(list(range(8)))
    bad = [
        (lambda: blk.qk_norm_rope(q, k, pos), ValueError),                                  # gains missing
        (lambda: blk.qk_norm_rope(q.float(), k, pos, g, g), ValueError),
        (lambda: blk.qk_norm_rope(q.cpu(), k, pos, g, g), ValueError),
        (lambda: blk.qk_norm_rope(q, k, pos.long(), g, g), ValueError),
        (lambda: blk.qk_norm_rope(q, k, pos[:7], g, g), ValueError),
        (lambda: blk.qk_norm_rope(q, k[:, :1], pos, g, g), ValueError),
        (lambda: blk.qk_norm_rope(q, k, torch.stack([pos, pos]), g, g, sections=[64]), ValueError),
        (lambda: blk.qk_norm_rope(q, k, torch.stack([pos, pos]), g, g, sections=[32, 31]), 1),
        (lambda: blk.qk_norm_rope(q, k, torch.stack([pos, pos]), g, g, sections=[65, -1]), 1),
        (lambda: blk.qk_norm_rope(q, k, torch.stack([pos, pos]), g, g, sections=[31, 33], interleaved=True), 1),
        (lambda: blk.qk_norm_rope(q, k, pos, g, g, q_out=torch.zeros(1, 4, D, dtype=torch.bfloat16, device=DEV).expand(8, 4, D)), 1),
        (lambda: blk.qk_norm_rope(q, k, pos, g, g, q_out=q.as_strided((8, 4, D), (D, 8 * D, 1))), 1),  # in place, other strides
        (lambda: blk.attn_packed(q, k, k, ints([0, 8]), out=q), 1),
        (lambda: blk.attn_packed(q, k[:, :1].expand(8, 2, D), k, ints([0, 8])), 2),
        (lambda: blk.attn_packed(q, k, k, torch.tensor([0, 8], device=DEV)), ValueError),
        (lambda: blk.attn_packed(q[..., ::2], k, k, ints([0, 8])), ValueError),
        (lambda: blk.attn_packed(torch.zeros(8, 4, D + 1, dtype=torch.bfloat16, device=DEV)[..., 1:], k, k, ints([0, 8])), 3),
        (lambda: blk.kv4_store(blk.kv4_cache(3, 4), k, k), 1),                                # 8 rows, 3 sequences
        (lambda: blk.kv4_store(dict(blk.kv4_cache(8, 4), k=torch.zeros(8, 2, 4, 32, dtype=torch.uint8, device=DEV)), k, k), ValueError),
        (lambda: blk.kv4_load(blk.kv4_cache(8, 4), k_out=k, v_out=k), 1),
        (lambda: blk.attn_decode_kv4(q, blk.kv4_cache(8, 4), out=q), 1),
        (lambda: blk.attn_decode_kv4(q, blk.kv4_cache(7, 4)), ValueError),
    ]
    f32 = block(4, 2, "f32", 64)
    x = torch.zeros(8, 4, 64, device=DEV)
    bad += [(lambda: f32.attn_packed(x, x[:, :2], x[:, :2], ints([0, 8])), 2)]
    for i, (call, want) in enumerate(bad):
        if want is ValueError:
            with pytest.raises(ValueError):
                call()
        else:
            with pytest.raises(BlkError) as e:
                call()
            assert e.value.status == want, (i, str(e.value))
    # the C calls, with too small a workspace
    from llama_family_decoder_gb300 import binding as b
    L = b.lib()
    r = lambda t: b.head_rows(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    o = torch.empty_like(q)
    cu = ints([0, 8])
    args = (blk.handle, r(q), r(k), r(k), 8, cu.data_ptr(), 1, r(o))
    assert L.blk_attn_packed_workspace_bytes(blk.handle, 8, 1) == 0  # a small batch needs none
    assert L.blk_attn_packed(*args, None, 0, None) == 0
    assert L.blk_attn_packed(*args[:5], None, *args[6:], None, 0, None) == 1
    assert L.blk_attn_packed(*args[:4], -1, *args[5:], None, 0, None) == 1
    many = ints([0] * 9000 + [8])
    need = L.blk_attn_packed_workspace_bytes(blk.handle, 8, 9000)
    assert need > 0
    ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    args = (*args[:5], many.data_ptr(), 9000, args[7])
    assert L.blk_attn_packed(*args, ws.data_ptr(), need - 1, None) == 7
    assert L.blk_attn_packed(*args, None, need, None) == 7
    assert L.blk_attn_packed(*args, ws.data_ptr() + 8, need, None) == 3
    assert L.blk_attn_packed(*args, ws.data_ptr(), need, None) == 0
    kv4 = lambda c: b.kv4_cache_struct(*[c[x].data_ptr() for x in ("k", "k_scale", "v", "v_scale")], c["k"].shape[2],  # noqa: E731
                                       c["lens"].data_ptr())
    c = blk.kv4_cache(8, 4)
    assert L.blk_attn_decode_kv4_workspace_bytes(blk.handle, 8, 4) == 0  # few pairs, few keys: none
    assert L.blk_attn_decode_kv4(blk.handle, r(q), kv4(c), 8, r(o), None, 0, None) == 0
    q, o, c = randn(1, 500, 4, D), randn(1, 500, 4, D), blk.kv4_cache(500, 4)
    need = L.blk_attn_decode_kv4_workspace_bytes(blk.handle, 500, 4)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert L.blk_attn_decode_kv4(blk.handle, r(q), kv4(c), 500, r(o), ws.data_ptr(), need - 1, None) == 7
    assert L.blk_attn_decode_kv4(blk.handle, r(q), kv4(c), 500, r(o), None, need, None) == 7
    assert L.blk_attn_decode_kv4(blk.handle, r(q), kv4(c), 500, r(o), ws.data_ptr(), need, None) == 0
    torch.cuda.synchronize()


def test_far_rows_and_slots():
    """Rows more than 2^31 elements apart and slots behind 2^31 bytes give what near ones do, and
    nothing else is written."""
    n, H, Hkv, cap, lens = 70, 4, 2, 1 << 25, [40, 30]
    blk = block(H, Hkv, qk_norm=True)
    step = (1 << 25) + 64
    far = torch.zeros(n * step, dtype=torch.bfloat16, device=DEV)

    def rows(first, heads):
        return far.as_strided((n, heads, D), (step, D, 1), first * D)

    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    fq, fk, fv, fo = rows(0, H), rows(H, Hkv), rows(H + Hkv, Hkv), rows(H + 2 * Hkv, H)
    for a, b in ((fq, q), (fk, k), (fv, v)):
        a.copy_(b)
    pos, g, cu = ints(list(range(n))), randn(4, 2, D), cu_of(lens)
    q, k = blk.qk_norm_rope(q, k, pos, g[0], g[1])
    blk.qk_norm_rope(fq, fk, pos, g[0], g[1], q_out=fq, k_out=fk)
    assert torch.equal(fq, q) and torch.equal(fk, k)
    o = blk.attn_packed(q, k, v, cu)
    blk.attn_packed(fq, fk, fv, cu, out=fo)
    assert torch.equal(fo, o)
    near, big = blk.kv4_cache(2, 64), blk.kv4_cache(2, cap)  # 2^25 slots of 64 bytes: a plane of 2^31
    starts = ints([cap - 64, cap - 50])
    blk.kv4_store(near, k, v, cu)
    blk.kv4_store(big, fk, fv, cu, starts=starts)
    assert big["lens"].tolist() == [cap - 24, cap - 20]
    for x in ("k", "k_scale", "v", "v_scale"):
        for b, (f, m) in enumerate(zip(starts.tolist(), lens)):
            assert torch.equal(big[x][b, :, f:f + m], near[x][b, :, :m])
            assert not big[x][b, :, f + m:].any() and not big[x][b, :, f - 64:f].any()
    kk, vv = blk.kv4_load(near, cu, n)
    blk.kv4_load(big, cu, n, starts=starts, k_out=fk, v_out=fv)
    assert torch.equal(fk, kk) and torch.equal(fv, vv)
    assert blk.last_status() == 0
    used = (2 * H + 2 * Hkv) * D
    assert not far.as_strided((n - 1, 4096), (step, 1), used).any()  # behind each row's channels


def test_short_and_long_way_agree(monkeypatch):
    """The compiled argument handling takes every plain call, and what it leaves out (here: all of
    them) gives the same to the bit; it keeps no argument or output alive."""
    import sys

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    H, Hkv, lens = 8, 2, [5, 0, 70, 1]
    n = sum(lens)
    blk = block(H, Hkv, qk_norm=True)
    qkv, g, cu = randn(1, n, H + 2 * Hkv, D), randn(2, 2, D), cu_of(lens)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    pos, axes, q1, starts = ints(list(range(n))), ints([list(range(n))] * 3), randn(3, len(lens), H, D), ints([3, 0, 1, 0])

    def calls():
        c = blk.kv4_cache(len(lens), 90)
        res = [*blk.qk_norm_rope(q, k, pos, g[0], g[1]),
               *blk.qk_norm_rope(q, k, axes, g[0], g[1], sections=[24, 20, 20], interleaved=True),
               *blk.qk_norm_rope(q, k, axes, g[0], g[1], sections=(24, 20, 20)),
               blk.attn_packed(q, k, v, cu)]
        assert blk.kv4_store(c, k, v, cu, host_lens_max=70) is None
        blk.kv4_store(c, q1[:, :Hkv], q1[:, Hkv:2 * Hkv])
        blk.kv4_store(c, k, v, cu, starts=starts)
        return res + [*blk.kv4_load(c, cu, n, starts=starts), *blk.kv4_load(c), blk.attn_decode_kv4(q1, c),
                      *[c[x] for x in ("k", "k_scale", "v", "v_scale", "lens")]]

    fast, taken = blk._fast, []

    class Counted:
        def __getattr__(self, name):
            return lambda *a: (taken.append((r := getattr(fast, name)(*a)) is not None), r)[1]

    held = [q, k, v, cu, pos, axes, q1, starts, g]
    before = [sys.getrefcount(x) for x in held]
    monkeypatch.setattr(blk, "_fast", Counted())
    short = calls()
    assert len(taken) == 10 and all(taken)
    monkeypatch.setattr(blk, "_fast", Nothing())
    long = calls()
    for a, b in zip(short, long, strict=True):
        assert torch.equal(a, b) and a.shape == b.shape and a.stride() == b.stride()
    assert before == [sys.getrefcount(x) for x in held]
    # given outputs come back as they are
    monkeypatch.setattr(blk, "_fast", fast)
    out = torch.empty_like(short[6])
    count = sys.getrefcount(out)
    assert blk.attn_packed(q, k, v, cu, out=out) is out and torch.equal(out, short[6])
    assert sys.getrefcount(out) == count
    # a closed handle is refused
    blk.close()
    with pytest.raises(BlkError) as e:
        blk.attn_packed(q, k, v, cu)
    assert e.value.status == 1

"""Packed calls on inputs that are not all numbers, and on lists of sequences that are not valid."""
import numpy as np
import pytest
import torch

from llama_family_decoder_gb300 import BlkError
from tests.helpers import np64
from tests.test_gpu_packed import (D, DEV, U, attn_ref, block, check_decode, check_packed, cu_of, filled_cache, ints, randn,
                                   values)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ NaN and infinities in q and k

@pytest.mark.parametrize("H,Hkv,lens", [(4, 2, [100, 37, 260]), (32, 8, [900, 50, 700]), (3, 3, [300])])  # keys split; not; split
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("which,bad", [("q", float("nan")), ("q", float("inf")), ("k", float("nan")), ("k", float("inf")),
                                       ("k", -float("inf"))])
def test_attn_packed_nan_and_infinities(H, Hkv, lens, window, which, bad):
    """A query whose score of a visible key is NaN or +inf, or whose scores are all -inf, gets NaN, as
    the formula does; every other row what it gets from the numbers alone."""
    n = sum(lens)
    blk = block(H, Hkv, sliding_window=window)
    x = {"q": randn(1, n, H, D), "k": randn(2, n, Hkv, D), "v": randn(3, n, Hkv, D)}
    for row, head, channel in ((0, 0, 3), (70, Hkv - 1, 127), (n - 20, 0, 64)):
        x[which][row, head, channel] = bad
    out = blk.attn_packed(x["q"], x["k"], x["v"], cu_of(lens))
    assert blk.last_status() == 0
    at, seen = 0, 0
    with np.errstate(invalid="ignore"):
        for m in lens:
            sl = slice(at, at + m)
            ref, mag = attn_ref(*(np64(x[c][sl]) for c in "qkv"), window)
            got, nan = np64(out[sl]), np.isnan(ref)
            assert np.array_equal(np.isnan(got), nan)
            err = np.abs(got - ref)[~nan]
            # the two roundings to bf16 of p and the output, and 2e-4 for the scores (see test_gpu_packed)
            assert np.all(err <= ((U + 2e-4) * mag + U * np.abs(ref))[~nan])
            seen += nan.sum()
            at += m
    assert seen > 0  # the corner is there


# ------------------------------------------------------------------ lists that are not valid

# cu_seqlens of 200 rows, and how it is read
BAD_LISTS = [([0, 60, 500], [0, 60, 200]), ([-5, -1, 50], [0, 0, 50]), ([-7, 20, 60], [0, 20, 60]), ([0, 250, 300], [0, 200, 200]),
             ([*range(180), 201], [*range(180), 200]), ([0] * 1500 + [150, 2**31 - 1], [0] * 1500 + [150, 200]),
             ([-2**31] * 1500 + [150, 190], [0] * 1500 + [150, 190])]


@pytest.mark.parametrize("cu,read", BAD_LISTS)
@pytest.mark.parametrize("append", [False, True])
def test_kv4_lists_outside_the_rows_are_clamped(cu, read, append):
    """The lengths move by the rows that were stored, and the status word says INVALID_ARG."""
    B, n, Hkv, cap = len(cu) - 1, 200, 2, 700
    blk = block(Hkv, Hkv)
    k, v = randn(1, n, Hkv, D), randn(2, n, Hkv, D)
    first = [3 + b % 5 for b in range(B)]
    caches = []
    for c in (cu, read):
        cache = blk.kv4_cache(B, cap)
        for x in ("k", "v", "k_scale", "v_scale"):
            cache[x].view(torch.uint8).fill_(0xA5)
        cache["lens"].copy_(ints(first))
        blk.kv4_store(cache, k, v, ints(c), starts=None if append else ints(first))
        assert blk.last_status() == (1 if c is cu else 0)
        assert cache["lens"].tolist() == [f + b - a for f, a, b in zip(first, read, read[1:])]
        caches.append(cache)
    for x in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(caches[0][x].view(torch.uint8), caches[1][x].view(torch.uint8))
    outs = []
    for c in (cu, read):
        out = torch.full((2, n, Hkv, D), 3.0, dtype=torch.bfloat16, device=DEV)
        blk.kv4_load(caches[1], ints(c), n, starts=ints(first), k_out=out[0], v_out=out[1])
        assert blk.last_status() == (1 if c is cu else 0)
        outs.append(out)
    assert torch.equal(*outs)
    assert torch.equal(outs[0][0, read[0]:read[-1]].cpu(), values(k[read[0]:read[-1]]).bfloat16())


@pytest.mark.parametrize("cu", [[0, 100, 50, 200], [0, 60, 20], [200, 0], [*range(100), 0, *range(100, 1500)]])
@pytest.mark.parametrize("append", [False, True])
def test_kv4_lists_that_fall_move_no_length(cu, append):
    B, n, Hkv, cap = len(cu) - 1, 200, 2, 400
    blk = block(Hkv, Hkv)
    k, v = randn(1, n, Hkv, D), randn(2, n, Hkv, D)
    cache = blk.kv4_cache(B, cap)
    first = [3 + b % 5 for b in range(B)]
    cache["lens"].copy_(ints(first))
    blk.kv4_store(cache, k, v, ints(cu), starts=None if append else ints([9] * B))
    assert blk.last_status() == 1 and cache["lens"].tolist() == first
    for x in ("k", "v", "k_scale", "v_scale"):  # the slots in use are as they were
        for b in range(min(B, 50)):
            assert not cache[x][b, :, :first[b]].any()
    blk.kv4_load(cache, ints(cu), n)
    assert blk.last_status() == 1


def test_kv4_load_of_packed_rows_needs_their_number():
    """cu_seqlens is on the device: without `rows` the call would have to guess how many there are."""
    blk = block(2, 2)
    k = randn(1, 10, 2, D)
    cache, cu = blk.kv4_cache(2, 8), ints([0, 3, 10])
    blk.kv4_store(cache, k, k, cu)
    with pytest.raises(ValueError):
        blk.kv4_load(cache, cu)
    out = torch.empty_like(k[:2])
    with pytest.raises(ValueError):
        blk.kv4_load(cache, cu, k_out=out, v_out=out.clone())
    assert torch.equal(blk.kv4_load(cache, cu, 10)[0].cpu(), values(k).bfloat16())
    assert torch.equal(blk.kv4_load(cache)[1].cpu(), values(k[[0, 3]]).bfloat16())


def running(cu, rows):
    return np.clip(np.maximum.accumulate(cu), 0, rows).tolist()


@pytest.mark.parametrize("cu", [[0, 100, 50, 200], [0, 200, 0, 200, 0], [150, 30, 170, 20], [-9, 60, 500, 40], [200, 0],
                                [*range(60), 0, 150, *range(60, 160)], [0, 200] * 1500 + [0], [*range(100), 0] * 30])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (16, 1)])
def test_attn_packed_lists_that_fall(cu, H, Hkv):
    """Sequences that claim the same rows are read as ones that do not: the first one keeps them."""
    n = 200
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    out = torch.full((2, n, H, D), 3.0, dtype=torch.bfloat16, device=DEV)
    read = running(cu, n)
    blk.attn_packed(q, k, v, ints(cu), out=out[0])
    assert blk.last_status() == 1
    blk.attn_packed(q, k, v, ints(read), out=out[1])
    assert blk.last_status() == 0
    assert torch.equal(out[0], out[1])
    check_packed(out[0], q, k, v, np.diff(read).tolist(), read[0])


def test_attn_packed_more_claims_than_32_bits_count():
    """2^19 sequences that each claim all rows, 2^13 tiles of them: read as one."""
    n, H, Hkv = 1 << 17, 16, 1
    blk = block(H, Hkv)
    q, k, v = randn(1, n, H, D), randn(2, n, Hkv, D), randn(3, n, Hkv, D)
    want = blk.attn_packed(q, k, v, ints([0, n]))
    assert blk.last_status() == 0
    cu = ints([0, n]).repeat(1 << 19)
    assert torch.equal(blk.attn_packed(q, k, v, cu), want)
    assert blk.last_status() == 1


# ------------------------------------------------------------------ shares of nothing

@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 1), (4, 4), (5, 1), (8, 1), (9, 1), (12, 1), (16, 1)])
@pytest.mark.parametrize("cap", [130, 4000, 12000])
def test_attn_decode_kv4_more_ctas_than_tiles(H, Hkv, cap):
    """Short sequences in caches that clusters of 8 and of 16 CTAs work on: most or all of a
    cluster's CTAs have no keys, and groups of any size leave half a warp over in filling their shares."""
    for lens in ([0], [1], [129], [0, 128, 1, 0]):
        blk = block(H, Hkv)
        c, k, v = filled_cache(blk, 1, Hkv, cap, lens)
        q = randn(9, len(lens), H, D)
        check_decode(blk.attn_decode_kv4(q, c), q, k, v, lens)
        assert blk.last_status() == 0


# ------------------------------------------------------------------ large scores, exactly known

@pytest.mark.parametrize("H,Hkv,lens", [(4, 2, [200, 130]), (3, 3, [300]), (32, 8, [900, 50, 700])])  # keys split; split; not
@pytest.mark.parametrize("top,slope", [(90, 0), (90, 1), (12, 0), (12, 1), (4, 1)])
@pytest.mark.parametrize("window", [0, 150])
def test_attn_packed_large_scores_of_whole_numbers(H, Hkv, lens, top, slope, window):
    """Scores in the thousands, most rows one-hot or nearly so, and references that move from tile to
    tile (with a slope, later keys score higher and higher).

    q and k are whole numbers up to 90: every product and every partial sum of 128 of them is below
    128 * 90^2 < 2^24, so a raw score x has no rounding at all. A probability is 2^(x c - m), c =
    log2(e) / sqrt(128) to within 2^-22 of itself, m a number that is the same for all keys of a row (or
    is moved by its exact difference): x c - m is one fused operation, off by 2^-24 of its own size.
    A key that counts has x c within 30 of the largest (2^-30 of the weight), m within 8 of that: at most
    38 * 2^-24 + 30 * 2^-22 in the exponent, and 2^-22 for the exponential: below 2e-5 of a probability, so
    the bound of ordinary scores (2e-4) holds, and keys that lead alone are exact to the roundings."""
    n = sum(lens)
    blk = block(H, Hkv, sliding_window=window)
    g = torch.Generator(device=DEV).manual_seed(7)
    q = torch.randint(-top, top + 1, (n, H, D), generator=g, device=DEV).float()
    k = torch.randint(-top, top + 1, (n, Hkv, D), generator=g, device=DEV).float()
    if slope:  # the first 32 channels carry it: q positive there, k's part grows with the key's place
        q[..., :32] = q[..., :32].abs()
        place = torch.cat([torch.linspace(0, 1, m, device=DEV) for m in lens])
        k[..., :32] = (k[..., :32].abs() * place[:, None, None]).round()
    q, k, v = q.bfloat16(), k.bfloat16(), randn(3, n, Hkv, D)
    out = blk.attn_packed(q, k, v, cu_of(lens))
    assert blk.last_status() == 0
    check_packed(out, q, k, v, lens, window=window)


def test_kv4_store_refuses_lists_that_overlap_the_lengths():
    """The lengths are written while other blocks still read their first slots or the list."""
    blk = block(2, 2)
    k, shared = randn(1, 4, 2, D), ints([0, 1, 2, 3, 4, 5, 6, 7, 8])
    cache = blk.kv4_cache(4, 20)
    cache["lens"] = shared[2:6]
    for kw in (dict(starts=shared[1:5]), dict(starts=shared[3:7]), dict(cu_seqlens=shared[0:5]), dict(cu_seqlens=shared[4:9]),
               dict(cu_seqlens=shared[2:7], starts=shared[:4].clone())):
        with pytest.raises(BlkError) as e:
            blk.kv4_store(cache, k, k, **kw)
        assert e.value.status == 1
    assert shared.tolist() == list(range(9))
    blk.kv4_store(cache, k, k, starts=cache["lens"])  # an append
    blk.kv4_store(cache, k[:2], k[:2], ints([0, 1, 1, 1, 2]), starts=shared[2:6])
    assert shared.tolist() == [0, 1, 4, 4, 5, 7, 6, 7, 8]
    cache["lens"] = shared[4:8]
    blk.kv4_store(cache, k, k, starts=shared[:4])  # beside them
    assert shared.tolist() == [0, 1, 4, 4, 1, 2, 5, 5, 8] and blk.last_status() == 0


def test_qk_norm_rope_refuses_an_output_over_the_other_input():
    """In place means q over q and k over k: a warp may still read k while another writes q's rows there."""
    blk = block(2, 2, qk_norm=True)
    q, k, g, pos = randn(1, 8, 2, D), randn(2, 8, 2, D), randn(3, D), ints(list(range(8)))
    want = blk.qk_norm_rope(q, k, pos, g, g)
    for args, kw in (((q, k), dict(q_out=k)), ((q, k), dict(k_out=q)), ((q, k), dict(q_out=k, k_out=q)),
                     ((q, q), dict(q_out=q)), ((q, q), dict(k_out=q))):
        with pytest.raises(BlkError) as e:
            blk.qk_norm_rope(*args, pos, g, g, **kw)
        assert e.value.status == 1
    blk.qk_norm_rope(q, k, pos, g, g, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_kv4_append_to_very_many_sequences():
    """More sequences than the blocks that move the lengths on have threads, and more than a block copies."""
    B, Hkv, cap = 100_000, 1, 4
    blk = block(Hkv, Hkv)
    k, v = randn(1, B, Hkv, D), randn(2, B, Hkv, D)
    cache = blk.kv4_cache(B, cap)
    cu = torch.arange(B + 1, device=DEV, dtype=torch.int32)
    blk.kv4_store(cache, k, v, cu)
    blk.kv4_store(cache, v, k, cu)
    assert blk.last_status() == 0 and torch.all(cache["lens"] == 2)
    ko, vo = blk.kv4_load(cache, cu, B, starts=cache["lens"] - 1)
    assert torch.equal(ko.cpu(), values(v).bfloat16()) and torch.equal(vo.cpu(), values(k).bfloat16())
    cu[-1] = B + 7
    blk.kv4_store(cache, k, v, cu)
    assert blk.last_status() == 1 and torch.all(cache["lens"] == 3)
    cu[70_000] = 3
    blk.kv4_store(cache, k, v, cu)
    assert blk.last_status() == 1 and torch.all(cache["lens"] == 3)

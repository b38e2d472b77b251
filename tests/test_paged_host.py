"""What the calls of the paged cache check on the host before anything is launched (no GPU)."""
import types

import pytest
import torch

from llama_family_decoder_gb300 import binding as b

CALLS = [("paged_append", 4), ("attn_paged", 2), ("verify_drafts", 4), ("paged_keep", 2)]


def test_without_a_handle_nothing_is_looked_at():
    lib = b.lib()
    r = b.head_rows(0x1000, 512, 128)
    c = b.paged_cache_struct(0x1000, 0x2000, 0x3000, 0x4000, 4, 16, 2)
    assert len(c) == 48 and len(b.rope_layout_struct(0x1000, 128, 64, 0)) == 24  # the C structs' sizes
    assert lib.blk_paged_append(None, r, r, r, 1, None, None, 1, c, None, None, None, r, -1, None) == 1
    assert lib.blk_attn_paged(None, r, 1, None, None, 1, c, r, None, 0, None) == 1
    assert lib.blk_verify_drafts(None, 4096, 8, None, 0, 1, 8, 4096, None, None, 4096, 4096, 1, 4096, 4096, 4096, None) == 1
    assert lib.blk_paged_keep(None, c, 1, 4096, None, None, None, 1, 0, None) == 1
    assert b"NULL handle" in lib.blk_last_error_message()
    assert lib.blk_rope_table(None, 64, 8, 4096, None) == 1
    assert lib.blk_attn_paged_workspace_bytes(None, 8, 0, 0, 8, c) == 0


def test_compiled_argument_handling_leaves_what_is_not_plain():
    f = b.fastcall()
    blk = f.block(0, 4, 2, 128, 1, 0, 0, 0)
    x = torch.zeros(8, 4, 128, dtype=torch.bfloat16)
    for first in (None, blk, 3, "block"):
        for a in (None, x, "x", {}, {"k": x}, [], [x], [{}]):
            assert f.paged_append(first, *[a] * 12) is None
            assert f.attn_paged(first, *[a] * 5) is None
            assert f.verify_drafts(first, *[a] * 7) is None
            assert f.paged_keep(first, *[a] * 5) is None
    assert f.attn_paged() is None and f.paged_keep(blk) is None  # not the number of arguments


@pytest.mark.parametrize("call,n_args", CALLS)
def test_a_stream_of_another_device_is_refused(monkeypatch, call, n_args):
    blk = object.__new__(b.DecoderBlock)
    blk.handle = None
    blk._torch, blk._dev, blk._device = torch, 0, torch.device("cuda", 0)
    blk._fast = types.SimpleNamespace(**{call: lambda *a: "ran on another stream"})
    blk._block = None
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: torch.no_grad())  # any context: nothing is launched here
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        getattr(blk, call)(*[None] * n_args, stream=other)

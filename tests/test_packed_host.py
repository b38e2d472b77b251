"""What the packed calls' host side does before anything is launched (no GPU)."""
import types

import pytest
import torch

from llama_family_decoder_gb300 import binding


def bare_block(monkeypatch, dev=0):
    """A DecoderBlock without a handle, whose own calls are recorded; `dev` is current."""
    blk = object.__new__(binding.DecoderBlock)
    blk.handle = None
    blk._torch, blk._dev, blk._device = torch, dev, torch.device("cuda", dev)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: dev)
    return blk


@pytest.mark.parametrize("call,n_args", [("qk_norm_rope", 3), ("attn_packed", 4), ("kv4_store", 3), ("kv4_load", 1),
                                         ("attn_decode_kv4", 2)])
def test_a_stream_of_another_device_is_refused(monkeypatch, call, n_args):
    """... and not dropped for the current stream of the handle's device."""
    blk = bare_block(monkeypatch)
    blk._fast = types.SimpleNamespace(**{call: lambda *a: "ran on another stream"})
    blk._block = None
    monkeypatch.setattr(torch.cuda, "stream", lambda s: torch.no_grad())  # any context: nothing is launched here
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    with pytest.raises(ValueError, match="stream"):
        getattr(blk, call)(*[None] * n_args, stream=other)


def test_only_the_packed_calls_need_their_compiled_module(monkeypatch):
    """A handle, and every call but the packed ones, works without _fastcall.so; those say what is missing."""
    def missing():
        raise ImportError("_fastcall is not there")

    made = []
    monkeypatch.setattr(binding, "lib", lambda: types.SimpleNamespace(blk_create=lambda d, h: made.append(d) or 0,
                                                                      blk_workspace_bytes=lambda *a: 64))
    monkeypatch.setattr(binding, "fastcall", missing)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    blk = binding.DecoderBlock(hidden=256, n_heads=2, n_kv_heads=1, head_dim=128, ffn=512)
    assert len(made) == 1 and blk.workspace_bytes(1, 1) == 64
    for call, n in (("qk_norm_rope", 3), ("attn_packed", 4), ("kv4_store", 3), ("kv4_load", 1), ("attn_decode_kv4", 2)):
        with pytest.raises(ImportError, match="_fastcall"):
            getattr(blk, call)(*[None] * n)


def test_the_compiled_module_is_rebuilt_for_another_torch_or_python(monkeypatch, tmp_path):
    """Times of files say nothing about these: an install may keep older ones."""
    import os
    import sysconfig

    from llama_family_decoder_gb300 import build
    runs = []

    class Ran:  # a compiler that writes its output file
        returncode, stdout, stderr = 0, "", ""

        def __init__(self, cmd, **kw):
            runs.append(cmd)
            with open(cmd[cmd.index("-o") + 1], "w"):
                pass

        def communicate(self):
            return "", None

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libblk.so"))
    monkeypatch.setattr(build, "FAST_OBJ", str(tmp_path / "fastcall.o"))
    monkeypatch.setattr(build, "FAST", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build.subprocess, "Popen", Ran)
    monkeypatch.setattr(build.subprocess, "run", Ran)

    def compiled():
        del runs[:]
        build.build()
        return sum(build.FAST_SRC in cmd for cmd in runs), sum(build.FAST in cmd for cmd in runs)

    assert compiled() == (1, 1) and compiled() == (0, 0)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0+other")
        assert compiled() == (1, 1) and compiled() == (0, 0)
    assert compiled() == (1, 1)
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".other-abi.so")
        assert compiled() == (1, 1)
    # a compiler found on the search path only: its includes are beside it, not under "include"
    there = tmp_path / "cuda" / "bin"
    there.mkdir(parents=True)
    (there / "nvcc").write_text("")
    os.chmod(there / "nvcc", 0o755)
    monkeypatch.setattr(build, "_nvcc", lambda: "nvcc")
    monkeypatch.setenv("PATH", str(there))
    assert compiled() == (1, 1)
    assert str(tmp_path / "cuda" / "include") in next(cmd for cmd in runs if build.FAST_SRC in cmd)

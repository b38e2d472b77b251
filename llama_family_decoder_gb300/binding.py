"""Thin ctypes binding of libblk (include/blk.h): argument marshalling only.

PyTorch provides device memory and streams; every step of the block runs in
the library's CUDA kernels. There is no fallback: if libblk.so is missing the
first call raises, and so does the first packed call if _fastcall.so, which
handles these calls' arguments, is.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from ctypes import POINTER, c_char_p, c_float, c_int, c_longlong, c_size_t, c_void_p

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libblk.so")

BLK_OK = 0
STATUS_NAMES = {0: "BLK_OK", 1: "BLK_ERR_INVALID_ARG", 2: "BLK_ERR_UNSUPPORTED", 3: "BLK_ERR_ALIGNMENT",
                4: "BLK_ERR_CACHE_FULL", 5: "BLK_ERR_CUDA", 6: "BLK_ERR_TIMEOUT", 7: "BLK_ERR_WORKSPACE"}
ACTS = {"silu": 0, "swiglu": 0, "relu2": 1, "xielu": 2}
DTYPES = {"f32": 0, "fp32": 0, "float32": 0, "bf16": 1, "bfloat16": 1}


class blk_desc(ctypes.Structure):
    _fields_ = [("hidden", c_int), ("n_heads", c_int), ("n_kv_heads", c_int), ("head_dim", c_int), ("ffn", c_int),
                ("rope_theta", c_float), ("eps", c_float), ("act", c_int), ("xielu_alpha_p", c_float),
                ("xielu_alpha_n", c_float), ("xielu_beta", c_float), ("xielu_eps", c_float), ("qk_norm", c_int),
                ("dtype", c_int), ("max_batch", c_int), ("max_seq", c_int), ("rope_type", c_int),
                ("rope_factor", c_float), ("rope_orig_max_pos", c_int), ("rope_low", c_float), ("rope_high", c_float),
                ("sliding_window", c_int), ("no_rope", c_int), ("attn_gate", c_int), ("sandwich_norm", c_int)]

ROPE_TYPES = {"yarn": 1, "llama3": 2}


class blk_weights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("ln1_g", "wq", "wk", "wv", "q_norm_g", "k_norm_g", "wo", "ln2_g",
                                         "w_gate", "w_up", "w_down", "prepared", "w_attn_gate", "post_attn_g",
                                         "post_mlp_g")]


class blk_kv_cache(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("capacity", c_int), ("lens", c_void_p)]


class blk_model(ctypes.Structure):
    _fields_ = [("embed", c_void_p), ("layers", POINTER(blk_weights)), ("n_layers", c_int), ("norm_g", c_void_p),
                ("lm_head", c_void_p), ("vocab", c_int)]


TAP_NAMES = ("attention_queries", "attention_keys", "attention_values", "attention_head_outputs",
             "attention_output", "layer_mid", "mlp_neurons", "mlp_output")


class blk_taps(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in TAP_NAMES]


# blk_head_rows (pointer, row and head stride in elements) and blk_kv4_cache as bytes: packing
# them costs a tenth of building ctypes structures, which these short calls would feel
head_rows = struct.Struct("@Pqq").pack
kv4_cache_struct = struct.Struct("@PPPPiP").pack  # k, k_scale, v, v_scale, capacity, lens


class blk_rope_axes(ctypes.Structure):
    _fields_ = [("n_axes", c_int), ("sections", c_int * 4), ("interleaved", c_int)]


# blk_paged_cache (k, v, pages, lens, n_pages, page_size, max_pages) and blk_rope_layout (table, dims, max_pos,
# interleaved), likewise
paged_cache_struct = struct.Struct("@PPPPiii4x").pack
rope_layout_struct = struct.Struct("@Piii4x").pack


_ROWS = _KV4 = _PAGED = _LAYOUT = c_char_p  # see head_rows, kv4_cache_struct, paged_cache_struct and rope_layout_struct

# name -> (restype, argtypes); the exported symbols of include/blk.h
SIGNATURES = {
    "blk_create": (c_int, [POINTER(blk_desc), POINTER(c_void_p)]),
    "blk_destroy": (c_int, [c_void_p]),
    "blk_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int, c_int]),
    "blk_forward": (c_int, [c_void_p, c_void_p, c_int, c_int, POINTER(blk_weights), POINTER(blk_kv_cache), c_int,
                            c_void_p, c_void_p, c_size_t, POINTER(blk_taps), c_void_p]),
    "blk_forward_masked": (c_int, [c_void_p, c_void_p, c_int, c_int, c_void_p, POINTER(blk_weights), c_void_p,
                                   c_void_p, c_size_t, POINTER(blk_taps), c_void_p]),
    "blk_rmsnorm": (c_int, [c_void_p, c_void_p, c_int, c_int, c_float, c_void_p, c_int, c_void_p]),
    "blk_qkv_rope": (c_int, [c_void_p, c_void_p, POINTER(blk_weights), c_int, c_int, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_void_p, c_size_t, c_void_p]),
    "blk_attn_gqa": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_void_p, c_void_p,
                             c_void_p, c_size_t, c_void_p]),
    "blk_mlp": (c_int, [c_void_p, c_void_p, c_void_p, POINTER(blk_weights), c_int, c_void_p, c_void_p, c_size_t,
                        c_void_p]),
    "blk_qk_norm_rope": (c_int, [c_void_p, _ROWS, _ROWS, c_int, c_void_p, POINTER(blk_rope_axes), c_void_p, c_void_p,
                                 _ROWS, _ROWS, c_void_p]),
    "blk_attn_packed_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int]),
    "blk_attn_packed": (c_int, [c_void_p, _ROWS, _ROWS, _ROWS, c_int, c_void_p, c_int, _ROWS, c_void_p, c_size_t,
                                c_void_p]),
    "blk_kv4_store": (c_int, [c_void_p, _ROWS, _ROWS, c_int, c_void_p, c_void_p, c_int, _KV4, c_int,
                              c_void_p]),
    "blk_kv4_load": (c_int, [c_void_p, _KV4, c_void_p, c_void_p, c_int, c_int, _ROWS, _ROWS,
                             c_void_p]),
    "blk_attn_decode_kv4_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int]),
    "blk_attn_decode_kv4": (c_int, [c_void_p, _ROWS, _KV4, c_int, _ROWS, c_void_p, c_size_t,
                                    c_void_p]),
    "blk_rope_table": (c_int, [c_void_p, c_int, c_int, c_void_p, c_void_p]),
    "blk_paged_append": (c_int, [c_void_p, _ROWS, _ROWS, _ROWS, c_int, c_void_p, c_void_p, c_int, _PAGED, _LAYOUT,
                                 c_void_p, c_void_p, _ROWS, c_int, c_void_p]),
    "blk_attn_paged_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int, c_int, c_int, _PAGED]),
    "blk_attn_paged": (c_int, [c_void_p, _ROWS, c_int, c_void_p, c_void_p, c_int, _PAGED, _ROWS, c_void_p, c_size_t,
                               c_void_p]),
    "blk_verify_drafts": (c_int, [c_void_p, c_void_p, c_longlong, c_void_p, c_longlong, c_int, c_int, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p,
                                  c_void_p]),
    "blk_paged_keep": (c_int, [c_void_p, _PAGED, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int,
                               c_void_p]),
    "blk_model_paged_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int, c_int, c_int, _PAGED, c_int, c_int]),
    "blk_model_forward_paged": (c_int, [c_void_p, POINTER(blk_model), c_void_p, c_int, c_void_p, c_void_p, c_void_p,
                                        c_int, _PAGED, c_float, c_int, c_void_p, c_void_p, c_size_t, c_void_p]),
    "blk_stage_workspace_bytes": (c_size_t, [c_void_p, c_int]),
    "blk_last_status": (c_int, [c_void_p]),
    "blk_xielu_effective": (None, [c_float, c_float, c_float, POINTER(c_float), POINTER(c_float)]),
    "blk_error_string": (c_char_p, [c_int]),
    "blk_last_error_message": (c_char_p, []),
    "blk_debug_set_wait_timeout_ns": (None, [c_longlong]),
    "blk_debug_last_status": (c_int, []),
    "blk_version": (c_char_p, []),
    "blk_profile_enable": (c_int, [c_void_p, c_int]),
    "blk_profile_collect": (c_int, [c_void_p, POINTER(ctypes.c_double), POINTER(c_longlong), c_int]),
    "blk_profile_stage_name": (c_char_p, [c_void_p, c_int]),
    "blk_profile_reset": (None, [c_void_p]),
    "blk_debug_gemm_bf16": (c_int, [c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int, c_int,
                                    c_void_p]),
    "blk_forward_graph_create": (c_int, [c_void_p, c_void_p, c_int, c_int, POINTER(blk_weights),
                                         POINTER(blk_kv_cache), c_int, c_void_p, c_void_p, c_size_t,
                                         POINTER(blk_taps), POINTER(c_void_p)]),
    "blk_graph_launch": (c_int, [c_void_p, c_void_p]),
    "blk_graph_destroy": (c_int, [c_void_p]),
    "blk_prepared_bytes": (c_size_t, [c_void_p]),
    "blk_prepare_weights": (c_int, [c_void_p, POINTER(blk_weights), c_void_p, c_size_t, c_void_p]),
    "blk_attn_decode_noalloc": (c_int, [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int, c_int, c_int,
                                        c_void_p, c_void_p]),
    "blk_model_workspace_bytes": (c_size_t, [c_void_p, c_int, c_int, c_int]),
    "blk_model_forward": (c_int, [c_void_p, POINTER(blk_model), c_void_p, c_int, c_int, POINTER(blk_kv_cache), c_int,
                                  c_void_p, c_void_p, c_size_t, c_void_p]),
}

_lib_handle = None


def lib():
    """Loads libblk.so (once). Raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(python -m llama_family_decoder_gb300.build)")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib_handle = h
    return _lib_handle


_fast_module = None


def fastcall():
    """The compiled argument handling of the packed calls (csrc/fastcall.cpp), built with the
    library and linked to it."""
    global _fast_module
    if _fast_module is None:
        import torch  # noqa: F401  (its libraries, which the module uses)
        lib()
        from . import _fastcall
        _fast_module = _fastcall
    return _fast_module


class BlkError(RuntimeError):
    def __init__(self, status, msg=""):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")


def _check(status):
    if status != BLK_OK:
        raise BlkError(status, lib().blk_last_error_message().decode())


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _on_stream(device, stream):
    """The device and stream that a call's own tensors (outputs, workspace) are made on and
    its kernels run on: the given stream, or the device's current one."""
    import torch
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError(f"stream: one of {device}, where the handle is, is wanted, got one of {stream.device}")
    return torch.cuda.stream(stream)


def _check_tensor(t, name, dtype, dev, shape):
    """The packed calls' check of a tensor: type, device (its number) and shape."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name}: {dtype} {list(shape)} on cuda:{dev} is wanted, got {t.dtype} {list(t.shape)} "
                         f"on {t.device}")


def _contiguous(t, name, dtype, dev, shape):
    """The address of a contiguous tensor of this type and shape."""
    _check_tensor(t, name, dtype, dev, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def xielu_effective(raw_alpha_p, raw_alpha_n, beta=0.5):
    ap, an = c_float(), c_float()
    lib().blk_xielu_effective(raw_alpha_p, raw_alpha_n, beta, ctypes.byref(ap), ctypes.byref(an))
    return ap.value, an.value


def set_wait_timeout_ns(ns: int):
    lib().blk_debug_set_wait_timeout_ns(int(ns))


def make_weights_struct(w: dict) -> blk_weights:
    """Page-named weight tensors (input_layernorm, q_proj, ...) -> blk_weights.

    The "afmoe" weights: attn_gate_proj (the attention gate), post_attn_norm and
    post_mlp_norm (the sandwich post-norms); post_attention_layernorm stays the
    MLP's input norm."""
    g = w.get
    return blk_weights(_ptr(g("input_layernorm")), _ptr(g("q_proj")), _ptr(g("k_proj")), _ptr(g("v_proj")),
                       _ptr(g("q_norm")), _ptr(g("k_norm")), _ptr(g("o_proj")), _ptr(g("post_attention_layernorm")),
                       _ptr(g("gate_proj")), _ptr(g("up_proj")), _ptr(g("down_proj")), _ptr(g("prepared")),
                       _ptr(g("attn_gate_proj")), _ptr(g("post_attn_norm")), _ptr(g("post_mlp_norm")))


class DecoderBlock:
    """One decoder block handle (blk_create) and its calls."""

    def __init__(self, hidden, n_heads, n_kv_heads, head_dim, ffn, act="silu", dtype="bf16", qk_norm=False,
                 rope_theta=10000.0, eps=1e-5, xielu_alpha_p=0.8, xielu_alpha_n=0.8, xielu_beta=0.5,
                 xielu_eps=-1e-6, max_batch=64, max_seq=4096, rope_scaling=None, sliding_window=0, use_rope=True,
                 attn_gate=False, sandwich_norm=False):
        # rope_scaling: None, or (kind, factor, original_max_position, low, high), kind "yarn" | "llama3"
        rs = (ROPE_TYPES[rope_scaling[0]], *rope_scaling[1:]) if rope_scaling else (0, 1.0, 0, 0.0, 0.0)
        self.desc = blk_desc(hidden, n_heads, n_kv_heads, head_dim, ffn, rope_theta, eps, ACTS[act],
                             xielu_alpha_p, xielu_alpha_n, xielu_beta, xielu_eps, int(bool(qk_norm)), DTYPES[dtype],
                             max_batch, max_seq, rs[0], float(rs[1]), int(rs[2]), float(rs[3]), float(rs[4]),
                             int(sliding_window), int(not use_rope), int(bool(attn_gate)), int(bool(sandwich_norm)))
        h = c_void_p()
        _check(lib().blk_create(ctypes.byref(self.desc), ctypes.byref(h)))
        self.handle = h
        self._ws = None
        import torch
        self._torch = torch
        self._dev = torch.cuda.current_device()  # where the handle's tables live
        self._device = torch.device("cuda", self._dev)
        self._dtype = torch.bfloat16 if self.desc.dtype == 1 else torch.float32
        self._sizes = n_heads, n_kv_heads, head_dim
        self._axes = {}  # (sections, interleaved) -> blk_rope_axes
        # the current stream's handle, without building a Stream object where torch has the short way
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda dev: torch.cuda.current_stream(dev).cuda_stream)

    @classmethod
    def from_workload(cls, wl, max_batch=None, max_seq=None):
        return cls(wl.hidden_size, wl.num_heads, wl.num_kv_heads, wl.head_dim, wl.intermediate_size,
                   act=wl.hidden_act, dtype=wl.dtype, qk_norm=wl.qk_norm, rope_theta=wl.rope_theta,
                   eps=wl.rms_norm_eps, xielu_alpha_p=wl.xielu_alpha_p, xielu_alpha_n=wl.xielu_alpha_n,
                   max_batch=max_batch or wl.batch, max_seq=max_seq or wl.cache_len + wl.seq,
                   rope_scaling=wl.rope_scaling, sliding_window=wl.sliding_window, use_rope=wl.use_rope,
                   attn_gate=wl.attn_gate, sandwich_norm=wl.sandwich_norm)

    @functools.cached_property
    def _fast(self):
        """The packed calls' short way, loaded at the first of them; what it returns None for takes the
        long one."""
        return fastcall()

    @functools.cached_property
    def _block(self):
        return fastcall().block(self.handle.value, *self._sizes, self.desc.dtype == 1, self._dev, self.desc.qk_norm,
                                self.desc.no_rope) if self.handle else None

    def close(self):
        if self.handle:
            self._block = None  # the short way is closed with the handle
            lib().blk_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prepare(self, weights, stream=None):
        """fp16 copies of wo / w_gate / w_up (blk_prepare_weights); returns weights plus 'prepared'."""
        import torch
        buf = torch.empty(max(lib().blk_prepared_bytes(self.handle), 16), dtype=torch.uint8,
                          device=weights["o_proj"].device)
        wst = make_weights_struct(weights)
        _check(lib().blk_prepare_weights(self.handle, ctypes.byref(wst), _ptr(buf), buf.numel(), _stream_ptr(stream)))
        return dict(weights, prepared=buf)

    def model_workspace_bytes(self, batch, seq, decode=False):
        return lib().blk_model_workspace_bytes(self.handle, batch, seq, int(bool(decode)))

    def workspace_bytes(self, batch, seq, decode=False):
        return lib().blk_workspace_bytes(self.handle, batch, seq, int(decode))

    def stage_workspace_bytes(self, rows):
        return lib().blk_stage_workspace_bytes(self.handle, rows)

    def _workspace(self, nbytes, device):
        import torch
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
        return self._ws

    def forward(self, x, weights, cache=None, out=None, workspace=None, taps=None, stream=None, host_lens_max=-1,
                attention_mask=None):
        """out = block(x); x [B, T, D] device tensor. cache: dict(k, v, lens): T new tokens per
        sequence after lens[b] cached positions (a decode step for T == 1, a prefill chunk for
        T > 1, which needs host_lens_max = max(lens)). attention_mask: device int32 [B, T] of a
        padded prefill batch (blk_forward_masked; zeros are padding)."""
        import torch
        B, T, _ = x.shape
        if out is None:
            out = torch.empty_like(x)
        need = self.workspace_bytes(B, T, cache is not None)
        if workspace is None:
            workspace = self._workspace(need, x.device)
        ws_bytes = workspace.numel() * workspace.element_size()
        wst = weights if isinstance(weights, blk_weights) else make_weights_struct(weights)
        kvc = None
        if cache is not None:
            kvc = blk_kv_cache(_ptr(cache["k"]), _ptr(cache["v"]), cache["k"].shape[2], _ptr(cache["lens"]))
        tp = None
        if taps:
            tp = blk_taps(*[_ptr(taps.get(n)) for n in TAP_NAMES])
        if attention_mask is not None:
            if cache is not None:
                raise ValueError("attention_mask: prefill batches only")
            _check(lib().blk_forward_masked(self.handle, _ptr(x), B, T, _ptr(attention_mask), ctypes.byref(wst),
                                            _ptr(out), _ptr(workspace), ws_bytes,
                                            ctypes.byref(tp) if tp is not None else None, _stream_ptr(stream)))
            return out
        _check(lib().blk_forward(self.handle, _ptr(x), B, T, ctypes.byref(wst),
                                 ctypes.byref(kvc) if kvc is not None else None, int(host_lens_max), _ptr(out),
                                 _ptr(workspace), ws_bytes, ctypes.byref(tp) if tp is not None else None,
                                 _stream_ptr(stream)))
        return out

    def model_forward(self, tokens, layers, embed, norm_g, lm_head, caches=None, host_lens_max=-1, logits=None,
                      workspace=None, stream=None):
        """logits [B, T, vocab] of the model around this block's shape: embed[tokens], the
        layers (a list of weight dicts), the final norm and lm_head. tokens: device int32
        [B, T]. caches: None, or one dict(k, v, lens) per layer (T new tokens after lens)."""
        import torch
        B, T = tokens.shape
        vocab = embed.shape[0]
        if logits is None:
            logits = torch.empty(B, T, vocab, dtype=embed.dtype, device=tokens.device)
        need = lib().blk_model_workspace_bytes(self.handle, B, T, int(caches is not None))
        if workspace is None:
            workspace = self._workspace(need, tokens.device)
        wls = (blk_weights * len(layers))(*[make_weights_struct(w) for w in layers])
        m = blk_model(_ptr(embed), wls, len(layers), _ptr(norm_g), _ptr(lm_head), vocab)
        kvs = None
        if caches is not None:
            kvs = (blk_kv_cache * len(caches))(*[blk_kv_cache(_ptr(c["k"]), _ptr(c["v"]), c["k"].shape[2],
                                                              _ptr(c["lens"])) for c in caches])
        _check(lib().blk_model_forward(self.handle, ctypes.byref(m), _ptr(tokens), B, T, kvs, host_lens_max,
                                       _ptr(logits), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream_ptr(stream)))
        return logits

    def forward_graph(self, x, weights, out, workspace, cache=None, taps=None, host_lens_max=-1):
        """Records blk_forward for these exact buffers into a CUDA graph (ForwardGraph)."""
        B, T, _ = x.shape
        wst = weights if isinstance(weights, blk_weights) else make_weights_struct(weights)
        kvc = None
        if cache is not None:
            kvc = blk_kv_cache(_ptr(cache["k"]), _ptr(cache["v"]), cache["k"].shape[2], _ptr(cache["lens"]))
        tp = blk_taps(*[_ptr(taps.get(n)) for n in TAP_NAMES]) if taps else None
        g = c_void_p()
        _check(lib().blk_forward_graph_create(self.handle, _ptr(x), B, T, ctypes.byref(wst),
                                              ctypes.byref(kvc) if kvc is not None else None, int(host_lens_max),
                                              _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                              ctypes.byref(tp) if tp is not None else None, ctypes.byref(g)))
        return ForwardGraph(g, keep=(x, weights, out, workspace, cache, taps, wst, kvc, tp))

    def qkv_rope(self, y, weights, batch, seq, q, k, v, pos0=None, stream=None):
        need = self.stage_workspace_bytes(batch * seq)
        ws = self._workspace(need, y.device)
        wst = make_weights_struct(weights)
        _check(lib().blk_qkv_rope(self.handle, _ptr(y), ctypes.byref(wst), batch, seq, _ptr(pos0), _ptr(q), _ptr(k),
                                  _ptr(v), _ptr(ws), ws.numel(), _stream_ptr(stream)))

    def attn_gqa(self, q, k, v, o, kv_lens=None, stream=None):
        B, H, Tq, _ = q.shape
        kv_stride = k.shape[2]
        ws = self._workspace(self.stage_workspace_bytes(B * Tq), q.device)
        _check(lib().blk_attn_gqa(self.handle, _ptr(q), _ptr(k), _ptr(v), B, Tq, kv_stride, _ptr(kv_lens), _ptr(o),
                                  _ptr(ws), ws.numel(), _stream_ptr(stream)))

    # Packed, mixed-length batches and the 4-bit cache. Outputs not passed, and every
    # workspace, are made for the call on its stream: calls on several streams, and captured
    # graphs, share none.

    def _rows(self, t, name, shape):
        """A [rows, heads, d] tensor, of any row and head strides, as blk_head_rows."""
        if t.dtype is not self._dtype or t.get_device() != self._dev or t.shape != shape:
            _check_tensor(t, name, self._dtype, self._dev, shape)
        rs, hs, cs = t.stride()
        if cs != 1:
            raise ValueError(f"{name}: the channels must be contiguous")
        return head_rows(t.data_ptr(), rs, hs)

    def _out(self, t, name, shape):
        """An output and its blk_head_rows: the given tensor, or a new one."""
        if t is not None:
            return t, self._rows(t, name, shape)
        t = self._torch.empty(shape, dtype=self._dtype, device=self._device)
        return t, head_rows(t.data_ptr(), shape[1] * shape[2], shape[2])

    def _int32(self, t, name, n):
        return None if t is None else _contiguous(t, name, self._torch.int32, self._dev, (n,))

    def _elsewhere(self, stream):
        """Whether a call has to switch to its stream or to the handle's device first."""
        return stream is not None or self._torch.cuda.current_device() != self._dev

    def qk_norm_rope(self, q, k, positions, q_gain=None, k_gain=None, sections=None, interleaved=False, q_out=None,
                     k_out=None, stream=None):
        """Per-head RMSNorm (a qk_norm handle, with gains [d]) and rotary of packed rows q [N, H, d]
        and k [N, Hkv, d], of any row and head strides. positions: int32 [N], or [axes, N] with
        `sections`, the rotary pairs of each axis (one after the other, or interleaved). Returns
        (q_out, k_out), [N, heads, d]; pass q and k as outputs to work in place."""
        if stream is None:
            r = self._fast.qk_norm_rope(self._block, q, k, positions, q_gain, k_gain, sections, interleaved, q_out, k_out)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.qk_norm_rope(q, k, positions, q_gain, k_gain, sections, interleaved, q_out, k_out)
        H, Hkv, d = self._sizes
        n = q.shape[0]
        axes = pos = gq = gk = None
        if not self.desc.no_rope:
            n_axes = 1
            if sections is not None:
                key = (*sections, bool(interleaved))
                axes = self._axes.get(key)
                n_axes = len(key) - 1
                if axes is None:
                    if not 1 <= n_axes <= 4:
                        raise ValueError("sections: 1 to 4 position axes")
                    axes = self._axes[key] = blk_rope_axes(n_axes, (c_int * 4)(*sections), int(key[-1]))
            shape = (n,) if n_axes == 1 and positions.dim() == 1 else (n_axes, n)
            pos = _contiguous(positions, "positions", self._torch.int32, self._dev, shape)
        if self.desc.qk_norm:
            if q_gain is None or k_gain is None:
                raise ValueError("q_gain, k_gain: the handle norms queries and keys")
            gq = _contiguous(q_gain, "q_gain", self._dtype, self._dev, (d,))
            gk = _contiguous(k_gain, "k_gain", self._dtype, self._dev, (d,))
        qs, ks = (n, H, d), (n, Hkv, d)
        qi, ki = self._rows(q, "q", qs), self._rows(k, "k", ks)
        q_out, qo = self._out(q_out, "q_out", qs)
        k_out, ko = self._out(k_out, "k_out", ks)
        _check(lib().blk_qk_norm_rope(self.handle, qi, ki, n, pos, axes, gq, gk, qo, ko, self._raw_stream(self._dev)))
        return q_out, k_out

    def attn_packed(self, q, k, v, cu_seqlens, out=None, stream=None):
        """Causal attention over packed whole prompts: q [N, H, d], k, v [N, Hkv, d], of any row and
        head strides; cu_seqlens int32 [B + 1]: sequence b is rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1.
        Returns out [N, H, d]; rows of no sequence are left as they were (undefined in an out
        made here)."""
        if stream is None:
            r = self._fast.attn_packed(self._block, q, k, v, cu_seqlens, out)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.attn_packed(q, k, v, cu_seqlens, out)
        H, Hkv, d = self._sizes
        n, batch = q.shape[0], cu_seqlens.numel() - 1
        qs, ks = (n, H, d), (n, Hkv, d)
        cu = self._int32(cu_seqlens, "cu_seqlens", batch + 1)
        qi, ki, vi = self._rows(q, "q", qs), self._rows(k, "k", ks), self._rows(v, "v", ks)
        out, o = self._out(out, "out", qs)
        nbytes = lib().blk_attn_packed_workspace_bytes(self.handle, n, batch)
        ws = self._torch.empty(nbytes, dtype=self._torch.uint8, device=self._device) if nbytes else None
        _check(lib().blk_attn_packed(self.handle, qi, ki, vi, n, cu, batch, o, ws.data_ptr() if nbytes else None,
                                     nbytes, self._raw_stream(self._dev)))
        return out

    def kv4_cache(self, batch, capacity):
        """An empty KV cache in 4 bits: dict(k, k_scale, v, v_scale, lens)."""
        torch = self._torch
        n = (batch, self._sizes[1], capacity)
        c = {"lens": torch.zeros(batch, dtype=torch.int32, device=self._device)}
        for x in ("k", "v"):
            c[x] = torch.zeros(*n, 64, dtype=torch.uint8, device=self._device)
            c[x + "_scale"] = torch.zeros(*n, 8, dtype=torch.bfloat16, device=self._device)
        return c

    def _kv4(self, cache):
        torch, dev = self._torch, self._dev
        batch, Hkv, cap, _ = cache["k"].shape
        if Hkv != self._sizes[1]:
            raise ValueError(f"cache: {self._sizes[1]} KV heads are wanted, got {Hkv}")
        codes, scales = (batch, Hkv, cap, 64), (batch, Hkv, cap, 8)
        return kv4_cache_struct(_contiguous(cache["k"], "cache k", torch.uint8, dev, codes),
                                _contiguous(cache["k_scale"], "cache k_scale", torch.bfloat16, dev, scales),
                                _contiguous(cache["v"], "cache v", torch.uint8, dev, codes),
                                _contiguous(cache["v_scale"], "cache v_scale", torch.bfloat16, dev, scales), cap,
                                _contiguous(cache["lens"], "cache lens", torch.int32, dev, (batch,))), batch

    def kv4_store(self, cache, k, v, cu_seqlens=None, starts=None, host_lens_max=-1, stream=None):
        """Quantises rows k, v [N, Hkv, 128] into the cache: sequence b's rows (cu_seqlens as in
        attn_packed; None: row b alone) to slots starts[b], ... (None: lens[b], an append), and sets
        lens[b] behind them. host_lens_max: the largest new length, to have the capacity checked
        here; else rows that do not fit are left out and last_status() says so."""
        if stream is None and self._fast.kv4_store(self._block, cache, k, v, cu_seqlens, starts, host_lens_max):
            return
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.kv4_store(cache, k, v, cu_seqlens, starts, host_lens_max)
        c, batch = self._kv4(cache)
        n = k.shape[0]
        shape = (n, *self._sizes[1:])
        _check(lib().blk_kv4_store(self.handle, self._rows(k, "k", shape), self._rows(v, "v", shape), n,
                                   self._int32(cu_seqlens, "cu_seqlens", batch + 1),
                                   self._int32(starts, "starts", batch), batch, c, host_lens_max,
                                   self._raw_stream(self._dev)))

    def kv4_load(self, cache, cu_seqlens=None, rows=None, starts=None, k_out=None, v_out=None, stream=None):
        """The values of the cache's slots starts[b], ... (None: 0, ...) as packed bf16 rows (k, v)
        [rows, Hkv, 128]: the rows that cu_seqlens gives each sequence (None: one each). cu_seqlens
        is on the device, so with it the number of rows is wanted."""
        if stream is None:
            r = self._fast.kv4_load(self._block, cache, cu_seqlens, rows, starts, k_out, v_out)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.kv4_load(cache, cu_seqlens, rows, starts, k_out, v_out)
        if cu_seqlens is not None and rows is None:
            raise ValueError("rows: how many packed rows cu_seqlens stands for is wanted")
        c, batch = self._kv4(cache)
        n = batch if rows is None else rows
        shape = (n, *self._sizes[1:])
        cu, st = self._int32(cu_seqlens, "cu_seqlens", batch + 1), self._int32(starts, "starts", batch)
        k_out, ko = self._out(k_out, "k_out", shape)
        v_out, vo = self._out(v_out, "v_out", shape)
        _check(lib().blk_kv4_load(self.handle, c, cu, st, batch, n, ko, vo, self._raw_stream(self._dev)))
        return k_out, v_out

    def attn_decode_kv4(self, q, cache, out=None, stream=None):
        """One query per sequence, q [B, H, 128], over the lens[b] slots of the 4-bit cache (the last
        sliding_window of them). Returns out [B, H, 128]; a sequence without keys gets zeros."""
        if stream is None:
            r = self._fast.attn_decode_kv4(self._block, q, cache, out)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.attn_decode_kv4(q, cache, out)
        c, batch = self._kv4(cache)
        H, _, d = self._sizes
        qi = self._rows(q, "q", (batch, H, d))
        out, o = self._out(out, "out", (batch, H, d))
        nbytes = lib().blk_attn_decode_kv4_workspace_bytes(self.handle, batch, cache["k"].shape[2])
        ws = self._torch.empty(nbytes, dtype=self._torch.uint8, device=self._device) if nbytes else None
        _check(lib().blk_attn_decode_kv4(self.handle, qi, c, batch, o, ws.data_ptr() if nbytes else None, nbytes,
                                         self._raw_stream(self._dev)))
        return out

    # Speculative decoding over a paged cache: a step's new rows (one token, a chain or a tree of drafts)
    # are appended, attend, and are verified; what is kept of them then moves lens.

    def paged_cache(self, batch, capacity, page_size=64, n_pages=None, shared=None):
        """An empty paged KV cache of this handle's type: dict(k, v, pages, lens), each sequence with pages
        of its own for `capacity` slots. n_pages: pages to make instead, with the page table filled with
        -1 for the caller to deal them out. shared: another layer's cache, whose pages and lens this one uses."""
        torch = self._torch
        if shared is not None:
            return dict(shared, k=torch.zeros_like(shared["k"]), v=torch.zeros_like(shared["v"]))
        per = -(-capacity // page_size)
        if n_pages is None:
            n_pages = batch * per
            pages = torch.arange(n_pages, dtype=torch.int32, device=self._device).view(batch, per)
        else:
            pages = torch.full((batch, per), -1, dtype=torch.int32, device=self._device)
        shape = (n_pages, self._sizes[1], page_size, self._sizes[2])
        return {"k": torch.zeros(shape, dtype=self._dtype, device=self._device),
                "v": torch.zeros(shape, dtype=self._dtype, device=self._device),
                "pages": pages, "lens": torch.zeros(batch, dtype=torch.int32, device=self._device)}

    def rope_table(self, dims=None, max_pos=None, stream=None):
        """The (cos, sin) table [max_pos, dims / 2, 2] of the handle's rotary over the first `dims` channels
        of a head, for paged_append's rope_table."""
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.rope_table(dims, max_pos)
        dims = self._sizes[2] if dims is None else dims
        max_pos = self.desc.max_seq if max_pos is None else max_pos
        if dims < 2 or dims % 2 or max_pos <= 0:
            raise ValueError("dims, max_pos: an even number of channels and a positive number of positions")
        t = self._torch.empty(max_pos, dims // 2, 2, dtype=self._torch.float32, device=self._device)
        _check(lib().blk_rope_table(self.handle, dims, max_pos, t.data_ptr(), self._raw_stream(self._dev)))
        return t

    def _paged(self, cache):
        torch, dev = self._torch, self._dev
        if cache["k"].dim() != 4 or cache["pages"].dim() != 2:
            raise ValueError("cache: k is [pages, KV heads, page_size, d] and pages [batch, max_pages]")
        n_pages, _, page_size, _ = cache["k"].shape
        batch, max_pages = cache["pages"].shape
        shape = (n_pages, self._sizes[1], page_size, self._sizes[2])
        return paged_cache_struct(_contiguous(cache["k"], "cache k", self._dtype, dev, shape),
                                  _contiguous(cache["v"], "cache v", self._dtype, dev, shape),
                                  _contiguous(cache["pages"], "cache pages", torch.int32, dev, (batch, max_pages)),
                                  _contiguous(cache["lens"], "cache lens", torch.int32, dev, (batch,)),
                                  n_pages, page_size, max_pages), batch

    def paged_append(self, cache, q, k, v, cu_seqlens=None, depths=None, q_gain=None, k_gain=None, rope_table=None,
                     interleaved=False, q_out=None, host_lens_max=-1, stream=None):
        """Per-head RMSNorm (a qk_norm handle, with gains [d]) and rotary of rows q [N, H, d] and k [N, Hkv, d], of any
        row and head strides like v [N, Hkv, d]; keys and values go behind the paged cache's lens, which do
        not move. Row i of sequence b (cu_seqlens as in attn_packed; None: row b alone) has position
        lens[b] + depths[row] (None: lens[b] + i). rope_table: fp32 [max_pos, dims / 2, 2] (rope_table()), None: the
        handle's; interleaved: pairs of neighbouring channels. Returns q_out [N, H, d]; pass q to work in
        place. host_lens_max: the largest slot behind a row, to have the capacity checked here."""
        if stream is None:
            r = self._fast.paged_append(self._block, cache, q, k, v, cu_seqlens, depths, q_gain, k_gain, rope_table,
                                        interleaved, q_out, host_lens_max)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.paged_append(cache, q, k, v, cu_seqlens, depths, q_gain, k_gain, rope_table, interleaved,
                                         q_out, host_lens_max)
        H, Hkv, d = self._sizes
        n = q.shape[0]
        c, batch = self._paged(cache)
        layout = gq = gk = None
        if not self.desc.no_rope and (rope_table is not None or interleaved):
            at, dims, max_pos = None, d, self.desc.max_seq
            if rope_table is not None:
                max_pos, half = rope_table.shape[0], rope_table.shape[1] if rope_table.dim() == 3 else 0
                at, dims = _contiguous(rope_table, "rope_table", self._torch.float32, self._dev, (max_pos, half, 2)), 2 * half
            layout = rope_layout_struct(at or 0, dims, max_pos, int(bool(interleaved)))
        if self.desc.qk_norm:
            if q_gain is None or k_gain is None:
                raise ValueError("q_gain, k_gain: the handle norms queries and keys")
            gq = _contiguous(q_gain, "q_gain", self._dtype, self._dev, (d,))
            gk = _contiguous(k_gain, "k_gain", self._dtype, self._dev, (d,))
        qs, ks = (n, H, d), (n, Hkv, d)
        qi, ki, vi = self._rows(q, "q", qs), self._rows(k, "k", ks), self._rows(v, "v", ks)
        cu, dp = self._int32(cu_seqlens, "cu_seqlens", batch + 1), self._int32(depths, "depths", n)
        q_out, qo = self._out(q_out, "q_out", qs)
        _check(lib().blk_paged_append(self.handle, qi, ki, vi, n, cu, dp, batch, c, layout, gq, gk, qo, host_lens_max,
                                      self._raw_stream(self._dev)))
        return q_out

    def attn_paged(self, q, cache, cu_seqlens=None, parents=None, out=None, stream=None):
        """Attention of the appended rows q [N, H, 128], of any row and head strides, over the paged cache: row i of
        sequence b sees the slots below lens[b] and its ancestors' and its own. parents: int32 [N], each row's
        parent within its sequence (-1: none), at most 64 rows a sequence; None: chains. Returns out
        [N, H, 128]; rows of no sequence are left as they were (undefined in an out made here)."""
        if stream is None:
            r = self._fast.attn_paged(self._block, q, cache, cu_seqlens, parents, out)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.attn_paged(q, cache, cu_seqlens, parents, out)
        H, _, d = self._sizes
        n = q.shape[0]
        c, batch = self._paged(cache)
        qi = self._rows(q, "q", (n, H, d))
        cu, up = self._int32(cu_seqlens, "cu_seqlens", batch + 1), self._int32(parents, "parents", n)
        out, o = self._out(out, "out", (n, H, d))
        nbytes = lib().blk_attn_paged_workspace_bytes(self.handle, n, cu is not None, up is not None, batch, c)
        ws = self._torch.empty(nbytes, dtype=self._torch.uint8, device=self._device) if nbytes else None
        _check(lib().blk_attn_paged(self.handle, qi, n, cu, up, batch, c, o, ws.data_ptr() if nbytes else None, nbytes,
                                    self._raw_stream(self._dev)))
        return out

    def _probs(self, t, name, shape):
        """Rows of probabilities (address, row stride), of any row stride."""
        _check_tensor(t, name, self._torch.float32, self._dev, shape)
        if t.stride(1) != 1 and shape[1] > 1:
            raise ValueError(f"{name}: the vocabulary must be contiguous")
        return t.data_ptr(), t.stride(0)

    def verify_drafts(self, target, tokens, u, u_next, cu_seqlens=None, parents=None, draft=None, stream=None):
        """Speculative sampling over each sequence's rows, row 0 its last token and the others drafts: target fp32
        [N, vocab], the target's probabilities of what follows each row; draft None (candidates without
        probabilities), or likewise the distribution each row's children were drawn from; tokens int32 [N]; u fp32 [N]
        and u_next [B], uniform in [0, 1). cu_seqlens and parents as in attn_paged, at most 64 rows a sequence.
        Returns int32 (counts [B], path [N], next [B]): how many rows stay, which (-1 behind them), and the
        token that follows."""
        if stream is None:
            r = self._fast.verify_drafts(self._block, target, tokens, u, u_next, cu_seqlens, parents, draft)
            if r is not None:
                return r
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.verify_drafts(target, tokens, u, u_next, cu_seqlens, parents, draft)
        torch, dev = self._torch, self._dev
        if target.dim() != 2:
            raise ValueError("target: [rows, vocab] is wanted")
        n, vocab = target.shape
        batch = u_next.numel()
        t, t_row = self._probs(target, "target", (n, vocab))
        g, g_row = (None, 0) if draft is None else self._probs(draft, "draft", (n, vocab))
        tok, up = self._int32(tokens, "tokens", n), self._int32(parents, "parents", n)
        if tok is None:
            raise ValueError("tokens: the rows' tokens are wanted")
        cu = self._int32(cu_seqlens, "cu_seqlens", batch + 1)
        ua, un = _contiguous(u, "u", torch.float32, dev, (n,)), _contiguous(u_next, "u_next", torch.float32, dev, (batch,))
        counts, path, nxt = (torch.empty(k, dtype=torch.int32, device=self._device) for k in (batch, n, batch))
        _check(lib().blk_verify_drafts(self.handle, t, t_row, g, g_row, n, vocab, tok, up, cu, ua, un, batch,
                                       counts.data_ptr(), path.data_ptr(), nxt.data_ptr(), self._raw_stream(dev)))
        return counts, path, nxt

    def paged_keep(self, caches, counts, path=None, cu_seqlens=None, starts=None, stream=None):
        """Keeps the first counts[b] rows of path (int32 [B] and [N], as from verify_drafts) of each sequence: their keys
        and values move to the slots from starts[b] (None: lens[b]) on in every layer's cache (a list; they
        share pages and lens), and lens[b] behind them. path None: lens alone moves by counts (whole
        prompts, a chain's first rows)."""
        if stream is None and self._fast.paged_keep(self._block, caches, counts, path, cu_seqlens, starts):
            return
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.paged_keep(caches, counts, path, cu_seqlens, starts)
        structs = [self._paged(c) for c in caches]
        if not structs:
            raise ValueError("caches: one at least")
        batch, n = structs[0][1], 0 if path is None else path.shape[0]
        _check(lib().blk_paged_keep(self.handle, b"".join(s for s, _ in structs), len(structs),
                                    self._int32(counts, "counts", batch), self._int32(path, "path", n),
                                    self._int32(cu_seqlens, "cu_seqlens", batch + 1), self._int32(starts, "starts", batch),
                                    batch, n, self._raw_stream(self._dev)))

    def model_forward_paged(self, tokens, layers, embed, norm_g, lm_head, caches, cu_seqlens=None, depths=None,
                            parents=None, temperature=None, out=None, host_lens_max=-1, stream=None):
        """The model (as in model_forward) over new rows of paged caches, one per layer (paged_cache, shared): tokens
        int32 [N], packed by cu_seqlens, are appended behind lens, which do not move, and attend (paged_append,
        attn_paged; a tree's rows need depths and parents). Returns the logits, bf16 [N, vocab], or with a
        temperature the probabilities softmax(logits / temperature), fp32 [N, vocab] (0: all on the largest)."""
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.model_forward_paged(tokens, layers, embed, norm_g, lm_head, caches, cu_seqlens, depths, parents,
                                                temperature, out, host_lens_max)
        torch, dev = self._torch, self._dev
        if len(caches) != len(layers) or not caches:
            raise ValueError("caches: one for each layer")
        if temperature is not None and not temperature >= 0:
            raise ValueError("temperature: 0 or more")
        n, vocab = tokens.shape[0], embed.shape[0]
        structs = [self._paged(c) for c in caches]
        batch = structs[0][1]
        tok = self._int32(tokens, "tokens", n)
        cu = self._int32(cu_seqlens, "cu_seqlens", batch + 1)
        dp, up = self._int32(depths, "depths", n), self._int32(parents, "parents", n)
        for t, name, shape in ((embed, "embed", (vocab, self.desc.hidden)), (lm_head, "lm_head", (vocab, self.desc.hidden)),
                               (norm_g, "norm_g", (self.desc.hidden,))):
            _contiguous(t, name, self._dtype, dev, shape)
        dtype = self._dtype if temperature is None else torch.float32
        if out is None:
            out = torch.empty(n, vocab, dtype=dtype, device=self._device)
        else:
            _contiguous(out, "out", dtype, dev, (n, vocab))
        wls = (blk_weights * len(layers))(*[make_weights_struct(w) for w in layers])
        m = blk_model(_ptr(embed), wls, len(layers), _ptr(norm_g), _ptr(lm_head), vocab)
        nbytes = lib().blk_model_paged_workspace_bytes(self.handle, n, cu is not None, up is not None, batch, structs[0][0],
                                                       vocab, temperature is not None)
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self._device)
        _check(lib().blk_model_forward_paged(self.handle, ctypes.byref(m), tok, n, cu, dp, up, batch,
                                             b"".join(s for s, _ in structs), -1.0 if temperature is None else temperature,
                                             host_lens_max, out.data_ptr(), ws.data_ptr(), nbytes, self._raw_stream(dev)))
        return out

    def model_verify(self, tokens, layers, embed, norm_g, lm_head, caches, u, u_next, cu_seqlens=None, depths=None,
                     parents=None, temperature=1.0, draft=None, host_lens_max=-1, stream=None):
        """A step of speculative decoding: the model over each sequence's last token and its drafts
        (model_forward_paged), their verification with the given random numbers (verify_drafts), and the kept
        rows moved behind lens in every layer's cache (paged_keep). Returns (counts, path, next). A sequence whose rows
        pass its page list (status CACHE_FULL) is left alone; what is returned for it means nothing."""
        if self._elsewhere(stream):
            with _on_stream(self._device, stream):
                return self.model_verify(tokens, layers, embed, norm_g, lm_head, caches, u, u_next, cu_seqlens, depths, parents,
                                         temperature, draft, host_lens_max)
        p = self.model_forward_paged(tokens, layers, embed, norm_g, lm_head, caches, cu_seqlens, depths, parents, temperature,
                                     host_lens_max=host_lens_max)
        counts, path, token = self.verify_drafts(p, tokens, u, u_next, cu_seqlens, parents, draft)
        self.paged_keep(caches, counts, path, cu_seqlens)
        return counts, path, token

    def mlp(self, resid, h_normed, weights, out, stream=None):
        rows = resid.numel() // resid.shape[-1]
        ws = self._workspace(self.stage_workspace_bytes(rows), resid.device)
        wst = make_weights_struct(weights)
        _check(lib().blk_mlp(self.handle, _ptr(resid), _ptr(h_normed), ctypes.byref(wst), rows, _ptr(out), _ptr(ws),
                             ws.numel(), _stream_ptr(stream)))

    def last_status(self):
        return lib().blk_last_status(self.handle)

    def profile(self, on=True):
        _check(lib().blk_profile_enable(self.handle, int(bool(on))))

    def profile_reset(self):
        lib().blk_profile_reset(self.handle)

    def profile_collect(self):
        """Waits for the last profiled forward; returns {stage: (total_ms, launches)}."""
        n_max = 24
        ms = (ctypes.c_double * n_max)()
        ln = (c_longlong * n_max)()
        n = lib().blk_profile_collect(self.handle, ms, ln, n_max)
        if n < 0:
            raise BlkError(5, "profiling is off or a CUDA error occurred")
        return {lib().blk_profile_stage_name(self.handle, i).decode(): (ms[i], ln[i]) for i in range(n)}


class ForwardGraph:
    """A recorded blk_forward (blk_graph); launch() replays it on a stream."""

    def __init__(self, handle, keep):
        self.handle = handle
        self._keep = keep  # the buffers the graph reads and writes stay alive with it

    def launch(self, stream=None):
        _check(lib().blk_graph_launch(self.handle, _stream_ptr(stream)))

    def close(self):
        if self.handle:
            lib().blk_graph_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rmsnorm(x, g, eps=1e-5, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty_like(x)
    n = x.shape[-1]
    rows = x.numel() // n
    dt = 1 if x.dtype == torch.bfloat16 else 0
    _check(lib().blk_rmsnorm(_ptr(x), _ptr(g), rows, n, eps, _ptr(out), dt, _stream_ptr(stream)))
    return out


def debug_gemm_bf16(a, b, bn=256, split_k=1, out=None, stream=None, pair=False):
    """c = a @ b.T on the bare tcgen05 GEMM (bf16 out), or fp32 split-K partials [split, N, M];
    pair: CTA pairs with 256-row tiles."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        if split_k == 1:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
        else:
            out = torch.empty(split_k, M, N, dtype=torch.float32, device=a.device)
    _check(lib().blk_debug_gemm_bf16(_ptr(a), _ptr(b), _ptr(out), M, N, K, bn, split_k, 1 if pair else 0,
                                     _stream_ptr(stream)))
    return out


def attn_decode_noalloc(q, k, v, kv_lens, o, stream=None):
    """Decode attention through blk_attn_decode_noalloc (no workspace, no handle).

    q [B, H, 1, d], k/v [B, Hkv, kv_stride, d], kv_lens int32 [B], o [B, 1, H, d]; bf16 on the device.
    """
    B, H = q.shape[0], q.shape[1]
    Hkv, kv_stride, d = k.shape[1], k.shape[2], k.shape[3]
    _check(lib().blk_attn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_lens), B, H, Hkv, d, kv_stride, _ptr(o),
                                         _stream_ptr(stream)))
    return o

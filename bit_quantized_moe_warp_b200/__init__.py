"""Python binding of the B200 routed-expert MoE layer (libstrata_moe.so).

Argument marshalling only: every function below forwards to the C ABI of
``include/strata_moe.h`` with the same name; tensors may be passed as torch
tensors (their ``data_ptr()``) or as integer device addresses. Every step of
the layer runs in the library's sm_100a kernels. Importing this package fails
loudly when the shared library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# STRATA_MOE_LIB selects another build of the same library (e.g. the checked build,
# libstrata_moe_checked.so)
LIB_PATH = os.environ.get("STRATA_MOE_LIB") or os.path.join(_HERE, "libstrata_moe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_quantized_moe_warp_b200.build` "
                      "(or __graft_entry__.build())")

_lib = ctypes.CDLL(LIB_PATH)

# status codes (include/strata_moe.h)
STRATA_OK = 0
STRATA_ERR_INVALID_ARG = -1
STRATA_ERR_UNSUPPORTED = -2
STRATA_ERR_CUDA = -3
STRATA_ERR_OOM = -4
STRATA_ERR_TOO_MANY_TOKENS = -5
STRATA_ERR_BAD_BLOB = -6
STRATA_ERR_TIMEOUT = -7
STRATA_ERR_BOUNDS = -8

STRATA_FMT_Q2_0_TILED = 1
STRATA_FMT_Q4_0_TILED = 2
STRATA_ACCUMULATE = 1
STRATA_FORCE_PREFILL = 2
STRATA_DECODE_MAX_TOKENS = 16
STRATA_Q2_TILE_BYTES = 1280
STRATA_Q4_TILE_BYTES = 2304
STRATA_KV4_BLOCK = 32  # include/strata_kv.h
# include/strata_attn.h
STRATA_ROPE_HALF = 0
STRATA_ROPE_INTERLEAVED = 1
STRATA_ROPE_SCALE_NONE = 0
STRATA_ROPE_SCALE_LINEAR = 1
STRATA_ROPE_SCALE_NTK = 2
STRATA_ROPE_SCALE_YARN = 3
STRATA_ROPE_MAX_HEAD_DIM = 256
FORMAT_OF_BITS = {2: STRATA_FMT_Q2_0_TILED, 4: STRATA_FMT_Q4_0_TILED}


class strata_moe_desc(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("weight_format", ctypes.c_int32), ("flags", ctypes.c_uint32), ("router_bias", ctypes.c_void_p)]


class strata_rope_desc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_max_position", ctypes.c_int32), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("attn_factor", ctypes.c_double)]


class strata_kv4_cache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("n_kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class strata_kv4_attn_desc(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("max_q_len", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_tokens", ctypes.c_int64), ("q_token_stride", ctypes.c_int64),
                ("out_token_stride", ctypes.c_int64), ("window", ctypes.c_int32), ("scale", ctypes.c_float)]


class StrataError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_lib.strata_status_string(status).decode()} ({status}): {msg}")
        self.status = status


V, I32, SZ, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int64
DP = ctypes.POINTER(strata_moe_desc)
_SIGS = {
    "strata_q2_matrix_bytes": (SZ, [I32, I32]),
    "strata_q4_matrix_bytes": (SZ, [I32, I32]),
    "strata_moe_expert_bytes": (SZ, [DP]),
    "strata_moe_expert_blob_bytes": (SZ, [DP]),
    "strata_moe_workspace_bytes": (SZ, [DP]),
    "strata_moe_layer_create": (I32, [DP, V, SZ, ctypes.POINTER(V)]),
    "strata_moe_layer_destroy": (I32, [V]),
    "strata_moe_forward": (I32, [V, V, V, V, V, I32, V]),
    "strata_moe_router_logits": (I32, [V, V, V, V, I32, V]),
    "strata_moe_route": (I32, [V, V, V, I32, V]),
    "strata_moe_experts": (I32, [V, V, V, V, I32, V]),
    "strata_moe_get_routing": (I32, [V, V, V, V, V, V, V]),
    "strata_moe_route_noalloc": (I32, [DP, V, V, I32, V, V, V, V, V, V]),
    "strata_moe_stack_forward": (I32, [V, I32, V, V, V, V, I32, ctypes.c_float, V]),
    "strata_rmsnorm_bf16": (I32, [V, V, I32, I32, ctypes.c_float, V]),
    "strata_moe_set_stage_events": (I32, [V, V, I32]),
    "strata_moe_check_status": (I32, [V]),
    "strata_q2_pack": (I32, [V, V, I32, I32, V]),
    "strata_q4_pack": (I32, [V, V, I32, I32, V]),
    "strata_moe_pack_expert": (I32, [DP, V, V, V, V, V, V, V]),
    "strata_moe_pack_expert_device": (I32, [DP, V, V, V, V, V, V, V, V]),
    "strata_selftest_wait_timeout": (I32, [ctypes.c_uint64, V]),
    "strata_selftest_bounds_check": (I32, [V]),
    "strata_is_checked_build": (I32, []),
    "strata_kv4_code_bytes": (SZ, [ctypes.c_int64, I32]),
    "strata_kv4_scale_bytes": (SZ, [ctypes.c_int64, I32]),
    "strata_kv4_encode": (I32, [V, ctypes.c_int64, I32, V, V, V]),
    "strata_kv4_decode": (I32, [V, V, ctypes.c_int64, I32, V, V]),
    "strata_rope_create": (I32, [ctypes.POINTER(strata_rope_desc), ctypes.POINTER(V)]),
    "strata_rope_destroy": (I32, [V]),
    "strata_rope_apply": (I32, [V, V, I64, I64, V, I64, I32, V, I64, I64, V]),
    "strata_kv4_append": (I32, [V, V, V, I64, V, I64, V, V, I64, V]),
    "strata_kv4_copy_pages": (I32, [V, I32, V, V, I64, V]),
    "strata_kv4_attention_workspace_bytes": (SZ, [V, I32]),
    "strata_kv4_attention": (I32, [V, V, V, V, V, V, V, V, V, V, SZ, V]),
    "strata_selftest_attention_timeout": (I32, [V, V, V, V, V, V, V, V, SZ, I32, I32, I32, V]),
    "strata_status_string": (ctypes.c_char_p, [I32]),
    "strata_last_error": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, device=None):
    if stream is None:
        import torch
        if device is None:
            return torch.cuda.current_stream().cuda_stream
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the same handle without building a Stream
        return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _making_on(stream, device):
    """Context for what a call allocates itself: it belongs to the stream that the call's kernels run on, so that a
    fill comes before them, and a block given back on return goes to nobody who does not come after them."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _host_i32(v):
    """A host list of int32 as a CPU tensor (which keeps its memory) and its length."""
    import torch
    t = v if isinstance(v, torch.Tensor) else torch.as_tensor(v)
    if t.get_device() >= 0 or t.dim() != 1 or (t.numel() and (t.is_floating_point() or t.is_complex())):
        raise ValueError("page lists are one-dimensional host arrays of whole numbers")
    if t.dtype != torch.int32 or not t.is_contiguous():
        if t.numel() and (int(t.max()) > 0x7fffffff or int(t.min()) < -0x80000000):
            raise ValueError("page numbers are int32")
        t = t.to(torch.int32).contiguous()
    return t, t.numel()


def _on(device, call, *args):
    """call(*args) with GPU `device` (an index) current; a status that is not OK raises."""
    import torch
    if torch.cuda.current_device() == device:
        status = call(*args)
    else:
        with torch.cuda.device(device):
            status = call(*args)
    if status != STRATA_OK:
        _check(status)


def _check(status: int):
    if status != STRATA_OK:
        raise StrataError(status, _lib.strata_last_error().decode(errors="replace"))


def make_desc(d_model, d_ff, n_experts, top_k, max_tokens, flags=0, router_bias=None, bits=2) -> strata_moe_desc:
    """Layer descriptor; bits = 2 or 4 picks the weight format."""
    return strata_moe_desc(d_model, d_ff, n_experts, top_k, max_tokens, 32, FORMAT_OF_BITS.get(bits, 0), flags,
                           _ptr(router_bias))


# ---------------------------------------------------------------- C ABI


def strata_q2_matrix_bytes(rows, K):
    return _lib.strata_q2_matrix_bytes(rows, K)


def strata_q4_matrix_bytes(rows, K):
    return _lib.strata_q4_matrix_bytes(rows, K)


def strata_moe_expert_bytes(desc):
    return _lib.strata_moe_expert_bytes(ctypes.byref(desc))


def strata_moe_expert_blob_bytes(desc):
    return _lib.strata_moe_expert_blob_bytes(ctypes.byref(desc))


def strata_moe_workspace_bytes(desc):
    return _lib.strata_moe_workspace_bytes(ctypes.byref(desc))


def strata_moe_layer_create(desc, workspace=None, workspace_bytes=0):
    h = ctypes.c_void_p()
    _check(_lib.strata_moe_layer_create(ctypes.byref(desc), _ptr(workspace), workspace_bytes, ctypes.byref(h)))
    return h.value


def strata_moe_layer_destroy(layer):
    _check(_lib.strata_moe_layer_destroy(layer))


def strata_moe_forward(layer, x, router_w, expert_blob, y, n_tokens, stream=None):
    _check(_lib.strata_moe_forward(layer, _ptr(x), _ptr(router_w), _ptr(expert_blob), _ptr(y), n_tokens,
                                   _stream(stream)))


def strata_moe_router_logits(layer, x, router_w, logits, n_tokens, stream=None):
    _check(_lib.strata_moe_router_logits(layer, _ptr(x), _ptr(router_w), _ptr(logits), n_tokens, _stream(stream)))


def strata_moe_route(layer, x, router_w, n_tokens, stream=None):
    _check(_lib.strata_moe_route(layer, _ptr(x), _ptr(router_w), n_tokens, _stream(stream)))


def strata_moe_experts(layer, x, expert_blob, y, n_tokens, stream=None):
    _check(_lib.strata_moe_experts(layer, _ptr(x), _ptr(expert_blob), _ptr(y), n_tokens, _stream(stream)))


def strata_moe_get_routing(layer, topk_idx=None, topk_w=None, expert_offsets=None, token_list=None,
                           pair_slot=None, stream=None):
    _check(_lib.strata_moe_get_routing(layer, _ptr(topk_idx), _ptr(topk_w), _ptr(expert_offsets),
                                       _ptr(token_list), _ptr(pair_slot), _stream(stream)))


def strata_moe_route_noalloc(desc, x, router_w, n_tokens, topk_idx, topk_w, expert_offsets, token_list,
                             pair_slot, stream=None):
    _check(_lib.strata_moe_route_noalloc(ctypes.byref(desc), _ptr(x), _ptr(router_w), n_tokens, _ptr(topk_idx),
                                         _ptr(topk_w), _ptr(expert_offsets), _ptr(token_list), _ptr(pair_slot),
                                         _stream(stream)))


def strata_moe_stack_forward(layer, router_w, router_bias, expert_blobs, x_resid, n_tokens, rms_eps,
                             stream=None):
    n = len(router_w)
    W = (ctypes.c_void_p * n)(*[_ptr(w) for w in router_w])
    B = None if router_bias is None else (ctypes.c_void_p * n)(*[_ptr(b) for b in router_bias])
    X = (ctypes.c_void_p * n)(*[_ptr(b) for b in expert_blobs])
    _check(_lib.strata_moe_stack_forward(layer, n, ctypes.cast(W, V), None if B is None else ctypes.cast(B, V),
                                         ctypes.cast(X, V), _ptr(x_resid), n_tokens, float(rms_eps),
                                         _stream(stream)))


def strata_kv4_code_bytes(n_rows, head_dim):
    return _lib.strata_kv4_code_bytes(n_rows, head_dim)


def strata_kv4_scale_bytes(n_rows, head_dim):
    return _lib.strata_kv4_scale_bytes(n_rows, head_dim)


def strata_kv4_encode(x, n_rows, head_dim, codes, scales, stream=None):
    """bf16 rows [n_rows, head_dim] -> 4-bit codes [n_rows, head_dim/2] and fp16 scales [n_rows, head_dim/32]."""
    _check(_lib.strata_kv4_encode(_ptr(x), n_rows, head_dim, _ptr(codes), _ptr(scales), _stream(stream)))


def strata_kv4_decode(codes, scales, n_rows, head_dim, out, stream=None):
    """4-bit codes and fp16 scales of n_rows rows -> bf16 rows [n_rows, head_dim]."""
    _check(_lib.strata_kv4_decode(_ptr(codes), _ptr(scales), n_rows, head_dim, _ptr(out), _stream(stream)))


def strata_rope_create(desc):
    h = ctypes.c_void_p()
    _check(_lib.strata_rope_create(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def strata_rope_destroy(rope):
    _check(_lib.strata_rope_destroy(rope))


def strata_rope_apply(rope, x, x_token_stride, x_head_stride, positions, n_tokens, n_heads, out, out_token_stride,
                      out_head_stride, stream=None):
    _check(_lib.strata_rope_apply(rope, _ptr(x), x_token_stride, x_head_stride, _ptr(positions), n_tokens, n_heads,
                                  _ptr(out), out_token_stride, out_head_stride, _stream(stream)))


def strata_kv4_append(cache, rope, k, k_token_stride, v, v_token_stride, positions, slots, n_tokens, stream=None):
    _check(_lib.strata_kv4_append(ctypes.addressof(cache), rope, _ptr(k), k_token_stride, _ptr(v), v_token_stride,
                                  _ptr(positions), _ptr(slots), n_tokens, _stream(stream)))


def strata_kv4_copy_pages(caches, src, dst, stream=None):
    """caches: a ctypes array of strata_kv4_cache (or a list of them); src, dst: host page lists (CPU int32
    tensors, numpy arrays or sequences)."""
    if not isinstance(caches, ctypes.Array):
        caches = (strata_kv4_cache * len(caches))(*caches)
    s, n = _host_i32(src)
    d, m = _host_i32(dst)
    if n != m:
        raise ValueError(f"{n} source pages and {m} destinations")
    _check(_lib.strata_kv4_copy_pages(ctypes.addressof(caches), len(caches), _ptr(s), _ptr(d), n, _stream(stream)))


def strata_kv4_attention_workspace_bytes(cache, n_q_heads):
    return _lib.strata_kv4_attention_workspace_bytes(ctypes.addressof(cache), n_q_heads)


def strata_kv4_attention(cache, desc, rope, positions, q, q_offsets, kv_lens, block_table, out, workspace,
                         workspace_bytes, stream=None):
    _check(_lib.strata_kv4_attention(ctypes.addressof(cache), ctypes.addressof(desc), rope, _ptr(positions), _ptr(q),
                                     _ptr(q_offsets), _ptr(kv_lens), _ptr(block_table), _ptr(out), _ptr(workspace),
                                     workspace_bytes, _stream(stream)))


def strata_selftest_attention_timeout(cache, desc, q, q_offsets, kv_lens, block_table, out, workspace, workspace_bytes,
                                      role, every, piece, stream=None):
    _check(_lib.strata_selftest_attention_timeout(ctypes.addressof(cache), ctypes.addressof(desc), _ptr(q),
                                                  _ptr(q_offsets), _ptr(kv_lens), _ptr(block_table), _ptr(out),
                                                  _ptr(workspace), workspace_bytes, role, every, piece,
                                                  _stream(stream)))


def strata_rmsnorm_bf16(x, out, n_tokens, d, eps, stream=None):
    _check(_lib.strata_rmsnorm_bf16(_ptr(x), _ptr(out), n_tokens, d, float(eps), _stream(stream)))


def strata_moe_set_stage_events(layer, events):
    """events: five torch.cuda.Event (timing enabled) or raw handles; [] clears."""
    import torch
    handles = []
    for e in events:
        if isinstance(e, torch.cuda.Event):
            if e.cuda_event == 0:
                e.record()
            handles.append(e.cuda_event)
        else:
            handles.append(int(e))
    arr = (ctypes.c_void_p * max(1, len(handles)))(*handles)
    _check(_lib.strata_moe_set_stage_events(layer, ctypes.cast(arr, V), len(handles)))


def strata_moe_check_status(layer):
    _check(_lib.strata_moe_check_status(layer))


def strata_q2_pack(codes, scales_fp16, rows, K, dst):
    """Host packer: numpy arrays (uint8 codes, uint16/float16 scales, uint8 dst)."""
    import numpy as np
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    s = np.ascontiguousarray(np.asarray(scales_fp16).view(np.uint16))
    _check(_lib.strata_q2_pack(c.ctypes.data, s.ctypes.data, rows, K, dst.ctypes.data))


def strata_q4_pack(codes, scales_fp16, rows, K, dst):
    """Host packer of the 4-bit format (codes 0..15), arguments as strata_q2_pack."""
    import numpy as np
    c = np.ascontiguousarray(codes, dtype=np.uint8)
    s = np.ascontiguousarray(np.asarray(scales_fp16).view(np.uint16))
    _check(_lib.strata_q4_pack(c.ctypes.data, s.ctypes.data, rows, K, dst.ctypes.data))


def strata_moe_pack_expert(desc, gc, gs, uc, us, dc, ds, dst):
    """Host packer of one expert (numpy arrays)."""
    import numpy as np
    a = [np.ascontiguousarray(v, dtype=np.uint8) for v in (gc, uc, dc)]
    s = [np.ascontiguousarray(np.asarray(v).view(np.uint16)) for v in (gs, us, ds)]
    _check(_lib.strata_moe_pack_expert(ctypes.byref(desc), a[0].ctypes.data, s[0].ctypes.data, a[1].ctypes.data,
                                       s[1].ctypes.data, a[2].ctypes.data, s[2].ctypes.data, dst.ctypes.data))


def strata_moe_pack_expert_device(desc, gc, gs, uc, us, dc, ds, dst, stream=None):
    _check(_lib.strata_moe_pack_expert_device(ctypes.byref(desc), _ptr(gc), _ptr(gs), _ptr(uc), _ptr(us),
                                              _ptr(dc), _ptr(ds), _ptr(dst), _stream(stream)))


def strata_selftest_wait_timeout(timeout_ns, stream=None):
    return _lib.strata_selftest_wait_timeout(int(timeout_ns), _stream(stream))


def strata_selftest_bounds_check(stream=None):
    return _lib.strata_selftest_bounds_check(_stream(stream))


def strata_is_checked_build():
    return _lib.strata_is_checked_build()


def strata_status_string(status):
    return _lib.strata_status_string(status).decode()


def strata_last_error():
    return _lib.strata_last_error().decode(errors="replace")


# ---------------------------------------------------------------- handle


class MoELayer:
    """Owns a layer handle (and keeps the desc's bias tensor alive)."""

    def __init__(self, d_model, d_ff, n_experts, top_k, max_tokens, flags=0, router_bias=None, workspace=None,
                 bits=2):
        self._bias = router_bias
        self.desc = make_desc(d_model, d_ff, n_experts, top_k, max_tokens, flags, router_bias, bits)
        nbytes = strata_moe_workspace_bytes(self.desc) if workspace is not None else 0
        self.handle = strata_moe_layer_create(self.desc, workspace, nbytes)

    def close(self):
        if self.handle:
            strata_moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, router_w, blob, y, n_tokens, stream=None):
        strata_moe_forward(self.handle, x, router_w, blob, y, n_tokens, stream)

    def router_logits(self, x, router_w, logits, n_tokens, stream=None):
        strata_moe_router_logits(self.handle, x, router_w, logits, n_tokens, stream)

    def route(self, x, router_w, n_tokens, stream=None):
        strata_moe_route(self.handle, x, router_w, n_tokens, stream)

    def experts(self, x, blob, y, n_tokens, stream=None):
        strata_moe_experts(self.handle, x, blob, y, n_tokens, stream)

    def routing(self, n_tokens, stream=None):
        """Routing of the last call as torch tensors."""
        import torch
        k, E = self.desc.top_k, self.desc.n_experts
        dev = torch.device("cuda")
        idx = torch.empty((n_tokens, k), dtype=torch.int32, device=dev)
        w = torch.empty((n_tokens, k), dtype=torch.float32, device=dev)
        off = torch.empty(E + 1, dtype=torch.int32, device=dev)
        tl = torch.empty(n_tokens * k, dtype=torch.int32, device=dev)
        sl = torch.empty(n_tokens * k, dtype=torch.int32, device=dev)
        strata_moe_get_routing(self.handle, idx, w, off, tl, sl, stream)
        return idx, w, off, tl, sl

    def stack_forward(self, router_w, router_bias, blobs, x_resid, n_tokens, eps, stream=None):
        strata_moe_stack_forward(self.handle, router_w, router_bias, blobs, x_resid, n_tokens, eps, stream)

    def check_status(self):
        strata_moe_check_status(self.handle)

    def pack_expert_device(self, gc, gs, uc, us, dc, ds, dst, stream=None):
        strata_moe_pack_expert_device(self.desc, gc, gs, uc, us, dc, ds, dst, stream)


def _need(t, name, dtype, device):
    """The entry points take raw pointers: refuse a tensor of another type or device (an index) than they will read."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} is on {t.device}, not on {f'GPU {device}' if device >= 0 else 'a GPU'}")


def _int32(v, name):
    """v, if a 32-bit field of the library's structures holds it: ctypes would keep the low bits of a wider one."""
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name} {v} is not an int32")
    return v


def _rotary(rope, positions, n, device):
    """Handle of a Rope and address of its rows' positions; (None, None), the library's "no rotation", without one."""
    if rope is None:
        return None, None
    if rope.handle is None:
        raise ValueError("the Rope is closed")
    if positions is None:
        raise ValueError("rope needs positions")
    import torch
    _need(positions, "positions", torch.int32, device)
    if positions.shape != (n,) or not positions.is_contiguous():
        raise ValueError(f"positions {tuple(positions.shape)}")
    return rope.handle, positions.data_ptr()


class Rope:
    """Rotary positions of head rows: the table of frequencies (include/strata_attn.h)."""

    LAYOUTS = {"half": STRATA_ROPE_HALF, "interleaved": STRATA_ROPE_INTERLEAVED}
    SCALINGS = {"none": STRATA_ROPE_SCALE_NONE, "linear": STRATA_ROPE_SCALE_LINEAR, "ntk": STRATA_ROPE_SCALE_NTK,
                "yarn": STRATA_ROPE_SCALE_YARN}

    def __init__(self, head_dim, rotary_dim=None, theta=10000.0, layout="half", scaling="none", factor=1.0,
                 original_max_position=0, beta_fast=0.0, beta_slow=0.0, attn_factor=0.0):
        self.handle = None
        self.head_dim = head_dim
        self.desc = strata_rope_desc(_int32(head_dim, "head_dim"),
                                     _int32(head_dim if rotary_dim is None else rotary_dim, "rotary_dim"),
                                     self.LAYOUTS.get(layout, -1), self.SCALINGS.get(scaling, -1), theta, factor,
                                     _int32(original_max_position, "original_max_position"), beta_fast, beta_slow,
                                     attn_factor)
        self.handle = strata_rope_create(self.desc)

    def close(self):
        if self.handle:
            strata_rope_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def apply(self, x, positions, out=None, stream=None):
        """x [tokens, heads, head_dim] bf16 (token by token or head by head), positions int32 [tokens]; out may be x.
        An `out` that the call makes belongs to `stream`, like any tensor made under torch.cuda.stream."""
        import torch
        if self.handle is None:
            raise ValueError("the Rope is closed")
        n, heads, D = x.shape
        dev = x.get_device()
        if out is None:
            with _making_on(stream, dev):
                out = torch.empty((n, heads, D), dtype=x.dtype, device=x.device)
        _need(x, "x", torch.bfloat16, dev)
        _need(out, "out", torch.bfloat16, dev)
        _need(positions, "positions", torch.int32, dev)
        if D != self.head_dim or out.shape != x.shape or positions.shape != (n,):
            raise ValueError(f"x {tuple(x.shape)}, out {tuple(out.shape)}, positions {tuple(positions.shape)}, "
                             f"head_dim {self.head_dim}")
        (xt, xh, x1), (ot, oh, o1) = x.stride(), out.stride()
        if x1 != 1 or o1 != 1 or not positions.is_contiguous():
            raise ValueError("the values of a row and the positions must be contiguous")
        _on(dev, _lib.strata_rope_apply, self.handle, x.data_ptr(), xt, xh, positions.data_ptr(), n, heads,
            out.data_ptr(), ot, oh, _stream(stream, dev))
        return out


class Kv4Cache:
    """One layer's paged 4-bit KV cache over four tensors (kept alive): codes uint8 [pages, kv_heads, page_size,
    head_dim / 2] and scales fp16 [pages, kv_heads, page_size, head_dim / 32], of keys and of values."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        import torch
        pages, heads, page, half = k_codes.shape
        self.device, self.index = k_codes.device, k_codes.get_device()
        for name, t, dtype, last in (("k_codes", k_codes, torch.uint8, half), ("v_codes", v_codes, torch.uint8, half),
                                     ("k_scales", k_scales, torch.float16, half // 16),
                                     ("v_scales", v_scales, torch.float16, half // 16)):
            _need(t, name, dtype, self.index)
            if tuple(t.shape) != (pages, heads, page, last) or not t.is_contiguous():
                raise ValueError(f"{name} {tuple(t.shape)} does not fit codes {tuple(k_codes.shape)}")
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        self.desc = strata_kv4_cache(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), pages, heads, page,
                                     2 * half)
        self._desc = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, n_pages, page_size, n_kv_heads, head_dim, device="cuda"):
        """A cache of new, uninitialised pages."""
        import torch
        shape = (n_pages, n_kv_heads, page_size)
        return cls(*(torch.empty((*shape, last), dtype=dtype, device=device)
                     for last, dtype in 2 * ((head_dim // 2, torch.uint8), (head_dim // 32, torch.float16))))

    def append(self, k, v, slots, rope=None, positions=None, stream=None):
        """k, v [tokens, kv_heads, head_dim] bf16 (any token stride) into slots int64 [tokens] (page * page_size +
        slot; negative: dropped), k through `rope` at positions int32 [tokens]."""
        import torch
        n = k.shape[0]
        D, dev = self.head_dim, self.index
        _need(k, "k", torch.bfloat16, dev)
        _need(v, "v", torch.bfloat16, dev)
        _need(slots, "slots", torch.int64, dev)
        if k.shape != (n, self.n_kv_heads, D) or v.shape != k.shape or slots.shape != (n,):
            raise ValueError(f"k {tuple(k.shape)}, v {tuple(v.shape)}, slots {tuple(slots.shape)}")
        (kt, kh, k1), (vt, vh, v1) = k.stride(), v.stride()
        if n and ((kh, k1) != (D, 1) or (vh, v1) != (D, 1) or not slots.is_contiguous()):
            raise ValueError("the heads of a token and the slots must be contiguous")
        handle, where = _rotary(rope, positions, n, dev)
        _on(dev, _lib.strata_kv4_append, self._desc, handle, k.data_ptr(), kt, v.data_ptr(), vt, where, slots.data_ptr(),
            n, _stream(stream, dev))

    def attention_workspace(self, n_q_heads):
        """A workspace for attention() with n_q_heads query heads, whatever the sequences."""
        import torch
        n = strata_kv4_attention_workspace_bytes(self.desc, _int32(n_q_heads, "n_q_heads"))
        if n == 0:
            raise ValueError(f"{n_q_heads} query heads over {self.n_kv_heads} KV heads")
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attention(self, q, q_offsets, kv_lens, block_table, out=None, *, max_q_len, scale=None, window=0, rope=None,
                  positions=None, workspace=None, stream=None):
        """Causal attention of q [tokens, heads, head_dim] bf16 (any token stride). Sequence b: query rows
        q_offsets[b] .. q_offsets[b + 1] - 1, the last of its kv_lens[b] cached tokens, on pages block_table[b]
        (all int32); max_q_len its longest query run. Rows outside every sequence stay as they are in `out`. Without
        `out` the call makes one of zeros; it, and a workspace that the call makes, belong to `stream`, like any
        tensor made under torch.cuda.stream."""
        import torch
        n, heads, D = q.shape
        dev = self.index
        if out is None:
            with _making_on(stream, dev):
                out = torch.zeros((n, heads, D), dtype=q.dtype, device=self.device)
        _need(q, "q", torch.bfloat16, dev)
        _need(out, "out", torch.bfloat16, dev)
        for name, t in (("q_offsets", q_offsets), ("kv_lens", kv_lens), ("block_table", block_table)):
            _need(t, name, torch.int32, dev)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        B = kv_lens.shape[0]
        if D != self.head_dim or out.shape != q.shape or q_offsets.shape != (B + 1,) or \
                block_table.dim() != 2 or block_table.shape[0] != B:
            raise ValueError(f"q {tuple(q.shape)}, out {tuple(out.shape)}, q_offsets {tuple(q_offsets.shape)}, "
                             f"kv_lens {tuple(kv_lens.shape)}, block_table {tuple(block_table.shape)}")
        (qt, qh, q1), (ot, oh, o1) = q.stride(), out.stride()
        if n and ((qh, q1) != (D, 1) or (oh, o1) != (D, 1)):
            raise ValueError("the heads of a token must be contiguous")
        handle, where = _rotary(rope, positions, n, dev)
        if workspace is None:
            with _making_on(stream, dev):
                workspace = self.attention_workspace(heads)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"the workspace is on {workspace.device}, not contiguous on GPU {dev}")
        desc = strata_kv4_attn_desc(B, heads, _int32(max_q_len, "max_q_len"), block_table.shape[1], n, qt, ot,
                                    _int32(window, "window"),
                                    D ** -0.5 if scale is None else scale)
        _on(dev, _lib.strata_kv4_attention, self._desc, ctypes.addressof(desc), handle, where, q.data_ptr(),
            q_offsets.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream, dev))
        return out


class Kv4CacheSet:
    """Several caches of one shape (a model's layers), whose pages are copied together."""

    def __init__(self, caches):
        self.caches = list(caches)
        if len({c.device for c in self.caches}) > 1:
            raise ValueError("the caches of a set are on one device")
        self.descs = (strata_kv4_cache * len(self.caches))(*(c.desc for c in self.caches))

    def copy_pages(self, src, dst, stream=None):
        """Page src[i] -> dst[i] in every cache; src and dst are host lists (see strata_kv4_copy_pages)."""
        if not self.caches:
            return
        s, n = _host_i32(src)
        d, m = _host_i32(dst)
        if n != m:
            raise ValueError(f"{n} source pages and {m} destinations")
        dev = self.caches[0].index
        _on(dev, _lib.strata_kv4_copy_pages, ctypes.addressof(self.descs), len(self.caches), s.data_ptr(), d.data_ptr(),
            n, _stream(stream, dev))

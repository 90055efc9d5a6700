"""Python binding of the S^2-Attn C ABI (include/s2attn.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch tensors
(device memory, contiguous [B,N,H,D]); shapes are read off the tensors, pointers and
the current CUDA stream are passed through, and a non-zero status raises
S2AttnError.  All arithmetic runs in the CUDA library libs2attn.so; if that library
is missing, every call raises -- there is no fallback.
"""
import array
import ctypes
import os

__all__ = [
    "S2AttnError", "capi", "library_path",
    "s2attn_fwd", "s2attn_bwd", "s2attn_bwd_workspace_bytes", "s2attn_bwd_preprocess", "s2attn_bwd_main",
    "s2attn_bwd_dq_convert", "s2attn_bwd_noalloc", "s2attn_decode", "s2attn_decode_workspace_bytes", "s2attn_fwd_f32", "s2attn_bwd_f32", "rope_pi_apply", "rope_pi_apply_offset",
    "lora_proj_fwd", "lora_proj_workspace_bytes", "lora_proj_bwd", "lora_proj_bwd_workspace_bytes",
    "s2attn_halo_rows", "s2attn_halo_lse",
    "rope_inv_freq", "qk_norm_rope_fwd", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_bytes",
    "s2attn_tree_mask", "s2attn_tree_decode", "s2attn_tree_decode_workspace_bytes",
    "s2attn_cache_append", "s2attn_cache_copy_pages",
    "get_device_error", "clear_device_error", "s2attn_selftest_bounded_wait",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
# S2ATTN_LIBRARY selects another build of the library, e.g. libs2attn_debug.so (bounds-checked)
library_path = os.environ.get("S2ATTN_LIBRARY") or os.path.join(_HERE, "libs2attn.so")

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "workspace", -4: "CUDA error",
          -5: "device timeout", -6: "device index out of range"}


class S2AttnError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: status {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


_lib = None


def capi():
    """The loaded C library (ctypes), with argument types declared."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"CUDA library not built: {library_path} is missing "
                           "(run: python -m shifted_sparse_attention_s2attn_b200._build)")
    lib = ctypes.CDLL(library_path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sig = {
        "s2attn_version": ([], I),
        "s2attn_status_string": ([I], ctypes.c_char_p),
        "s2attn_fwd": ([P, P, P, P, P, I, I, I, I, I, I, P], I),
        "s2attn_bwd_workspace_bytes": ([I, I, I, I], Z),
        "s2attn_bwd": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P], I),
        "s2attn_bwd_preprocess": ([P, P, P, P, I, I, I, I, P], I),
        "s2attn_bwd_main": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P], I),
        "s2attn_bwd_dq_convert": ([P, P, I, I, I, I, P], I),
        "s2attn_bwd_noalloc": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P], I),
        "s2attn_decode_workspace_bytes": ([I, I, I, I, I], Z),
        "s2attn_decode": ([P, P, P, P, P, I, I, I, I, I, P, Z, P], I),
        "s2attn_fwd_f32": ([P, P, P, P, P, I, I, I, I, I, I, P], I),
        "s2attn_bwd_f32": ([P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P], I),
        "rope_pi_apply": ([P, P, I, I, I, I, F, F, P], I),
        "rope_pi_apply_offset": ([P, P, I, I, I, I, I, F, F, P], I),
        "lora_proj_workspace_bytes": ([I, I, I, I, I], Z),
        "lora_proj_fwd": ([P, P, P, P, P, I, I, I, I, I, F, I, I, I, F, F, P, Z, P], I),
        "lora_proj_bwd_workspace_bytes": ([I, I, I, I, I], Z),
        "lora_proj_bwd": ([P, P, P, P, P, P, P, P, I, I, I, I, I, F, P, Z, P], I),
        "s2attn_halo_rows": ([ctypes.POINTER(P), ctypes.POINTER(P), I, I, I, I, I, I, I, I, P], I),
        "s2attn_halo_lse": ([ctypes.POINTER(P), ctypes.POINTER(P), I, I, I, I, I, I, I, P], I),
        "rope_inv_freq": ([P, P, I, F, I, F, I, F, F], I),
        "qk_norm_rope_fwd": ([P] * 8 + [I] * 8 + [F, F, I, I, P], I),
        "qk_norm_rope_bwd_workspace_bytes": ([I], Z),
        "qk_norm_rope_bwd": ([P] * 12 + [I] * 8 + [F, F, I, I, P, Z, P], I),
        "s2attn_tree_mask": ([P, P, P, I, I, P], I),
        "s2attn_tree_decode_workspace_bytes": ([I, I, I, I, I], Z),
        "s2attn_tree_decode": ([P] * 11 + [I] * 9 + [P, Z, P], I),
        "s2attn_cache_append": ([P] * 8 + [I] * 9 + [P], I),
        "s2attn_cache_copy_pages": ([P, I, P, I, I, Z, P], I),
        "s2attn_get_device_error": ([ctypes.POINTER(I)], I),
        "s2attn_clear_device_error": ([], I),
        "s2attn_selftest_bounded_wait": ([ctypes.c_uint, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise S2AttnError(fn, rc)


def _bnhd(t, name):
    if t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B,N,H,D] tensor")
    return tuple(t.shape)


# The C entry points see only pointers, so the binding checks every tensor a call reads or
# writes: first that each is contiguous with exactly the elements its role covers and the
# expected dtype (_extent), then that all of them live on a CUDA device (_on_cuda).

def _extent(t, name, numel, dtype):
    if t is None or not t.is_contiguous() or t.numel() != numel or t.dtype != dtype:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {numel} elements")


def _on_cuda(**tensors):
    for name, t in tensors.items():
        if t is not None and t.device.type != "cuda":
            raise ValueError(f"{name} must be on a CUDA device")


def _workspace(t):
    if t is None or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    _on_cuda(workspace=t)


def _attn_args(dtype, shape, **tensors):
    """Checks the [B,N,H,D] tensors (q's element count) and the [B,H,N] lse/delta of an
    attention call (dq_acc: fp32 with q's element count), then their device."""
    B, N, H, D = shape
    for name, t in tensors.items():
        if name in ("lse", "delta"):
            _extent(t, name, B * H * N, _torch().float32)
        elif name == "dq_acc":
            _extent(t, name, B * N * H * D, _torch().float32)
        else:
            _extent(t, name, B * N * H * D, dtype)
    _on_cuda(**tensors)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def s2attn_fwd(q, k, v, o, lse, G, shift_heads, stream=None):
    """bf16 forward: o <- S^2-Attn(q, k, v), lse <- [B,H,N] fp32 log-sum-exp."""
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().bfloat16, (B, N, H, D), q=q, k=k, v=v, o=o, lse=lse)
    _check("s2attn_fwd", capi().s2attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, N, H, D, G,
                                           shift_heads, _stream(stream)))


def s2attn_bwd_workspace_bytes(B, N, H, D):
    return int(capi().s2attn_bwd_workspace_bytes(B, N, H, D))


def s2attn_bwd(q, k, v, o, dout, lse, dq, dk, dv, G, shift_heads, workspace, stream=None):
    """bf16 backward into dq, dk, dv.  workspace: a uint8 device tensor of at least
    s2attn_bwd_workspace_bytes(B,N,H,D) bytes, 256-byte aligned."""
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().bfloat16, (B, N, H, D), q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv)
    _workspace(workspace)
    _check("s2attn_bwd", capi().s2attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                                           _ptr(dk), _ptr(dv), B, N, H, D, G, shift_heads, _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)))


def s2attn_bwd_preprocess(o, dout, delta, dq_acc, stream=None):
    B, N, H, D = _bnhd(o, "o")
    _attn_args(_torch().bfloat16, (B, N, H, D), o=o, dout=dout, delta=delta, dq_acc=dq_acc)
    _check("s2attn_bwd_preprocess", capi().s2attn_bwd_preprocess(_ptr(o), _ptr(dout), _ptr(delta), _ptr(dq_acc),
                                                                 B, N, H, D, _stream(stream)))


def s2attn_bwd_main(q, k, v, dout, lse, delta, dq_acc, dk, dv, G, shift_heads, stream=None):
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().bfloat16, (B, N, H, D), q=q, k=k, v=v, dout=dout, lse=lse, delta=delta, dq_acc=dq_acc,
               dk=dk, dv=dv)
    _check("s2attn_bwd_main", capi().s2attn_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse), _ptr(delta),
                                                     _ptr(dq_acc), _ptr(dk), _ptr(dv), B, N, H, D, G, shift_heads,
                                                     _stream(stream)))


def s2attn_bwd_dq_convert(dq_acc, dq, stream=None):
    B, N, H, D = _bnhd(dq, "dq")
    _attn_args(_torch().bfloat16, (B, N, H, D), dq=dq, dq_acc=dq_acc)
    _check("s2attn_bwd_dq_convert", capi().s2attn_bwd_dq_convert(_ptr(dq_acc), _ptr(dq), B, N, H, D,
                                                                 _stream(stream)))


def s2attn_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, G, shift_heads, stream=None):
    """bf16 backward without a caller workspace: for callers that cannot allocate device
    memory.  Uses the library's fixed device scratch (S2ATTN_NOALLOC_SCRATCH_BYTES per
    device, shared by all calls; overlapping calls race)."""
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().bfloat16, (B, N, H, D), q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv)
    _check("s2attn_bwd_noalloc", capi().s2attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout),
                                                           _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, N, H, D, G,
                                                           shift_heads, _stream(stream)))


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def s2attn_halo_rows(xs, bufs, to_buf, G, shift_heads, stream=None):
    """Rows [0, G/2) of the shifted heads of each bf16 [B,N,H,D] tensor in xs to (to_buf=True)
    or from (False) the matching contiguous [B, G/2, shift_heads, D] buffer in bufs; one launch."""
    if not xs or len(xs) != len(bufs):
        raise ValueError("xs and bufs must be non-empty lists of equal length")
    B, N, H, D = _bnhd(xs[0], "x")
    bf16 = _torch().bfloat16
    for i, (x, b) in enumerate(zip(xs, bufs)):
        _extent(x, f"x[{i}]", B * N * H * D, bf16)
        _extent(b, f"buf[{i}]", B * (G // 2) * shift_heads * D, bf16)
    for x, b in zip(xs, bufs):
        _on_cuda(x=x, buf=b)
    _check("s2attn_halo_rows", capi().s2attn_halo_rows(_ptr_array(xs), _ptr_array(bufs), len(xs), int(bool(to_buf)),
                                                       B, N, H, D, G, shift_heads, _stream(stream)))


def s2attn_halo_lse(lses, bufs, to_buf, G, shift_heads, stream=None):
    """The same rows of fp32 [B,H,N] tensors (softmax statistics) to or from [B, shift_heads, G/2]
    buffers; one launch."""
    if not lses or len(lses) != len(bufs):
        raise ValueError("lses and bufs must be non-empty lists of equal length")
    if lses[0].dim() != 3:
        raise ValueError("lse must be a [B,H,N] tensor")
    B, H, N = tuple(lses[0].shape)
    f32 = _torch().float32
    for i, (x, b) in enumerate(zip(lses, bufs)):
        _extent(x, f"lse[{i}]", B * H * N, f32)
        _extent(b, f"buf[{i}]", B * shift_heads * (G // 2), f32)
    for x, b in zip(lses, bufs):
        _on_cuda(lse=x, buf=b)
    _check("s2attn_halo_lse", capi().s2attn_halo_lse(_ptr_array(lses), _ptr_array(bufs), len(lses),
                                                     int(bool(to_buf)), B, N, H, G, shift_heads, _stream(stream)))


def s2attn_decode_workspace_bytes(B, M, N, H, D):
    return int(capi().s2attn_decode_workspace_bytes(B, M, N, H, D))


def s2attn_decode(q, k, v, o, lse, workspace, stream=None):
    """Decoding step of full causal attention: q [B,M,H,D] (query m at position N-M+m)
    against k, v [B,N,H,D]; o [B,M,H,D] bf16 and lse [B,H,M] fp32 are written.
    workspace: a uint8 device tensor of at least s2attn_decode_workspace_bytes bytes."""
    B, M, H, D = _bnhd(q, "q")
    Bk, N, Hk, Dk = _bnhd(k, "k")
    if (Bk, Hk, Dk) != (B, H, D):
        raise ValueError("k must be [B,N,H,D] with q's B, H and D")
    bf16 = _torch().bfloat16
    _extent(q, "q", B * M * H * D, bf16)
    _extent(k, "k", B * N * H * D, bf16)
    _extent(v, "v", B * N * H * D, bf16)
    _extent(o, "o", B * M * H * D, bf16)
    _extent(lse, "lse", B * H * M, _torch().float32)
    _on_cuda(q=q, k=k, v=v, o=o, lse=lse)
    _workspace(workspace)
    _check("s2attn_decode", capi().s2attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, M, N, H, D,
                                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                 _stream(stream)))


def s2attn_fwd_f32(q, k, v, o, lse, G, shift_heads, stream=None):
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().float32, (B, N, H, D), q=q, k=k, v=v, o=o, lse=lse)
    _check("s2attn_fwd_f32", capi().s2attn_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, N, H, D, G,
                                                   shift_heads, _stream(stream)))


def s2attn_bwd_f32(q, k, v, o, dout, lse, dq, dk, dv, G, shift_heads, workspace, stream=None):
    B, N, H, D = _bnhd(q, "q")
    _attn_args(_torch().float32, (B, N, H, D), q=q, k=k, v=v, o=o, dout=dout, lse=lse, dq=dq, dk=dk, dv=dv)
    _workspace(workspace)
    _check("s2attn_bwd_f32", capi().s2attn_bwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                                   _ptr(dq), _ptr(dk), _ptr(dv), B, N, H, D, G, shift_heads,
                                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                   _stream(stream)))


def rope_pi_apply(q, k, pos_scale, base=10000.0, stream=None):
    """In-place RoPE with position interpolation on bf16 q and/or k ([B,N,H,D])."""
    ref = q if q is not None else k
    B, N, H, D = _bnhd(ref, "q/k")
    for name, t in (("q", q), ("k", k)):
        if t is not None:
            _extent(t, name, B * N * H * D, _torch().bfloat16)
    _on_cuda(q=q, k=k)
    _check("rope_pi_apply", capi().rope_pi_apply(_ptr(q), _ptr(k), B, N, H, D, float(pos_scale), float(base),
                                                 _stream(stream)))


def rope_pi_apply_offset(q, k, pos0, pos_scale, base=10000.0, stream=None):
    """In-place RoPE-PI on bf16 q and/or k whose row t is the token at position pos0 + t."""
    ref = q if q is not None else k
    B, N, H, D = _bnhd(ref, "q/k")
    for name, t in (("q", q), ("k", k)):
        if t is not None:
            _extent(t, name, B * N * H * D, _torch().bfloat16)
    _on_cuda(q=q, k=k)
    _check("rope_pi_apply_offset", capi().rope_pi_apply_offset(_ptr(q), _ptr(k), B, N, H, D, int(pos0),
                                                               float(pos_scale), float(base), _stream(stream)))


def lora_proj_workspace_bytes(T, K, n_out, parts, r):
    return int(capi().lora_proj_workspace_bytes(T, K, n_out, parts, r))


def lora_proj_fwd(x, w, lora_a, lora_b, y, parts, scaling, rope_parts=0, head_dim=128, seq_len=None,
                  pos_scale=1.0, base=10000.0, workspace=None, stream=None):
    """LoRA-adapted projections: y[p] = x W_p^T + scaling (x A_p^T) B_p^T for p < parts, RoPE-PI
    on the first rope_parts parts.  x: [..., K] (T rows), w: [parts*n_out, K], lora_a:
    [parts*r, K] and lora_b: [parts*n_out, r] (both None for r = 0), y: [parts, T, n_out]
    (or any contiguous tensor of that many elements); all bf16 on the device.  workspace:
    uint8 device tensor of lora_proj_workspace_bytes(T, K, n_out, parts, r) bytes (r > 0)."""
    import torch
    if (lora_a is None) != (lora_b is None):
        raise ValueError("lora_a and lora_b are given together (or both None for no adapter)")
    for t, name in ((x, "x"), (w, "w"), (y, "y"), (lora_a, "lora_a"), (lora_b, "lora_b")):
        if t is None:
            continue
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16")
    # The C entry point sees only pointers: every extent it will read or write is checked here.
    K = x.shape[-1]
    T = x.numel() // K
    if parts < 1 or w.dim() != 2 or w.shape[1] != K or w.shape[0] % parts:
        raise ValueError("w must be [parts*n_out, K] with x's K")
    n_out = w.shape[0] // parts
    r = 0
    if lora_a is not None:
        if lora_a.dim() != 2 or lora_a.shape[1] != K or lora_a.shape[0] % parts:
            raise ValueError("lora_a must be [parts*r, K]")
        r = lora_a.shape[0] // parts
        if tuple(lora_b.shape) != (parts * n_out, r):
            raise ValueError("lora_b must be [parts*n_out, r]")
    if y.numel() != parts * T * n_out:
        raise ValueError("y must hold parts * T * n_out elements")
    _on_cuda(x=x, w=w, y=y, lora_a=lora_a, lora_b=lora_b)
    if r > 0:
        _workspace(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("lora_proj_fwd", capi().lora_proj_fwd(
        _ptr(x), _ptr(w), _ptr(lora_a), _ptr(lora_b), _ptr(y), T, K, n_out, parts, r, float(scaling),
        int(rope_parts), int(head_dim), int(seq_len if seq_len is not None else T), float(pos_scale), float(base),
        _ptr(workspace), ws_bytes, _stream(stream)))


def lora_proj_bwd_workspace_bytes(T, K, n_out, parts, r):
    return int(capi().lora_proj_bwd_workspace_bytes(T, K, n_out, parts, r))


def lora_proj_bwd(x, w, lora_a, lora_b, dy, dx, d_lora_a, d_lora_b, parts, scaling, workspace, stream=None):
    """Backward of lora_proj_fwd (W frozen): dx [T, K], d_lora_a [parts*r, K], d_lora_b
    [parts*n_out, r] from dy [parts, T, n_out] (the gradient before RoPE; rope_pi_apply with
    -pos_scale takes dq, dk back through it)."""
    torch = _torch()
    K = x.shape[-1]
    T = x.numel() // K
    if parts < 1 or w.dim() != 2 or w.shape[1] != K or w.shape[0] % parts:
        raise ValueError("w must be [parts*n_out, K] with x's K")
    n_out = w.shape[0] // parts
    r = 0 if lora_a is None else lora_a.shape[0] // parts
    bf = torch.bfloat16
    _extent(x, "x", T * K, bf)
    _extent(w, "w", parts * n_out * K, bf)
    _extent(dy, "dy", parts * T * n_out, bf)
    _extent(dx, "dx", T * K, bf)
    if r:
        _extent(lora_a, "lora_a", parts * r * K, bf)
        _extent(lora_b, "lora_b", parts * n_out * r, bf)
        _extent(d_lora_a, "d_lora_a", parts * r * K, bf)
        _extent(d_lora_b, "d_lora_b", parts * n_out * r, bf)
    _on_cuda(x=x, w=w, dy=dy, dx=dx, lora_a=lora_a, lora_b=lora_b, d_lora_a=d_lora_a, d_lora_b=d_lora_b)
    _workspace(workspace)
    _check("lora_proj_bwd", capi().lora_proj_bwd(
        _ptr(x), _ptr(w), _ptr(lora_a), _ptr(lora_b), _ptr(dy), _ptr(dx), _ptr(d_lora_a), _ptr(d_lora_b),
        T, K, n_out, parts, r, float(scaling), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


# The calls below launch on the device of their tensors, which must be one, whatever the current
# device is; without a `stream` they take that device's current stream.  They are made once or
# more per layer and token, so their checks are kept to a few attribute reads a tensor.

def _fit(t, name, shape, dtype, dev):
    """A contiguous tensor of this shape and dtype on device `dev` (an index, -1 for the host)."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        where = f"cuda:{dev}" if dev >= 0 else "the host"
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {where} "
                         "like the other tensors")


def _call_on(dev, fn, stream, *args):
    """Calls the C entry point `fn` with device `dev` current; the stream is its last argument."""
    torch = _torch()
    if dev < 0:
        raise ValueError(f"{fn}: the tensors must be on a CUDA device")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream if isinstance(stream, int) else stream.cuda_stream
    call = getattr(_lib or capi(), fn)
    if torch._C._cuda_getDevice() == dev:
        rc = call(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, raw)
    if rc != 0:
        raise S2AttnError(fn, rc)


def _adr(t):
    return None if t is None else t.data_ptr()


_dtype_codes = {}


def _dtype_code(dtype, name, f32):
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
    code = _dtype_codes.get(dtype, 3)
    if code > (2 if f32 else 1):
        raise ValueError(f"{name} must be bf16{', fp16 or fp32' if f32 else ' or fp16'}")
    return code


def _scratch(t, dev):
    """Address and bytes of a workspace."""
    if t is None or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the others")
    return t.data_ptr(), t.numel() * t.element_size()


_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_inv_freq(R, base=10000.0, scaling="none", factor=1.0, original_len=4096, beta_fast=32.0, beta_slow=1.0):
    """(inv_freq [R/2] fp32 on the host, attn_factor) for a context stretched by `factor`: scaling
    "none", "linear" (position interpolation), "ntk" (a larger base) or "yarn" (by wavelength)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    if R < 2 or R % 2 or R > 256:
        raise ValueError("R must be even, 2 to 256")
    out = _torch().empty(R // 2, dtype=_torch().float32)
    af = ctypes.c_float(0.0)
    _check("rope_inv_freq", capi().rope_inv_freq(_ptr(out), ctypes.byref(af), R, base, _SCALINGS[scaling], factor,
                                                 original_len, beta_fast, beta_slow))
    return out, af.value


def _norm_rope_ref(q, k, names, norm, wq, wk, inv_freq, positions, pos0):
    """Checks what a call's sides share, q and k being the tensors that give their sizes; q's (or
    without it k's) shape, type and device."""
    ref = k if q is None else q
    if ref is None:
        raise ValueError(f"{names[0]} or {names[1]} must be given")
    shape, dtype, dev = ref.shape, ref.dtype, ref.get_device()
    # (the C calls' sizes are 32-bit)
    if len(shape) != 4 or shape[0] * shape[1] >= 2 ** 30 or shape[2] >= 2 ** 31 or shape[3] >= 2 ** 31:
        raise ValueError(f"{names[0]} and {names[1]} must be [B,N,H,D] with B*N below 2^30, H and D below 2^31")
    if wq is not None:
        _fit(wq, "wq", shape[3:], dtype, dev)
    if wk is not None:
        _fit(wk, "wk", shape[3:], dtype, dev)
    if not norm and (wq is not None or wk is not None):
        raise ValueError("wq and wk are only used with norm=True")
    f32 = _torch().float32
    if inv_freq.dim() != 1 or inv_freq.dtype is not f32 or inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous fp32 vector on the device of the other tensors")
    if positions is not None:
        _fit(positions, "positions", shape[:2], _torch().int32, dev)
    elif not -2 ** 31 <= pos0 < 2 ** 31 - shape[1]:
        raise ValueError("pos0 is outside the range of positions")
    return shape, dtype, dev


def _norm_rope_k_shape(shape, k, name):
    if k.dim() != 4 or k.shape[2] >= 2 ** 31:
        raise ValueError(f"{name} must be [B,N,H,D] with H below 2^31")
    return shape[0], shape[1], k.shape[2], shape[3]


def qk_norm_rope_fwd(q, k, q_out, k_out, inv_freq, wq=None, wk=None, norm=True, eps=1e-6, positions=None, pos0=0,
                     attn_factor=1.0, interleaved=False, stream=None):
    """RMS norm of every head of q [B,N,Hq,D] and k [B,N,Hk,D] (norm=False: none) and the rotary
    embedding of its first 2*len(inv_freq) elements, in one pass, into q_out and k_out (which
    may be q and k).  q with q_out, or k with k_out, may be None.  wq, wk [D] (None: 1);
    positions [B,N] int32 (None: pos0 + row); bf16, fp16 or fp32."""
    shape, dtype, dev = _norm_rope_ref(q, k, ("q", "k"), norm, wq, wk, inv_freq, positions, pos0)
    if (q is None) != (q_out is None) or (k is None) != (k_out is None):
        raise ValueError("q and q_out, and k and k_out, must be given together")
    Hq = Hk = 0
    if q is not None:
        Hq = shape[2]
        _fit(q, "q", shape, dtype, dev)
        _fit(q_out, "q_out", shape, dtype, dev)
    if k is not None:
        k_shape = _norm_rope_k_shape(shape, k, "k")
        Hk = k_shape[2]
        _fit(k, "k", k_shape, dtype, dev)
        _fit(k_out, "k_out", k_shape, dtype, dev)
    _call_on(dev, "qk_norm_rope_fwd", stream, _adr(q), _adr(k), _adr(wq), _adr(wk), _adr(positions),
             inv_freq.data_ptr(), _adr(q_out), _adr(k_out), shape[0], shape[1], Hq, Hk, shape[3], 2 * inv_freq.numel(),
             bool(interleaved), bool(norm), eps, attn_factor, 0 if positions is not None else pos0,
             _dtype_code(dtype, "q/k", True))


def qk_norm_rope_bwd_workspace_bytes(D):
    return int(capi().qk_norm_rope_bwd_workspace_bytes(D))


def qk_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, inv_freq, wq=None, wk=None, dwq=None, dwk=None, norm=True, eps=1e-6,
                     positions=None, pos0=0, attn_factor=1.0, interleaved=False, workspace=None, stream=None):
    """Backward of qk_norm_rope_fwd: dq, dk (which may be dq_out, dk_out) and, where given, dwq, dwk
    [D].  q, k are the forward's inputs (norm=False: may be None).  workspace: a uint8 device
    tensor of qk_norm_rope_bwd_workspace_bytes(D) bytes, needed with dwq or dwk."""
    shape, dtype, dev = _norm_rope_ref(dq_out, dk_out, ("dq_out", "dk_out"), norm, wq, wk, inv_freq, positions, pos0)
    if (dq_out is None) != (dq is None) or (dk_out is None) != (dk is None):
        raise ValueError("dq_out and dq, and dk_out and dk, must be given together")
    if not norm:
        q = k = None
    elif (q is None) != (dq is None) or (k is None) != (dk is None):
        raise ValueError("with norm=True q must be given with dq, and k with dk")
    Hq = Hk = 0
    if dq_out is not None:
        Hq = shape[2]
        _fit(dq_out, "dq_out", shape, dtype, dev)
        _fit(dq, "dq", shape, dtype, dev)
        if norm:
            _fit(q, "q", shape, dtype, dev)
    if dk_out is not None:
        k_shape = _norm_rope_k_shape(shape, dk_out, "dk_out")
        Hk = k_shape[2]
        _fit(dk_out, "dk_out", k_shape, dtype, dev)
        _fit(dk, "dk", k_shape, dtype, dev)
        if norm:
            _fit(k, "k", k_shape, dtype, dev)
    ws, ws_bytes = None, 0
    if dwq is not None or dwk is not None:
        if not norm or (dwq is not None and dq is None) or (dwk is not None and dk is None):
            raise ValueError("dwq and dwk need norm=True and their side's gradient")
        if dwq is not None:
            _fit(dwq, "dwq", shape[3:], dtype, dev)
        if dwk is not None:
            _fit(dwk, "dwk", shape[3:], dtype, dev)
        ws, ws_bytes = _scratch(workspace, dev)
    _call_on(dev, "qk_norm_rope_bwd", stream, _adr(q), _adr(k), _adr(dq_out), _adr(dk_out), _adr(wq), _adr(wk),
             _adr(positions), inv_freq.data_ptr(), _adr(dq), _adr(dk), _adr(dwq), _adr(dwk), shape[0], shape[1], Hq, Hk,
             shape[3], 2 * inv_freq.numel(), bool(interleaved), bool(norm), eps, attn_factor,
             0 if positions is not None else pos0, _dtype_code(dtype, "q/k", True), ws, ws_bytes)


def s2attn_tree_mask(parents, mask, depth=None, stream=None):
    """Ancestor masks of trees of drafted tokens: parents [B,M] int32 (-1: follows the cache) ->
    mask [B,M,ceil(M/64)] int64 (bit j: j is m or an ancestor) and depth [B,M] int32."""
    torch = _torch()
    if parents.dim() != 2 or parents.numel() >= 2 ** 31:
        raise ValueError("parents must be [B,M] with fewer than 2^31 nodes")
    B, M = parents.shape
    dev = parents.get_device()
    _fit(parents, "parents", (B, M), torch.int32, dev)
    _fit(mask, "mask", (B, M, (M + 63) // 64), torch.int64, dev)
    if depth is not None:
        _fit(depth, "depth", (B, M), torch.int32, dev)
    _call_on(dev, "s2attn_tree_mask", stream, parents.data_ptr(), mask.data_ptr(), _adr(depth), B, M)


def s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D):
    return int(capi().s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D))


def _paged(k_pages, v_pages, page_table, cache_len, B, Hkv, D, dtype, dev):
    """Checks a paged cache; its pages, page size and table width."""
    int32 = _torch().int32
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages must be [n_pages,page_size,Hkv,D] and page_table [B,table_width]")
    n_pages, page_size, _, _ = k_pages.shape
    if n_pages * page_size >= 2 ** 31 or page_table.shape[1] >= 2 ** 31:
        raise ValueError("a pool must have fewer than 2^31 rows")
    shape = (n_pages, page_size, Hkv, D)
    _fit(k_pages, "k_pages", shape, dtype, dev)
    _fit(v_pages, "v_pages", shape, dtype, dev)
    width = page_table.shape[1]
    _fit(page_table, "page_table", (B, width), int32, dev)
    _fit(cache_len, "cache_len", (B,), int32, dev)
    return n_pages, page_size, width


def s2attn_tree_decode(q, k_new, v_new, k_pages, v_pages, page_table, cache_len, o, lse, workspace, tree_mask=None,
                       new_len=None, stream=None):
    """Attention of drafted tokens (q [B,M,H,D], k_new, v_new [B,M,Hkv,D]) over the paged cache
    (k_pages, v_pages [n_pages,page_size,Hkv,D], page_table [B,width] and cache_len [B] int32) and
    over each other by tree_mask [B,M,ceil(M/64)] int64 (None: token m sees j <= m), into o like q
    and lse [B,H,M] fp32.  new_len [B] int32: drafted tokens of each sequence (None: M); the
    other rows of o and lse stay.  bf16 or fp16.  workspace: a uint8 device tensor of
    s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D) bytes, one per call in flight."""
    torch = _torch()
    if q.dim() != 4 or k_new.dim() != 4:
        raise ValueError("q must be [B,M,H,D] and k_new [B,M,Hkv,D]")
    B, M, H, D = q.shape
    Hkv = k_new.shape[2]
    if B >= 2 ** 31 or M >= 2 ** 31 or H >= 2 ** 31 or D >= 2 ** 31 or Hkv >= 2 ** 31:
        raise ValueError("every size of q and k_new must be below 2^31")
    dtype, dev = q.dtype, q.get_device()
    code = _dtype_code(dtype, "q", False)
    _fit(q, "q", (B, M, H, D), dtype, dev)
    _fit(o, "o", (B, M, H, D), dtype, dev)
    _fit(k_new, "k_new", (B, M, Hkv, D), dtype, dev)
    _fit(v_new, "v_new", (B, M, Hkv, D), dtype, dev)
    n_pages, page_size, width = _paged(k_pages, v_pages, page_table, cache_len, B, Hkv, D, dtype, dev)
    _fit(lse, "lse", (B, H, M), torch.float32, dev)
    if tree_mask is not None:
        _fit(tree_mask, "tree_mask", (B, M, (M + 63) // 64), torch.int64, dev)
    if new_len is not None:
        _fit(new_len, "new_len", (B,), torch.int32, dev)
    ws, ws_bytes = _scratch(workspace, dev)
    _call_on(dev, "s2attn_tree_decode", stream, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
             v_pages.data_ptr(), page_table.data_ptr(), cache_len.data_ptr(), _adr(new_len), _adr(tree_mask),
             o.data_ptr(), lse.data_ptr(), B, M, H, Hkv, D, n_pages, page_size, width, code, ws, ws_bytes)


def s2attn_cache_append(k_new, v_new, k_pages, v_pages, page_table, cache_len, rows=None, n_rows=None, stream=None):
    """Writes rows of k_new, v_new [B,M,Hkv,D] into the sequences' pages: for j < n_rows[b] row
    rows[b][j] goes to position cache_len[b] + j.  rows [B,A] int32 (None: row j, all M);
    n_rows [B] int32 (None: A).  cache_len is not changed.  bf16, fp16 or fp32."""
    torch = _torch()
    if k_new.dim() != 4:
        raise ValueError("k_new must be [B,M,Hkv,D]")
    B, M, Hkv, D = k_new.shape
    if B * M >= 2 ** 30 or Hkv >= 2 ** 31 or D >= 2 ** 31:
        raise ValueError("k_new must have fewer than 2^30 rows, and Hkv and D below 2^31")
    dtype, dev = k_new.dtype, k_new.get_device()
    _dtype_code(dtype, "k_new", True)
    _fit(k_new, "k_new", (B, M, Hkv, D), dtype, dev)
    _fit(v_new, "v_new", (B, M, Hkv, D), dtype, dev)
    n_pages, page_size, width = _paged(k_pages, v_pages, page_table, cache_len, B, Hkv, D, dtype, dev)
    A = M
    if rows is not None:
        if rows.dim() != 2 or rows.numel() >= 2 ** 30:
            raise ValueError("rows must be [B,A] with B*A below 2^30")
        A = rows.shape[1]
        _fit(rows, "rows", (B, A), torch.int32, dev)
    if n_rows is not None:
        _fit(n_rows, "n_rows", (B,), torch.int32, dev)
    _call_on(dev, "s2attn_cache_append", stream, k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(),
             v_pages.data_ptr(), page_table.data_ptr(), cache_len.data_ptr(), _adr(rows), _adr(n_rows), B, M, A, Hkv, D,
             n_pages, page_size, width, k_new.element_size())


def s2attn_cache_copy_pages(pools, pairs, stream=None):
    """Copies pages inside every tensor of `pools` ([n_pages, page_size, Hkv, D], one shape and dtype,
    at most 128): for (src, dst) in pairs (host integers) page src to page dst.  No page may be
    written twice, or both read and written."""
    if not pools:
        raise ValueError("pools must be a non-empty list")
    ref = pools[0]
    shape, dtype, dev = ref.shape, ref.dtype, ref.get_device()
    if len(shape) < 2 or shape[0] >= 2 ** 31:
        raise ValueError("a pool must be [n_pages, ...] with fewer than 2^31 pages")
    for t in pools:
        if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            _fit(t, "every pool", shape, dtype, dev)
    addresses = array.array("Q", [t.data_ptr() for t in pools])
    flat = array.array("i", bytes(8 * len(pairs)))
    if len(pairs):
        src, dst = zip(*pairs, strict=True)      # a pair of any other length raises ValueError
        try:
            flat[0::2], flat[1::2] = array.array("i", src), array.array("i", dst)
        except OverflowError:
            raise ValueError("a page number does not fit 32 bits") from None
    n_pages = shape[0]
    _call_on(dev, "s2attn_cache_copy_pages", stream, addresses.buffer_info()[0], len(pools), flat.buffer_info()[0],
             len(pairs), n_pages,
             ref.numel() // max(n_pages, 1) * ref.element_size())


def get_device_error():
    """(status, detail) of the current device's error word; synchronize first."""
    d = ctypes.c_int(0)
    rc = capi().s2attn_get_device_error(ctypes.byref(d))
    return rc, d.value


def clear_device_error():
    _check("s2attn_clear_device_error", capi().s2attn_clear_device_error())


def s2attn_selftest_bounded_wait(timeout_us, stream=None):
    """Runs a kernel whose bounded wait must time out (see include/s2attn.h)."""
    _check("s2attn_selftest_bounded_wait", capi().s2attn_selftest_bounded_wait(int(timeout_us), _stream(stream)))

"""Thin Python binding of libtreeverify (ctypes).

Each function carries the name of the C entry point it calls and only
marshals arguments: it checks tensor placement/dtype/contiguity, passes raw
pointers, sizes and the current CUDA stream, and raises :class:`TVError` on a
non-zero status.  Every step of the computation runs in the library's
kernels; there is no Python or CPU fallback, and a missing library raises.
"""

from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtreeverify.so")

TV_F32, TV_BF16 = 0, 1
TV_ATTN_AUTO, TV_ATTN_SIMT, TV_ATTN_TCGEN05 = 0, 1, 2
TV_ATTN_PUBLISH_ALL = 4
TV_ATTN_ROPE_Q = 8
TV_ATTN_CTA_PAIRS = 16
TV_ATTN_WORKSPACE_ZEROED = 32
TV_SAMPLE_AUTO, TV_SAMPLE_CLUSTER, TV_SAMPLE_SINGLE_CTA, TV_SAMPLE_STREAM, TV_SAMPLE_GRID = 0, 1, 2, 3, 4
TV_DEV_BAD_TOPOLOGY, TV_DEV_BAD_TOKEN, TV_DEV_OUT_OVERFLOW, TV_DEV_BAD_POSITION, TV_DEV_TIMEOUT = 1, 2, 4, 8, 16
TV_DEV_BAD_BLOCK = 32
TV_DEV_BAD_OFFSETS = 64
TV_MAX_TOP_K = 32
STATUS_NAMES = {0: "TV_OK", -1: "TV_ERR_INVALID_ARG", -2: "TV_ERR_MISSING_PARENT", -3: "TV_ERR_TOO_MANY_NODES",
                -4: "TV_ERR_UNSUPPORTED", -5: "TV_ERR_WORKSPACE", -6: "TV_ERR_CUDA"}

# exported symbol -> (restype, argtypes)
_I32, _I64, _P, _SZ, _F, _D = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "tv_last_error": (ctypes.c_char_p, []),
    "tv_version": (ctypes.c_int, []),
    "tv_tree_build": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P, _P, _P, _P]),
    "tv_tree_mask": (ctypes.c_int, [_P, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _P]),
    "tv_rope_table": (ctypes.c_int, [_P, _I32, _I32, _D, _P]),
    "tv_rope_apply": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P]),
    "tv_tree_attn_workspace_size": (ctypes.c_int, [_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
    "tv_tree_attn_verify": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _I64, _I32, _I32,
                                           _I32, _I32, _I32, _I32, _F, _P, _P, _P, _SZ, _I32, _I32, _P, _P]),
    "tv_tree_attn_verify_static": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _I64, _I32,
                                                  _I32, _I32, _I32, _I32, _I32, _F, _P, _P, _I32, _I32, _P, _P]),
    "tv_tree_attn_static_workspace_bytes": (ctypes.c_size_t, []),
    "tv_tree_attn_verify_rope": (ctypes.c_int, [_P, _P, _P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _I64, _P, _I32,
                                                _I32, _I32, _I32, _I32, _I32, _I32, _F, _P, _P, _P, _SZ, _I32, _I32,
                                                _P, _P]),
    "tv_tree_prepare": (ctypes.c_int, [_P, _I64, _P, _P, _I32, _I32, _P, _P, _P, _P, _I32, _P, _I32, _I32, _I32,
                                       _P, _I32, _P, _P]),
    "tv_tree_accept_greedy": (ctypes.c_int, [_P, _P, _P, _P, _I64, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _P, _P]),
    "tv_tree_accept_sample": (ctypes.c_int, [_P, _P, _P, _P, _I64, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _I32,
                                             _I32, _P, _SZ, _P, _P]),
    "tv_accept_sample_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I32]),
    "tv_accept_sample_uses_grid": (ctypes.c_int, [_I32, _I32, _I32, _I32, _SZ, _P]),
    "tv_chain_accept_sample": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _I32, _I32, _P, _SZ,
                                              _P, _P]),
    "tv_kv_commit": (ctypes.c_int, [_P, _P, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _I32, _P, _I32, _I32, _I32,
                                    _I32, _I32, _P, _P]),
    "tv_kv_append": (ctypes.c_int, [_P, _I64, _P, _I64, _I32, _P, _I64, _P, _I64, _P, _I32, _P, _P, _I64, _I32, _P,
                                    _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P]),
    "tv_decode_attn_workspace_size": (ctypes.c_int, [_I32, _I32, _I32, _I32, _I32, _P]),
    "tv_decode_attn": (ctypes.c_int, [_P, _I64, _P, _P, _I64, _I32, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _F,
                                      _F, _I32, _I32, _P, _P, _P, _P, _SZ, _I32, _I32, _P, _P]),
    "tv_token_logprobs": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P]),
}


class TVError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_lib = None


def lib():
    """The loaded library (raises if it was not built).  The environment
    variable TREEVERIFY_LIB names another build to load instead (the
    development build with test hooks)."""
    global _lib
    if _lib is None:
        path = os.environ.get("TREEVERIFY_LIB") or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with speculative_decoding_tree_attn_gb300.build")
        h = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(h, name)
            f.restype, f.argtypes = res, args
        _lib = h
    return _lib


def _check(fn, code):
    if code != 0:
        raise TVError(fn, code, lib().tv_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t, name, dtypes):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# torch's own raw calls, without the objects that torch.cuda makes (8 us of a call's 20); a torch that lacks the names
# has the public ones
_device_now = getattr(torch._C, "_cuda_getDevice", None) or (lambda: torch.cuda.current_device())
_stream_now = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _current():
    """Current device and its current stream's handle; no tensor is on device -2."""
    if not torch.cuda.is_initialized():
        return -2, 0
    dev = _device_now()
    return dev, _stream_now(dev)


def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    want = "x".join("*" if n is None else str(n) for n in shape)
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {want}, got {t.dtype} {tuple(t.shape)}"
                     + ("" if t.is_contiguous() else ", not contiguous"))


def _arg(t, name, dtype, shape, dev, Tensor=torch.Tensor):
    """Address of a contiguous tensor of exactly this type and shape on device dev."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _arg_rows(t, name, dtype, shape, dev, Tensor=torch.Tensor):
    """Address and row stride of a tensor [T, H, D] whose rows are contiguous (any stride between them)."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        _refuse(t, name, dtype, shape, dev)
    rows, inner, last = t.stride()
    if (last != 1 and shape[2] > 1 or inner != shape[2] and shape[1] > 1) and t.numel():
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), rows


def _rows(t, name, dev):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        _refuse(t, name, "float32 or bfloat16", (None,) * 3, dev)
    return t.shape[0]


def _arg_cache(k_cache, v_cache, block_table, B, dev):
    """Addresses and sizes of a paged cache [num_blocks, Hkv, block_size, D] and its block table [B, max_blocks]."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.dtype not in (torch.float32, torch.bfloat16):
        _refuse(k_cache, "k_cache", "float32 or bfloat16", (None,) * 4, dev)
    shape = k_cache.shape
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        _refuse(block_table, "block_table", torch.int32, (B, None), dev)
    width = block_table.shape[1]
    dt = k_cache.dtype
    return (_arg(k_cache, "k_cache", dt, shape, dev), _arg(v_cache, "v_cache", dt, shape, dev), shape, dt,
            _arg(block_table, "block_table", torch.int32, (B, width), dev), width)


def _arg_batch(seq_lens, dev):
    """Address and length of seq_lens [B]."""
    if not isinstance(seq_lens, torch.Tensor):
        _refuse(seq_lens, "seq_lens", torch.int32, (None,), dev)
    B = seq_lens.numel()
    return _arg(seq_lens, "seq_lens", torch.int32, (B,), dev), B


def _arg_status(status, dev):
    return None if status is None else _arg(status, "status", torch.int32, status.shape, dev)


def _code(dtype):
    if dtype == torch.float32:
        return TV_F32
    if dtype == torch.bfloat16:
        return TV_BF16
    raise ValueError(f"unsupported dtype {dtype}")


def tv_version():
    return lib().tv_version()


def tv_tree_build(paths, max_nodes=64):
    """Rank paths -> (parent, depth, mask (uint64), path_to_node, n_nodes) on the host."""
    ranks = np.array([r for p in paths for r in p], dtype=np.int32)
    offsets = np.zeros(len(paths) + 1, dtype=np.int32)
    offsets[1:] = np.cumsum([len(p) for p in paths])
    parent = np.zeros(max_nodes, dtype=np.int32)
    depth = np.zeros(max_nodes, dtype=np.int32)
    mask = np.zeros(max_nodes, dtype=np.uint64)
    p2n = np.zeros(max(len(paths), 1), dtype=np.int32)
    n = np.zeros(1, dtype=np.int32)
    _check("tv_tree_build", lib().tv_tree_build(_ptr(ranks) if ranks.size else None, _ptr(offsets), len(paths),
                                                max_nodes, _ptr(parent), _ptr(depth), _ptr(mask), _ptr(p2n), _ptr(n)))
    k = int(n[0])
    return parent[:k].copy(), depth[:k].copy(), mask[:k].copy(), p2n[:len(paths)].copy(), k


def tv_tree_mask(parent, seq_lens, status=None, mask=None, depth=None, pos=None, stream=None, n_nodes=None):
    """parent int32 [N] (shared) or [B, N]; seq_lens int32 [B]; n_nodes int32 [B]
    (optional, ragged trees: nodes >= n_nodes[b] absent) -> (mask int64 [B, N]
    holding the uint64 rows, depth int32 [B, N], pos int32 [B, N])."""
    _dev(parent, "parent", (torch.int32,))
    _dev(seq_lens, "seq_lens", (torch.int32,))
    if n_nodes is not None:
        _dev(n_nodes, "n_nodes", (torch.int32,))
    B = seq_lens.numel()
    N = parent.shape[-1]
    bstride = 0 if parent.dim() == 1 else parent.stride(0)
    dev = seq_lens.device
    mask = torch.empty(B, N, dtype=torch.int64, device=dev) if mask is None else mask
    depth = torch.empty(B, N, dtype=torch.int32, device=dev) if depth is None else depth
    pos = torch.empty(B, N, dtype=torch.int32, device=dev) if pos is None else pos
    _check("tv_tree_mask", lib().tv_tree_mask(_ptr(parent), bstride, _ptr(seq_lens), _ptr(n_nodes), B, N, _ptr(mask),
                                              _ptr(depth), _ptr(pos), _ptr(status), _stream(stream)))
    return mask, depth, pos


def tv_rope_table(max_pos, head_dim, base=10000.0, device="cuda", stream=None):
    cs = torch.empty(max_pos, 2, head_dim // 2, dtype=torch.float32, device=device)
    _check("tv_rope_table", lib().tv_rope_table(_ptr(cs), max_pos, head_dim, float(base), _stream(stream)))
    return cs


def tv_rope_apply(q, k_tree, pos, cos_sin, status=None, stream=None):
    """Rotates q [B, N, Hq, D] and k_tree [B, N, Hkv, D] in place at pos [B, N]."""
    _dev(q, "q", (torch.float32, torch.bfloat16))
    if k_tree is not None:
        _dev(k_tree, "k_tree", (q.dtype,))
    _dev(pos, "pos", (torch.int32,))
    _dev(cos_sin, "cos_sin", (torch.float32,))
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2] if k_tree is not None else 1
    _check("tv_rope_apply", lib().tv_rope_apply(_ptr(q), _ptr(k_tree), _ptr(pos), _ptr(cos_sin), cos_sin.shape[0],
                                                B, N, Hq, Hkv, D, _code(q.dtype), _ptr(status), _stream(stream)))


def tv_tree_attn_workspace_size(B, N, Hq, Hkv, head_dim, dtype, block_size, num_ctas=0, flags=0):
    out = ctypes.c_size_t(0)
    _check("tv_tree_attn_workspace_size",
           lib().tv_tree_attn_workspace_size(B, N, Hq, Hkv, head_dim, _code(dtype), block_size, num_ctas, flags,
                                             ctypes.addressof(out)))
    return out.value


def alloc_workspace(nbytes, device="cuda"):
    """A 256-byte aligned workspace tensor of at least nbytes, zeroed (so it
    can be passed with TV_ATTN_WORKSPACE_ZEROED until a call times out)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def tv_tree_attn_verify(q, k_cache, v_cache, block_table, seq_lens, k_tree, v_tree, mask, *, scale=None,
                        out=None, lse=None, workspace=None, num_ctas=0, flags=0, status=None, stream=None):
    """Tree attention; returns out [B, N, Hq, D].  mask is int64 [B, N] (uint64 rows)
    or [N] (shared)."""
    dts = (torch.float32, torch.bfloat16)
    _dev(q, "q", dts)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_tree", k_tree), ("v_tree", v_tree)):
        _dev(t, name, (q.dtype,))
    _dev(block_table, "block_table", (torch.int32,))
    _dev(seq_lens, "seq_lens", (torch.int32,))
    _dev(mask, "mask", (torch.int64,))
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    num_blocks, _, block_size, _ = k_cache.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(tv_tree_attn_workspace_size(B, N, Hq, Hkv, D, q.dtype, block_size, num_ctas,
                                                                flags), q.device)
    mstride = 0 if mask.dim() == 1 else mask.stride(0)
    _check("tv_tree_attn_verify",
           lib().tv_tree_attn_verify(_ptr(q), _ptr(k_cache), _ptr(v_cache), num_blocks, block_size, _ptr(block_table),
                                     block_table.shape[1], _ptr(seq_lens), _ptr(k_tree), _ptr(v_tree), _ptr(mask),
                                     mstride, B, N, Hq, Hkv, D, _code(q.dtype), scale, _ptr(out), _ptr(lse),
                                     _ptr(workspace), workspace.numel(), num_ctas, flags, _ptr(status),
                                     _stream(stream)))
    return out


def tv_tree_attn_verify_rope(q, k_cache, v_cache, block_table, seq_lens, k_tree, v_tree, mask, cos_sin, *,
                             scale=None, out=None, lse=None, workspace=None, num_ctas=0, flags=0, status=None,
                             stream=None):
    """Tree attention with Q rotated as it is loaded (q unrotated and left as
    it is; k_tree already rotated); returns out [B, N, Hq, D], the same bits as
    tv_rope_apply followed by tv_tree_attn_verify."""
    dts = (torch.float32, torch.bfloat16)
    _dev(q, "q", dts)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_tree", k_tree), ("v_tree", v_tree)):
        _dev(t, name, (q.dtype,))
    _dev(block_table, "block_table", (torch.int32,))
    _dev(seq_lens, "seq_lens", (torch.int32,))
    _dev(mask, "mask", (torch.int64,))
    _dev(cos_sin, "cos_sin", (torch.float32,))
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    num_blocks, _, block_size, _ = k_cache.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = alloc_workspace(tv_tree_attn_workspace_size(B, N, Hq, Hkv, D, q.dtype, block_size, num_ctas,
                                                                flags | TV_ATTN_ROPE_Q), q.device)
    mstride = 0 if mask.dim() == 1 else mask.stride(0)
    _check("tv_tree_attn_verify_rope",
           lib().tv_tree_attn_verify_rope(_ptr(q), _ptr(k_cache), _ptr(v_cache), num_blocks, block_size,
                                          _ptr(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(k_tree),
                                          _ptr(v_tree), _ptr(mask), mstride, _ptr(cos_sin), cos_sin.shape[0], B, N,
                                          Hq, Hkv, D, _code(q.dtype), scale, _ptr(out), _ptr(lse), _ptr(workspace),
                                          workspace.numel(), num_ctas, flags, _ptr(status), _stream(stream)))
    return out


def tv_tree_prepare(parent, seq_lens, k_tree=None, cos_sin=None, *, q=None, n_nodes=None, status=None, mask=None,
                    depth=None, pos=None, stream=None):
    """tv_tree_mask plus the rotation of k_tree [B, N, Hkv, D] and/or q
    [B, N, Hq, D] in place at pos, in one launch; returns (mask, depth, pos)
    like tv_tree_mask."""
    _dev(parent, "parent", (torch.int32,))
    _dev(seq_lens, "seq_lens", (torch.int32,))
    if n_nodes is not None:
        _dev(n_nodes, "n_nodes", (torch.int32,))
    B = seq_lens.numel()
    N = parent.shape[-1]
    bstride = 0 if parent.dim() == 1 else parent.stride(0)
    dev = seq_lens.device
    mask = torch.empty(B, N, dtype=torch.int64, device=dev) if mask is None else mask
    depth = torch.empty(B, N, dtype=torch.int32, device=dev) if depth is None else depth
    pos = torch.empty(B, N, dtype=torch.int32, device=dev) if pos is None else pos
    Hq = Hkv = D = dt = max_pos = 0
    for t, nm in ((q, "q"), (k_tree, "k_tree")):
        if t is not None:
            _dev(t, nm, (torch.float32, torch.bfloat16))
            _dev(cos_sin, "cos_sin", (torch.float32,))
            D, dt, max_pos = t.shape[3], _code(t.dtype), cos_sin.shape[0]
    if q is not None:
        Hq = q.shape[2]
    if k_tree is not None:
        Hkv = k_tree.shape[2]
    _check("tv_tree_prepare",
           lib().tv_tree_prepare(_ptr(parent), bstride, _ptr(seq_lens), _ptr(n_nodes), B, N, _ptr(mask),
                                 _ptr(depth), _ptr(pos), _ptr(q), Hq, _ptr(k_tree), Hkv, D, dt, _ptr(cos_sin),
                                 max_pos, _ptr(status), _stream(stream)))
    return mask, depth, pos


def tv_tree_attn_static_workspace_bytes():
    return lib().tv_tree_attn_static_workspace_bytes()


def tv_tree_attn_verify_static(q, k_cache, v_cache, block_table, seq_lens, k_tree, v_tree, mask, *, scale=None,
                               out=None, lse=None, num_ctas=0, flags=0, status=None, stream=None):
    """Tree attention without a caller workspace (the library's fixed scratch
    array is used); same arguments and result as tv_tree_attn_verify."""
    dts = (torch.float32, torch.bfloat16)
    _dev(q, "q", dts)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache), ("k_tree", k_tree), ("v_tree", v_tree)):
        _dev(t, name, (q.dtype,))
    _dev(block_table, "block_table", (torch.int32,))
    _dev(seq_lens, "seq_lens", (torch.int32,))
    _dev(mask, "mask", (torch.int64,))
    B, N, Hq, D = q.shape
    Hkv = k_tree.shape[2]
    num_blocks, _, block_size, _ = k_cache.shape
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    mstride = 0 if mask.dim() == 1 else mask.stride(0)
    _check("tv_tree_attn_verify_static",
           lib().tv_tree_attn_verify_static(_ptr(q), _ptr(k_cache), _ptr(v_cache), num_blocks, block_size,
                                            _ptr(block_table), block_table.shape[1], _ptr(seq_lens), _ptr(k_tree),
                                            _ptr(v_tree), _ptr(mask), mstride, B, N, Hq, Hkv, D, _code(q.dtype),
                                            scale, _ptr(out), _ptr(lse), num_ctas, flags, _ptr(status),
                                            _stream(stream)))
    return out


def _accept_outputs(B, out_cols, device, out, n_out, path):
    if out is None:
        out = torch.empty(B, out_cols, dtype=torch.int32, device=device)
    if n_out is None:
        n_out = torch.empty(B, dtype=torch.int32, device=device)
    if path is None:
        path = torch.empty(B, out_cols, dtype=torch.int32, device=device)
    return out, n_out, path


def tv_tree_accept_greedy(tokens, parent, *, logits=None, target_argmax=None, n_nodes=None, out_cols=None,
                          out=None, n_out=None, path=None, status=None, stream=None):
    """Greedy walk; returns (out [B, out_cols], n_out [B], path [B, out_cols])."""
    _dev(tokens, "tokens", (torch.int32,))
    _dev(parent, "parent", (torch.int32,))
    B, N = tokens.shape
    if logits is not None:
        _dev(logits, "logits", (torch.float32,))
        V = logits.shape[-1]
    else:
        _dev(target_argmax, "target_argmax", (torch.int32,))
        V = 1
    out_cols = N if out_cols is None else out_cols
    out, n_out, path = _accept_outputs(B, out_cols, tokens.device, out, n_out, path)
    bstride = 0 if parent.dim() == 1 else parent.stride(0)
    _check("tv_tree_accept_greedy",
           lib().tv_tree_accept_greedy(_ptr(logits), _ptr(target_argmax), _ptr(tokens), _ptr(parent), bstride,
                                       _ptr(n_nodes), B, N, V, _ptr(out), _ptr(n_out), _ptr(path), out_cols,
                                       _ptr(status), _stream(stream)))
    return out, n_out, path


def tv_accept_sample_workspace_size(B, N, V):
    """Bytes of the grid sampler's workspace (tv_tree_accept_sample and
    tv_chain_accept_sample with N = K + 1)."""
    return int(lib().tv_accept_sample_workspace_size(B, N, V))


def tv_accept_sample_uses_grid(B, N, V, flags=0, workspace_bytes=0):
    """Whether a sampler call with these sizes, flags and workspace size takes
    the grid sampler (queries the current device)."""
    g = ctypes.c_int32(0)
    _check("tv_accept_sample_uses_grid",
           lib().tv_accept_sample_uses_grid(B, N, V, int(flags), int(workspace_bytes), ctypes.addressof(g)))
    return bool(g.value)


def _ws(workspace):
    if workspace is None:
        return None, 0
    _dev(workspace, "workspace", (torch.uint8,))
    return workspace, workspace.numel()


def tv_tree_accept_sample(p, q, tokens, parent, u_accept, u_final, *, n_nodes=None, out_cols=None, out=None,
                          n_out=None, path=None, flags=0, workspace=None, status=None, stream=None):
    """Stochastic walk; returns (out [B, out_cols], n_out [B], path [B, out_cols]).
    flags: TV_SAMPLE_AUTO / TV_SAMPLE_CLUSTER / TV_SAMPLE_SINGLE_CTA / TV_SAMPLE_STREAM /
    TV_SAMPLE_GRID; workspace: uint8 device tensor of
    tv_accept_sample_workspace_size(B, N, V) bytes (alloc_workspace), or None."""
    _dev(p, "p", (torch.float32,))
    _dev(q, "q", (torch.float32,))
    _dev(tokens, "tokens", (torch.int32,))
    _dev(parent, "parent", (torch.int32,))
    _dev(u_accept, "u_accept", (torch.float32,))
    _dev(u_final, "u_final", (torch.float32,))
    B, N, V = p.shape
    out_cols = N if out_cols is None else out_cols
    out, n_out, path = _accept_outputs(B, out_cols, p.device, out, n_out, path)
    bstride = 0 if parent.dim() == 1 else parent.stride(0)
    ws, ws_bytes = _ws(workspace)
    _check("tv_tree_accept_sample",
           lib().tv_tree_accept_sample(_ptr(p), _ptr(q), _ptr(tokens), _ptr(parent), bstride, _ptr(n_nodes),
                                       _ptr(u_accept), _ptr(u_final), B, N, V, _ptr(out), _ptr(n_out), _ptr(path),
                                       out_cols, int(flags), _ptr(ws), ws_bytes, _ptr(status), _stream(stream)))
    return out, n_out, path


def tv_chain_accept_sample(p, q, draft, u, u_final, *, num_draft=None, out_cols=None, out=None, n_out=None,
                           flags=0, workspace=None, status=None, stream=None):
    """The verifier page's chain walk, read in place: p float32 [B, K + 1, V],
    q float32 [B, K, V], draft int32 [B, K], u float32 [B, K], u_final float32
    [B], num_draft int32 [B] (optional), workspace as in tv_tree_accept_sample
    (N = K + 1).  Returns (out [B, out_cols] -1 padded, n_out [B] =
    accepted + 1); allocates nothing when out and n_out are given."""
    _dev(p, "p", (torch.float32,))
    _dev(q, "q", (torch.float32,))
    _dev(draft, "draft", (torch.int32,))
    _dev(u, "u", (torch.float32,))
    _dev(u_final, "u_final", (torch.float32,))
    if num_draft is not None:
        _dev(num_draft, "num_draft", (torch.int32,))
    B, K1, V = p.shape
    K = K1 - 1
    if tuple(q.shape) != (B, K, V) or tuple(draft.shape) != (B, K) or tuple(u.shape) != (B, K):
        raise ValueError("tv_chain_accept_sample: q [B, K, V], draft and u [B, K] with p [B, K + 1, V]")
    out_cols = K1 if out_cols is None else out_cols
    out, n_out, _ = _accept_outputs(B, out_cols, p.device, out, n_out, False)
    ws, ws_bytes = _ws(workspace)
    _check("tv_chain_accept_sample",
           lib().tv_chain_accept_sample(_ptr(p), _ptr(q), _ptr(draft), _ptr(num_draft), _ptr(u), _ptr(u_final), B,
                                        K, V, _ptr(out), _ptr(n_out), out_cols, int(flags), _ptr(ws), ws_bytes,
                                        _ptr(status), _stream(stream)))
    return out, n_out


def verify_chain(draft, q, p, num_draft, u, u_final, *, flags=0, out=None, n_out=None, workspace=None, status=None,
                 stream=None):
    """The verifier page's verify(draft, q, p, num_draft, u, u_final) call:
    draft int32 [B, K] (draft j drawn from q[:, j]); q float32 [B, K, V]; p
    float32 [B, K + 1, V] (the target after each prefix, the last row for the
    bonus); num_draft int32 [B] (ragged); u float32 [B, K] (one uniform per
    test); u_final float32 [B].  Returns (out int32 [B, K + 1] -1 padded,
    n_out int32 [B] = accepted + 1).  Marshalling only, through
    tv_chain_accept_sample: the arrays are read in place, and with out and
    n_out given nothing is allocated."""
    return tv_chain_accept_sample(p, q, draft, u, u_final, num_draft=num_draft, out=out, n_out=n_out, flags=flags,
                                  workspace=workspace, status=status, stream=stream)


def accept_greedy(parent, tokens, target_argmax, *, n_nodes=None, status=None, stream=None):
    """The mask page's accept_greedy(parent, tokens, target_argmax) on top of
    tv_tree_accept_greedy: parent int32 [N] or [B, N], tokens int32 [B, N],
    target_argmax int32 [B, N] (the target's choice after each node).  Returns
    (out, n_out, path) like tv_tree_accept_greedy."""
    return tv_tree_accept_greedy(tokens, parent, target_argmax=target_argmax, n_nodes=n_nodes, status=status,
                                 stream=stream)


def tv_kv_commit(k_cache, v_cache, block_table, seq_lens, k_tree, v_tree, path, n_out, *, new_seq_lens=None,
                 status=None, stream=None):
    """Copy the accepted path's tree K/V rows into the paged cache (in place);
    returns new_seq_lens int32 [B] = seq_lens + n_out."""
    for t, nm in ((k_cache, "k_cache"), (v_cache, "v_cache"), (k_tree, "k_tree"), (v_tree, "v_tree")):
        _dev(t, nm, (torch.float32, torch.bfloat16))
    for t, nm in ((block_table, "block_table"), (seq_lens, "seq_lens"), (path, "path"), (n_out, "n_out")):
        _dev(t, nm, (torch.int32,))
    num_blocks, Hkv, bs, D = k_cache.shape
    B, N = k_tree.shape[0], k_tree.shape[1]
    if new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
    _check("tv_kv_commit",
           lib().tv_kv_commit(_ptr(k_cache), _ptr(v_cache), num_blocks, bs, _ptr(block_table), block_table.shape[1],
                              _ptr(seq_lens), _ptr(new_seq_lens), _ptr(k_tree), _ptr(v_tree), _ptr(path),
                              path.shape[1], _ptr(n_out), B, N, Hkv, D, _code(k_cache.dtype), _ptr(status),
                              _stream(stream)))
    return new_seq_lens


def tv_kv_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, *, cos_sin=None, q=None, q_out=None,
                 cu_new=None, new_seq_lens=None, status=None, stream=None):
    """Put new tokens' K/V rows [T, Hkv, D] into the paged cache (in place), keys
    rotated with cos_sin (None: stored as given) at the positions that follow
    seq_lens; q [T, Hq, D] is rotated into q_out (may be q).  Rows of k_new, v_new,
    q and q_out may be strided.  cu_new int32 [B + 1]: packed offsets; None: T / B
    tokens each.  Returns (q_out, new_seq_lens int32 [B])."""
    if stream is not None:  # under it, so that what the call allocates is ordered and reused with its work
        with torch.cuda.stream(stream):
            return tv_kv_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, cos_sin=cos_sin, q=q, q_out=q_out,
                                cu_new=cu_new, new_seq_lens=new_seq_lens, status=status)
    dev, st = _current()
    lens, B = _arg_batch(seq_lens, dev)
    kc, vc, (num_blocks, Hkv, bs, D), dt, table, width = _arg_cache(k_cache, v_cache, block_table, B, dev)
    T = _rows(k_new, "k_new", dev)
    k, k_stride = _arg_rows(k_new, "k_new", dt, (T, Hkv, D), dev)
    v, v_stride = _arg_rows(v_new, "v_new", dt, (T, Hkv, D), dev)
    cs = qp = qo = cu = None
    Hq = max_pos = q_stride = out_stride = 0
    if cos_sin is not None:
        max_pos = _rows(cos_sin, "cos_sin", dev)
        cs = _arg(cos_sin, "cos_sin", torch.float32, (max_pos, 2, D // 2), dev)
    if q is not None:
        _rows(q, "q", dev)
        Hq = q.shape[1]
        qp, q_stride = _arg_rows(q, "q", dt, (T, Hq, D), dev)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
            qo, out_stride = q_out.data_ptr(), Hq * D
        else:
            qo, out_stride = _arg_rows(q_out, "q_out", dt, (T, Hq, D), dev)
    if cu_new is not None:
        cu = _arg(cu_new, "cu_new", torch.int32, (B + 1,), dev)
    if new_seq_lens is None:
        new_seq_lens = torch.empty_like(seq_lens)
        new = new_seq_lens.data_ptr()
    else:
        new = _arg(new_seq_lens, "new_seq_lens", torch.int32, (B,), dev)
    code = lib().tv_kv_append(qp, q_stride, qo, out_stride, Hq, k, k_stride, v, v_stride, cu, T, kc, vc, num_blocks, bs,
                              table, width, lens, new, cs, max_pos, B, Hkv, D,
                              TV_F32 if dt is torch.float32 else TV_BF16, _arg_status(status, dev), st)
    if code:
        _check("tv_kv_append", code)
    return q_out, new_seq_lens


def tv_decode_attn_workspace_size(Hq, Hkv, head_dim, dtype, num_ctas=0):
    out = ctypes.c_size_t(0)
    _check("tv_decode_attn_workspace_size",
           lib().tv_decode_attn_workspace_size(Hq, Hkv, head_dim, _code(dtype), num_ctas, ctypes.addressof(out)))
    return out.value


def tv_decode_attn(q, k_cache, v_cache, block_table, seq_lens, *, scale=None, softcap=0.0, window=0, n_sink=0,
                   slopes=None, out=None, lse=None, workspace=None, num_ctas=0, flags=0, status=None, stream=None):
    """Attention of one new token per request over the paged cache (which holds
    its K/V already); returns out [B, Hq, D].  q [B, Hq, D] may be strided
    between requests; softcap, window / n_sink and slopes as in the header;
    lse float32 [B, Hq] is filled when given."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return tv_decode_attn(q, k_cache, v_cache, block_table, seq_lens, scale=scale, softcap=softcap, window=window,
                                  n_sink=n_sink, slopes=slopes, out=out, lse=lse, workspace=workspace,
                                  num_ctas=num_ctas, flags=flags, status=status)
    if (window | n_sink | num_ctas | flags) >> 31 not in (0, -1):  # ctypes would take them modulo 2^32
        raise ValueError(f"window {window}, n_sink {n_sink}, num_ctas {num_ctas} or flags {flags} does not fit 32 bits")
    dev, st = _current()
    lens, B = _arg_batch(seq_lens, dev)
    kc, vc, (num_blocks, Hkv, bs, D), dt, table, width = _arg_cache(k_cache, v_cache, block_table, B, dev)
    _rows(q, "q", dev)
    Hq = q.shape[1]
    qp, q_stride = _arg_rows(q, "q", dt, (B, Hq, D), dev)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=dt, device=q.device)
        op = out.data_ptr()
    else:
        op = _arg(out, "out", dt, (B, Hq, D), dev)
    if workspace is None:
        # the call clears the counters, the first 16 KiB of up to 16 MiB
        workspace = torch.empty(tv_decode_attn_workspace_size(Hq, Hkv, D, dt, num_ctas), dtype=torch.uint8, device=q.device)
        flags &= ~TV_ATTN_WORKSPACE_ZEROED
    n_ws = workspace.numel()
    code = lib().tv_decode_attn(qp, q_stride, kc, vc, num_blocks, bs, table, width, lens, B, Hq, Hkv, D,
                                TV_F32 if dt is torch.float32 else TV_BF16,
                                1.0 / math.sqrt(D) if scale is None else scale, softcap, window, n_sink,
                                None if slopes is None else _arg(slopes, "slopes", torch.float32, (Hq,), dev), op,
                                None if lse is None else _arg(lse, "lse", torch.float32, (B, Hq), dev),
                                _arg(workspace, "workspace", torch.uint8, (n_ws,), dev), n_ws, num_ctas, flags,
                                _arg_status(status, dev), st)
    if code:
        _check("tv_decode_attn", code)
    return out


def tv_token_logprobs(logits, tokens, *, node=None, top_k=0, logprob=None, entropy=None, top_ids=None,
                      top_logprobs=None, status=None, stream=None):
    """Log probabilities of tokens [B, C] under rows node [B, C] (None: row c) of
    logits [B, N, V] (float32 or bf16); returns (logprob, entropy [B, C] float32,
    top_ids int32, top_logprobs float32 [B, C, top_k]).  tokens and node may be
    out and path of tv_tree_accept_*: -1 is no entry."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return tv_token_logprobs(logits, tokens, node=node, top_k=top_k, logprob=logprob, entropy=entropy,
                                     top_ids=top_ids, top_logprobs=top_logprobs, status=status)
    if top_k >> 31 not in (0, -1):
        raise ValueError(f"top_k {top_k} does not fit 32 bits")
    dev, st = _current()
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3 or logits.dtype not in (torch.float32, torch.bfloat16):
        _refuse(logits, "logits", "float32 or bfloat16", (None,) * 3, dev)
    B, N, V = logits.shape
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 2:
        _refuse(tokens, "tokens", torch.int32, (B, None), dev)
    C = tokens.shape[1]
    f32, where = torch.float32, logits.device
    x = _arg(logits, "logits", logits.dtype, (B, N, V), dev)
    tok = _arg(tokens, "tokens", torch.int32, (B, C), dev)
    row = None if node is None else _arg(node, "node", torch.int32, (B, C), dev)
    k = max(top_k, 0)

    def output(t, name, dtype, shape):  # given, or made here
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=where)
            return t, t.data_ptr()
        return t, _arg(t, name, dtype, shape, dev)

    logprob, p_lp = output(logprob, "logprob", f32, (B, C))
    entropy, p_ent = output(entropy, "entropy", f32, (B, C))
    top_ids, p_ids = output(top_ids, "top_ids", torch.int32, (B, C, k))
    top_logprobs, p_top = output(top_logprobs, "top_logprobs", f32, (B, C, k))
    code = lib().tv_token_logprobs(x, tok, row, B, N, C, V, TV_F32 if logits.dtype is f32 else TV_BF16, p_lp, p_ent, top_k,
                                   p_ids, p_top, _arg_status(status, dev), st)
    if code:
        _check("tv_token_logprobs", code)
    return logprob, entropy, top_ids, top_logprobs

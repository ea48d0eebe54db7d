"""Binding of the attention entry points of libfmoe.so (see include/fmoe_attn.h for the
contract): a paged key/value cache in the library's 4-bit format, single-token attention
over it and causal attention over packed prompts.

Functions keep the C names and take torch CUDA tensors; tensors are checked for type, shape
and layout, everything else by the library.  `error` is an int32 or uint32 tensor of one
element for the device-side error bits, or None."""
from __future__ import annotations

import ctypes

import torch

from . import fmoe

DEVERR_BAD_SLOT = 0x10
DEVERR_BAD_POSITION = 0x20
DEVERR_BAD_PAGE = 0x40
DEVERR_BAD_LENGTH = 0x80

TILE_TOKENS = 16

# every symbol include/fmoe_attn.h declares
EXPORTS = ["fmoe_kv_page_bytes", "fmoe_kv_append", "fmoe_kv_gather", "fmoe_attn_decode", "fmoe_attn_workspace_bytes",
           "fmoe_attn_prompt"]


class fmoe_attn_config(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_tokens", ctypes.c_int)]

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, page_tokens: int = 64):
        super().__init__(q_heads, kv_heads, head_dim, page_tokens)
        self.ref = ctypes.byref(self)


_lib = None


def lib():
    global _lib
    if _lib is None:
        L = fmoe.lib()
        vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        cfg = ctypes.POINTER(fmoe_attn_config)
        L.fmoe_kv_page_bytes.restype = sz
        L.fmoe_kv_page_bytes.argtypes = [cfg]
        L.fmoe_attn_workspace_bytes.restype = sz
        L.fmoe_attn_workspace_bytes.argtypes = [cfg]
        L.fmoe_kv_append.argtypes = [cfg, vp, i64, vp, i64, vp, i64, i32, vp, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp]
        L.fmoe_kv_gather.argtypes = [cfg, vp, i64, vp, i32, i32, vp, vp, i64, vp, vp, vp, vp]
        L.fmoe_attn_decode.argtypes = [cfg, vp, i64, vp, i64, vp, i32, vp, i32, f32, vp, vp, sz, vp, vp]
        L.fmoe_attn_prompt.argtypes = [cfg, vp, i64, vp, i64, vp, i64, vp, vp, i32, i64, i64, f32, vp, vp, vp]
        _lib = L
    return _lib


def _stream(stream, t) -> int:
    """The raw stream handle to launch on; the tensors' device has to be the current one.
    (torch.cuda.current_stream() takes 3 us, as long as a small call's launch.)"""
    d = t.get_device()
    if d != torch._C._cuda_getDevice():
        _refuse(f"the tensors are on device {d}, which is not the current one")
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream


def _refuse(what: str):
    raise fmoe.FmoeError(1, what)


def _rows(t, heads: int, dim: int, what: str):
    """(pointer, row stride, rows) of a bf16 [rows][heads][dim] tensor whose heads are contiguous."""
    shape, stride = t.shape, t.stride()
    if (t.dtype is not torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != dim or stride[2] != 1
            or (stride[1] != dim and heads > 1) or not t.is_cuda):
        _refuse(f"{what}: bf16 [rows][{heads}][{dim}] with contiguous heads on the GPU is wanted")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * dim, shape[0]


def _whole(t, heads: int, dim: int, what: str):
    p, stride, n = _rows(t, heads, dim, what)
    if stride != heads * dim:
        _refuse(f"{what}: contiguous rows are wanted")
    return p, n


def _ints(t, dtype, shape, what: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        _refuse(f"{what}: contiguous {dtype} {tuple(shape)} on the GPU is wanted")
    return t.data_ptr()


def _error(t):
    if t is None:
        return None
    if t.element_size() != 4 or t.numel() != 1 or not t.is_cuda:
        _refuse("error: one 32-bit word on the GPU is wanted")
    return t.data_ptr()


def _pages(cfg, cache):
    """Pointer and page count of a cache tensor: uint8, contiguous, whole pages."""
    size = cfg.page_bytes = getattr(cfg, "page_bytes", None) or fmoe_kv_page_bytes(cfg)
    n = cache.numel()
    if cache.dtype is not torch.uint8 or not cache.is_contiguous() or not size or n % size or not cache.is_cuda:
        _refuse(f"cache: contiguous uint8 pages of {size} bytes on the GPU are wanted")
    return cache.data_ptr(), n // size


def fmoe_kv_page_bytes(cfg: fmoe_attn_config) -> int:
    return lib().fmoe_kv_page_bytes(cfg.ref)


def fmoe_attn_workspace_bytes(cfg: fmoe_attn_config) -> int:
    return lib().fmoe_attn_workspace_bytes(cfg.ref)


def attn_workspace(cfg: fmoe_attn_config, device="cuda"):
    """A zeroed workspace for fmoe_attn_decode."""
    return torch.zeros(fmoe_attn_workspace_bytes(cfg), dtype=torch.uint8, device=device)


def kv_cache(cfg: fmoe_attn_config, pages: int, device="cuda"):
    """An empty cache of `pages` pages."""
    return torch.zeros(pages, fmoe_kv_page_bytes(cfg), dtype=torch.uint8, device=device)


def rope_table(positions: int, rotary: int, theta: float = 10000.0, device="cuda"):
    """fp32 [positions][2][rotary/2]: cosines and sines of position * theta^(-2i/rotary),
    from angles in fp64 (in fp32 a far position's angle is off by whole radians' worth)."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64, device=device)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * theta ** (-i / rotary)
    return torch.stack([a.cos(), a.sin()], 1).float().contiguous()


def fmoe_kv_append(cfg: fmoe_attn_config, q, k, v, rope, positions, slots, cache, q_out=None, k_out=None, error=None,
                   stream=None):
    """Rotates q and k [T][heads][D], writes k and v into the cache's slots, the rotated q and
    k to q_out and k_out.  rope fp32 [positions][2][rotary/2] or None (no rotation); q and
    q_out may be None together, k_out may be None."""
    D, H, KV = cfg.head_dim, cfg.q_heads, cfg.kv_heads
    kp, ks, T = _rows(k, KV, D, "k")
    vp, vs, n = _rows(v, KV, D, "v")
    qp, qs = None, 0
    qo = ko = pos = table = None
    known = rotary = 0
    if q is not None:
        qp, qs, m = _rows(q, H, D, "q")
        n = n if m == T else -1
    if q_out is not None:
        qo, m = _whole(q_out, H, D, "q_out")
        n = n if m == T else -1
    if k_out is not None:
        ko, m = _whole(k_out, KV, D, "k_out")
        n = n if m == T else -1
    if n != T:
        _refuse("q, k, v, q_out and k_out have as many rows as each other")
    if rope is not None:
        known, two, rotary = rope.shape
        rotary *= 2
        if rope.dtype is not torch.float32 or two != 2 or not rope.is_contiguous() or not rope.is_cuda:
            _refuse("rope: contiguous fp32 [positions][2][rotary/2] on the GPU is wanted")
        table = rope.data_ptr()
        pos = _ints(positions, torch.int32, (T,), "positions")
    cp, pages = _pages(cfg, cache)
    st = lib().fmoe_kv_append(cfg.ref, qp, qs, kp, ks, vp, vs, T, table, known, rotary, pos,
                              _ints(slots, torch.int64, (T,), "slots"), cp, pages, qo, ko, _error(error),
                              _stream(stream, cache))
    fmoe._check(st, "fmoe_kv_append")


def fmoe_kv_gather(cfg: fmoe_attn_config, cache, page_table, cu, k_out, v_out, first=None, error=None, stream=None):
    """Cached tokens as packed bf16 rows [rows][kv_heads][D]: sequence s's tokens from first[s]
    (0 without `first`) on into rows cu[s] .. cu[s+1] - 1."""
    D, KV = cfg.head_dim, cfg.kv_heads
    kp, n = _whole(k_out, KV, D, "k_out")
    vp, m = _whole(v_out, KV, D, "v_out")
    if n != m:
        _refuse("k_out and v_out have as many rows as each other")
    seqs, width = page_table.shape
    cp, pages = _pages(cfg, cache)
    st = lib().fmoe_kv_gather(cfg.ref, cp, pages, _ints(page_table, torch.int32, (seqs, width), "page_table"), width, seqs,
                              None if first is None else _ints(first, torch.int32, (seqs,), "first"),
                              _ints(cu, torch.int32, (seqs + 1,), "cu"), n, kp, vp, _error(error), _stream(stream, cache))
    fmoe._check(st, "fmoe_kv_gather")


def fmoe_attn_decode(cfg: fmoe_attn_config, q, cache, page_table, lens, out, scale, workspace, error=None, stream=None):
    """out[s] = attention of the single query row q[s] [q_heads][D] over the first lens[s]
    cached tokens of the sequence."""
    D, H = cfg.head_dim, cfg.q_heads
    qp, qs, seqs = _rows(q, H, D, "q")
    op, n = _whole(out, H, D, "out")
    width = page_table.shape[-1]
    if n != seqs or workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or not workspace.is_cuda:
        _refuse("q and out have as many rows as each other; workspace: contiguous uint8 on the GPU is wanted")
    cp, pages = _pages(cfg, cache)
    st = lib().fmoe_attn_decode(cfg.ref, qp, qs, cp, pages, _ints(page_table, torch.int32, (seqs, width), "page_table"),
                                width, _ints(lens, torch.int32, (seqs,), "lens"), seqs, scale, op, workspace.data_ptr(),
                                workspace.numel(), _error(error), _stream(stream, q))
    fmoe._check(st, "fmoe_attn_decode")
    return out


def fmoe_attn_prompt(cfg: fmoe_attn_config, q, k, v, cu_q, cu_k, out, scale, error=None, stream=None):
    """Causal attention of packed sequences: q and out [q_rows][q_heads][D], k and v
    [k_rows][kv_heads][D], row offsets cu_q and cu_k int32 [seqs + 1]."""
    D, H, KV = cfg.head_dim, cfg.q_heads, cfg.kv_heads
    qp, qs, n = _rows(q, H, D, "q")
    kp, ks, m = _rows(k, KV, D, "k")
    vp, vs, mv = _rows(v, KV, D, "v")
    op, no = _whole(out, H, D, "out")
    seqs = cu_q.shape[0] - 1
    if mv != m or no != n:
        _refuse("k and v, and q and out, have as many rows as each other")
    st = lib().fmoe_attn_prompt(cfg.ref, qp, qs, kp, ks, vp, vs, _ints(cu_q, torch.int32, (seqs + 1,), "cu_q"),
                                _ints(cu_k, torch.int32, (seqs + 1,), "cu_k"), seqs, n, m, scale, op, _error(error),
                                _stream(stream, q))
    fmoe._check(st, "fmoe_attn_prompt")
    return out

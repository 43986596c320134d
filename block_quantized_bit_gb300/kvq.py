"""Thin ctypes binding of libkvq (``include/kvq.h``), with the same entry-point names.

Argument marshalling only: torch tensors are passed as raw device pointers plus sizes, and the
current torch CUDA stream as the ``stream`` argument.  Every step of the store and the decode runs
in libkvq's CUDA kernels.  If the library has not been built, importing works but every call raises
``RuntimeError`` -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")

KVQ_FP8_E4M3 = 1
KVQ_Q8_0 = 2
KVQ_FP8_E4M3_UNSCALED = 3
KVQ_FP8_E5M2_UNSCALED = 4
KIND = {"fp8_e4m3": KVQ_FP8_E4M3, "q8_0": KVQ_Q8_0, "fp8_e4m3_unscaled": KVQ_FP8_E4M3_UNSCALED,
        "fp8_e5m2_unscaled": KVQ_FP8_E5M2_UNSCALED}
KVQ_OUT_BF16 = 0
KVQ_OUT_F32 = 1

STATUS = {0: "KVQ_OK", -1: "KVQ_EINVAL", -2: "KVQ_EKIND", -3: "KVQ_EHEADDIM", -4: "KVQ_EALIGN",
          -5: "KVQ_EWORKSPACE", -6: "KVQ_EARCH", -7: "KVQ_ECUDA", -8: "KVQ_EUNSUPPORTED", -9: "KVQ_ETIMEOUT",
          -10: "KVQ_ENOPAGES"}

EXPORTS = ["kvq_pool_bytes", "kvq_scale_bytes", "kvq_bytes_per_token", "kvq_num_pages", "kvq_store",
           "kvq_decode_workspace_bytes", "kvq_decode_workspace_bytes_ex", "kvq_decode_path",
           "kvq_decode_sparse_workspace_bytes", "kvq_decode_sparse", "kvq_decode", "kvq_decode_ex",
           "kvq_workspace_status", "kvq_encode_probe", "kvq_quantize_probe", "kvq_dequant_probe", "kvq_strerror",
           "kvq_device_check", "kvq_version", "kvq_decode_noalloc", "kvq_noalloc_status", "kvq_wait_probe",
           "kvq_extend_workspace_bytes", "kvq_extend", "kvq_store_act_quant", "kvq_store_unscaled",
           "kvq_bytes_per_token_ex", "kvq_num_pages_ex", "kvq_exp2_probe", "kvq_extend_workspace_bytes_ex",
           "kvq_extend_ex", "kvq_extend_path", "kvq_pages_workspace_bytes", "kvq_pages_copy", "kvq_pages_fork",
           "kvq_pages_resize", "kvq_pages_compact", "kvq_tree_workspace_bytes", "kvq_tree",
           "kvq_prompt_workspace_bytes", "kvq_prompt"]


class kvq_layout(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("v_dim", ctypes.c_int32), ("mla", ctypes.c_int32)]


class kvq_decode_options(ctypes.Structure):
    _fields_ = [("pages_per_split", ctypes.c_int32), ("path", ctypes.c_int32)]


class kvq_extend_options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("precise_p", ctypes.c_int32)]


class kvq_prompt_strides(ctypes.Structure):
    _fields_ = [(x + "_" + y, ctypes.c_int64) for x in ("q", "k", "v", "out") for y in ("token", "head")]


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (where, STATUS.get(status, status), strerror(status)))


_lib = None


def lib():
    """The loaded libkvq (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkvq.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        LP = ctypes.POINTER(kvq_layout)
        OP = ctypes.POINTER(kvq_decode_options)
        EP = ctypes.POINTER(kvq_extend_options)
        sig = {
            "kvq_pool_bytes": (sz, [LP]),
            "kvq_scale_bytes": (sz, [LP]),
            "kvq_bytes_per_token": (ctypes.c_double, [LP]),
            "kvq_num_pages": (i64, [LP, sz]),
            "kvq_bytes_per_token_ex": (ctypes.c_double, [LP, i32]),
            "kvq_num_pages_ex": (i64, [LP, i32, sz]),
            "kvq_store": (i32, [P, P, P, P, P, i64, LP, i32, P]),
            "kvq_decode_workspace_bytes": (sz, [LP, i32, i32, i32]),
            "kvq_decode_workspace_bytes_ex": (sz, [LP, i32, i32, i32, OP]),
            "kvq_decode_path": (i32, [LP, i32, i32, i32, OP]),
            "kvq_decode_sparse_workspace_bytes": (sz, [LP, i32, i32, i32]),
            "kvq_decode_sparse": (i32, [P, P, P, P, i32, P, P, i32, i32, i32, ctypes.c_float, P, i32, P, sz, LP,
                                        i32, P]),
            "kvq_decode": (i32, [P, P, P, P, i32, P, i32, i32, ctypes.c_float, P, i32, P, sz, LP, i32, P]),
            "kvq_extend_workspace_bytes": (sz, []),
            "kvq_store_act_quant": (i32, [P, P, P, P, i64, i32, LP, i32, P]),
            "kvq_store_unscaled": (i32, [P, P, P, P, i64, LP, i32, P]),
            "kvq_extend": (i32, [P, P, P, P, i32, P, P, i32, i32, i32, ctypes.c_float, P, i32, P, sz, LP, i32, P]),
            "kvq_decode_ex": (i32, [P, P, P, P, i32, P, i32, i32, ctypes.c_float, P, i32, P, sz, LP, i32, OP, P]),
            "kvq_workspace_status": (i32, [P, P]),
            "kvq_encode_probe": (i32, [i32, P, P, i64, P]),
            "kvq_dequant_probe": (i32, [i32, P, P, P, i64, P]),
            "kvq_quantize_probe": (i32, [i32, P, i64, P, i64, P, P]),
            "kvq_strerror": (ctypes.c_char_p, [i32]),
            "kvq_device_check": (i32, []),
            "kvq_version": (ctypes.c_char_p, []),
            "kvq_decode_noalloc": (i32, [P, P, P, P, i32, P, i32, i32, ctypes.c_float, P, i32, LP, i32, P]),
            "kvq_wait_probe": (i32, [P, P]),
            "kvq_noalloc_status": (i32, [P]),
            "kvq_exp2_probe": (i32, [P, P, i64, P]),
            "kvq_extend_workspace_bytes_ex": (sz, [LP, i32, i32, i32, EP]),
            "kvq_extend_path": (i32, [LP, i32, i32, i32, EP]),
            "kvq_extend_ex": (i32, [P, P, P, P, i32, P, P, i32, i32, i32, ctypes.c_float, P, i32, P, sz, LP, i32,
                                    EP, P]),
            "kvq_prompt_workspace_bytes": (sz, []),
            "kvq_prompt": (i32, [P, P, P, P, i32, i32, i32, i32, i32, ctypes.c_float, P, i32,
                                 ctypes.POINTER(kvq_prompt_strides), P, sz, P]),
            "kvq_tree_workspace_bytes": (sz, [LP, i32, i32, i32, i32, i32]),
            "kvq_tree": (i32, [P, P, P, P, i32, P, P, P, i32, i32, i32, i32, ctypes.c_float, P, i32, P, sz, LP, i32, i32,
                               P]),
            "kvq_pages_workspace_bytes": (sz, [LP, i32, i32]),
            "kvq_pages_copy": (i32, [P, P, P, P, i32, LP, i32, P]),
            "kvq_pages_fork": (i32, [P, i32, P, i32, P, P, P, i32, P, P, P, sz, LP, P]),
            "kvq_pages_resize": (i32, [P, i32, P, i32, P, P, P, i32, P, sz, LP, P]),
            "kvq_pages_compact": (i32, [P, P, P, i32, P, P, P, i32, i32, P, P, P, sz, LP, i32, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().kvq_strerror(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise KvqError(status, where)


def _kind(kind) -> int:
    return KIND[kind] if isinstance(kind, str) else int(kind)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


@dataclass
class Layout:
    """Python view of ``kvq_layout``."""
    num_pages: int
    page_size: int
    num_kv_heads: int
    head_dim: int
    v_dim: int
    mla: bool = False

    def c(self) -> kvq_layout:
        return kvq_layout(self.num_pages, self.page_size, self.num_kv_heads, self.head_dim, self.v_dim,
                          int(bool(self.mla)))

    @property
    def n_kv(self) -> int:
        return 1 if self.mla else 2

    def codes_shape(self):
        return (self.num_pages, self.n_kv, self.num_kv_heads, self.page_size, self.head_dim)

    def scales_shape(self):
        return (self.num_pages, self.n_kv, self.num_kv_heads, self.page_size, self.head_dim // 32)


# ---------------------------------------------------------------------------- cost model
def kvq_pool_bytes(layout: Layout) -> int:
    return lib().kvq_pool_bytes(ctypes.byref(layout.c()))


def kvq_scale_bytes(layout: Layout) -> int:
    return lib().kvq_scale_bytes(ctypes.byref(layout.c()))


def kvq_bytes_per_token(layout: Layout) -> float:
    return lib().kvq_bytes_per_token(ctypes.byref(layout.c()))


def kvq_num_pages(layout: Layout, budget_bytes: int) -> int:
    return lib().kvq_num_pages(ctypes.byref(layout.c()), int(budget_bytes))


def kvq_bytes_per_token_ex(layout: Layout, kind) -> float:
    return lib().kvq_bytes_per_token_ex(ctypes.byref(layout.c()), _kind(kind))


def kvq_num_pages_ex(layout: Layout, kind, budget_bytes: int) -> int:
    return lib().kvq_num_pages_ex(ctypes.byref(layout.c()), _kind(kind), int(budget_bytes))


def alloc_pool(layout: Layout, device="cuda"):
    """(codes uint8, scales as int16 bit patterns) tensors of the pool's shapes on ``device``."""
    codes = torch.empty(layout.codes_shape(), dtype=torch.uint8, device=device)
    scales = torch.empty(layout.scales_shape(), dtype=torch.int16, device=device)
    return codes, scales


# ---------------------------------------------------------------------------- store
def kvq_store(pool: torch.Tensor, scales: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor],
              slot_mapping: torch.Tensor, layout: Layout, kind, stream=None):
    """Quantize rows ``k`` / ``v`` ([T, Hkv, D] bf16) and scatter them to ``slot_mapping`` ([T] int64)."""
    _check(lib().kvq_store(_ptr(pool), _ptr(scales), _ptr(k), _ptr(v), _ptr(slot_mapping), int(k.shape[0]),
                           ctypes.byref(layout.c()), _kind(kind), _stream(stream)), "kvq_store")


# ---------------------------------------------------------------------------- decode
def _opts(pages_per_split=0, path=0):
    return kvq_decode_options(int(pages_per_split), int(path))


def kvq_decode_workspace_bytes(layout: Layout, batch: int, num_q_heads: int, max_pages_per_seq: int,
                               pages_per_split=0, path=0) -> int:
    o = _opts(pages_per_split, path)
    return lib().kvq_decode_workspace_bytes_ex(ctypes.byref(layout.c()), int(batch), int(num_q_heads),
                                               int(max_pages_per_seq), ctypes.byref(o))


def kvq_decode_path(layout: Layout, batch: int, num_q_heads: int, max_pages_per_seq: int, pages_per_split=0,
                    path=0) -> int:
    """1 (CUDA cores, one launch) or 2 (tensor cores + merge, two launches); negative status if none."""
    o = _opts(pages_per_split, path)
    return lib().kvq_decode_path(ctypes.byref(layout.c()), int(batch), int(num_q_heads), int(max_pages_per_seq),
                                 ctypes.byref(o))


def alloc_workspace(layout: Layout, batch, num_q_heads, max_pages_per_seq, device="cuda", **opts):
    n = kvq_decode_workspace_bytes(layout, batch, num_q_heads, max_pages_per_seq, **opts)
    if n == 0:
        raise KvqError(-1, "kvq_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_decode(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, layout: Layout, kind,
               sm_scale: float = 1.0, pages_per_split: int = 0, path: int = 0, stream=None):
    """Decode attention; writes ``out`` ([B, Hq, v_dim], bf16 or float32)."""
    if out.dtype == torch.bfloat16:
        od = KVQ_OUT_BF16
    elif out.dtype == torch.float32:
        od = KVQ_OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    o = _opts(pages_per_split, path)
    _check(lib().kvq_decode_ex(_ptr(q), _ptr(pool), _ptr(scales), _ptr(block_table), int(block_table.shape[1]),
                               _ptr(seq_lens), int(seq_lens.shape[0]), int(q.shape[1]), float(sm_scale), _ptr(out),
                               od, _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                               ctypes.byref(layout.c()), _kind(kind), ctypes.byref(o), _stream(stream)),
           "kvq_decode")


def kvq_decode_noalloc(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, out: torch.Tensor, layout: Layout, kind, sm_scale: float = 1.0,
                       stream=None):
    """kvq_decode without a workspace argument, for callers that cannot allocate device memory.

    The split-K scratch is the library's fixed device array (KVQ_NOALLOC_SCRATCH_BYTES); calls that
    overlap on the GPU share it and race.
    """
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_decode_noalloc(_ptr(q), _ptr(pool), _ptr(scales), _ptr(block_table), int(block_table.shape[1]),
                                    _ptr(seq_lens), int(seq_lens.shape[0]), int(q.shape[1]), float(sm_scale),
                                    _ptr(out), od, ctypes.byref(layout.c()), _kind(kind), _stream(stream)),
           "kvq_decode_noalloc")


def alloc_sparse_workspace(layout: Layout, batch: int, num_q_heads: int, topk: int, device="cuda"):
    n = lib().kvq_decode_sparse_workspace_bytes(ctypes.byref(layout.c()), int(batch), int(num_q_heads), int(topk))
    if n == 0:
        raise KvqError(-1, "kvq_decode_sparse_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_decode_sparse(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, indices: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                      layout: Layout, kind, sm_scale: float = 1.0, stream=None):
    """Sparse (top-K) decode over the columns ``indices`` ([B, topk] int32, -1 = masked) selects."""
    if out.dtype == torch.bfloat16:
        od = KVQ_OUT_BF16
    elif out.dtype == torch.float32:
        od = KVQ_OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    B, Hq = q.shape[0], q.shape[1]
    topk = indices.shape[1] if indices.dim() == 2 else 0
    _check(lib().kvq_decode_sparse(_ptr(q), _ptr(pool), _ptr(scales), _ptr(block_table), int(block_table.shape[1]),
                                   _ptr(seq_lens), _ptr(indices), int(topk), int(B), int(Hq), float(sm_scale),
                                   _ptr(out), od, _ptr(workspace), int(workspace.numel() * workspace.element_size()),
                                   ctypes.byref(layout.c()),
                                   _kind(kind), _stream(stream)), "kvq_decode_sparse")


def kvq_store_unscaled(pool: torch.Tensor, k: torch.Tensor, v, slot_mapping: torch.Tensor, layout: Layout, kind,
                       stream=None):
    """Store into an unscaled fp8 pool (kind "fp8_e4m3_unscaled" or "fp8_e5m2_unscaled"): the plain cast."""
    _check(lib().kvq_store_unscaled(_ptr(pool), _ptr(k), None if v is None else _ptr(v), _ptr(slot_mapping),
                                    int(k.shape[0]), ctypes.byref(layout.c()), _kind(kind), _stream(stream)),
           "kvq_store_unscaled")


def kvq_store_act_quant(pool: torch.Tensor, scales: torch.Tensor, kv: torch.Tensor, slot_mapping: torch.Tensor,
                        layout: Layout, kind, rope_dim: int = 64, stream=None):
    """The MLA store fused with the model's per-64 E4M3 rounding of the latent: kv is bf16 [T, head_dim]."""
    _check(lib().kvq_store_act_quant(_ptr(pool), _ptr(scales), _ptr(kv), _ptr(slot_mapping), int(kv.shape[0]),
                                     int(rope_dim), ctypes.byref(layout.c()), _kind(kind), _stream(stream)),
           "kvq_store_act_quant")


def _extend_opts(path, precise_p=False):
    if path is None and not precise_p:
        return None
    return ctypes.byref(kvq_extend_options(int(path or 0), 1 if precise_p else 0))


def alloc_extend_workspace(device="cuda", layout: Optional[Layout] = None, total_q=0, num_q_heads=1,
                           max_pages_per_seq=1, path=None, precise_p=False):
    """The extend's workspace for these sizes and kernel choice (path None or 0: automatic; 1: each new
    token's prefix on the CUDA-core decode; 2: the flash kernel / the MLA tensor-core decode; precise_p: P
    carried to 16 bits or more).  Without a layout: the flash kernel's status word."""
    if layout is None:
        n = lib().kvq_extend_workspace_bytes()
    else:
        n = lib().kvq_extend_workspace_bytes_ex(ctypes.byref(layout.c()), int(total_q), int(num_q_heads),
                                                int(max_pages_per_seq), _extend_opts(path, precise_p))
        if n == 0:
            raise KvqError(-1, "kvq_extend_workspace_bytes_ex")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_extend_path(layout: Layout, total_q, num_q_heads, max_pages_per_seq, path=None, precise_p=False) -> int:
    """3 (flash kernel), 4 (flash, P as two bf16 terms), 1 or 2 (prefixes on the CUDA-core / tensor-core
    decode), or a negative status."""
    return lib().kvq_extend_path(ctypes.byref(layout.c()), int(total_q), int(num_q_heads), int(max_pages_per_seq),
                                 _extend_opts(path, precise_p))


def kvq_extend(q: torch.Tensor, pool: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
               seq_lens: torch.Tensor, q_start: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
               layout: Layout, kind, sm_scale: float = 1.0, stream=None, path=None, precise_p=False):
    """Extend (prefill) attention: the q rows q_start[b] .. q_start[b+1]-1 ([total_q, Hq, D] bf16) are the
    last new tokens of sequence b and attend causally over the pool; out is [total_q, Hq, Dv].  path None
    (and no precise_p) calls kvq_extend (automatic), else kvq_extend_ex with those options."""
    if out.dtype == torch.bfloat16:
        od = KVQ_OUT_BF16
    elif out.dtype == torch.float32:
        od = KVQ_OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    total_q, Hq = q.shape[0], q.shape[1]
    B = seq_lens.numel()
    args = (_ptr(q), _ptr(pool), _ptr(scales), _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
            _ptr(q_start), int(total_q), int(B), int(Hq), float(sm_scale), _ptr(out), od, _ptr(workspace),
            int(workspace.numel() * workspace.element_size()), ctypes.byref(layout.c()), _kind(kind))
    opts = _extend_opts(path, precise_p)
    if opts is None:
        _check(lib().kvq_extend(*args, _stream(stream)), "kvq_extend")
    else:
        _check(lib().kvq_extend_ex(*args, opts, _stream(stream)), "kvq_extend_ex")


# ---------------------------------------------------------------------------- checked marshalling
# The calls below belong to loops of short GPU work, so what they marshal is checked and passed as plain
# integers, and a layout's C struct is built once.
_I32, _I64, _U8, _BF16 = torch.int32, torch.int64, torch.uint8, torch.bfloat16
_layouts: dict = {}


def _layout_info(L: Layout):
    """(pointer to the C struct, code bytes, scales) of a layout."""
    key = (L.num_pages, L.page_size, L.num_kv_heads, L.head_dim, L.v_dim, L.mla)
    info = _layouts.get(key)
    if info is None:
        if len(_layouts) >= 1024:
            _layouts.clear()
        info = _layouts[key] = (ctypes.byref(L.c()), math.prod(L.codes_shape()), math.prod(L.scales_shape()))
    return info


def _check_args(names, types, *tensors):
    """The tensors (named, of these types) must be dense and on the current CUDA device, whose index is returned."""
    device = tensors[0].get_device()
    for t, dtype in zip(tensors, types):
        if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device:
            break
    else:
        if device >= 0 and device == torch.cuda.current_device():
            return device
    for name, t, dtype in zip(names, tensors, types):
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    raise ValueError("every tensor must be on the current CUDA device, got " +
                     ", ".join("%s on %s" % (name, t.device) for name, t in zip(names, tensors)))


def _raw_stream(stream, device):
    if stream is None:  # (torch.cuda.current_stream() builds an object, 3 us)
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _check_pool(pool, scales, info, kind, device):
    """The kind's number and the scales' address (None for the unscaled kinds); pool and scales must hold the layout's
    pages."""
    k = _kind(kind)
    if pool.dtype is not _U8:
        raise TypeError("pool must be torch.uint8, got %s" % pool.dtype)
    if pool.numel() < info[1] or not pool.is_contiguous():
        raise ValueError("pool must be contiguous and hold the layout's %d codes" % info[1])
    if k == KVQ_FP8_E4M3 or k == KVQ_Q8_0:
        if scales is None or scales.numel() < info[2] or scales.dtype.itemsize != 2 or not scales.is_contiguous():
            raise ValueError("scales must be contiguous and hold the layout's %d scales of 16 bits" % info[2])
        if scales.get_device() != device:
            raise ValueError("scales is on %s, not on the current CUDA device" % scales.device)
    else:
        scales = None
    if pool.get_device() != device:
        raise ValueError("pool is on %s, not on the current CUDA device" % pool.device)
    return k, None if scales is None else scales.data_ptr()


def _out_dtype(out):
    if out.dtype is torch.bfloat16:
        return KVQ_OUT_BF16
    if out.dtype is torch.float32:
        return KVQ_OUT_F32
    raise TypeError("out must be bfloat16 or float32")


# ---------------------------------------------------------------------------- whole prompts
def alloc_prompt_workspace(device="cuda"):
    return torch.empty(lib().kvq_prompt_workspace_bytes(), dtype=torch.uint8, device=device)


def kvq_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_start: torch.Tensor, out: torch.Tensor,
               workspace: torch.Tensor, sm_scale: float = 1.0, stream=None):
    """Causal attention over packed prompts: rows q_start[b] .. q_start[b+1]-1 of q ([total, Hq, D] bf16) and k / v
    ([total, Hkv, D] bf16) are sequence b.  Writes out ([total, Hq, D], bf16 or float32).  q, k, v and out may be
    strided between tokens and heads (slices of one projection)."""
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [total, Hq, D], k and v [total, Hkv, D]")
    if out.shape != q.shape or q_start.numel() < 1:
        raise ValueError("out must have q's shape and q_start batch + 1 entries")
    od = _out_dtype(out)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        st = [t.stride() for t in (q, k, v, out)]
        if q.shape[2] > 1 and any(s[2] != 1 for s in st):
            raise ValueError("the last dimension of q, k, v and out must be dense")
        strides = ctypes.byref(kvq_prompt_strides(*[x for s in st for x in s[:2]]))
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype is not _BF16:
            raise TypeError("%s must be %s, got %s" % (name, _BF16, t.dtype))
    device = _check_args(("q_start", "workspace"), (_I32, _U8), q_start, workspace)
    if not (q.get_device() == k.get_device() == v.get_device() == out.get_device() == device):
        raise ValueError("every tensor must be on the current CUDA device")
    status = lib().kvq_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_start.data_ptr(), q.shape[0],
                              q_start.numel() - 1, q.shape[1], k.shape[1], q.shape[2], sm_scale, out.data_ptr(), od,
                              strides, workspace.data_ptr(), workspace.numel(), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_prompt")


# ---------------------------------------------------------------------------- drafted tokens
_TREE_NAMES = ("q", "block_table", "seq_lens", "q_start", "tree_mask", "out", "workspace")


def alloc_tree_workspace(layout: Layout, batch: int, total_q: int, num_q_heads: int, max_pages_per_seq: int,
                         path: int = 0, device="cuda"):
    n = lib().kvq_tree_workspace_bytes(ctypes.byref(layout.c()), int(batch), int(total_q), int(num_q_heads),
                                       int(max_pages_per_seq), int(path))
    if n == 0:
        raise KvqError(-1, "kvq_tree_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_tree(q: torch.Tensor, pool: torch.Tensor, scales: Optional[torch.Tensor], block_table: torch.Tensor,
             seq_lens: torch.Tensor, q_start: torch.Tensor, tree_mask: torch.Tensor, out: torch.Tensor,
             workspace: torch.Tensor, layout: Layout, kind, sm_scale: float = 1.0, path: int = 0, stream=None):
    """Attention of drafted tokens: the q rows q_start[b] .. q_start[b+1]-1 ([total_q, Hq, D] bf16) are the last
    stored tokens of sequence b; each sees the tokens before them and the drafted ones in its row of tree_mask
    ([total_q, words] int64).  Writes out ([total_q, Hq, v_dim], bf16 or float32).  path: 0 automatic, 1 CUDA cores
    with P in fp32, 2 tensor cores."""
    B = seq_lens.numel()
    if q.dim() != 3 or q.shape[2] != layout.head_dim or out.shape != (q.shape[0], q.shape[1], layout.v_dim):
        raise ValueError("q must be [total_q, heads, head_dim] and out [total_q, heads, v_dim]")
    if tree_mask.dim() != 2 or tree_mask.shape[0] != q.shape[0] or q_start.numel() != B + 1:
        raise ValueError("tree_mask must be [total_q, words] and q_start [batch + 1]")
    _check_tables(block_table, seq_lens, None, layout)
    od = _out_dtype(out)
    info = _layout_info(layout)
    device = _check_args(_TREE_NAMES, (_BF16, _I32, _I32, _I32, _I64, out.dtype, _U8), q, block_table, seq_lens, q_start,
                         tree_mask, out, workspace)
    k, sc = _check_pool(pool, scales, info, kind, device)
    st = lib().kvq_tree(q.data_ptr(), pool.data_ptr(), sc,
                        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), q_start.data_ptr(),
                        tree_mask.data_ptr(), tree_mask.shape[1], q.shape[0], B, q.shape[1], sm_scale, out.data_ptr(), od,
                        workspace.data_ptr(), workspace.numel(), info[0], k, path,
                        _raw_stream(stream, device))
    if st:
        raise KvqError(st, "kvq_tree")


# ---------------------------------------------------------------------------- pages
_FORK_NAMES = ("block_table", "seq_lens", "page_refs", "src", "dst", "copy_src", "copy_dst", "workspace")
_FORK_TYPES = (_I32,) * 7 + (_U8,)
_RESIZE_NAMES = ("block_table", "seq_lens", "page_refs", "seqs", "new_lens", "workspace")
_RESIZE_TYPES = (_I32,) * 5 + (_U8,)
_COMPACT_NAMES = ("block_table", "seq_lens", "q_start", "keep", "new_lens", "workspace", "page_refs")
_COMPACT_TYPES = (_I32, _I32, _I32, _I64, _I32, _U8, _I32)


def alloc_pages_workspace(layout: Layout, n: int, max_pages_per_seq: int, device="cuda"):
    """Workspace of kvq_pages_fork and kvq_pages_resize for n list entries (kvq_pages_compact takes it too)."""
    b = lib().kvq_pages_workspace_bytes(ctypes.byref(layout.c()), int(n), int(max_pages_per_seq))
    if b == 0:
        raise KvqError(-1, "kvq_pages_workspace_bytes")
    return torch.empty(b, dtype=torch.uint8, device=device)


def kvq_pages_copy(pool: torch.Tensor, scales: Optional[torch.Tensor], src: torch.Tensor, dst: torch.Tensor,
                   layout: Layout, kind, stream=None):
    """Page dst[i] of the pool becomes a copy of page src[i] (int32 lists; pairs with -1 are skipped)."""
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst must have one entry per copy")
    info = _layout_info(layout)
    device = _check_args(("src", "dst"), (_I32, _I32), src, dst)
    k, sc = _check_pool(pool, scales, info, kind, device)
    st = lib().kvq_pages_copy(pool.data_ptr(), sc, src.data_ptr(), dst.data_ptr(), n, info[0], k,
                              _raw_stream(stream, device))
    if st:
        raise KvqError(st, "kvq_pages_copy")


def _check_tables(block_table, seq_lens, page_refs, layout: Layout):
    if block_table.dim() != 2 or seq_lens.numel() != block_table.shape[0]:
        raise ValueError("block_table must be [batch, max_pages] and seq_lens [batch]")
    if page_refs is not None and page_refs.numel() < layout.num_pages:
        raise ValueError("page_refs needs one count per page")


def kvq_pages_fork(block_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor, src: torch.Tensor,
                   dst: torch.Tensor, copy_src: torch.Tensor, copy_dst: torch.Tensor, workspace: torch.Tensor,
                   layout: Layout, stream=None):
    """Rows dst continue rows src (int32 lists, parents read as before the call); the copies of partly filled
    last pages that kvq_pages_copy must then make in every layer are written to copy_src / copy_dst."""
    n = src.numel()
    if dst.numel() != n or copy_src.numel() != n or copy_dst.numel() != n:
        raise ValueError("src, dst, copy_src and copy_dst must have the same length")
    _check_tables(block_table, seq_lens, page_refs, layout)
    device = _check_args(_FORK_NAMES, _FORK_TYPES, block_table, seq_lens, page_refs, src, dst, copy_src, copy_dst,
                         workspace)
    batch, max_pages = block_table.shape
    st = lib().kvq_pages_fork(block_table.data_ptr(), max_pages, seq_lens.data_ptr(), batch, page_refs.data_ptr(),
                              src.data_ptr(), dst.data_ptr(), n, copy_src.data_ptr(), copy_dst.data_ptr(),
                              workspace.data_ptr(), workspace.numel(), _layout_info(layout)[0], _raw_stream(stream, device))
    if st:
        raise KvqError(st, "kvq_pages_fork")


def kvq_pages_resize(block_table: torch.Tensor, seq_lens: torch.Tensor, page_refs: torch.Tensor, seqs: torch.Tensor,
                     new_lens: torch.Tensor, workspace: torch.Tensor, layout: Layout, stream=None):
    """Rows seqs get room for new_lens tokens (int32 lists): pages are taken or released; 0 frees a row."""
    n = seqs.numel()
    if new_lens.numel() != n:
        raise ValueError("seqs and new_lens must have the same length")
    _check_tables(block_table, seq_lens, page_refs, layout)
    device = _check_args(_RESIZE_NAMES, _RESIZE_TYPES, block_table, seq_lens, page_refs, seqs, new_lens, workspace)
    batch, max_pages = block_table.shape
    st = lib().kvq_pages_resize(block_table.data_ptr(), max_pages, seq_lens.data_ptr(), batch, page_refs.data_ptr(),
                                seqs.data_ptr(), new_lens.data_ptr(), n, workspace.data_ptr(), workspace.numel(),
                                _layout_info(layout)[0], _raw_stream(stream, device))
    if st:
        raise KvqError(st, "kvq_pages_resize")


def kvq_pages_compact(pool: torch.Tensor, scales: Optional[torch.Tensor], block_table: torch.Tensor,
                      seq_lens: torch.Tensor, q_start: torch.Tensor, keep: torch.Tensor, new_lens: torch.Tensor,
                      workspace: torch.Tensor, layout: Layout, kind, page_refs: Optional[torch.Tensor] = None,
                      stream=None):
    """Of the last q_start[b+1] - q_start[b] tokens of sequence b, those whose bit is set in keep ([B, words]
    int64) move together; new_lens ([B] int32) receives the tokens that remain."""
    B = seq_lens.numel()
    if keep.dim() != 2 or keep.shape[0] != B or q_start.numel() != B + 1 or new_lens.numel() != B:
        raise ValueError("keep must be [batch, words], q_start [batch + 1] and new_lens [batch]")
    _check_tables(block_table, seq_lens, page_refs, layout)
    info = _layout_info(layout)
    device = _check_args(_COMPACT_NAMES, _COMPACT_TYPES, block_table, seq_lens, q_start, keep, new_lens, workspace,
                         *(() if page_refs is None else (page_refs,)))
    k, sc = _check_pool(pool, scales, info, kind, device)
    st = lib().kvq_pages_compact(pool.data_ptr(), sc, block_table.data_ptr(),
                                 block_table.shape[1], seq_lens.data_ptr(), q_start.data_ptr(), keep.data_ptr(),
                                 keep.shape[1], B, new_lens.data_ptr(),
                                 None if page_refs is None else page_refs.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), info[0], k, _raw_stream(stream, device))
    if st:
        raise KvqError(st, "kvq_pages_compact")


def kvq_workspace_status(workspace: torch.Tensor, stream=None) -> int:
    return lib().kvq_workspace_status(_ptr(workspace), _stream(stream))


def kvq_noalloc_status(stream=None) -> int:
    """Status word the last kvq_decode_noalloc left in the library's scratch (0 = KVQ_OK)."""
    return lib().kvq_noalloc_status(_stream(stream))


# ---------------------------------------------------------------------------- probes
def kvq_encode_probe(kind, y: torch.Tensor, codes: torch.Tensor, stream=None):
    _check(lib().kvq_encode_probe(_kind(kind), _ptr(y), _ptr(codes), int(y.numel()), _stream(stream)),
           "kvq_encode_probe")


def kvq_quantize_probe(kind, x_bits: torch.Tensor, s_bits: torch.Tensor, codes: torch.Tensor, stream=None):
    """codes[i * nx + j] = the store's code of bf16 x[j] against nonzero fp16 scale s[i]."""
    _check(lib().kvq_quantize_probe(_kind(kind), _ptr(x_bits), int(x_bits.numel()), _ptr(s_bits), int(s_bits.numel()),
                                    _ptr(codes), _stream(stream)), "kvq_quantize_probe")


def kvq_dequant_probe(kind, codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor, stream=None):
    _check(lib().kvq_dequant_probe(_kind(kind), _ptr(codes), _ptr(scales), _ptr(out), int(codes.numel()),
                                   _stream(stream)), "kvq_dequant_probe")


def kvq_exp2_probe(x: torch.Tensor, y: torch.Tensor, stream=None):
    """y = 2^x by the extend kernel's FMA-pipe exponential (float32 device tensors of equal size)."""
    _check(lib().kvq_exp2_probe(_ptr(x), _ptr(y), int(x.numel()), _stream(stream)), "kvq_exp2_probe")


def kvq_wait_probe(workspace: torch.Tensor, stream=None):
    """One bounded wait that never completes: afterwards kvq_workspace_status(workspace) is KVQ_ETIMEOUT."""
    _check(lib().kvq_wait_probe(_ptr(workspace), _stream(stream)), "kvq_wait_probe")


def kvq_device_check() -> int:
    return lib().kvq_device_check()


def kvq_version() -> str:
    return lib().kvq_version().decode()

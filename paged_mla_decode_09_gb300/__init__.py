"""Paged MLA decode for GB300: Python binding of the C ABI in include/mla_decode.h,
include/mla_kv_pack.h, include/mla_sparse.h, include/mla_cascade.h,
include/mla_prefill.h, include/mla_evict.h, include/mla_tree.h,
include/mla_verify.h, include/mla_pages.h and include/mla_rope.h.

The functions here only marshal arguments (torch tensors -> device
pointers, shapes -> ``mla_dims``), those of a speculative step through a
compiled module (csrc/binding.cpp); every step of the decode runs in the
CUDA library.  There is no CPU fallback: if the library is missing or the
device is not sm_103a, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from .build import LIB_PATH, binding_path, build_library

MLA_OK = 0
MLA_KV_BF16 = 0
MLA_KV_FP8_E4M3 = 1
MLA_DEV_BAD_PAGE_ID = 1
MLA_DEV_BAD_SEQ_LEN = 2
MLA_DEV_TIMEOUT = 4
MLA_DEV_INTERNAL = 8
MLA_DEV_BAD_INDEX = 16
MLA_DEV_BAD_PREFIX = 32
MLA_DEV_BAD_QUERY_RANGE = 64
MLA_DEV_BAD_TREE = 128
MLA_DEV_BAD_PROBS = 256
MLA_DEV_NO_PAGES = 512
MLA_DEV_BAD_REFS = 1024
MLA_TREE_MAX_NODES = 256

ENTRY_POINTS = (
    "mla_decode_workspace_size",
    "mla_decode",
    "mla_decode_profiled",
    "mla_query_status",
    "mla_gather_rows",
    "mla_selftest_wait_timeout",
    "mla_status_string",
    "mla_decode_launch_shape",
    "mla_decode_noalloc",
    "mla_kv_pack",
    "mla_decode_sparse_workspace_size",
    "mla_decode_sparse",
    "mla_decode_sparse_query_status",
    "mla_decode_cascade_workspace_size",
    "mla_decode_cascade",
    "mla_decode_cascade_query_status",
    "mla_prefill_workspace_size",
    "mla_prefill",
    "mla_decode_window_workspace_size",
    "mla_decode_window",
    "mla_attn_mass_workspace_size",
    "mla_attn_mass",
    "mla_evict_workspace_size",
    "mla_evict",
    "mla_decode_tree_workspace_size",
    "mla_decode_tree",
    "mla_tree_commit",
    "mla_verify",
    "mla_page_resize_workspace_size",
    "mla_page_resize",
    "mla_page_fork_workspace_size",
    "mla_page_fork",
    "mla_rope_frequencies",
    "mla_rope_frequencies_by_index",
    "mla_rope_plan_init",
    "mla_rope_pack",
)


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


class MlaDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class MlaKvPackDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_new", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class MlaPrefillDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
    ]


class MlaEvictDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("mass_cols", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("budget", ctypes.c_int32),
        ("num_sinks", ctypes.c_int32),
        ("num_recent", ctypes.c_int32),
    ]


class MlaTreeCommitDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_layers", ctypes.c_int32),
        ("path_cols", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("layer_stride", ctypes.c_int64),
    ]


class MlaVerifyDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("vocab", ctypes.c_int32),
        ("path_cols", ctypes.c_int32),
        ("target_stride", ctypes.c_int64),
        ("draft_stride", ctypes.c_int64),
    ]


class MlaPageResizeDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("table_stride", ctypes.c_int32),
        ("out_stride", ctypes.c_int32),
    ]


class MlaPageForkDims(ctypes.Structure):
    _fields_ = [
        ("sources", ctypes.c_int32),
        ("children", ctypes.c_int32),
        ("num_layers", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("table_stride", ctypes.c_int32),
        ("out_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("layer_stride", ctypes.c_int64),
    ]


class MlaRopePlan(ctypes.Structure):
    _fields_ = [
        ("turn", ctypes.c_uint64 * 32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("amplitude", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class MlaRopeDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("total_q", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages_per_req", ctypes.c_int32),
        ("page_table_stride", ctypes.c_int32),
        ("kv_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
    ]


_lib = None


def load_library(path: str | None = None, build: bool = False) -> ctypes.CDLL:
    """Load (optionally building first) the CUDA library; raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if build:
        build_library()
    if not os.path.exists(p):
        raise RuntimeError(
            f"CUDA library {p} is missing: build it with __graft_entry__.build() or "
            "`python -m paged_mla_decode_09_gb300.build` (there is no CPU fallback)"
        )
    lib = ctypes.CDLL(p)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(MlaDims)
    lib.mla_decode_workspace_size.argtypes = [D, ctypes.c_int]
    lib.mla_decode_workspace_size.restype = SZ
    dec_args = [D, P, P, P, P, P, I32, ctypes.c_float, ctypes.c_float, P, P, P, SZ, P]
    lib.mla_decode.argtypes = dec_args
    lib.mla_decode.restype = ctypes.c_int
    lib.mla_decode_profiled.argtypes = dec_args + [ctypes.POINTER(P)]
    lib.mla_decode_profiled.restype = ctypes.c_int
    lib.mla_query_status.argtypes = [P, P, ctypes.POINTER(I32)]
    lib.mla_query_status.restype = ctypes.c_int
    lib.mla_gather_rows.argtypes = [D, P, P, P, P, P, P, P]
    lib.mla_gather_rows.restype = ctypes.c_int
    lib.mla_selftest_wait_timeout.argtypes = [P, ctypes.c_uint32, P]
    lib.mla_selftest_wait_timeout.restype = ctypes.c_int
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_decode_launch_shape.argtypes = [D, ctypes.c_int, ctypes.POINTER(I32), ctypes.POINTER(I32)]
    lib.mla_decode_launch_shape.restype = ctypes.c_int
    lib.mla_decode_noalloc.argtypes = [D, P, P, P, P, P, I32, ctypes.c_float, ctypes.c_float, P, P, P, P]
    lib.mla_decode_noalloc.restype = ctypes.c_int
    lib.mla_kv_pack.argtypes = [ctypes.POINTER(MlaKvPackDims), P, P, P, ctypes.c_float, P, P, P]
    lib.mla_kv_pack.restype = ctypes.c_int
    lib.mla_decode_sparse_workspace_size.argtypes = [D, I32, ctypes.c_int]
    lib.mla_decode_sparse_workspace_size.restype = SZ
    lib.mla_decode_sparse.argtypes = [D, P, P, P, P, P, P, I32, I32, ctypes.c_float, ctypes.c_float, P, P, P, SZ, P]
    lib.mla_decode_sparse.restype = ctypes.c_int
    lib.mla_decode_sparse_query_status.argtypes = [D, I32, P, P, ctypes.POINTER(I32)]
    lib.mla_decode_sparse_query_status.restype = ctypes.c_int
    lib.mla_decode_cascade_workspace_size.argtypes = [D, I32, ctypes.c_int]
    lib.mla_decode_cascade_workspace_size.restype = SZ
    lib.mla_decode_cascade.argtypes = [D, P, P, P, P, P, I32, I32, ctypes.c_float, ctypes.c_float, P, P, P, SZ, P]
    lib.mla_decode_cascade.restype = ctypes.c_int
    lib.mla_decode_cascade_query_status.argtypes = [D, I32, P, P, ctypes.POINTER(I32)]
    lib.mla_decode_cascade_query_status.restype = ctypes.c_int
    PD = ctypes.POINTER(MlaPrefillDims)
    F = ctypes.c_float
    lib.mla_prefill_workspace_size.argtypes = [PD, ctypes.c_int]
    lib.mla_prefill_workspace_size.restype = SZ
    lib.mla_prefill.argtypes = [PD, P, P, P, P, P, P, I32, I32, F, F, P, P, P, SZ, P]
    lib.mla_prefill.restype = ctypes.c_int
    lib.mla_decode_window_workspace_size.argtypes = [D, ctypes.c_int]
    lib.mla_decode_window_workspace_size.restype = SZ
    lib.mla_decode_window.argtypes = [D, P, P, P, P, P, I32, I32, F, F, P, P, P, SZ, P]
    lib.mla_decode_window.restype = ctypes.c_int
    lib.mla_attn_mass_workspace_size.argtypes = [D, ctypes.c_int]
    lib.mla_attn_mass_workspace_size.restype = SZ
    lib.mla_attn_mass.argtypes = [D, P, P, P, P, P, P, I32, F, F, P, P, I32, P, SZ, P]
    lib.mla_attn_mass.restype = ctypes.c_int
    lib.mla_evict_workspace_size.argtypes = [I32, I32]
    lib.mla_evict_workspace_size.restype = SZ
    lib.mla_evict.argtypes = [ctypes.POINTER(MlaEvictDims), P, P, P, P, P, P, P, P, P, P, SZ, P]
    lib.mla_evict.restype = ctypes.c_int
    lib.mla_decode_tree_workspace_size.argtypes = [PD, ctypes.c_int]
    lib.mla_decode_tree_workspace_size.restype = SZ
    lib.mla_decode_tree.argtypes = [PD, P, P, P, P, P, P, P, F, F, P, P, P, SZ, P]
    lib.mla_decode_tree.restype = ctypes.c_int
    lib.mla_tree_commit.argtypes = [ctypes.POINTER(MlaTreeCommitDims), P, P, P, P, P, P, P, P, P]
    lib.mla_tree_commit.restype = ctypes.c_int
    lib.mla_verify.argtypes = [ctypes.POINTER(MlaVerifyDims), P, P, P, P, P, P, P, P, P, P, P, P]
    lib.mla_verify.restype = ctypes.c_int
    lib.mla_page_resize_workspace_size.argtypes = [I32, I32, I32]
    lib.mla_page_resize_workspace_size.restype = SZ
    lib.mla_page_resize.argtypes = [ctypes.POINTER(MlaPageResizeDims), P, P, P, P, P, P, SZ, P]
    lib.mla_page_resize.restype = ctypes.c_int
    lib.mla_page_fork_workspace_size.argtypes = [I32, I32, I32, I32]
    lib.mla_page_fork_workspace_size.restype = SZ
    lib.mla_page_fork.argtypes = [ctypes.POINTER(MlaPageForkDims), P, P, P, P, P, P, P, P, SZ, P]
    lib.mla_page_fork.restype = ctypes.c_int
    DP, R = ctypes.POINTER(ctypes.c_double), ctypes.POINTER(MlaRopePlan)
    for f in (lib.mla_rope_frequencies, lib.mla_rope_frequencies_by_index):
        f.argtypes = [I32, ctypes.c_double, ctypes.c_double, I32, ctypes.c_double, ctypes.c_double, DP]
        f.restype = ctypes.c_int
    lib.mla_rope_plan_init.argtypes = [I32, I32, F, DP, R]
    lib.mla_rope_plan_init.restype = ctypes.c_int
    lib.mla_rope_pack.argtypes = [ctypes.POINTER(MlaRopeDims), R, P, P, P, P, P, P, F, P, P, P, P]
    lib.mla_rope_pack.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


_fast = None


def _binding():
    """The compiled fast path of the calls of a speculative step
    (csrc/binding.cpp): each of its functions makes the C call, or returns
    None where a tensor is not what the call takes."""
    global _fast
    if _fast is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries are loaded first)

        load_library()
        path = binding_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path}, the binding for this Python and torch, is missing: build it with "
                               "__graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_binding", loader))
        loader.exec_module(module)
        _fast = module
    return _fast


def _refuse(call, explain, device, *tensors):
    """The binding found a tensor that the call does not take: say which."""
    explain(*tensors)
    _check_current_device(device)
    raise ValueError(f"{call}: the arguments do not have the shapes, types and layouts the library expects")


def status_string(code: int) -> str:
    try:
        return load_library().mla_status_string(int(code)).decode()
    except RuntimeError:
        return "library not loaded"


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def kv_dtype_code(kv_cache) -> int:
    import torch

    if kv_cache.dtype == torch.bfloat16:
        return MLA_KV_BF16
    if kv_cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MLA_KV_FP8_E4M3
    raise TypeError(f"unsupported cache dtype {kv_cache.dtype}")


def make_dims(q_nope, kv_cache, page_table) -> MlaDims:
    B, Q, H, _ = q_nope.shape
    return MlaDims(
        batch=B,
        num_heads=H,
        q_len=Q,
        page_size=int(kv_cache.shape[1]),
        num_pages=int(kv_cache.shape[0]),
        max_pages_per_req=int(page_table.shape[1]),
        page_table_stride=int(page_table.stride(0)),
        kv_dtype=kv_dtype_code(kv_cache),
    )


def mla_decode_workspace_size(dims: MlaDims, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_decode_workspace_size(ctypes.byref(dims), dev)
    if n == 0:
        raise MlaError(-1, "mla_decode_workspace_size")
    return int(n)


def mla_decode_launch_shape(dims: MlaDims, device: int | None = None):
    import torch

    dev = torch.cuda.current_device() if device is None else device
    c, s = ctypes.c_int32(), ctypes.c_int32()
    rc = load_library().mla_decode_launch_shape(ctypes.byref(dims), dev, ctypes.byref(c), ctypes.byref(s))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_launch_shape")
    return c.value, s.value


def _check_cuda(*tensors):
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (the decode runs only on the GPU)")


def _check_layout(name, t, shape, dtypes):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_cache_and_table(kv_cache, page_table, seq_lens, B):
    import torch

    if kv_cache.dim() != 3 or kv_cache.shape[2] != 576 or not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be a contiguous [num_pages, page_size, 576] tensor")
    kv_dtype_code(kv_cache)  # raises for other element types
    if (page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B
            or page_table.stride(1) != 1 or page_table.stride(0) < page_table.shape[1]):
        raise ValueError("page_table must be an int32 [B, max_pages] tensor with unit column stride")
    _check_layout("seq_lens", seq_lens, (B,), (torch.int32,))


def _check_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace):
    """The shapes, element types and layouts the C ABI assumes.  It receives
    bare pointers, so a tensor that does not match (a broadcast view, another
    dtype, a transposed copy) would be read or written with the wrong extent.
    One combined test on the fast path (it runs on every call); the detailed
    checks below name what is wrong."""
    import torch

    bf16, i32 = torch.bfloat16, torch.int32
    s = q_nope.shape
    if len(s) == 4:
        B, Q, H = s[0], s[1], s[2]
        dev = q_nope.get_device()
        if (s[3] == 512 and q_nope.dtype is bf16 and q_nope.is_contiguous()
                and q_pe.dtype is bf16 and q_pe.shape == (B, Q, H, 64) and q_pe.is_contiguous()
                and out.dtype is bf16 and out.shape == s and out.is_contiguous()
                and lse.dtype is torch.float32 and lse.shape == (B, Q, H) and lse.is_contiguous()
                and seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
                and page_table.dtype is i32 and page_table.dim() == 2 and page_table.shape[0] == B
                and page_table.stride(1) == 1 and page_table.stride(0) >= page_table.shape[1]
                and kv_cache.dim() == 3 and kv_cache.shape[2] == 576 and kv_cache.is_contiguous()
                and kv_cache.dtype in (bf16, torch.uint8, torch.float8_e4m3fn) and workspace.is_contiguous()
                and q_pe.get_device() == dev and out.get_device() == dev and lse.get_device() == dev
                and seq_lens.get_device() == dev and page_table.get_device() == dev
                and kv_cache.get_device() == dev and workspace.get_device() == dev):
            return
    _explain_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    raise ValueError("decode tensors do not have the shapes, types and layouts the library expects")


def _explain_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace):
    import torch

    if q_nope.dim() != 4 or q_nope.shape[3] != 512:
        raise ValueError(f"q_nope must be [B, q_len, H, 512], got {list(q_nope.shape)}")
    B, Q, H, _ = q_nope.shape
    _check_layout("q_nope", q_nope, (B, Q, H, 512), (torch.bfloat16,))
    _check_layout("q_pe", q_pe, (B, Q, H, 64), (torch.bfloat16,))
    _check_layout("out", out, (B, Q, H, 512), (torch.bfloat16,))
    _check_layout("lse", lse, (B, Q, H), (torch.float32,))
    _check_cache_and_table(kv_cache, page_table, seq_lens, B)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    for t in (q_pe, kv_cache, page_table, seq_lens, out, lse, workspace):
        if t.device != q_nope.device:
            raise ValueError("all tensors must be on one device")


def mla_decode(q_nope, q_pe, kv_cache, page_table, seq_lens, q_len, scale, kv_scale, out, lse, workspace,
               stream=None, events=None) -> None:
    """Enqueue one decode step (see include/mla_decode.h).  Raises MlaError on a host-side error.

    ``events``: optional 4 torch.cuda.Event objects (already recorded once)
    to time the schedule / attention / combine launches.
    """
    _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    _check_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    if int(q_len) != q_nope.shape[1]:
        raise ValueError(f"q_len {q_len} does not match q_nope's second dimension {q_nope.shape[1]}")
    dims = make_dims(q_nope, kv_cache, page_table)
    lib = load_library()
    args = [ctypes.byref(dims), _ptr(q_nope), _ptr(q_pe), _ptr(kv_cache), _ptr(page_table), _ptr(seq_lens),
            int(q_len), float(scale), float(kv_scale), _ptr(out), _ptr(lse), _ptr(workspace),
            ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream_handle(stream)]
    if events is None:
        rc = lib.mla_decode(*args)
    else:
        arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in events])
        rc = lib.mla_decode_profiled(*args, arr)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode")


def mla_query_status(workspace, stream=None) -> int:
    st = ctypes.c_int32(0)
    rc = load_library().mla_query_status(_ptr(workspace), _stream_handle(stream), ctypes.byref(st))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_query_status")
    return st.value


def timeout_diagnostics(workspace) -> dict:
    """Words 0..3 of the workspace: status bits and, after a device timeout,
    which wait gave up (tag, page counter, cluster, rank, warp)."""
    import torch

    w = workspace[:16].view(torch.int32).cpu().tolist()
    return {"status": w[0], "wait_tag": w[1], "page_counter": w[2], "cluster": w[3] >> 16,
            "rank": (w[3] >> 8) & 0xFF, "warp": w[3] & 0xFF}


def mla_gather_rows(kv_cache, page_table, seq_lens, row_offsets, rows_out, workspace, q_len: int = 1,
                    stream=None) -> None:
    _check_cuda(kv_cache, page_table, seq_lens, row_offsets, rows_out, workspace)
    dims = MlaDims(batch=int(seq_lens.shape[0]), num_heads=1, q_len=q_len, page_size=int(kv_cache.shape[1]),
                   num_pages=int(kv_cache.shape[0]), max_pages_per_req=int(page_table.shape[1]),
                   page_table_stride=int(page_table.stride(0)), kv_dtype=kv_dtype_code(kv_cache))
    rc = load_library().mla_gather_rows(ctypes.byref(dims), _ptr(kv_cache), _ptr(page_table), _ptr(seq_lens),
                                        _ptr(row_offsets), _ptr(rows_out), _ptr(workspace), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_gather_rows")


def mla_selftest_wait_timeout(workspace, timeout_us: int, stream=None) -> None:
    rc = load_library().mla_selftest_wait_timeout(_ptr(workspace), int(timeout_us), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_selftest_wait_timeout")


def _check_kv_pack_tensors(rows, page_table, seq_lens, kv_cache, status):
    import torch

    if rows.dim() != 3 or rows.shape[2] != 576 or not rows.is_contiguous() or rows.dtype != torch.bfloat16:
        raise ValueError("rows must be a contiguous bf16 [B, num_new, 576] tensor")
    _check_cache_and_table(kv_cache, page_table, seq_lens, rows.shape[0])
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor of at least one element")
    for t in (page_table, seq_lens, kv_cache, status):
        if t.device != rows.device:
            raise ValueError("all tensors must be on one device")


def mla_kv_pack(rows, page_table, seq_lens, kv_scale, kv_cache, status, stream=None) -> None:
    """Enqueue the cache write of a step's new rows (see include/mla_kv_pack.h).

    rows: bf16 [B, num_new, 576]; kv_cache: bf16 or uint8 (e4m3 codes)
    [num_pages, 64, 576]; status: int32 [1] on the device (flags OR-ed in).
    Raises MlaError on a host-side error.
    """
    _check_cuda(rows, page_table, seq_lens, kv_cache, status)
    _check_kv_pack_tensors(rows, page_table, seq_lens, kv_cache, status)
    B, N, _ = rows.shape
    dims = MlaKvPackDims(batch=B, num_new=N, num_pages=int(kv_cache.shape[0]),
                         max_pages_per_req=int(page_table.shape[1]), page_table_stride=int(page_table.stride(0)),
                         kv_dtype=kv_dtype_code(kv_cache))
    rc = load_library().mla_kv_pack(ctypes.byref(dims), _ptr(rows), _ptr(page_table), _ptr(seq_lens),
                                    float(kv_scale), _ptr(kv_cache), _ptr(status), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_kv_pack")


def mla_decode_sparse_workspace_size(dims: MlaDims, topk: int, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_decode_sparse_workspace_size(ctypes.byref(dims), int(topk), dev)
    if n == 0:
        raise MlaError(-1, "mla_decode_sparse_workspace_size")
    return int(n)


def _check_indices(indices, q_nope):
    import torch

    if (indices.dim() != 3 or tuple(indices.shape[:2]) != tuple(q_nope.shape[:2]) or not indices.is_contiguous()
            or indices.dtype != torch.int32 or indices.device != q_nope.device):
        raise ValueError("indices must be a contiguous int32 [B, q_len, topk] tensor")


def mla_decode_sparse(q_nope, q_pe, kv_cache, page_table, seq_lens, indices, scale, kv_scale, out, lse, workspace,
                      stream=None) -> None:
    """Enqueue a top-k decode (see include/mla_sparse.h); indices: int32
    [B, q_len, topk] token positions, -1 = unused."""
    _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, indices, out, lse, workspace)
    _check_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    _check_indices(indices, q_nope)
    B, Q, topk = indices.shape
    dims = make_dims(q_nope, kv_cache, page_table)
    rc = load_library().mla_decode_sparse(
        ctypes.byref(dims), _ptr(q_nope), _ptr(q_pe), _ptr(kv_cache), _ptr(page_table), _ptr(seq_lens),
        _ptr(indices), int(topk), int(Q), float(scale), float(kv_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_sparse")


def mla_decode_sparse_query_status(q_nope, kv_cache, page_table, topk: int, workspace, stream=None) -> int:
    dims = make_dims(q_nope, kv_cache, page_table)
    st = ctypes.c_int32(0)
    rc = load_library().mla_decode_sparse_query_status(ctypes.byref(dims), int(topk), _ptr(workspace),
                                                        _stream_handle(stream), ctypes.byref(st))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_sparse_query_status")
    return st.value


def mla_decode_cascade_workspace_size(dims: MlaDims, prefix_pages: int, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_decode_cascade_workspace_size(ctypes.byref(dims), int(prefix_pages), dev)
    if n == 0:
        raise MlaError(-1, "mla_decode_cascade_workspace_size")
    return int(n)


def mla_decode_cascade(q_nope, q_pe, kv_cache, page_table, seq_lens, prefix_pages, scale, kv_scale, out, lse,
                       workspace, stream=None) -> None:
    """Enqueue a cascade decode over a shared prefix (see include/mla_cascade.h)."""
    _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    _check_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    dims = make_dims(q_nope, kv_cache, page_table)
    rc = load_library().mla_decode_cascade(
        ctypes.byref(dims), _ptr(q_nope), _ptr(q_pe), _ptr(kv_cache), _ptr(page_table), _ptr(seq_lens),
        int(prefix_pages), int(q_nope.shape[1]), float(scale), float(kv_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        ctypes.c_size_t(workspace.numel() * workspace.element_size()), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_cascade")


def mla_decode_cascade_query_status(q_nope, kv_cache, page_table, prefix_pages: int, workspace, stream=None) -> int:
    dims = make_dims(q_nope, kv_cache, page_table)
    st = ctypes.c_int32(0)
    rc = load_library().mla_decode_cascade_query_status(ctypes.byref(dims), int(prefix_pages), _ptr(workspace),
                                                         _stream_handle(stream), ctypes.byref(st))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_cascade_query_status")
    return st.value


# ---- prompt chunks and windows (include/mla_prefill.h) ----
#
# Each call first runs one combined test of everything it passes on (it runs
# on every call; a small step is bound by it); the functions below it name
# what is wrong when that test fails.

class _Torch:
    """What the tests below need of torch, looked up once (importing torch, or
    its attributes, on every call costs microseconds)."""

    torch = None

    @classmethod
    def load(cls):
        import torch

        cls.bf16, cls.f32, cls.i32 = torch.bfloat16, torch.float32, torch.int32
        cls.cache_codes = {torch.bfloat16: MLA_KV_BF16, torch.uint8: MLA_KV_FP8_E4M3,
                           torch.float8_e4m3fn: MLA_KV_FP8_E4M3}
        cls.device, cls.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        cls.torch = torch
        return cls


def _t():
    return _Torch if _Torch.torch is not None else _Torch.load()


def _fits(t, shape, dtype, dev) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _cache_fits(kv_cache, page_table, seq_lens, B, dev, T) -> bool:
    c, p = kv_cache.shape, page_table.shape
    return (len(c) == 3 and c[2] == 576 and kv_cache.get_device() == dev and kv_cache.dtype in T.cache_codes
            and kv_cache.is_contiguous() and _fits(seq_lens, (B,), T.i32, dev) and page_table.dtype is T.i32
            and len(p) == 2 and p[0] == B and page_table.get_device() == dev and page_table.stride(1) == 1
            and page_table.stride(0) >= p[1])


def _check_current_device(dev):
    """The library runs on the current device; a tensor elsewhere would be
    read through a pointer of another device."""
    now = _t().device()
    if dev != now:
        raise ValueError(f"tensors must be on the current CUDA device {now}, got cuda:{dev}")


def _int32_arg(name, v, low=0):
    v = int(v)
    if not low <= v <= 2**31 - 1:
        raise ValueError(f"{name} must be between {low} and 2**31 - 1, got {v}")
    return v


def _stream_int(stream, dev):
    return _t().raw_stream(dev) if stream is None else stream.cuda_stream


def make_prefill_dims(q_nope, kv_cache, page_table, seq_lens) -> MlaPrefillDims:
    T, H, _ = q_nope.shape
    c = kv_cache.shape
    return MlaPrefillDims(seq_lens.shape[0], H, T, c[1], c[0], page_table.shape[1], page_table.stride(0),
                          kv_dtype_code(kv_cache))


def _decode_dims(s, kv_cache, page_table, T) -> MlaDims:
    """make_dims for tensors that passed their tests (s: q_nope's shape)."""
    c = kv_cache.shape
    return MlaDims(s[0], s[2], s[1], c[1], c[0], page_table.shape[1], page_table.stride(0),
                   T.cache_codes[kv_cache.dtype])


def mla_prefill_workspace_size(dims: MlaPrefillDims, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_prefill_workspace_size(ctypes.byref(dims), dev)
    if n == 0:
        raise MlaError(-1, "mla_prefill_workspace_size")
    return int(n)


def _check_prefill_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace):
    import torch

    if q_nope.dim() != 3 or q_nope.shape[2] != 512:
        raise ValueError(f"q_nope must be [total_q, H, 512], got {list(q_nope.shape)}")
    T, H, _ = q_nope.shape
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _check_layout("q_nope", q_nope, (T, H, 512), (torch.bfloat16,))
    _check_layout("q_pe", q_pe, (T, H, 64), (torch.bfloat16,))
    _check_layout("out", out, (T, H, 512), (torch.bfloat16,))
    _check_layout("lse", lse, (T, H), (torch.float32,))
    _check_layout("cu_q_lens", cu_q_lens, (B + 1,), (torch.int32,))
    _check_cache_and_table(kv_cache, page_table, seq_lens, B)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    for t in (q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace):
        if t.device != q_nope.device:
            raise ValueError("all tensors must be on one device")


def _prefill_fits(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace) -> bool:
    t = _t()
    s, dev = q_nope.shape, q_nope.get_device()
    if dev < 0 or len(s) != 3 or s[2] != 512 or seq_lens.dim() != 1:
        return False
    T, H, B = s[0], s[1], seq_lens.shape[0]
    return (_fits(q_nope, s, t.bf16, dev) and _fits(q_pe, (T, H, 64), t.bf16, dev) and _fits(out, s, t.bf16, dev)
            and _fits(lse, (T, H), t.f32, dev) and _fits(cu_q_lens, (B + 1,), t.i32, dev)
            and _cache_fits(kv_cache, page_table, seq_lens, B, dev, t) and workspace.get_device() == dev
            and workspace.is_contiguous())


def mla_prefill(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, window, num_sinks, scale, kv_scale, out, lse,
                workspace, stream=None) -> None:
    """Enqueue the attention of chunks of new tokens over the paged cache (see
    include/mla_prefill.h): q_nope [total_q, H, 512], cu_q_lens int32 [B + 1];
    window 0 = none, else a sliding window plus num_sinks first tokens."""
    if not _prefill_fits(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace):
        _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace)
        _check_prefill_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace)
        raise ValueError("prefill tensors do not have the shapes, types and layouts the library expects")
    dev = q_nope.get_device()
    _check_current_device(dev)
    dims = make_prefill_dims(q_nope, kv_cache, page_table, seq_lens)
    rc = load_library().mla_prefill(
        ctypes.byref(dims), q_nope.data_ptr(), q_pe.data_ptr(), kv_cache.data_ptr(), page_table.data_ptr(),
        seq_lens.data_ptr(), cu_q_lens.data_ptr(), _int32_arg("window", window), _int32_arg("num_sinks", num_sinks),
        float(scale), float(kv_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        _stream_int(stream, dev))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_prefill")


def mla_decode_window_workspace_size(dims: MlaDims, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_decode_window_workspace_size(ctypes.byref(dims), dev)
    if n == 0:
        raise MlaError(-1, "mla_decode_window_workspace_size")
    return int(n)


def mla_decode_window(q_nope, q_pe, kv_cache, page_table, seq_lens, window, num_sinks, scale, kv_scale, out, lse,
                      workspace, stream=None) -> None:
    """Enqueue a decode over a sliding window of `window` tokens and num_sinks
    first tokens (see include/mla_prefill.h); tensors as for mla_decode."""
    t = _t()
    s, dev = q_nope.shape, q_nope.get_device()
    if not (dev >= 0 and len(s) == 4 and s[3] == 512 and _fits(q_nope, s, t.bf16, dev)
            and _fits(q_pe, (s[0], s[1], s[2], 64), t.bf16, dev) and _fits(out, s, t.bf16, dev)
            and _fits(lse, s[:3], t.f32, dev) and _cache_fits(kv_cache, page_table, seq_lens, s[0], dev, t)
            and workspace.get_device() == dev and workspace.is_contiguous()):
        _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
        _check_decode_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, out, lse, workspace)
    _check_current_device(dev)
    dims = _decode_dims(s, kv_cache, page_table, t)
    rc = load_library().mla_decode_window(
        ctypes.byref(dims), q_nope.data_ptr(), q_pe.data_ptr(), kv_cache.data_ptr(), page_table.data_ptr(),
        seq_lens.data_ptr(), _int32_arg("window", window, 1), _int32_arg("num_sinks", num_sinks), float(scale),
        float(kv_scale),
        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream_int(stream, dev))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_window")


# ---- attention mass and eviction (include/mla_evict.h) ----

def mla_attn_mass_workspace_size(dims: MlaDims, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_attn_mass_workspace_size(ctypes.byref(dims), dev)
    if n == 0:
        raise MlaError(-1, "mla_attn_mass_workspace_size")
    return int(n)


def _check_mass_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, mass, mass_out, workspace):
    import torch

    if q_nope.dim() != 4 or q_nope.shape[3] != 512:
        raise ValueError(f"q_nope must be [B, q_len, H, 512], got {list(q_nope.shape)}")
    B, Q, H, _ = q_nope.shape
    _check_layout("q_nope", q_nope, (B, Q, H, 512), (torch.bfloat16,))
    _check_layout("q_pe", q_pe, (B, Q, H, 64), (torch.bfloat16,))
    _check_layout("lse", lse, (B, Q, H), (torch.float32,))
    _check_cache_and_table(kv_cache, page_table, seq_lens, B)
    if mass_out.dim() != 2:
        raise ValueError("mass_out must be [B, mass_cols]")
    _check_layout("mass_out", mass_out, (B, mass_out.shape[1]), (torch.float32,))
    if mass is not None:
        _check_layout("mass", mass, tuple(mass_out.shape), (torch.float32,))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    for t in (q_pe, kv_cache, page_table, seq_lens, lse, mass_out, workspace) + (() if mass is None else (mass,)):
        if t.device != q_nope.device:
            raise ValueError("all tensors must be on one device")


def _mass_fits(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, mass, mass_out, workspace) -> bool:
    t = _t()
    s, o, dev = q_nope.shape, mass_out.shape, q_nope.get_device()
    if dev < 0 or len(s) != 4 or s[3] != 512 or len(o) != 2 or o[0] != s[0]:
        return False
    return (_fits(q_nope, s, t.bf16, dev) and _fits(q_pe, (s[0], s[1], s[2], 64), t.bf16, dev)
            and _fits(lse, s[:3], t.f32, dev) and _fits(mass_out, o, t.f32, dev)
            and (mass is None or _fits(mass, o, t.f32, dev))
            and _cache_fits(kv_cache, page_table, seq_lens, s[0], dev, t) and workspace.get_device() == dev
            and workspace.is_contiguous())


def mla_attn_mass(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, num_fresh, scale, kv_scale, mass, mass_out,
                  workspace, stream=None) -> None:
    """Enqueue the accumulation of the softmax weights that a step's queries
    gave to every cached token (see include/mla_evict.h): mass (None: zeros)
    and mass_out fp32 [B, mass_cols]; the last num_fresh tokens start at 0."""
    if not _mass_fits(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, mass, mass_out, workspace):
        _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, mass_out, workspace)
        if mass is not None:
            _check_cuda(mass)
        _check_mass_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, lse, mass, mass_out, workspace)
        raise ValueError("mass tensors do not have the shapes, types and layouts the library expects")
    dev = q_nope.get_device()
    _check_current_device(dev)
    dims = _decode_dims(q_nope.shape, kv_cache, page_table, _t())
    rc = load_library().mla_attn_mass(
        ctypes.byref(dims), q_nope.data_ptr(), q_pe.data_ptr(), kv_cache.data_ptr(), page_table.data_ptr(),
        seq_lens.data_ptr(), lse.data_ptr(), _int32_arg("num_fresh", num_fresh), float(scale),
        float(kv_scale),
        None if mass is None else mass.data_ptr(), mass_out.data_ptr(), mass_out.shape[1], workspace.data_ptr(),
        workspace.nbytes, _stream_int(stream, dev))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_attn_mass")


def mla_evict_workspace_size(batch: int, budget: int) -> int:
    n = load_library().mla_evict_workspace_size(_int32_arg("batch", batch), _int32_arg("budget", budget))
    if n == 0:
        raise MlaError(-1, "mla_evict_workspace_size")
    return int(n)


def _check_evict_tensors(mass, positions, seq_lens, page_table, kv_cache, budget, new_lens, kept, mass_out,
                         positions_out, workspace):
    import torch

    if mass.dim() != 2:
        raise ValueError("mass must be [B, mass_cols]")
    B, cols = mass.shape
    _check_layout("mass", mass, (B, cols), (torch.float32,))
    _check_layout("mass_out", mass_out, (B, cols), (torch.float32,))
    if positions is not None:
        if positions_out is None:
            raise ValueError("positions_out is needed with positions")
        _check_layout("positions", positions, (B, cols), (torch.int32,))
        _check_layout("positions_out", positions_out, (B, cols), (torch.int32,))
    _check_cache_and_table(kv_cache, page_table, seq_lens, B)
    if kv_cache.shape[1] != 64:
        raise ValueError("kv_cache must have pages of 64 tokens")
    _check_layout("new_lens", new_lens, (B,), (torch.int32,))
    _check_layout("kept", kept, (B, budget), (torch.int32,))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    rest = (positions, positions_out) if positions is not None else ()
    for t in (seq_lens, page_table, kv_cache, new_lens, kept, mass_out, workspace) + rest:
        if t.device != mass.device:
            raise ValueError("all tensors must be on one device")


def _evict_fits(mass, positions, seq_lens, page_table, kv_cache, budget, new_lens, kept, mass_out, positions_out,
                workspace) -> bool:
    t = _t()
    s, dev = mass.shape, mass.get_device()
    if dev < 0 or len(s) != 2:
        return False
    if positions is not None:
        if positions_out is None or not (_fits(positions, s, t.i32, dev) and _fits(positions_out, s, t.i32, dev)):
            return False
    return (_fits(mass, s, t.f32, dev) and _fits(mass_out, s, t.f32, dev) and _fits(new_lens, s[:1], t.i32, dev)
            and _fits(kept, (s[0], budget), t.i32, dev) and _cache_fits(kv_cache, page_table, seq_lens, s[0], dev, t)
            and kv_cache.shape[1] == 64 and workspace.get_device() == dev and workspace.is_contiguous())


def mla_evict(mass, positions, seq_lens, page_table, kv_cache, budget, num_sinks, num_recent, new_lens, kept, mass_out,
              positions_out, workspace, stream=None) -> None:
    """Enqueue the eviction of every request's tokens beyond its budget (see
    include/mla_evict.h).  positions and positions_out may be None."""
    budget = _int32_arg("budget", budget, 1)
    if not _evict_fits(mass, positions, seq_lens, page_table, kv_cache, budget, new_lens, kept, mass_out,
                       positions_out, workspace):
        _check_cuda(mass, seq_lens, page_table, kv_cache, new_lens, kept, mass_out, workspace)
        if positions is not None and positions_out is not None:
            _check_cuda(positions, positions_out)
        _check_evict_tensors(mass, positions, seq_lens, page_table, kv_cache, budget, new_lens, kept, mass_out,
                             positions_out, workspace)
        raise ValueError("eviction tensors do not have the shapes, types and layouts the library expects")
    dev = mass.get_device()
    _check_current_device(dev)
    dims = MlaEvictDims(mass.shape[0], mass.shape[1], kv_cache.shape[0], page_table.shape[1], page_table.stride(0),
                        _t().cache_codes[kv_cache.dtype], budget, _int32_arg("num_sinks", num_sinks),
                        _int32_arg("num_recent", num_recent))
    pos = None if positions is None else positions.data_ptr()
    pos_out = None if positions is None else positions_out.data_ptr()
    rc = load_library().mla_evict(
        ctypes.byref(dims), mass.data_ptr(), pos, seq_lens.data_ptr(), page_table.data_ptr(), kv_cache.data_ptr(),
        new_lens.data_ptr(), kept.data_ptr(), mass_out.data_ptr(), pos_out, workspace.data_ptr(), workspace.nbytes,
        _stream_int(stream, dev))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_evict")


# ---- trees of drafted tokens (include/mla_tree.h, include/mla_verify.h) ----

def mla_decode_tree_workspace_size(dims: MlaPrefillDims, device: int | None = None) -> int:
    import torch

    dev = torch.cuda.current_device() if device is None else device
    n = load_library().mla_decode_tree_workspace_size(ctypes.byref(dims), dev)
    if n == 0:
        raise MlaError(-1, "mla_decode_tree_workspace_size")
    return int(n)


def mla_decode_tree(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, scale, kv_scale, out, lse,
                    workspace, stream=None) -> None:
    """Enqueue the attention of trees of drafted tokens (see
    include/mla_tree.h): tensors as for mla_prefill; parents int32 [total_q],
    each node's parent within its request, -1 = none."""
    rc = _binding().decode_tree(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, scale, kv_scale, out,
                                lse, workspace, stream)
    if rc is None:
        _refuse("mla_decode_tree", _explain_decode_tree, q_nope.get_device(), q_nope, q_pe, kv_cache, page_table,
                seq_lens, cu_q_lens, parents, out, lse, workspace)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_tree")


def _explain_decode_tree(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, out, lse, workspace):
    _check_cuda(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, parents, out, lse, workspace)
    _check_prefill_tensors(q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens, out, lse, workspace)
    _check_vectors(q_nope.device, parents=(parents, q_nope.shape[:1]))


def _check_vectors(device, **named):
    """name=(tensor, shape): contiguous int32 tensors on one device."""
    for name, (t, shape) in named.items():
        _check_layout(name, t, shape, (_t().i32,))
        if t.device != device:
            raise ValueError("all tensors must be on one device")


def _layers_of(kv_cache):
    """(layers, pages, page size, bytes between layers) of a cache
    [num_pages, 64, 576] or caches [num_layers, num_pages, 64, 576], or None."""
    s, k = kv_cache.shape, kv_cache.stride()
    if len(s) not in (3, 4) or s[-1] != 576 or s[-2] != 64 or kv_cache.dtype not in _t().cache_codes:
        return None
    if k[-1] != 1 or k[-2] != 576 or (s[-3] > 1 and k[-3] != 64 * 576):
        return None
    if len(s) == 3:
        return 1, s[0], 0
    return s[0], s[1], k[0] * kv_cache.element_size() if s[0] > 1 else 0


def _check_layers(kv_cache):
    if _layers_of(kv_cache) is None:
        raise ValueError("kv_cache must be bf16 or e4m3 [num_pages, 64, 576], or [num_layers, num_pages, 64, 576] "
                         "with contiguous layers")


def _check_table(name, table, rows):
    if (table.dtype != _t().i32 or table.dim() != 2 or (rows is not None and table.shape[0] != rows)
            or table.stride(1) != 1 or table.stride(0) < table.shape[1]):
        raise ValueError(f"{name} must be an int32 [{'rows' if rows is None else rows}, max_pages] tensor with unit "
                         "column stride")


def _check_devices(device, *tensors):
    for t in tensors:
        if t.device != device:
            raise ValueError("all tensors must be on one device")


def _check_status(status):
    if status.dtype != _t().i32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor of at least one element")


def _explain_tree_commit(kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, new_lens, status):
    _check_cuda(kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, new_lens, status)
    _check_layers(kv_cache)
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    if path.dim() != 2:
        raise ValueError("path must be [B, path_cols]")
    dev = kv_cache.device
    _check_vectors(dev, seq_lens=(seq_lens, (B,)), cu_q_lens=(cu_q_lens, (B + 1,)), path=(path, (B, path.shape[1])),
                   num_path=(num_path, (B,)), new_lens=(new_lens, (B,)))
    _check_table("page_table", page_table, B)
    _check_status(status)
    _check_devices(dev, page_table, status)


def mla_tree_commit(kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, new_lens, status, stream=None) -> None:
    """Enqueue the move of the accepted nodes' rows (see include/mla_tree.h).

    kv_cache: [num_pages, 64, 576], or one such cache per layer as
    [num_layers, num_pages, 64, 576]; path int32 [B, cols], num_path and
    new_lens int32 [B] (new_lens and status apart from the inputs); status int32 [1]."""
    tensors = kv_cache, page_table, seq_lens, cu_q_lens, path, num_path, new_lens, status
    rc = _binding().tree_commit(*tensors, stream)
    if rc is None:
        _refuse("mla_tree_commit", _explain_tree_commit, kv_cache.get_device(), *tensors)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_tree_commit")


def _check_probs(name, t, rows, vocab):
    if (t.dtype != _t().f32 or t.dim() != 2 or t.shape[0] != rows or t.shape[1] != vocab or t.stride(1) != 1
            or (rows > 1 and t.stride(0) < vocab)):
        raise ValueError(f"{name} must be an fp32 [total_q, vocab] tensor with unit column stride")


def _explain_verify(target, draft, tokens, parents, cu_q_lens, accept, sample, path, tokens_out, num_out, status):
    _check_cuda(target, tokens, parents, cu_q_lens, accept, sample, path, tokens_out, num_out, status)
    if target.dim() != 2:
        raise ValueError("target must be [total_q, vocab]")
    T, V = target.shape
    dev = target.device
    _check_probs("target", target, T, V)
    if draft is not None:
        _check_cuda(draft)
        _check_probs("draft", draft, T, V)
        _check_devices(dev, draft)
    B = sample.shape[0] if sample.dim() == 1 else -1
    if path.dim() != 2:
        raise ValueError("path must be [B, path_cols]")
    _check_layout("accept", accept, (T,), (_t().f32,))
    _check_layout("sample", sample, (B,), (_t().f32,))
    shape = (B, path.shape[1])
    _check_vectors(dev, tokens=(tokens, (T,)), parents=(parents, (T,)), cu_q_lens=(cu_q_lens, (B + 1,)),
                   path=(path, shape), tokens_out=(tokens_out, shape), num_out=(num_out, (B,)))
    _check_status(status)
    _check_devices(dev, accept, sample, status)


def mla_verify(target, draft, tokens, parents, cu_q_lens, accept, sample, path, tokens_out, num_out, status,
               stream=None) -> None:
    """Enqueue the verification of drafted tokens (see include/mla_verify.h).

    target and draft (None: fixed proposals) fp32 [total_q, vocab]; tokens,
    parents int32 and accept fp32 [total_q]; sample fp32 [B]; path and
    tokens_out int32 [B, cols], num_out int32 [B]; status int32 [1]."""
    tensors = target, draft, tokens, parents, cu_q_lens, accept, sample, path, tokens_out, num_out, status
    rc = _binding().verify(*tensors, stream)
    if rc is None:
        _refuse("mla_verify", _explain_verify, target.get_device(), *tensors)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_verify")


# ---- page operations (include/mla_pages.h) ----

def mla_page_resize_workspace_size(batch: int, max_pages: int, num_pages: int) -> int:
    n = load_library().mla_page_resize_workspace_size(_int32_arg("batch", batch), _int32_arg("max_pages", max_pages),
                                                      _int32_arg("num_pages", num_pages))
    if n == 0:
        raise MlaError(-1, "mla_page_resize_workspace_size")
    return int(n)


def _explain_page_resize(new_lens, page_table, page_refs, page_table_out, page_refs_out, workspace):
    _check_cuda(new_lens, page_table, page_refs, page_table_out, page_refs_out, workspace)
    B = new_lens.shape[0] if new_lens.dim() == 1 else -1
    dev = new_lens.device
    if page_refs.dim() != 1:
        raise ValueError("page_refs must be [num_pages]")
    _check_vectors(dev, new_lens=(new_lens, (B,)), page_refs=(page_refs, page_refs.shape),
                   page_refs_out=(page_refs_out, page_refs.shape))
    _check_table("page_table", page_table, B)
    _check_table("page_table_out", page_table_out, B)
    if page_table.shape != page_table_out.shape:
        raise ValueError("page_table and page_table_out must have the same shape")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check_devices(dev, page_table, page_table_out, workspace)


def mla_page_resize(new_lens, page_table, page_refs, page_table_out, page_refs_out, workspace, stream=None) -> None:
    """Enqueue handing out and freeing pages for the requests' new lengths (see
    include/mla_pages.h); page_table_out and page_refs_out may be the inputs."""
    tensors = new_lens, page_table, page_refs, page_table_out, page_refs_out, workspace
    rc = _binding().page_resize(*tensors, stream)
    if rc is None:
        _refuse("mla_page_resize", _explain_page_resize, new_lens.get_device(), *tensors)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_resize")


def mla_page_fork_workspace_size(sources: int, children: int, max_pages: int, num_pages: int) -> int:
    n = load_library().mla_page_fork_workspace_size(
        _int32_arg("sources", sources), _int32_arg("children", children), _int32_arg("max_pages", max_pages),
        _int32_arg("num_pages", num_pages))
    if n == 0:
        raise MlaError(-1, "mla_page_fork_workspace_size")
    return int(n)


def _explain_page_fork(src, seq_lens, page_table, page_refs, kv_cache, page_table_out, page_refs_out, workspace):
    _check_cuda(src, seq_lens, page_table, page_refs, kv_cache, page_table_out, page_refs_out, workspace)
    _check_layers(kv_cache)
    S = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    C = src.shape[0] if src.dim() == 1 else -1
    layers, pages, step = _layers_of(kv_cache)
    dev = kv_cache.device
    _check_vectors(dev, src=(src, (C,)), seq_lens=(seq_lens, (S,)), page_refs=(page_refs, (pages,)),
                   page_refs_out=(page_refs_out, (pages,)))
    _check_table("page_table", page_table, S)
    _check_table("page_table_out", page_table_out, C)
    if page_table.shape[1] != page_table_out.shape[1]:
        raise ValueError("page_table and page_table_out must have the same number of columns")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _check_devices(dev, page_table, page_table_out, workspace)


def mla_page_fork(src, seq_lens, page_table, page_refs, kv_cache, page_table_out, page_refs_out, workspace,
                  stream=None) -> None:
    """Enqueue the fork of requests (see include/mla_pages.h): child c continues
    request src[c] (int32 [children], -1 = an empty row); kv_cache as for
    mla_tree_commit; page_refs_out may be page_refs."""
    tensors = src, seq_lens, page_table, page_refs, kv_cache, page_table_out, page_refs_out, workspace
    rc = _binding().page_fork(*tensors, stream)
    if rc is None:
        _refuse("mla_page_fork", _explain_page_fork, kv_cache.get_device(), *tensors)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_fork")


# ---- rotary positions (include/mla_rope.h) ----

def mla_rope_frequencies(rotary_dim, base=10000.0, factor=1.0, original_len=0, fast=32.0, slow=1.0,
                         ramp="turns") -> list:
    """Radians a position of every rotated pair (see include/mla_rope.h).

    With a factor and an original_len, ramp says how the pairs between `fast`
    and `slow` turns pass from kept to stretched: "turns" (as published) or
    "index" (what DeepSeek-V3's configuration means by these parameters)."""
    lib = load_library()
    try:
        name = {"turns": "mla_rope_frequencies", "index": "mla_rope_frequencies_by_index"}[ramp]
    except (KeyError, TypeError):
        raise ValueError(f"ramp must be 'turns' or 'index', got {ramp!r}") from None
    out = (ctypes.c_double * 32)()
    rc = getattr(lib, name)(_int32_arg("rotary_dim", rotary_dim), float(base), float(factor),
                            _int32_arg("original_len", original_len), float(fast), float(slow), out)
    if rc != MLA_OK:
        raise MlaError(rc, name)
    return list(out)[:rotary_dim // 2]


def mla_rope_plan(rotary_dim, base=10000.0, factor=1.0, original_len=0, fast=32.0, slow=1.0, interleaved=True,
                  amplitude=1.0, frequencies=None, ramp="turns") -> MlaRopePlan:
    """The plan of a rotation: from base and scaling (see mla_rope_frequencies;
    the ramp has to be the one that the weights were trained with), or from the
    frequencies themselves (rotary_dim / 2 of them)."""
    if frequencies is None:
        frequencies = mla_rope_frequencies(rotary_dim, base, factor, original_len, fast, slow, ramp)
    elif len(frequencies) != rotary_dim // 2:
        raise ValueError(f"rotary_dim {rotary_dim} needs {rotary_dim // 2} frequencies, got {len(frequencies)}")
    plan = MlaRopePlan()
    rc = load_library().mla_rope_plan_init(_int32_arg("rotary_dim", rotary_dim), int(bool(interleaved)),
                                           float(amplitude), (ctypes.c_double * len(frequencies))(*frequencies),
                                           ctypes.byref(plan))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_rope_plan_init")
    return plan


def _explain_rope(q_pe, rows, positions, page_table, seq_lens, cu_q_lens, q_out, kv_cache, status):
    t = _t()
    _check_cuda(q_pe, rows, page_table, seq_lens, cu_q_lens, q_out, kv_cache, status)
    if q_pe.dim() != 3 or q_pe.shape[2] != 64 or q_pe.dtype != t.bf16 or q_pe.stride(2) != 1:
        raise ValueError("q_pe must be a bf16 [total_q, H, 64] tensor with unit stride in the last dimension")
    T, H, _ = q_pe.shape
    if tuple(rows.shape) != (T, 576) or rows.dtype != t.bf16 or rows.stride(1) != 1:
        raise ValueError("rows must be a bf16 [total_q, 576] tensor with unit stride in the last dimension")
    dev = q_pe.device
    _check_layout("q_out", q_out, (T, H, 64), (t.bf16,))
    B = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _check_cache_and_table(kv_cache, page_table, seq_lens, B)
    if kv_cache.shape[1] != 64:
        raise ValueError("kv_cache must have pages of 64 tokens")
    _check_vectors(dev, cu_q_lens=(cu_q_lens, (B + 1,)))
    if positions is not None:
        _check_cuda(positions)
        _check_vectors(dev, positions=(positions, (T,)))
    _check_status(status)
    _check_devices(dev, rows, q_out, kv_cache, page_table, seq_lens, status)


def mla_rope_pack(plan, q_pe, rows, positions, page_table, seq_lens, cu_q_lens, kv_scale, q_out, kv_cache, status,
                  stream=None) -> None:
    """Enqueue the rotation of a step's q_pe and k_pe and the cache write of its
    rows (see include/mla_rope.h).

    q_pe bf16 [total_q, H, 64] and rows bf16 [total_q, 576], with unit stride in
    the last dimension; positions int32 [total_q], or None: the tokens' slots;
    q_out bf16 [total_q, H, 64], contiguous (q_pe itself if that is)."""
    rc = _binding().rope_pack(plan, q_pe, rows, positions, page_table, seq_lens, cu_q_lens, kv_scale, q_out, kv_cache,
                              status, stream)
    if rc is None:
        if not isinstance(plan, MlaRopePlan):
            raise TypeError("plan must come from mla_rope_plan")
        _refuse("mla_rope_pack", _explain_rope, q_pe.get_device(), q_pe, rows, positions, page_table, seq_lens,
                cu_q_lens, q_out, kv_cache, status)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_rope_pack")


@dataclass
class DecodeBuffers:
    out: object
    lse: object
    workspace: object


def alloc_buffers(q_nope, kv_cache, page_table) -> DecodeBuffers:
    """torch allocations sized for one decode step (caller-owned memory)."""
    import torch

    B, Q, H, _ = q_nope.shape
    dims = make_dims(q_nope, kv_cache, page_table)
    ws = torch.empty(mla_decode_workspace_size(dims, q_nope.device.index), dtype=torch.uint8, device=q_nope.device)
    out = torch.empty(B, Q, H, 512, dtype=torch.bfloat16, device=q_nope.device)
    lse = torch.empty(B, Q, H, dtype=torch.float32, device=q_nope.device)
    return DecodeBuffers(out, lse, ws)


def decode(q_nope, q_pe, kv_cache, page_table, seq_lens, scale, kv_scale=1.0, buffers: DecodeBuffers | None = None,
           stream=None):
    """Convenience wrapper: allocates outputs/workspace if not given; returns (out, lse)."""
    if buffers is None:
        buffers = alloc_buffers(q_nope, kv_cache, page_table)
    mla_decode(q_nope, q_pe, kv_cache, page_table, seq_lens, q_nope.shape[1], scale, kv_scale, buffers.out,
               buffers.lse, buffers.workspace, stream)
    return buffers.out, buffers.lse

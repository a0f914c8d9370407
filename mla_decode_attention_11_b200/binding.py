"""Python binding of libmla_decode.so (ctypes; argument marshalling only).

Every step of MLA decode runs in the library's CUDA kernels.  PyTorch is used
here only to hold device memory, to name the current stream and to read
tensor pointers.  There is no fallback: if the library is missing or the
device is not an sm_100 GPU, the calls raise.

Entry points mirror include/mla_decode.h:
    mla_decode_plan, mla_decode_workspace_init, mla_decode_run,
    mla_decode_check, mla_status_string, mla_decode_set_debug,
    mla_decode_run_noalloc, mla_decode_run_sinks,
    the paged cache's mla_decode_plan_paged, mla_decode_run_paged,
    mla_decode_plan_paged_fp8, mla_decode_run_paged_fp8,
    mha_decode_plan_paged, mha_decode_run_paged, mla_decode_plan_prefix,
    mla_decode_run_prefix, mla_cache_append, mla_cache_append_prefix,
    mha_cache_append
plus the convenience wrappers ``mla_decode`` (device tensors in, device
tensors out) and ``mla_decode_host`` (host tensors in and out, with the
copies done here around the library call).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Tuple

import torch

from . import build as _build

D_QK = 576
D_V = 512

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_ALIGNMENT", 3: "MLA_ERR_UNSUPPORTED",
                4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_WORKSPACE", 7: "MLA_ERR_SEQLEN",
                8: "MLA_ERR_PAGE"}
MLA_KERNEL_TRANSPOSED = 1
MLA_KERNEL_PAIR = 2
MLA_KERNEL_MHA = 3
MLA_KERNEL_FP8 = 4
MLA_KERNEL_FP8_MMA = 5
MLA_KERNEL_FP8_PAIR = 6
MHA_D = 128
MLA_NOALLOC_SCRATCH_BYTES = 40 * 1024 * 1024

EXPORTED_SYMBOLS = ("mla_decode_plan", "mla_decode_plan_kernel", "mla_decode_plan_batch_invariant", "mla_decode_workspace_init", "mla_decode_run", "mla_decode_run_phase",
                    "mla_decode_check", "mla_decode_run_noalloc", "mla_decode_run_sinks",
                    "mla_status_string", "mla_decode_abi_version", "mla_decode_set_debug",
                    "mha_decode_plan", "mha_decode_run", "mha_decode_run_phase",
                    "mla_decode_plan_fp8", "mla_decode_plan_fp8_kernel", "mla_decode_run_fp8",
                    "mla_decode_run_fp8_phase",
                    "mla_decode_plan_paged", "mla_decode_run_paged", "mla_decode_plan_paged_fp8",
                    "mla_decode_run_paged_fp8", "mha_decode_plan_paged", "mha_decode_run_paged",
                    "mla_decode_plan_prefix", "mla_decode_run_prefix", "mla_cache_append", "mla_cache_append_prefix",
                    "mha_cache_append")


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)} ({status_string(code)})")


class mla_plan(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Sq", ctypes.c_int32), ("H", ctypes.c_int32), ("L_max", ctypes.c_int32),
                ("device", ctypes.c_int32), ("num_sms", ctypes.c_int32), ("kernel", ctypes.c_int32),
                ("group_rows", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("num_partitions", ctypes.c_int32), ("tile_kv", ctypes.c_int32), ("cta_threads", ctypes.c_int32),
                ("smem_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
                ("l2_prefetch_tiles", ctypes.c_int32), ("split_tiles", ctypes.c_int32),
                ("Hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("window", ctypes.c_int32), ("first_tokens", ctypes.c_int32),
                ("prefix_max", ctypes.c_int32), ("prefix_partitions", ctypes.c_int32),
                ("prefix_groups", ctypes.c_int32),
                ("reserved", ctypes.c_uint64 * 1)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if not k.startswith("reserved")}


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = True):
    """Load (building first if needed) libmla_decode.so; raises if it cannot."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise OSError(f"libmla_decode.so not built ({path}); run python -m mla_decode_attention_11_b200.build")
            _build.build()
        lib = ctypes.CDLL(path)
        c_i32, c_sz, c_vp, c_f = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
        lib.mla_decode_plan.restype = c_i32
        lib.mla_decode_plan.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(mla_plan),
                                        ctypes.POINTER(c_sz)]
        lib.mla_decode_plan_kernel.restype = c_i32
        lib.mla_decode_plan_kernel.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                               ctypes.POINTER(mla_plan), ctypes.POINTER(c_sz)]
        lib.mla_decode_plan_batch_invariant.restype = c_i32
        lib.mla_decode_plan_batch_invariant.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                                        ctypes.POINTER(mla_plan), ctypes.POINTER(c_sz)]
        lib.mla_decode_workspace_init.restype = c_i32
        lib.mla_decode_workspace_init.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_sz, c_vp]
        lib.mla_decode_run.restype = c_i32
        lib.mla_decode_run.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp, c_sz,
                                       c_vp]
        lib.mla_decode_run_sinks.restype = c_i32
        lib.mla_decode_run_sinks.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp, c_vp,
                                             c_sz, c_vp]
        lib.mla_decode_run_phase.restype = c_i32
        lib.mla_decode_run_phase.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp,
                                             c_sz, c_vp, c_i32]
        lib.mla_decode_run_noalloc.restype = c_i32
        lib.mla_decode_run_noalloc.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_i32,
                                               c_vp]
        lib.mha_decode_plan.restype = c_i32
        lib.mha_decode_plan.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(mla_plan),
                                        ctypes.POINTER(c_sz)]
        lib.mha_decode_run.restype = c_i32
        lib.mha_decode_run.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp, c_vp,
                                       c_sz, c_vp]
        lib.mha_decode_run_phase.restype = c_i32
        lib.mha_decode_run_phase.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp,
                                             c_vp, c_sz, c_vp, c_i32]
        lib.mla_decode_plan_fp8.restype = c_i32
        lib.mla_decode_plan_fp8.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, ctypes.POINTER(mla_plan),
                                            ctypes.POINTER(c_sz)]
        lib.mla_decode_plan_fp8_kernel.restype = c_i32
        lib.mla_decode_plan_fp8_kernel.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                                   ctypes.POINTER(mla_plan), ctypes.POINTER(c_sz)]
        lib.mla_decode_run_fp8.restype = c_i32
        lib.mla_decode_run_fp8.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_f, c_vp, c_f, c_vp, c_vp, c_vp,
                                           c_vp, c_sz, c_vp]
        lib.mla_decode_run_fp8_phase.restype = c_i32
        lib.mla_decode_run_fp8_phase.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp, c_f, c_vp, c_f, c_vp, c_vp,
                                                 c_vp, c_sz, c_vp, c_i32]
        pp, ps, c_i64 = ctypes.POINTER(mla_plan), ctypes.POINTER(c_sz), ctypes.c_int64
        lib.mla_decode_plan_paged.argtypes = [c_i32] * 9 + [pp, ps]
        lib.mla_decode_plan_paged_fp8.argtypes = [c_i32] * 9 + [pp, ps]
        lib.mha_decode_plan_paged.argtypes = [c_i32] * 10 + [pp, ps]
        lib.mla_decode_plan_prefix.argtypes = [c_i32] * 8 + [pp, ps]
        tail = [c_vp, c_i64, c_i32, c_vp, c_f, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]  # block_table .. stream
        lib.mla_decode_run_paged.argtypes = [pp, c_vp, c_vp, c_i32] + tail
        lib.mla_decode_run_paged_fp8.argtypes = [pp, c_vp, c_vp, c_i32, c_f] + tail
        lib.mha_decode_run_paged.argtypes = [pp, c_vp, c_vp, c_vp, c_i32] + tail
        lib.mla_decode_run_prefix.argtypes = [pp, c_vp, c_vp, c_i32, c_vp, c_i32, c_vp] + tail
        lib.mla_cache_append.argtypes = [c_vp, c_vp]
        lib.mla_cache_append_prefix.argtypes = [c_vp, c_vp, c_vp]
        lib.mha_cache_append.argtypes = [c_vp, c_vp]
        for fn in (lib.mla_decode_plan_paged, lib.mha_decode_plan_paged, lib.mla_decode_plan_prefix,
                   lib.mla_decode_plan_paged_fp8, lib.mla_decode_run_paged_fp8, lib.mla_decode_run_paged,
                   lib.mha_decode_run_paged, lib.mla_decode_run_prefix,
                   lib.mla_cache_append, lib.mla_cache_append_prefix, lib.mha_cache_append):
            fn.restype = c_i32
        lib.mla_decode_check.restype = c_i32
        lib.mla_decode_check.argtypes = [ctypes.POINTER(mla_plan), c_vp, c_vp]
        lib.mla_status_string.restype = ctypes.c_char_p
        lib.mla_status_string.argtypes = [c_i32]
        lib.mla_decode_abi_version.restype = c_i32
        lib.mla_decode_abi_version.argtypes = []
        lib.mla_decode_set_debug.restype = c_i32
        lib.mla_decode_set_debug.argtypes = [ctypes.c_uint64, c_i32]
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load_library().mla_status_string(int(code)).decode()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def mla_decode_plan(B: int, Sq: int, H: int, L_max: int, device: Optional[int] = None,
                    num_partitions: int = 0, kernel: int = 0) -> mla_plan:
    """Validate a shape and choose kernel / grid / workspace size.  device=None
    means the current CUDA device; device=-1 plans for a B200 without a GPU.
    kernel: 0 = automatic, MLA_KERNEL_TRANSPOSED or MLA_KERNEL_PAIR
    (mla_decode_plan_kernel)."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    ws = ctypes.c_size_t(0)
    lib = load_library()
    if kernel:
        rc = lib.mla_decode_plan_kernel(int(B), int(Sq), int(H), int(L_max), int(device), int(num_partitions),
                                        int(kernel), ctypes.byref(p), ctypes.byref(ws))
    else:
        rc = lib.mla_decode_plan(int(B), int(Sq), int(H), int(L_max), int(device), int(num_partitions),
                                 ctypes.byref(p), ctypes.byref(ws))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan")
    return p


def mla_decode_plan_batch_invariant(B: int, Sq: int, H: int, L_max: int, device: Optional[int] = None,
                                    split_tiles: int = 0) -> mla_plan:
    """A plan whose per-sequence results are bitwise independent of the rest of
    the batch: every sequence is cut into chunks of split_tiles KV tiles
    (0 = the library default) at fixed offsets (mla_decode_plan_batch_invariant)."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    ws = ctypes.c_size_t(0)
    rc = load_library().mla_decode_plan_batch_invariant(int(B), int(Sq), int(H), int(L_max), int(device),
                                                        int(split_tiles), ctypes.byref(p), ctypes.byref(ws))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan_batch_invariant")
    return p


def alloc_workspace(plan: mla_plan, device=None) -> torch.Tensor:
    """A zeroed uint8 device buffer of plan.workspace_bytes (torch allocates;
    the library never does)."""
    dev = torch.device("cuda", plan.device if plan.device >= 0 else torch.cuda.current_device())
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device=dev if device is None else device)
    return ws


def mla_decode_workspace_init(plan: mla_plan, workspace: torch.Tensor, stream=None) -> None:
    rc = load_library().mla_decode_workspace_init(ctypes.byref(plan), workspace.data_ptr(), workspace.numel(),
                                                  _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_workspace_init")


def _check_tensor(t: torch.Tensor, name: str, dtype, shape) -> None:
    if t.is_cuda and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def mla_decode_run(plan: mla_plan, q: torch.Tensor, kv: torch.Tensor, seqlens: torch.Tensor, softmax_scale: float,
                   out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Enqueue one decode on `stream` (default: torch's current stream)."""
    B, Sq, H, L = plan.B, plan.Sq, plan.H, plan.L_max
    _check_tensor(q, "q", torch.bfloat16, (B, Sq, H, D_QK))
    _check_tensor(kv, "kv", torch.bfloat16, (B, L, D_QK))
    _check_tensor(seqlens, "seqlens", torch.int32, (B,))
    _check_tensor(out, "out", torch.bfloat16, (B, Sq, H, D_V))
    _check_tensor(lse, "lse", torch.float32, (B, Sq, H))
    rc = load_library().mla_decode_run(ctypes.byref(plan), q.data_ptr(), kv.data_ptr(), seqlens.data_ptr(),
                                       float(softmax_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                       workspace.numel(), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run")


def mla_decode_run_sinks(plan: mla_plan, q: torch.Tensor, kv: torch.Tensor, seqlens: torch.Tensor,
                         softmax_scale: float, sinks: Optional[torch.Tensor], out: torch.Tensor, lse: torch.Tensor,
                         workspace: torch.Tensor, stream=None) -> None:
    """mla_decode_run with per-head attention-sink logits: sinks is a CUDA
    fp32 tensor [H] (units of the scaled scores) or None for no sinks."""
    B, Sq, H, L = plan.B, plan.Sq, plan.H, plan.L_max
    _check_tensor(q, "q", torch.bfloat16, (B, Sq, H, D_QK))
    _check_tensor(kv, "kv", torch.bfloat16, (B, L, D_QK))
    _check_tensor(seqlens, "seqlens", torch.int32, (B,))
    _check_tensor(out, "out", torch.bfloat16, (B, Sq, H, D_V))
    _check_tensor(lse, "lse", torch.float32, (B, Sq, H))
    if sinks is not None:
        _check_tensor(sinks, "sinks", torch.float32, (H,))
    rc = load_library().mla_decode_run_sinks(ctypes.byref(plan), q.data_ptr(), kv.data_ptr(), seqlens.data_ptr(),
                                             float(softmax_scale), sinks.data_ptr() if sinks is not None else None,
                                             out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                             workspace.numel(), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_sinks")


def mla_decode_run_phase(plan: mla_plan, q: torch.Tensor, kv: torch.Tensor, seqlens: torch.Tensor,
                         softmax_scale: float, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                         phase: int, stream=None) -> None:
    """One of the two launches of mla_decode_run (1 = main kernel, 2 = combine)."""
    rc = load_library().mla_decode_run_phase(ctypes.byref(plan), q.data_ptr(), kv.data_ptr(), seqlens.data_ptr(),
                                             float(softmax_scale), out.data_ptr(), lse.data_ptr(),
                                             workspace.data_ptr(), workspace.numel(), _stream_handle(stream),
                                             int(phase))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_phase")


def mla_decode_run_noalloc(plan: mla_plan, q: torch.Tensor, kv: torch.Tensor, seqlens: torch.Tensor,
                           softmax_scale: float, out: torch.Tensor, lse: torch.Tensor, wait_and_check: bool = False,
                           stream=None) -> None:
    """mla_decode_run for callers that may not allocate device memory while
    decoding (an engine whose KV cache took nearly all HBM at start-up, a C host
    without a device allocator): the library's own static scratch array of
    MLA_NOALLOC_SCRATCH_BYTES per device stands in for the workspace.  Calls on
    one device share that array, so calls that may overlap on the GPU race;
    make the first call on a device outside stream capture.  With
    wait_and_check the stream is synchronised and a recorded device fault
    raises, as mla_decode_check does."""
    B, Sq, H, L = plan.B, plan.Sq, plan.H, plan.L_max
    _check_tensor(q, "q", torch.bfloat16, (B, Sq, H, D_QK))
    _check_tensor(kv, "kv", torch.bfloat16, (B, L, D_QK))
    _check_tensor(seqlens, "seqlens", torch.int32, (B,))
    _check_tensor(out, "out", torch.bfloat16, (B, Sq, H, D_V))
    _check_tensor(lse, "lse", torch.float32, (B, Sq, H))
    rc = load_library().mla_decode_run_noalloc(ctypes.byref(plan), q.data_ptr(), kv.data_ptr(), seqlens.data_ptr(),
                                               float(softmax_scale), out.data_ptr(), lse.data_ptr(),
                                               int(bool(wait_and_check)), _stream_handle(stream))
    if rc != MLA_OK:
        what = "mla_decode_run_noalloc"
        if rc == 6:
            what += f" (plan needs more than the {MLA_NOALLOC_SCRATCH_BYTES} bytes of static scratch)"
        raise MlaError(rc, what)


def mla_decode_check(plan: mla_plan, workspace: torch.Tensor, stream=None) -> int:
    """Synchronise, read and clear the device status; raise on a recorded fault."""
    rc = load_library().mla_decode_check(ctypes.byref(plan), workspace.data_ptr(), _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_check")
    return rc


def mla_decode_set_debug(wait_timeout_ns: int = 0, stall_unit: int = -1) -> None:
    load_library().mla_decode_set_debug(int(wait_timeout_ns), int(stall_unit))


def mla_decode(q: torch.Tensor, kv: torch.Tensor, seqlens: torch.Tensor, softmax_scale: Optional[float] = None,
               num_partitions: int = 0, plan: Optional[mla_plan] = None,
               workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Device tensors in, (out bf16 [B,Sq,H,512], lse fp32 [B,Sq,H]) out."""
    B, Sq, H, _ = q.shape
    L = kv.shape[1]
    if softmax_scale is None:
        softmax_scale = D_QK ** -0.5
    if plan is None:
        plan = mla_decode_plan(B, Sq, H, L, device=q.device.index, num_partitions=num_partitions)
    if workspace is None:
        workspace = alloc_workspace(plan, device=q.device)
    out = torch.empty((B, Sq, H, D_V), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, Sq, H), dtype=torch.float32, device=q.device)
    mla_decode_run(plan, q, kv, seqlens, softmax_scale, out, lse, workspace)
    return out, lse


def mla_decode_host(q_host: torch.Tensor, kv_host: torch.Tensor, seqlens_host: torch.Tensor,
                    softmax_scale: float, plan: mla_plan, workspace: torch.Tensor,
                    dev_bufs: Optional[dict] = None, out_host: Optional[torch.Tensor] = None,
                    lse_host: Optional[torch.Tensor] = None, stream=None):
    """End-to-end call with HOST tensors: copy q / kv / seqlens to the device,
    run, copy out / lse back (pinned host buffers make the copies async)."""
    dev = workspace.device
    if dev_bufs is None:
        dev_bufs = {}
    B, Sq, H, L = plan.B, plan.Sq, plan.H, plan.L_max
    if "q" not in dev_bufs:
        dev_bufs["q"] = torch.empty((B, Sq, H, D_QK), dtype=torch.bfloat16, device=dev)
        dev_bufs["kv"] = torch.empty((B, L, D_QK), dtype=torch.bfloat16, device=dev)
        dev_bufs["seqlens"] = torch.empty((B,), dtype=torch.int32, device=dev)
        dev_bufs["out"] = torch.empty((B, Sq, H, D_V), dtype=torch.bfloat16, device=dev)
        dev_bufs["lse"] = torch.empty((B, Sq, H), dtype=torch.float32, device=dev)
    if out_host is None:
        out_host = torch.empty((B, Sq, H, D_V), dtype=torch.bfloat16, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty((B, Sq, H), dtype=torch.float32, pin_memory=True)
    dev_bufs["q"].copy_(q_host, non_blocking=True)
    dev_bufs["kv"].copy_(kv_host, non_blocking=True)
    dev_bufs["seqlens"].copy_(seqlens_host, non_blocking=True)
    mla_decode_run(plan, dev_bufs["q"], dev_bufs["kv"], dev_bufs["seqlens"], softmax_scale, dev_bufs["out"],
                   dev_bufs["lse"], workspace, stream=stream)
    out_host.copy_(dev_bufs["out"], non_blocking=True)
    lse_host.copy_(dev_bufs["lse"], non_blocking=True)
    return out_host, lse_host


# ---------------------------------------------------------------- MHA decode

def mha_decode_plan(B: int, Sq: int, H: int, Hkv: int, L_max: int, device: Optional[int] = None,
                    num_partitions: int = 0) -> mla_plan:
    """Plan an MHA decode (128-wide heads, H query heads over Hkv kv heads)."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    ws = ctypes.c_size_t(0)
    rc = load_library().mha_decode_plan(int(B), int(Sq), int(H), int(Hkv), int(L_max), int(device),
                                        int(num_partitions), ctypes.byref(p), ctypes.byref(ws))
    if rc != MLA_OK:
        raise MlaError(rc, "mha_decode_plan")
    return p


def mha_decode_run(plan: mla_plan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seqlens: torch.Tensor,
                   softmax_scale: float, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                   sinks: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue one MHA decode: q [B,Sq,H,128], k and v [B,L_max,Hkv,128] (bf16)."""
    B, Sq, H, L, Hkv = plan.B, plan.Sq, plan.H, plan.L_max, plan.Hkv
    _check_tensor(q, "q", torch.bfloat16, (B, Sq, H, MHA_D))
    _check_tensor(k, "k", torch.bfloat16, (B, L, Hkv, MHA_D))
    _check_tensor(v, "v", torch.bfloat16, (B, L, Hkv, MHA_D))
    _check_tensor(seqlens, "seqlens", torch.int32, (B,))
    _check_tensor(out, "out", torch.bfloat16, (B, Sq, H, MHA_D))
    _check_tensor(lse, "lse", torch.float32, (B, Sq, H))
    if sinks is not None:
        _check_tensor(sinks, "sinks", torch.float32, (H,))
    rc = load_library().mha_decode_run(ctypes.byref(plan), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       seqlens.data_ptr(), float(softmax_scale),
                                       sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                       lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                       _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mha_decode_run")


def mha_decode_run_phase(plan: mla_plan, q, k, v, seqlens, softmax_scale: float, out, lse, workspace, phase: int,
                         sinks=None, stream=None) -> None:
    """One launch of mha_decode_run (1 = main kernel, 2 = combine)."""
    rc = load_library().mha_decode_run_phase(ctypes.byref(plan), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                             seqlens.data_ptr(), float(softmax_scale),
                                             sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                             lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                             _stream_handle(stream), int(phase))
    if rc != MLA_OK:
        raise MlaError(rc, "mha_decode_run_phase")


# ---------------------------------------------------------------- FP8 latent cache

def mla_decode_plan_fp8(B: int, Sq: int, H: int, L_max: int, device: Optional[int] = None,
                        num_partitions: int = 0, kernel: int = 0) -> mla_plan:
    """A plan for a cache of E4M3 codes (mla_decode_plan_fp8_kernel).  kernel = 0
    picks the default: the codes as kind::f8f6f4 MMA operands on CTA pairs
    (MLA_KERNEL_FP8_PAIR) when Sq*H is a multiple of 128, else in the
    transposed orientation (MLA_KERNEL_FP8_MMA); MLA_KERNEL_FP8 selects the
    kernel that widens the codes to f16 in shared memory."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    ws = ctypes.c_size_t(0)
    rc = load_library().mla_decode_plan_fp8_kernel(int(B), int(Sq), int(H), int(L_max), int(device),
                                                   int(num_partitions), int(kernel), ctypes.byref(p),
                                                   ctypes.byref(ws))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan_fp8_kernel")
    return p


def _fp8_codes(kv_fp8: torch.Tensor) -> torch.Tensor:
    return kv_fp8.view(torch.uint8) if kv_fp8.dtype == torch.float8_e4m3fn else kv_fp8


def mla_decode_run_fp8(plan: mla_plan, q: torch.Tensor, kv_fp8: torch.Tensor, kv_scale: float,
                       seqlens: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse: torch.Tensor,
                       workspace: torch.Tensor, sinks: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue one decode over an FP8 cache: kv_fp8 is a CUDA tensor of E4M3
    codes [B, L_max, 576] (torch.uint8 or torch.float8_e4m3fn), kv_value =
    kv_scale * e4m3(code); sinks as in mla_decode_run_sinks."""
    B, Sq, H, L = plan.B, plan.Sq, plan.H, plan.L_max
    codes = _fp8_codes(kv_fp8)
    _check_tensor(q, "q", torch.bfloat16, (B, Sq, H, D_QK))
    _check_tensor(codes, "kv_fp8", torch.uint8, (B, L, D_QK))
    _check_tensor(seqlens, "seqlens", torch.int32, (B,))
    _check_tensor(out, "out", torch.bfloat16, (B, Sq, H, D_V))
    _check_tensor(lse, "lse", torch.float32, (B, Sq, H))
    if sinks is not None:
        _check_tensor(sinks, "sinks", torch.float32, (H,))
    rc = load_library().mla_decode_run_fp8(ctypes.byref(plan), q.data_ptr(), codes.data_ptr(), float(kv_scale),
                                           seqlens.data_ptr(), float(softmax_scale),
                                           sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                           lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                           _stream_handle(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_fp8")


def mla_decode_run_fp8_phase(plan: mla_plan, q: torch.Tensor, kv_fp8: torch.Tensor, kv_scale: float,
                             seqlens: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse: torch.Tensor,
                             workspace: torch.Tensor, phase: int, stream=None) -> None:
    """One of the two launches of mla_decode_run_fp8 (1 = main kernel, 2 = combine)."""
    codes = _fp8_codes(kv_fp8)
    rc = load_library().mla_decode_run_fp8_phase(ctypes.byref(plan), q.data_ptr(), codes.data_ptr(),
                                                 float(kv_scale), seqlens.data_ptr(), float(softmax_scale),
                                                 out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                                 workspace.numel(), _stream_handle(stream), int(phase))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_fp8_phase")


# ---------------------------------------------------------------- paged cache

def mla_decode_plan_paged(B: int, Sq: int, H: int, L_max: int, page_size: int, window: int = 0,
                          first_tokens: int = 0, device: Optional[int] = None, num_partitions: int = 0) -> mla_plan:
    """A plan for a latent cache in pages: query token t of a sequence of L keys
    sees the keys up to its position p = L - Sq + t, and with a window those of
    the last `window` positions or the `first_tokens` first ones."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    rc = load_library().mla_decode_plan_paged(int(B), int(Sq), int(H), int(L_max), int(page_size), int(window),
                                              int(first_tokens), int(device), int(num_partitions), ctypes.byref(p),
                                              None)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan_paged")
    return p


def mla_decode_plan_paged_fp8(B: int, Sq: int, H: int, L_max: int, page_size: int, window: int = 0,
                              first_tokens: int = 0, device: Optional[int] = None,
                              num_partitions: int = 0) -> mla_plan:
    """mla_decode_plan_paged for pages of E4M3 codes with one dequantisation scale."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    rc = load_library().mla_decode_plan_paged_fp8(int(B), int(Sq), int(H), int(L_max), int(page_size), int(window),
                                                  int(first_tokens), int(device), int(num_partitions),
                                                  ctypes.byref(p), None)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan_paged_fp8")
    return p


def mha_decode_plan_paged(B: int, Sq: int, H: int, Hkv: int, L_max: int, page_size: int, window: int = 0,
                          first_tokens: int = 0, device: Optional[int] = None, num_partitions: int = 0) -> mla_plan:
    """mla_decode_plan_paged for key and value pages of grouped kv heads (128 wide)."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    rc = load_library().mha_decode_plan_paged(int(B), int(Sq), int(H), int(Hkv), int(L_max), int(page_size),
                                              int(window), int(first_tokens), int(device), int(num_partitions),
                                              ctypes.byref(p), None)
    if rc != MLA_OK:
        raise MlaError(rc, "mha_decode_plan_paged")
    return p


def mla_decode_plan_prefix(B: int, Sq: int, H: int, L_max: int, prefix_max: int, page_size: int,
                           device: Optional[int] = None, num_partitions: int = 0) -> mla_plan:
    """A plan for a batch that shares a prefix of at most prefix_max keys; L_max
    is the most own keys a sequence has after it."""
    if device is None:
        device = torch.cuda.current_device()
    p = mla_plan()
    rc = load_library().mla_decode_plan_prefix(int(B), int(Sq), int(H), int(L_max), int(prefix_max), int(page_size),
                                               int(device), int(num_partitions), ctypes.byref(p), None)
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_plan_prefix")
    return p


# The current stream's handle without building a torch.cuda.Stream (3 us of the
# 10 to 15 that one of the calls below takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(device: int, stream) -> int:
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream_handle(stream)


def _device_of(t: torch.Tensor, name: str) -> int:
    """The tensor's device, which has to be the current one."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return device


def _check_on(t: torch.Tensor, name: str, dtype, shape, device: int) -> None:
    """_check_tensor, and that the tensor is on `device`."""
    if t.get_device() == device and t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return
    _check_tensor(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, which is not the current device")


def _check_table(t: torch.Tensor, name: str, rows: Optional[int], device: int) -> None:
    shape = t.shape
    if (t.get_device() == device and t.dtype == torch.int32 and len(shape) == (1 if rows is None else 2) and
            shape[-1] > 0 and (rows is None or shape[0] == rows) and (shape[-1] == 1 or t.stride()[-1] == 1)):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.dim() != (1 if rows is None else 2) or (rows is not None and shape[0] != rows) or shape[-1] < 1:
        raise ValueError(f"{name} must have shape {'(width,)' if rows is None else f'({rows}, width)'}, "
                         f"got {tuple(shape)}")
    if shape[-1] > 1 and t.stride()[-1] != 1:
        raise ValueError(f"{name}: the entries of a row must be contiguous")
    raise ValueError(f"{name} is on {t.device}, which is not the current device")


def _check_workspace(workspace: torch.Tensor, device: int) -> None:
    if workspace.get_device() != device:
        raise ValueError(f"workspace is on {workspace.device}, which is not the current device")


def _check_paged(plan, q, pages, seqlens, block_table, out, lse, sinks, workspace, d_key, d_value, page_row,
                 dtype=torch.bfloat16):
    """Checks what the paged decodes share; the current device's index."""
    device, B, Sq, H = _device_of(q, "q"), plan.B, plan.Sq, plan.H
    _check_on(q, "q", torch.bfloat16, (B, Sq, H, d_key), device)
    for name, p in pages:
        _check_on(p, name, dtype, (p.shape[0], plan.page_size, *page_row), device)
    _check_on(seqlens, "seqlens", torch.int32, (B,), device)
    _check_table(block_table, "block_table", B, device)
    _check_on(out, "out", torch.bfloat16, (B, Sq, H, d_value), device)
    _check_on(lse, "lse", torch.float32, (B, Sq, H), device)
    if sinks is not None:
        _check_on(sinks, "sinks", torch.float32, (H,), device)
    _check_workspace(workspace, device)
    return device


def mla_decode_run_paged(plan: mla_plan, q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                         seqlens: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse: torch.Tensor,
                         workspace: torch.Tensor, sinks: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue one decode over a paged cache: kv_pages bf16 [pages, page_size,
    576], block_table int32 [B, width] (rows may be strided), seqlens the
    lengths with the query tokens' own keys."""
    device = _check_paged(plan, q, (("kv_pages", kv_pages),), seqlens, block_table, out, lse, sinks, workspace,
                          D_QK, D_V, (D_QK,))
    rc = load_library().mla_decode_run_paged(ctypes.byref(plan), q.data_ptr(), kv_pages.data_ptr(), kv_pages.shape[0],
                                             block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                                             seqlens.data_ptr(), float(softmax_scale),
                                             sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                             lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                             _stream_on(device, stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_paged")


def mla_decode_run_paged_fp8(plan: mla_plan, q: torch.Tensor, kv_pages: torch.Tensor, kv_scale: float,
                             block_table: torch.Tensor, seqlens: torch.Tensor, softmax_scale: float,
                             out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                             sinks: Optional[torch.Tensor] = None, stream=None) -> None:
    """mla_decode_run_paged over pages of E4M3 codes (torch.uint8 or
    torch.float8_e4m3fn) that stand for code * kv_scale."""
    pages = _fp8_codes(kv_pages)
    device = _check_paged(plan, q, (("kv_pages", pages),), seqlens, block_table, out, lse, sinks, workspace,
                          D_QK, D_V, (D_QK,), torch.uint8)
    rc = load_library().mla_decode_run_paged_fp8(ctypes.byref(plan), q.data_ptr(), pages.data_ptr(), pages.shape[0],
                                                 float(kv_scale), block_table.data_ptr(), block_table.stride(0),
                                                 block_table.shape[1], seqlens.data_ptr(), float(softmax_scale),
                                                 sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                                 lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                                 _stream_on(device, stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_paged_fp8")


def mha_decode_run_paged(plan: mla_plan, q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         block_table: torch.Tensor, seqlens: torch.Tensor, softmax_scale: float, out: torch.Tensor,
                         lse: torch.Tensor, workspace: torch.Tensor, sinks: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Enqueue one MHA decode over key and value pages bf16 [pages, page_size, Hkv, 128]."""
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    device = _check_paged(plan, q, (("k_pages", k_pages), ("v_pages", v_pages)), seqlens, block_table, out, lse,
                          sinks, workspace, MHA_D, MHA_D, (plan.Hkv, MHA_D))
    rc = load_library().mha_decode_run_paged(ctypes.byref(plan), q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                             k_pages.shape[0], block_table.data_ptr(), block_table.stride(0),
                                             block_table.shape[1], seqlens.data_ptr(), float(softmax_scale),
                                             sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                             lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                             _stream_on(device, stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mha_decode_run_paged")


def mla_decode_run_prefix(plan: mla_plan, q: torch.Tensor, kv_pages: torch.Tensor, prefix_table: torch.Tensor,
                          prefix_len: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                          softmax_scale: float, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                          sinks: Optional[torch.Tensor] = None, stream=None) -> None:
    """Enqueue one decode of a batch with a shared prefix: prefix_table int32
    [width] the prefix's pages, prefix_len int32 [1] on the device, seqlens the
    sequences' own keys (the query tokens' among them), found in block_table."""
    device = _check_paged(plan, q, (("kv_pages", kv_pages),), seqlens, block_table, out, lse, sinks, workspace,
                          D_QK, D_V, (D_QK,))
    _check_table(prefix_table, "prefix_table", None, device)
    _check_on(prefix_len, "prefix_len", torch.int32, (1,), device)
    rc = load_library().mla_decode_run_prefix(ctypes.byref(plan), q.data_ptr(), kv_pages.data_ptr(), kv_pages.shape[0],
                                              prefix_table.data_ptr(), prefix_table.shape[0], prefix_len.data_ptr(),
                                              block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
                                              seqlens.data_ptr(), float(softmax_scale),
                                              sinks.data_ptr() if sinks is not None else None, out.data_ptr(),
                                              lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                              _stream_on(device, stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_decode_run_prefix")


def rope_table(num_positions: int, dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """The rotation table of the append calls: fp32 [num_positions, dim], row p
    the cosines, then the sines, of p * base^(-2i/dim), computed in 64 bits."""
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    angle = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


_FLT_MAX = torch.finfo(torch.float32).max
_APPEND = struct.Struct("=10iq10Q8qQfi")  # the fields of mla_append, in order


def _rows(t: torch.Tensor, name: str, shape, device: int) -> Tuple[int, int]:
    """Checks bf16 rows [T, (heads,) width] of any strides but the last; their (token, head) element strides, 0 where
    there is one token or head (or no head axis)."""
    stride = t.stride()
    if not (t.get_device() == device and t.dtype == torch.bfloat16 and t.shape == shape and stride[-1] == 1):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if stride[-1] != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return (stride[0] if shape[0] > 1 else 0), (stride[1] if len(shape) == 3 and shape[1] > 1 else 0)


def _query_rows(q_in, q_out, in_name, out_name, T, width, out_width, device):
    """Heads of the queries to rotate (0: none), and the strides of their rows."""
    if q_in is None and q_out is None:
        return 0, (0, 0), (0, 0)
    if q_in is None or q_out is None:
        raise ValueError("rotated queries need both their input and their output")
    H = q_in.shape[1] if q_in.dim() == 3 else -1
    in_strides = _rows(q_in, in_name, (T, H, width), device)
    out_strides = _rows(q_out, out_name, (T, H, out_width), device)
    if (T > 1 and out_strides[0] == 0) or (H > 1 and out_strides[1] == 0):  # (others that overlap: the library)
        raise ValueError("the rotated queries' rows must not share memory")
    return H, in_strides, out_strides


def _append(name, device, T, H, Hkv, k, v, cos_sin, rot, k_pages, v_pages, block_table, seqlens, cu_tokens, q_in, q_out,
            q_out_offset, strides, kv_scale, interleaved, workspace, stream, prefix_len=None):
    B = seqlens.shape[0]
    _check_on(seqlens, "seqlens", torch.int32, (B,), device)
    _check_table(block_table, "block_table", B, device)
    positions = cos_sin.shape[0]
    _check_on(cos_sin, "cos_sin", torch.float32, (positions, rot), device)
    if cu_tokens is not None:
        _check_on(cu_tokens, "cu_tokens", torch.int32, (B + 1,), device)
    if prefix_len is not None:
        _check_on(prefix_len, "prefix_len", torch.int32, (1,), device)
    if workspace is not None:
        _check_workspace(workspace, device)
        if workspace.data_ptr() == 0 or workspace.nbytes < 256:
            raise ValueError("workspace must be a decode plan's workspace")
    pages, page_size = k_pages.shape[0], k_pages.shape[1]
    args = _APPEND.pack(
        B, T, H, Hkv, rot, 1 if interleaved else 0, positions, page_size, pages, block_table.shape[1],
        block_table.stride()[0], cu_tokens.data_ptr() if cu_tokens is not None else 0, seqlens.data_ptr(),
        block_table.data_ptr(), cos_sin.data_ptr(), k.data_ptr(), v.data_ptr(), q_in.data_ptr() if H else 0,
        q_out.data_ptr() + q_out_offset if H else 0, k_pages.data_ptr(),
        v_pages.data_ptr() if v_pages is not None else 0, *strides,
        workspace.data_ptr() if workspace is not None else 0, kv_scale, 0)
    entry = getattr(_lib or load_library(), name)
    rc = (entry(args, _stream_on(device, stream)) if prefix_len is None else
          entry(args, prefix_len.data_ptr(), _stream_on(device, stream)))
    if rc != MLA_OK:
        raise MlaError(rc, name)


def _paged_shape(pages: torch.Tensor, *row) -> Tuple[int, ...]:
    """(pages, page_size, *row), with the first two those of the tensor."""
    shape = pages.shape
    return (shape[0], shape[1], *row) if len(shape) > 1 else row


def mla_cache_append(latent: torch.Tensor, k_rope: torch.Tensor, cos_sin: torch.Tensor, kv_pages: torch.Tensor,
                     block_table: torch.Tensor, seqlens: torch.Tensor, cu_tokens: Optional[torch.Tensor] = None,
                     q_rope: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                     kv_scale: Optional[float] = None, interleaved: bool = True,
                     workspace: Optional[torch.Tensor] = None, stream=None,
                     prefix_len: Optional[torch.Tensor] = None) -> None:
    """Append T new tokens to a latent cache: latent bf16 [T, 512] and the
    rotated k_rope bf16 [T, 64] become cache rows of kv_pages [pages, page_size,
    576] (bf16, or E4M3 codes of row / kv_scale), and the rotated q_rope bf16
    [T, H, 64] becomes columns 512.. of q [T, H, 576].

    cos_sin: fp32 [positions, 64] (rope_table).  seqlens int32 [B]: lengths with
    the new tokens; cu_tokens int32 [B + 1]: where each sequence's tokens start
    (None: T / B tokens each).  With a decode workspace, tokens without a
    position or page are reported by mla_decode_check.  A contiguous cache
    [B, L_max, 576] is a paged one with block_table[b] = [b].

    Behind a shared prefix (mla_decode_run_prefix), seqlens and block_table are
    the sequences' own and prefix_len int32 [1] is the decode's: rows and queries
    then turn by the angles of their positions behind the prefix."""
    device, T = _device_of(latent, "latent"), latent.shape[0]
    k_strides = _rows(latent, "latent", (T, D_V), device)
    v_strides = _rows(k_rope, "k_rope", (T, D_QK - D_V), device)
    fp8 = kv_pages.dtype in (torch.uint8, torch.float8_e4m3fn)
    if fp8 != (kv_scale is not None):
        raise ValueError("kv_scale goes with a cache of E4M3 codes (torch.uint8 or torch.float8_e4m3fn)")
    if fp8 and not 2.0 ** -149 <= kv_scale <= _FLT_MAX:  # 0 in fp32 would ask for bf16 rows
        raise ValueError("kv_scale must be positive and finite in fp32")
    _check_on(kv_pages, "kv_pages", kv_pages.dtype if fp8 else torch.bfloat16, _paged_shape(kv_pages, D_QK), device)
    H, in_strides, out_strides = _query_rows(q_rope, q, "q_rope", "q", T, D_QK - D_V, D_QK, device)
    _append("mla_cache_append" if prefix_len is None else "mla_cache_append_prefix", device, T, H, 1, latent, k_rope,
            cos_sin, D_QK - D_V, kv_pages, None, block_table, seqlens, cu_tokens, q_rope, q, 2 * D_V,
            (*k_strides, *v_strides, *in_strides, *out_strides), float(kv_scale) if fp8 else 0.0, interleaved, workspace,
            stream, prefix_len)


def mha_cache_append(k: torch.Tensor, v: torch.Tensor, cos_sin: torch.Tensor, k_pages: torch.Tensor,
                     v_pages: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor,
                     cu_tokens: Optional[torch.Tensor] = None, q_in: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, interleaved: bool = False,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Append T new tokens' keys (rotated) and values, bf16 [T, Hkv, 128], to
    k_pages and v_pages [pages, page_size, Hkv, 128], and rotate the queries
    q_in [T, H, 128] into q_out (which may be q_in).  cos_sin: fp32 [positions,
    n], n a multiple of 16 up to 128: the first n columns turn, the rest is
    copied.  Other arguments as mla_cache_append."""
    device, T, Hkv = _device_of(k, "k"), k.shape[0], k.shape[1] if k.dim() == 3 else -1
    k_strides = _rows(k, "k", (T, Hkv, MHA_D), device)
    v_strides = _rows(v, "v", (T, Hkv, MHA_D), device)
    _check_on(k_pages, "k_pages", torch.bfloat16, _paged_shape(k_pages, Hkv, MHA_D), device)
    _check_on(v_pages, "v_pages", torch.bfloat16, k_pages.shape, device)
    if cos_sin.dim() != 2:
        raise ValueError(f"cos_sin must have shape (positions, rotated columns), got {tuple(cos_sin.shape)}")
    H, in_strides, out_strides = _query_rows(q_in, q_out, "q_in", "q_out", T, MHA_D, MHA_D, device)
    _append("mha_cache_append", device, T, H, Hkv, k, v, cos_sin, cos_sin.shape[1], k_pages, v_pages, block_table,
            seqlens, cu_tokens, q_in, q_out, 0, (*k_strides, *v_strides, *in_strides, *out_strides), 0.0, interleaved,
            workspace, stream)

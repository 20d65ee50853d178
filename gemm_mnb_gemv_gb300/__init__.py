"""Python binding of libmnb (block-quantized INT4 MatMulNBits GEMV/GEMM for sm_103a).

Argument marshalling only: every entry point forwards raw device pointers, sizes and
the current CUDA stream to the C ABI declared in ``include/mnb.h``; all arithmetic runs
in the library's CUDA kernels.  PyTorch supplies device memory and streams.  When an
output tensor is not passed, the binding allocates it with torch before the call (pass
``out=`` to keep a call free of allocations, e.g. under CUDA-graph capture).

The names match the C entry points: ``mnb_dequant``, ``mnb_repacked_bytes``,
``mnb_repack``, ``mnb_gemv``, ``mnb_workspace_bytes``, ``mnb_gemm``,
``mnb_gemm_bias``, ``mnb_gemv_gate_up_swiglu``, ``mnb_workspace_bytes_f32``, ``mnb_gemm_f32``,
``mnb_dequant_gidx``,
``mnb_act_order_plan``, ``mnb_act_order_prepare``, ``mnb_act_order_gather``,
``mnb_act_order_workspace_bytes``, ``mnb_gemm_act_order``, ``mnb_gemm_act_order_noalloc``,
``mnb_kv4_cache_bytes``, ``mnb_kv4_append``, ``mnb_kv4_read``, ``mnb_kv4_attention_workspace_bytes``,
``mnb_kv4_attention`` (with ``MnbKv4Cache``, the handle of a cache, and ``mnb_kv4_cache_alloc``),
``mnb_lora_workspace_bytes``, ``mnb_lora`` (with ``MnbLoraPool``, the handle of a layer's adapters), ``mnb_softmax_workspace_bytes``,
``mnb_softmax``, ``mnb_verify_workspace_bytes``, ``mnb_verify``,
``mnb_set_programmatic_launch``,
``mnb_check_device_status``,
``mnb_last_error``,
``mnb_last_variant``, ``mnb_version``.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmnb.so")

MNB_OK, MNB_ERR_INVALID_ARG, MNB_ERR_UNSUPPORTED, MNB_ERR_MISALIGNED = 0, 1, 2, 3
MNB_ERR_CAPTURE, MNB_ERR_CUDA, MNB_ERR_TIMEOUT = 4, 5, 6
MNB_F16, MNB_F32 = 0, 1
STATUS_NAMES = {0: "MNB_OK", 1: "MNB_ERR_INVALID_ARG", 2: "MNB_ERR_UNSUPPORTED",
                3: "MNB_ERR_MISALIGNED", 4: "MNB_ERR_CAPTURE", 5: "MNB_ERR_CUDA",
                6: "MNB_ERR_TIMEOUT"}


class MnbError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class MnbWeight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("scales_dtype", ctypes.c_int32), ("zero_points", ctypes.c_void_p)]


class MnbKv4CacheArg(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32)]


class MnbRope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class MnbLoraPoolArg(ctypes.Structure):
    _fields_ = [("down", ctypes.c_void_p), ("up", ctypes.c_void_p), ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("count", ctypes.c_int32), ("max_rank", ctypes.c_int32)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libmnb.so (built in-tree by ``__graft_entry__.build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m gemm_mnb_gemv_gb300._build` "
                          "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    c_int, c_size, vp, i64 = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int64
    sigs = {
        "mnb_dequant": (c_int, [MnbWeight, c_int, c_int, c_int, vp, vp]),
        "mnb_repacked_bytes": (c_size, [c_int, c_int, c_int]),
        "mnb_repack": (c_int, [vp, c_int, c_int, c_int, vp, vp]),
        "mnb_gemv": (c_int, [vp, MnbWeight, c_int, c_int, c_int, vp, vp]),
        "mnb_workspace_bytes": (c_size, [c_int, c_int, c_int, c_int]),
        "mnb_gemm": (c_int, [vp, c_int, MnbWeight, vp, c_int, c_int, c_int, vp, c_size, vp, vp]),
        "mnb_gemv_gate_up_swiglu": (c_int, [vp, MnbWeight, MnbWeight, c_int, c_int, c_int, vp, vp]),
        "mnb_gemm_bias": (c_int, [vp, c_int, MnbWeight, vp, c_int, c_int, c_int, vp, c_int, vp, c_size, vp, vp]),
        "mnb_workspace_bytes_f32": (c_size, [c_int, c_int, c_int, c_int]),
        "mnb_gemm_f32": (c_int, [vp, c_int, MnbWeight, vp, c_int, c_int, c_int, vp, vp, c_size, vp, vp]),
        "mnb_dequant_gidx": (c_int, [MnbWeight, vp, c_int, c_int, c_int, vp, vp]),
        "mnb_act_order_plan": (c_int, [vp, c_int, c_int, vp, vp, vp]),
        "mnb_act_order_prepare": (c_int, [MnbWeight, c_int, c_int, c_int, vp, vp, c_int, vp, vp, vp, vp]),
        "mnb_act_order_gather": (c_int, [vp, c_int, c_int, vp, c_int, vp, vp]),
        "mnb_act_order_workspace_bytes": (c_size, [c_int, c_int]),
        "mnb_gemm_act_order": (c_int, [vp, c_int, MnbWeight, vp, vp, c_int, c_int, c_int, c_int, vp, c_int, vp,
                                       c_size, vp, vp]),
        "mnb_gemm_act_order_noalloc": (c_int, [vp, c_int, MnbWeight, vp, vp, c_int, c_int, c_int, c_int, vp,
                                               c_int, vp, vp]),
        "mnb_kv4_cache_bytes": (c_size, [c_int, c_int, c_int, c_int, c_int]),
        "mnb_kv4_append": (c_int, [vp, vp, vp, c_int, c_int, c_int, i64, i64, i64, vp, MnbRope, vp, MnbKv4CacheArg,
                                   vp, vp]),
        "mnb_kv4_read": (c_int, [MnbKv4CacheArg, vp, c_int, c_int, vp, vp, vp]),
        "mnb_kv4_attention_workspace_bytes": (c_size, [c_int, c_int, c_int, c_int, c_int, c_int]),
        "mnb_kv4_attention": (c_int, [vp, c_int, c_int, c_int, i64, MnbKv4CacheArg, vp, vp, vp, c_int, c_int,
                                      ctypes.c_float, c_int, c_int, vp, c_size, vp, vp, vp]),
        "mnb_lora_workspace_bytes": (c_size, [c_int]),
        "mnb_lora": (c_int, [vp, c_int, c_int, c_int, i64, MnbLoraPoolArg, vp, vp, i64, c_int, vp, c_size, vp, i64, vp]),
        "mnb_softmax_workspace_bytes": (c_size, [c_int, c_int]),
        "mnb_softmax": (c_int, [vp, c_int, c_int, c_int, i64, vp, vp, c_size, vp, vp]),
        "mnb_verify_workspace_bytes": (c_size, [c_int, c_int]),
        "mnb_verify": (c_int, [vp, i64, vp, i64, vp, vp, vp, vp, c_int, c_int, c_int, vp, c_size, vp, vp, vp]),
        "mnb_set_programmatic_launch": (None, [c_int]),
        "mnb_check_device_status": (c_int, []),
        "mnb_selftest_wait_timeout": (c_int, [ctypes.c_uint, vp]),
        "mnb_last_error": (ctypes.c_char_p, []),
        "mnb_last_variant": (ctypes.c_char_p, []),
        "mnb_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_dev(name, t, dtype=None):
    torch = _torch()
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _weight(packed, scales, zero_points) -> MnbWeight:
    torch = _torch()
    _check_dev("packed", packed, torch.uint8)
    _check_dev("scales", scales)
    _check_dev("zero_points", zero_points, torch.uint8)
    if scales.dtype == torch.float16:
        sd = MNB_F16
    elif scales.dtype == torch.float32:
        sd = MNB_F32
    else:
        raise TypeError("scales must be float16 or float32")
    return MnbWeight(packed.data_ptr(), scales.data_ptr(), sd,
                     zero_points.data_ptr() if zero_points is not None else None)


def _raise(status: int):
    if status != MNB_OK:
        raise MnbError(status, load_library().mnb_last_error().decode())


def mnb_last_error() -> str:
    return load_library().mnb_last_error().decode()


def mnb_last_variant() -> str:
    return load_library().mnb_last_variant().decode()


def mnb_version() -> str:
    return load_library().mnb_version().decode()


def mnb_set_programmatic_launch(enable: bool) -> None:
    load_library().mnb_set_programmatic_launch(1 if enable else 0)


def mnb_check_device_status() -> None:
    """Raises MnbError(MNB_ERR_TIMEOUT) if a device-side bounded wait gave up since the last check."""
    _raise(load_library().mnb_check_device_status())


def mnb_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launches the bounded-wait self-test kernel (its wait gives up after ``limit_us``)."""
    _raise(load_library().mnb_selftest_wait_timeout(limit_us, _stream_handle(stream)))


def mnb_repacked_bytes(K: int, N: int, block_size: int) -> int:
    return int(load_library().mnb_repacked_bytes(K, N, block_size))


def mnb_workspace_bytes(M: int, K: int, N: int, block_size: int) -> int:
    return int(load_library().mnb_workspace_bytes(M, K, N, block_size))


def mnb_dequant(packed, scales, zero_points, K: int, N: int, block_size: int, out=None, stream=None):
    """fp32 ``[K, N]`` dequantised weight (``out[k, n] = (code - zp) * scale``)."""
    torch = _torch()
    lib = load_library()
    w = _weight(packed, scales, zero_points)
    if out is None:
        out = torch.empty((K, N), dtype=torch.float32, device=packed.device)
    _check_dev("out", out, torch.float32)
    _raise(lib.mnb_dequant(w, K, N, block_size, _ptr(out), _stream_handle(stream)))
    return out


def mnb_repack(packed, K: int, N: int, block_size: int, out=None, stream=None):
    """uint8 repacked tensor-core operand (``mnb_repacked_bytes(K, N, bs)`` bytes)."""
    torch = _torch()
    lib = load_library()
    _check_dev("packed", packed, torch.uint8)
    if out is None:
        nbytes = mnb_repacked_bytes(K, N, block_size)
        if nbytes == 0:
            raise MnbError(MNB_ERR_INVALID_ARG, "mnb_repack: invalid shape")
        out = torch.empty(nbytes, dtype=torch.uint8, device=packed.device)
    _check_dev("out", out, torch.uint8)
    _raise(lib.mnb_repack(_ptr(packed), K, N, block_size, _ptr(out), _stream_handle(stream)))
    return out


def mnb_gemv(A, packed, scales, zero_points, K: int, N: int, block_size: int, out=None, stream=None):
    """fp16 ``[N]`` = A (fp16 ``[K]``) times the dequantised weight."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    w = _weight(packed, scales, zero_points)
    if out is None:
        out = torch.empty(N, dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemv(_ptr(A), w, K, N, block_size, _ptr(out), _stream_handle(stream)))
    return out


def mnb_gemm(A, packed, scales, zero_points, K: int, N: int, block_size: int, repacked=None,
             workspace=None, out=None, stream=None):
    """fp16 ``[M, N]`` = A (fp16 ``[M, K]``) times the dequantised weight."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    M = A.numel() // K
    w = _weight(packed, scales, zero_points)
    _check_dev("repacked", repacked, torch.uint8)
    need = mnb_workspace_bytes(M, K, N, block_size)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemm(_ptr(A), M, w, _ptr(repacked), K, N, block_size, _ptr(workspace), ws_bytes,
                        _ptr(out), _stream_handle(stream)))
    return out


MNB_BIAS_NONE, MNB_BIAS_FUSED, MNB_BIAS_AFTER_ROUND = 0, 1, 2


def mnb_gemm_bias(A, packed, scales, zero_points, K: int, N: int, block_size: int, bias, bias_mode: int,
                  repacked=None, workspace=None, out=None, stream=None):
    """``mnb_gemm`` plus a fp16 ``[N]`` bias: mode 1 = fp16(acc + b), mode 2 = fp16(fp16(acc) + b)."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    _check_dev("bias", bias, torch.float16)
    M = A.numel() // K
    w = _weight(packed, scales, zero_points)
    _check_dev("repacked", repacked, torch.uint8)
    need = mnb_workspace_bytes(M, K, N, block_size)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=A.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemm_bias(_ptr(A), M, w, _ptr(repacked), K, N, block_size, _ptr(bias), bias_mode,
                             _ptr(workspace), ws_bytes, _ptr(out), _stream_handle(stream)))
    return out


def mnb_gemv_gate_up_swiglu(A, gate, up, K: int, N: int, block_size: int, out=None, stream=None):
    """fp16 ``[N]`` = silu(A . gate^T) * (A . up^T); gate/up are (packed, scales, zero_points)."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    wg = _weight(*gate)
    wu = _weight(*up)
    if out is None:
        out = torch.empty(N, dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemv_gate_up_swiglu(_ptr(A), wg, wu, K, N, block_size, _ptr(out),
                                       _stream_handle(stream)))
    return out


# ---------------------------------------------------------------------------
# fp32 activations
# ---------------------------------------------------------------------------


def mnb_workspace_bytes_f32(M: int, K: int, N: int, block_size: int) -> int:
    return int(load_library().mnb_workspace_bytes_f32(M, K, N, block_size))


def mnb_gemm_f32(A, packed, scales, zero_points, K: int, N: int, block_size: int, repacked=None, bias=None,
                 workspace=None, out=None, stream=None):
    """fp32 ``[M, N]`` = A (fp32 ``[M, K]``) times the dequantised weight (+ fp32 bias ``[N]``)."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float32)
    _check_dev("bias", bias, torch.float32)
    _check_dev("repacked", repacked, torch.uint8)
    M = A.numel() // K
    w = _weight(packed, scales, zero_points)
    need = mnb_workspace_bytes_f32(M, K, N, block_size)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=A.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _check_dev("out", out, torch.float32)
    _raise(lib.mnb_gemm_f32(_ptr(A), M, w, _ptr(repacked), K, N, block_size, _ptr(bias), _ptr(workspace),
                            ws_bytes, _ptr(out), _stream_handle(stream)))
    return out


# ---------------------------------------------------------------------------
# Act-order (g_idx) weights
# ---------------------------------------------------------------------------


def mnb_dequant_gidx(packed, scales, zero_points, g_idx, K: int, N: int, block_size: int, out=None,
                     stream=None):
    """fp32 ``[K, N]`` with the scale and zero point of group ``g_idx[k]`` at column ``k``."""
    torch = _torch()
    lib = load_library()
    w = _weight(packed, scales, zero_points)
    _check_dev("g_idx", g_idx, torch.int32)
    if out is None:
        out = torch.empty((K, N), dtype=torch.float32, device=packed.device)
    _check_dev("out", out, torch.float32)
    _raise(lib.mnb_dequant_gidx(w, _ptr(g_idx), K, N, block_size, _ptr(out), _stream_handle(stream)))
    return out


def mnb_act_order_plan(g_idx, K: int, block_size: int):
    """Host-only: ``(K_prepared, perm, block_group)`` as int / int32 numpy arrays.

    ``g_idx`` is any host int sequence of length ``K`` (numpy array, list or CPU tensor).
    """
    import numpy as np
    lib = load_library()
    g = np.ascontiguousarray(np.asarray(g_idx), dtype=np.int32).reshape(-1)
    if g.size != K:
        raise MnbError(MNB_ERR_INVALID_ARG, f"mnb_act_order_plan: g_idx has {g.size} entries, expected {K}")
    kp = ctypes.c_int32(0)
    gp = g.ctypes.data_as(ctypes.c_void_p)
    _raise(lib.mnb_act_order_plan(gp, K, block_size, ctypes.byref(kp), None, None))
    perm = np.empty(max(kp.value, 1), dtype=np.int32)
    bg = np.empty(max(kp.value // block_size, 1), dtype=np.int32)
    _raise(lib.mnb_act_order_plan(gp, K, block_size, ctypes.byref(kp), perm.ctypes.data_as(ctypes.c_void_p),
                                  bg.ctypes.data_as(ctypes.c_void_p)))
    return kp.value, perm[:kp.value], bg[:kp.value // block_size]


def mnb_act_order_prepare(packed, scales, zero_points, K: int, N: int, block_size: int, perm, block_group,
                          K_prepared: int, packed_out=None, scales_out=None, zero_points_out=None, stream=None):
    """Prepared block weight ``(packed', scales', zero_points')`` (device tensors)."""
    torch = _torch()
    lib = load_library()
    w = _weight(packed, scales, zero_points)
    _check_dev("perm", perm, torch.int32)
    _check_dev("block_group", block_group, torch.int32)
    Gp = K_prepared // block_size
    dev = packed.device
    if packed_out is None:
        packed_out = torch.empty((N, K_prepared // 2), dtype=torch.uint8, device=dev)
    if scales_out is None:
        scales_out = torch.empty((N, Gp), dtype=scales.dtype, device=dev)
    if zero_points is not None and zero_points_out is None:
        zero_points_out = torch.empty((N, (Gp + 1) // 2), dtype=torch.uint8, device=dev)
    if zero_points is None:
        zero_points_out = None
    _raise(lib.mnb_act_order_prepare(w, K, N, block_size, _ptr(perm), _ptr(block_group), K_prepared,
                                     _ptr(packed_out), _ptr(scales_out), _ptr(zero_points_out),
                                     _stream_handle(stream)))
    return packed_out, scales_out, zero_points_out


def mnb_act_order_gather(A, K: int, perm, K_prepared: int, out=None, stream=None):
    """fp16 ``[M, K']`` with ``out[m, k'] = A[m, perm[k']]`` (0 where ``perm = -1``)."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    _check_dev("perm", perm, torch.int32)
    M = A.numel() // K
    if out is None:
        out = torch.empty((M, K_prepared), dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_act_order_gather(_ptr(A), M, K, _ptr(perm), K_prepared, _ptr(out), _stream_handle(stream)))
    return out


def mnb_act_order_workspace_bytes(M: int, K_prepared: int) -> int:
    return int(load_library().mnb_act_order_workspace_bytes(M, K_prepared))


def mnb_gemm_act_order(A, packed, scales, zero_points, perm, K: int, K_prepared: int, N: int, block_size: int,
                       repacked=None, bias=None, bias_mode: int = MNB_BIAS_NONE, workspace=None, out=None,
                       stream=None):
    """fp16 ``[M, N]`` for an act-order weight; ``packed/scales/zero_points/repacked`` are the prepared ones."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    _check_dev("perm", perm, torch.int32)
    _check_dev("bias", bias, torch.float16)
    _check_dev("repacked", repacked, torch.uint8)
    M = A.numel() // K
    w = _weight(packed, scales, zero_points)
    if workspace is None:
        # the gathered activation, then room for the small-M kernel's K-slice partials
        head = (mnb_act_order_workspace_bytes(M, K_prepared) + 15) // 16 * 16
        workspace = torch.empty(head + mnb_workspace_bytes(M, K_prepared, N, block_size), dtype=torch.uint8,
                                device=A.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemm_act_order(_ptr(A), M, w, _ptr(repacked), _ptr(perm), K, K_prepared, N, block_size,
                                  _ptr(bias), bias_mode, _ptr(workspace), ws_bytes, _ptr(out),
                                  _stream_handle(stream)))
    return out


def mnb_gemm_act_order_noalloc(A, packed, scales, zero_points, perm, K: int, K_prepared: int, N: int,
                               block_size: int, repacked=None, bias=None, bias_mode: int = MNB_BIAS_NONE, out=None,
                               stream=None):
    """``mnb_gemm_act_order`` with the library's static scratch (M * K' * 2 <= 8 MiB) instead of a
    workspace; pass ``out`` to keep the call free of allocations."""
    torch = _torch()
    lib = load_library()
    _check_dev("A", A, torch.float16)
    _check_dev("perm", perm, torch.int32)
    _check_dev("bias", bias, torch.float16)
    _check_dev("repacked", repacked, torch.uint8)
    M = A.numel() // K
    w = _weight(packed, scales, zero_points)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    _check_dev("out", out, torch.float16)
    _raise(lib.mnb_gemm_act_order_noalloc(_ptr(A), M, w, _ptr(repacked), _ptr(perm), K, K_prepared, N,
                                          block_size, _ptr(bias), bias_mode, _ptr(out), _stream_handle(stream)))
    return out


# ---------------------------------------------------------------------------
# Paged 4-bit key/value cache and attention
# ---------------------------------------------------------------------------


_INT_MAX = 2 ** 31 - 1


def _nearest(n: int) -> int:
    """``n``, or the C int nearest to it: ctypes would hand on its low 32 bits."""
    return max(-_INT_MAX, min(n, _INT_MAX))


def _size(n: int) -> int:
    """``n`` as a C int, -1 (which every entry point refuses) where it is none."""
    return n if -_INT_MAX <= n <= _INT_MAX else -1


def mnb_kv4_cache_bytes(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int) -> int:
    num_pages, page_size, kv_heads, head_dim, group_size = map(_size, (num_pages, page_size, kv_heads, head_dim, group_size))
    return int(load_library().mnb_kv4_cache_bytes(num_pages, page_size, kv_heads, head_dim, group_size))


class MnbKv4Cache:
    """Handle of a paged 4-bit key/value cache: ``pages`` is uint8 ``[num_pages, kv_heads, record bytes]``."""

    def __init__(self, pages, page_size: int, head_dim: int, group_size: int):
        torch = _torch()
        _check_dev("pages", pages, torch.uint8)
        if pages.dim() != 3:
            raise ValueError("pages must be [num_pages, kv_heads, record bytes]")
        num_pages, kv_heads, record = pages.shape
        need = mnb_kv4_cache_bytes(num_pages, page_size, kv_heads, head_dim, group_size)
        if need == 0:
            raise MnbError(MNB_ERR_INVALID_ARG, f"MnbKv4Cache: num_pages={num_pages} page_size={page_size} "
                           f"kv_heads={kv_heads} head_dim={head_dim} group_size={group_size}")
        if need != num_pages * kv_heads * record:
            raise ValueError(f"pages has records of {record} bytes, {need // (num_pages * kv_heads)} needed")
        self.pages, self.page_size, self.head_dim, self.group_size = pages, page_size, head_dim, group_size
        self.num_pages, self.kv_heads, self.device = num_pages, kv_heads, pages.get_device()
        # what tensors and the current device are compared with in each call: 1 to 2 us, for nothing where there is one GPU
        self.guard = self.device if _gpu_count() > 1 else None
        self.workspace_bytes = {}  # by (tokens, batch, q_heads, dtype)
        self.arg = MnbKv4CacheArg(pages.data_ptr(), num_pages, page_size, kv_heads, head_dim, group_size)


def mnb_kv4_cache_alloc(num_pages: int, page_size: int, kv_heads: int, head_dim: int, group_size: int,
                        device="cuda") -> MnbKv4Cache:
    """A new cache, zeroed (every element reads as 0)."""
    nbytes = mnb_kv4_cache_bytes(num_pages, page_size, kv_heads, head_dim, group_size)
    if nbytes == 0:
        raise MnbError(MNB_ERR_INVALID_ARG, f"mnb_kv4_cache_alloc: num_pages={num_pages} page_size={page_size} "
                       f"kv_heads={kv_heads} head_dim={head_dim} group_size={group_size}")
    torch = _torch()
    pages = torch.zeros((num_pages, kv_heads, nbytes // (num_pages * kv_heads)), dtype=torch.uint8, device=device)
    return MnbKv4Cache(pages, page_size, head_dim, group_size)


_ACT = {}  # torch dtype -> MNB_F16 / MNB_F32, filled on first use


def _act_dtype(name, t):
    if not _ACT:
        torch = _torch()
        _ACT.update({torch.float16: MNB_F16, torch.float32: MNB_F32})
    if t is None:
        raise TypeError(f"{name} must be a CUDA tensor, got None")
    code = _ACT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16 or float32, got {t.dtype}")
    return code


def _raw_stream(device: int, stream):
    """Handle of ``stream``, or of the current stream of the device."""
    if stream is not None:
        if stream.device.index != device:
            raise ValueError(f"stream is of {stream.device}, the cache on cuda:{device}")
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without building a Stream object: 3 us of a call
    return raw(device) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _gpu_count() -> int:
    return _torch().cuda.device_count()


def _current_device() -> int:
    return _torch()._C._cuda_getDevice()


def _call_on(device: int, fn, args) -> int:
    """Calls an entry point, which launches on the current device, with this device as that."""
    with _torch().cuda.device(device):
        return fn(*args)


def _refuse(name, t, dtype, guard):
    """Raises for a tensor that is missing, of another type or elsewhere."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor, got {None if t is None else type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if guard is not None and t.get_device() != guard:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{guard}")


def _token_rows(name, t, heads, D, dtype, guard):
    """Elements between the tokens of ``[T, heads, D]``, whose heads must lie one after the other."""
    if t is None or t.dtype != dtype or not t.is_cuda or guard is not None:
        _refuse(name, t, dtype, guard)
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{name} must be [tokens, {heads}, {D}], got {list(shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError(f"{name}: the heads of a token must lie one after the other")
    return s0 if shape[0] > 1 else heads * D


def _new(shape, dtype, device, stream):
    """A tensor of ``stream``'s own pool (the current stream's when None), so that it outlives the kernels on it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _index(name, t, dtype, shape, guard):
    """Address of a contiguous CUDA tensor of this type and shape."""
    if t is None or t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or guard is not None:
        _refuse(name, t, dtype, guard)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def mnb_kv4_append(cache: MnbKv4Cache, k, v, slots, q=None, positions=None, cos=None, sin=None,
                   interleaved: bool = False, q_out=None, stream=None):
    """Rotates, quantises and stores ``k`` and ``v`` (``[T, kv_heads, head_dim]``) at ``slots``; returns the rotated
    ``q`` (or None).  ``cos`` and ``sin`` are fp32 ``[rows, rot_dim / 2]``, None for no rotation."""
    torch = _torch()
    dt, Hk, D = _act_dtype("k", k), cache.kv_heads, cache.head_dim
    dtype = k.dtype
    dev, guard = cache.device, cache.guard
    ks, vs = _token_rows("k", k, Hk, D, dtype, guard), _token_rows("v", v, Hk, D, dtype, guard)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"v has {v.shape[0]} tokens, k has {T}")
    qs = Hq = 0
    qp = op = None
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T:
            raise ValueError(f"q must be [{T}, q_heads, {D}], got {list(q.shape)}")
        Hq = q.shape[1]
        qs = _token_rows("q", q, Hq, D, dtype, guard)
        if q_out is None:
            q_out = _new((T, Hq, D), dtype, q.device, stream)
        qp, op = q.data_ptr(), _index("q_out", q_out, dtype, (T, Hq, D), guard)
    if cos is None and sin is not None:
        raise TypeError("sin without cos")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError(f"cos must be [rows, rot_dim / 2], got {list(cos.shape)}")
        rows, half = cos.shape
        rope = MnbRope(_index("cos", cos, torch.float32, (rows, half), guard),
                       _index("sin", sin, torch.float32, (rows, half), guard), _nearest(rows), _size(2 * half), 1 if interleaved else 0)
        pp = _index("positions", positions, torch.int32, (T,), guard)
    else:
        rope, pp = MnbRope(None, None, 0, 0, 0), None
    args = (qp, k.data_ptr(), v.data_ptr(), dt, T, Hq, qs, ks, vs, pp, rope, _index("slots", slots, torch.int64, (T,), guard),
            cache.arg, op, _raw_stream(dev, stream))
    fn = load_library().mnb_kv4_append
    st = fn(*args) if guard is None or _current_device() == dev else _call_on(dev, fn, args)
    if st != MNB_OK:
        _raise(st)
    return q_out


def mnb_kv4_read(cache: MnbKv4Cache, slots, dtype=None, k_out=None, v_out=None, stream=None):
    """``(k, v)``, ``[T, kv_heads, head_dim]`` of ``dtype`` (float16 by default): what ``slots`` hold."""
    torch = _torch()
    if slots is None or slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    T = slots.shape[0]
    dev, guard = cache.device, cache.guard
    slots_at = _index("slots", slots, torch.int64, (T,), guard)
    shape = (T, cache.kv_heads, cache.head_dim)
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else torch.float16
    if k_out is None:
        k_out = _new(shape, dtype, slots.device, stream)
    if v_out is None:
        v_out = _new(shape, dtype, slots.device, stream)
    args = (cache.arg, slots_at, T, _act_dtype("k_out", k_out), _index("k_out", k_out, dtype, shape, guard),
            _index("v_out", v_out, dtype, shape, guard), _raw_stream(dev, stream))
    fn = load_library().mnb_kv4_read
    st = fn(*args) if guard is None or _current_device() == dev else _call_on(dev, fn, args)
    if st != MNB_OK:
        _raise(st)
    return k_out, v_out


def mnb_kv4_attention_workspace_bytes(T: int, batch: int, q_heads: int, kv_heads: int, head_dim: int,
                                      dtype: int = MNB_F16) -> int:
    T, batch, q_heads, kv_heads, head_dim, dtype = map(_size, (T, batch, q_heads, kv_heads, head_dim, dtype))
    return int(load_library().mnb_kv4_attention_workspace_bytes(T, batch, q_heads, kv_heads, head_dim, dtype))


_default_workspace = {}  # by device: of the calls on its default stream that want one


def mnb_kv4_attention(q, cache: MnbKv4Cache, q_start, kv_len, page_table, scale: float, causal: bool = True,
                      window: int = 0, workspace=None, out=None, lse=None, stream=None):
    """``[T, q_heads, head_dim]``: attention of ``q`` over the cached keys of ``batch`` sequences.

    ``q_start`` int32 ``[batch + 1]``, ``kv_len`` int32 ``[batch]``, ``page_table`` int32 ``[batch, pages]``.
    Without ``workspace``, calls on the device's default stream share one that is kept (the largest asked for so far, 43 MB
    at most for attention), and calls on other streams allocate theirs. One workspace may serve calls of several threads on one stream.
    """
    torch = _torch()
    if q is None or kv_len is None or page_table is None or q.dim() != 3 or kv_len.dim() != 1 or page_table.dim() != 2:
        raise ValueError("q, kv_len and page_table must be [tokens, q_heads, head_dim], [batch] and [batch, pages], got "
                         + ", ".join("None" if t is None else str(list(t.shape)) for t in (q, kv_len, page_table)))
    T, Hq, D = q.shape
    dtype, dt = q.dtype, _act_dtype("q", q)
    dev, guard = cache.device, cache.guard
    qs = _token_rows("q", q, Hq, cache.head_dim, dtype, guard)
    B = kv_len.shape[0]
    lib = load_library()
    raw_stream = _raw_stream(dev, stream)
    kept = workspace is None and stream is None and raw_stream == 0
    if workspace is None:
        need = cache.workspace_bytes.get((T, B, Hq, dt))
        if need is None:
            need = lib.mnb_kv4_attention_workspace_bytes(T, B, Hq, cache.kv_heads, D, dt)
            if len(cache.workspace_bytes) < 4096:
                cache.workspace_bytes[(T, B, Hq, dt)] = need
        if kept:
            # The default stream is never destroyed, orders all its calls and can't be captured, so one workspace serves
            # them in turn: 16 us a call of one token over 1000 keys against 20 us with one allocated in each.
            workspace = _default_workspace.get(dev)
            if workspace is None or workspace.numel() < need:
                workspace = _default_workspace[dev] = _new(need, torch.uint8, q.device, None)
        else:
            workspace = _new(need, torch.uint8, q.device, stream)
    else:
        _check_dev("workspace", workspace)
        if guard is not None:
            _refuse("workspace", workspace, workspace.dtype, guard)
    if out is None:
        out = _new((T, Hq, D), dtype, q.device, stream)
        op = out.data_ptr()
    else:
        op = _index("out", out, dtype, (T, Hq, D), guard)
    lp = None if lse is None else _index("lse", lse, torch.float32, (T, Hq), guard)
    stride = page_table.shape[1]
    args = (q.data_ptr(), dt, T, Hq, qs, cache.arg, _index("q_start", q_start, torch.int32, (B + 1,), guard),
            _index("kv_len", kv_len, torch.int32, (B,), guard),
            _index("page_table", page_table, torch.int32, (B, stride), guard), B, _size(stride), scale, 1 if causal else 0,
            _nearest(window), workspace.data_ptr(), workspace.nbytes, op, lp, raw_stream)
    fn = lib.mnb_kv4_attention
    st = fn(*args) if guard is None or _current_device() == dev else _call_on(dev, fn, args)
    if st != MNB_OK:
        _raise(st)
    return out


# ---------------------------------------------------------------------------
# What each request of a shared step has of its own: adapters, probabilities, drafted tokens
# ---------------------------------------------------------------------------


# A call's host time is most of a small one (13 us of softmax over 30 rows, whose kernel takes 3): what the checks look at is
# looked at in place, and only what is wrong goes through the functions that say so.

_gpus = None  # asked for once: 1 to 2 us of a call
_raw_stream_of = None  # handle of a device's current stream, without building a Stream object


def _guard_of(dev: int):
    """What tensors and the current device are compared with in each call: None where there is one GPU."""
    global _gpus
    if _gpus is None:
        _gpus = _gpu_count()
    return dev if _gpus > 1 else None


def _on(name, t, dtype, guard):
    """Raises for a tensor that is missing, of another type or on another GPU than the call's."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor, got {None if t is None else type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if guard is not None and t.get_device() != guard:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{guard}")


def _two_dims(name, t, what):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor, got {None if t is None else type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be {what}, got {list(t.shape)}")
    return t.shape


def _matrix(name, t, shape, dtype, guard):
    """Elements between the rows of a CUDA tensor of this type and shape whose rows are contiguous."""
    if getattr(t, "dtype", None) != dtype or not t.is_cuda or guard is not None:
        _on(name, t, dtype, guard)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must lie one after the other")
    return s0 if shape[0] > 1 else shape[1]


def _vector(name, t, dtype, shape, guard):
    """Address of a contiguous CUDA tensor of this type and shape."""
    if getattr(t, "dtype", None) != dtype or not t.is_cuda or guard is not None:
        _on(name, t, dtype, guard)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream_of(dev, stream):
    global _raw_stream_of
    if stream is None:
        if _raw_stream_of is None:
            torch = _torch()
            _raw_stream_of = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                              or (lambda device: torch.cuda.current_stream(device).cuda_stream))
        return _raw_stream_of(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream is of {stream.device}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _room(workspace, need, like, dev, stream, raw_stream, guard):
    """The workspace, or one of ``need`` bytes: the kept one on the default stream, as in the attention, else a new one of the
    stream's pool.  The caller holds it until the launch, so that no other allocation of the call gets its bytes."""
    torch = _torch()
    if workspace is not None:
        _check_dev("workspace", workspace)
        _on("workspace", workspace, workspace.dtype, guard)
        return workspace
    if need == 0:
        return None
    if stream is None and raw_stream == 0:
        workspace = _default_workspace.get(dev)
        if workspace is None or workspace.numel() < need:
            workspace = _default_workspace[dev] = _new(need, torch.uint8, like.device, None)
        return workspace
    return _new(need, torch.uint8, like.device, stream)


_room_bytes = {}  # (entry point, sizes) -> bytes


def _bytes_of(name, *sizes):
    key = (name, sizes)
    need = _room_bytes.get(key)
    if need is None:
        need = getattr(_lib, name)(*map(_size, sizes))
        if len(_room_bytes) < 4096:
            _room_bytes[key] = need
    return need


def _launch(fn, args, dev, guard):
    st = fn(*args) if guard is None or _current_device() == dev else _call_on(dev, fn, args)
    if st != MNB_OK:
        _raise(st)


class MnbLoraPool:
    """Handle of a layer's low-rank adapters: ``down`` fp16 ``[count, max_rank, K]``, ``up`` fp16 ``[count, N, max_rank]``,
    ``ranks`` int32 ``[count]`` (None: all ``max_rank``), ``scales`` fp32 ``[count]`` (None: 1)."""

    def __init__(self, down, up, ranks=None, scales=None):
        torch = _torch()
        for name, t in (("down", down), ("up", up)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a CUDA tensor, got {None if t is None else type(t).__name__}")
        if down.dim() != 3 or up.dim() != 3:
            raise ValueError("down and up must be [count, max_rank, K] and [count, N, max_rank]")
        self.device = down.get_device()
        self.guard = guard = _guard_of(self.device)
        count, max_rank, self.K = down.shape
        self.N = up.shape[1]
        if count < 1 or count > 1 << 20 or max_rank % 8 or not 8 <= max_rank <= 128 or max(self.K, self.N) > _INT_MAX:
            raise MnbError(MNB_ERR_INVALID_ARG, f"MnbLoraPool: count={count} max_rank={max_rank} K={self.K} N={self.N} (count "
                           "1..2^20, max_rank a multiple of 8 in 8..128, K and N below 2^31)")
        load_library()
        self.down, self.up, self.ranks, self.scales = down, up, ranks, scales
        self.arg = MnbLoraPoolArg(
            _vector("down", down, torch.float16, (count, max_rank, self.K), guard),
            _vector("up", up, torch.float16, (count, self.N, max_rank), guard),
            None if ranks is None else _vector("ranks", ranks, torch.int32, (count,), guard),
            None if scales is None else _vector("scales", scales, torch.float32, (count,), guard), count, max_rank)


def mnb_lora_workspace_bytes(M: int) -> int:
    return int(load_library().mnb_lora_workspace_bytes(_size(M)))


def mnb_lora(x, pool: MnbLoraPool, adapter, base=None, workspace=None, out=None, stream=None):
    """``[M, N]`` = ``base`` (None: zeros) + each row's adapter on ``x`` ``[M, K]``; ``adapter`` int32 ``[M]``, -1 for none.
    ``out`` may be ``base``.  A workspace is shared or allocated as in ``mnb_kv4_attention``."""
    torch = _torch_module or _torch()
    if not isinstance(pool, MnbLoraPool):
        raise TypeError(f"pool must be an MnbLoraPool, got {type(pool).__name__}")
    dev, guard, K, N = pool.device, pool.guard, pool.K, pool.N
    if type(x) is not torch.Tensor or not x.is_cuda or x.dim() != 2:
        _two_dims("x", x, f"[M, {K}]")
    M, cols = x.shape
    dtype = x.dtype
    dt = _ACT.get(dtype)
    if dt is None:
        dt = _act_dtype("x", x)
    xs, one = x.stride()
    if cols != K or one != 1 or M < 2 or guard is not None:
        xs = _matrix("x", x, (M, K), dtype, guard)
    shape = (M, N)
    bs, bp = 0, None
    if base is not None:
        bs, bp = _matrix("base", base, shape, dtype, guard), base.data_ptr()
    if out is None:
        out, os_ = x.new_empty(shape) if stream is None else _new(shape, dtype, x.device, stream), N
    else:
        os_ = _matrix("out", out, shape, dtype, guard)
    if type(adapter) is not torch.Tensor or adapter.dtype is not torch.int32 or not adapter.is_cuda or adapter.shape != (M,) or not (
            adapter.is_contiguous()) or guard is not None:
        _vector("adapter", adapter, torch.int32, (M,), guard)
    lib, raw_stream = _lib, _stream_of(dev, stream)
    wp, ws_bytes = None, 0
    if M > 256 or workspace is not None:
        workspace = _room(workspace, _bytes_of("mnb_lora_workspace_bytes", M), x, dev, stream, raw_stream, guard)
        if workspace is not None:
            wp, ws_bytes = workspace.data_ptr(), workspace.nbytes
    st = M if M <= _INT_MAX else -1
    args = (x.data_ptr(), dt, st, K, xs, pool.arg, adapter.data_ptr(), bp, bs, N, wp, ws_bytes, out.data_ptr(), os_, raw_stream)
    if guard is not None:
        _launch(lib.mnb_lora, args, dev, guard)
        return out
    st = lib.mnb_lora(*args)
    if st != MNB_OK:
        _raise(st)
    return out


def mnb_softmax_workspace_bytes(rows: int, V: int) -> int:
    return int(load_library().mnb_softmax_workspace_bytes(_size(rows), _size(V)))


def mnb_softmax(logits, temperature=None, workspace=None, out=None, stream=None):
    """fp32 ``[rows, V]``: softmax of ``logits / temperature`` (fp32 ``[rows]``, None: 1; 0: 1 at the largest logit).  A
    workspace is shared or allocated as in ``mnb_kv4_attention``."""
    torch = _torch_module or _torch()
    if type(logits) is not torch.Tensor or not logits.is_cuda or logits.dim() != 2:
        _two_dims("logits", logits, "[rows, V]")
    shape = logits.shape
    rows, V = shape
    dt = _ACT.get(logits.dtype)
    if dt is None:
        dt = _act_dtype("logits", logits)
    dev = logits.get_device()
    guard = _guard_of(dev) if _gpus != 1 else None
    stride, one = logits.stride()
    if one != 1 or rows < 2:
        stride = _matrix("logits", logits, shape, logits.dtype, guard)
    f32 = torch.float32
    tp = None if temperature is None else _vector("temperature", temperature, f32, (rows,), guard)
    lib, raw_stream = _lib or load_library(), _stream_of(dev, stream)
    if out is None:
        out = logits.new_empty(shape, dtype=f32) if stream is None else _new(shape, f32, logits.device, stream)
    else:
        _vector("out", out, f32, shape, guard)
    wp, ws_bytes = None, 0
    if V > 16377 or workspace is not None:
        workspace = _room(workspace, _bytes_of("mnb_softmax_workspace_bytes", rows, V), logits, dev, stream, raw_stream, guard)
        if workspace is not None:
            wp, ws_bytes = workspace.data_ptr(), workspace.nbytes
    args = (logits.data_ptr(), dt, _size(rows), _size(V), stride, tp, wp, ws_bytes, out.data_ptr(), raw_stream)
    if guard is not None:
        _launch(lib.mnb_softmax, args, dev, guard)
        return out
    st = lib.mnb_softmax(*args)
    if st != MNB_OK:
        _raise(st)
    return out


def mnb_verify_workspace_bytes(batch: int, V: int) -> int:
    return int(load_library().mnb_verify_workspace_bytes(_size(batch), _size(V)))


def mnb_verify(target, draft, draft_tokens, draft_start, u_accept, u_next, workspace=None, tokens=None, accepted=None, stream=None):
    """``(tokens, accepted)``: int32 ``[drafted + batch]`` in the order of ``target``'s rows (a sequence's accepted tokens, the
    next one, then -1) and int32 ``[batch]``.

    ``target`` fp32 ``[drafted + batch, V]``, ``draft`` fp32 ``[drafted, V]`` or None (each row 1 at its token),
    ``draft_tokens`` int32 and ``u_accept`` fp32 ``[drafted]``, ``draft_start`` int32 ``[batch + 1]``, ``u_next`` fp32 ``[batch]``.
    A workspace is shared or allocated as in ``mnb_kv4_attention``.
    """
    torch = _torch_module or _torch()
    tensor, f32, i32 = torch.Tensor, torch.float32, torch.int32
    if type(target) is not tensor or not target.is_cuda or target.dim() != 2:
        _two_dims("target", target, "[drafted + batch, V]")
    if not isinstance(draft_tokens, tensor) or not isinstance(u_next, tensor) or draft_tokens.dim() != 1 or u_next.dim() != 1:
        raise ValueError("target, draft_tokens and u_next must be [drafted + batch, V], [drafted] and [batch]")
    D, B = draft_tokens.shape[0], u_next.shape[0]
    rows, V = target.shape
    dev = target.get_device()
    guard = _guard_of(dev) if _gpus != 1 else None
    ts, one = target.stride()
    if rows != D + B or rows < 2 or one != 1 or target.dtype is not f32:
        ts = _matrix("target", target, (D + B, V), f32, guard)
    ds, dp = 0, None
    if draft is not None:
        ds, dp = _matrix("draft", draft, (D, V), f32, guard), draft.data_ptr()
    given = (_vector("draft_tokens", draft_tokens, i32, (D,), guard), _vector("draft_start", draft_start, i32, (B + 1,), guard),
             _vector("u_accept", u_accept, f32, (D,), guard), _vector("u_next", u_next, f32, (B,), guard))
    lib, raw_stream = _lib or load_library(), _stream_of(dev, stream)
    workspace = _room(workspace, _bytes_of("mnb_verify_workspace_bytes", B, V), target, dev, stream, raw_stream, guard)
    wp, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    if tokens is None:
        tokens = draft_tokens.new_empty(rows) if stream is None else _new((rows,), i32, target.device, stream)
    else:
        _vector("tokens", tokens, i32, (rows,), guard)
    if accepted is None:
        accepted = draft_tokens.new_empty(B) if stream is None else _new((B,), i32, target.device, stream)
    else:
        _vector("accepted", accepted, i32, (B,), guard)
    args = (target.data_ptr(), ts, dp, ds, *given, _size(B), _size(D), _size(V), wp, ws_bytes, tokens.data_ptr(), accepted.data_ptr(),
            raw_stream)
    if guard is not None:
        _launch(lib.mnb_verify, args, dev, guard)
        return tokens, accepted
    st = lib.mnb_verify(*args)
    if st != MNB_OK:
        _raise(st)
    return tokens, accepted

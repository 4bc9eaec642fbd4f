"""Thin ctypes binding of libmosaicq (include/mosaicq.h).

Argument marshalling only: every step of the decomposition, packing and
product runs inside the library (host C++ for packing, CUDA kernels for the
product). PyTorch supplies device memory and streams. There is no fallback:
if the library is missing or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmosaicq.so")

OK, INVALID_ARG, UNSUPPORTED, OUT_OF_MEMORY, CUDA, DEVICE_TIMEOUT = range(6)
PATH_AUTO, PATH_DECODE, PATH_PREFILL = range(3)
UNFUSED_NOALLOC_MAX_OUTPUTS = 2 * 1024 * 1024  # MQ_UNFUSED_NOALLOC_MAX_OUTPUTS
FP4_FORMATS = {"mxfp4": 0, "nvfp4": 1}  # mq_fp4_format
_PATHS = {"auto": PATH_AUTO, "decode": PATH_DECODE, "prefill": PATH_PREFILL}


class MQError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


class _PackOpts(ctypes.Structure):
    _fields_ = [("group_size", ctypes.c_int32), ("residual_density", ctypes.c_double),
                ("residual_blocks", ctypes.c_int32), ("block_fraction", ctypes.c_double),
                ("channel_weight", ctypes.c_void_p)]


class _Decomp(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("row_ptr", ctypes.c_void_p), ("col", ctypes.c_void_p),
                ("qr", ctypes.c_void_p), ("sr", ctypes.c_void_p)]


class _HostPacked(ctypes.Structure):
    _fields_ = [("qweight", ctypes.c_void_p), ("sz", ctypes.c_void_p),
                ("row_ptr", ctypes.c_void_p), ("col", ctypes.c_void_p),
                ("val", ctypes.c_void_p), ("rscale", ctypes.c_void_p)]


class _Info(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("nnz", ctypes.c_int64),
                ("group_size", ctypes.c_int32), ("device", ctypes.c_int32),
                ("device_bytes", ctypes.c_int64), ("max_row_nnz", ctypes.c_int64)]


class _Fp4Info(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("format", ctypes.c_int32), ("device", ctypes.c_int32), ("device_bytes", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmosaicq.so is not built ({LIB_PATH}); run "
                          "`python -m bit_gemm_w4_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    sig = {
        "mq_pack": ([vp, i64, i64, ctypes.POINTER(_PackOpts), vp, ctypes.POINTER(vp)], st),
        "mq_linear": ([vp, vp, i64, vp, vp], st),
        "mq_linear_path": ([vp, vp, i64, vp, vp, ctypes.c_int], st),
        "mq_linear_prefetch": ([vp, vp, i64, vp, vp, vp], st),
        "mq_linear_unfused": ([vp, vp, i64, vp, vp, ctypes.c_size_t, vp], st),
        "mq_linear_unfused_noalloc": ([vp, vp, i64, vp, vp], st),
        "mq_quantize_activations": ([vp, i64, i64, vp, vp, vp], st),
        "mq_selftest_bounded_wait": ([i64, ctypes.POINTER(ctypes.c_int32)], st),
        "mq_read_probe": ([vp, i64, vp, vp], st),
        "mq_w4a4_workspace_bytes": ([vp, i64], i64),
        "mq_linear_w4a4": ([vp, vp, i64, vp, vp, ctypes.c_size_t, vp], st),
        "mq_free": ([vp], None),
        "mq_residual_nnz": ([i64, i64, ctypes.POINTER(_PackOpts), ctypes.POINTER(i64)], st),
        "mq_pack_host": ([vp, i64, i64, ctypes.POINTER(_PackOpts), ctypes.POINTER(_HostPacked)], st),
        "mq_prefill_lists_host": ([i64, i64, vp, vp, vp, vp, vp], st),
        "mq_wide_lists_host": ([i64, i64, vp, vp, vp, vp, vp, vp, ctypes.POINTER(i64)], st),
        "mq_tile_lists_host": ([i64, i64, vp, vp, vp, vp, vp], st),
        "mq_pack_decomposed": ([ctypes.POINTER(_Decomp), vp, ctypes.POINTER(vp)], st),
        "mq_get_info": ([vp, ctypes.POINTER(_Info)], st),
        "mq_export": ([vp, ctypes.POINTER(_HostPacked)], st),
        "mq_export_blocks": ([vp, vp, vp, vp, ctypes.POINTER(i64)], st),
        "mq_block_tiles_host": ([ctypes.POINTER(_Decomp), vp, vp, vp, ctypes.POINTER(i64)], st),
        "mq_device_error": ([vp, vp, ctypes.POINTER(ctypes.c_int32)], st),
        "mq_fp4_code_bytes": ([i64], i64),
        "mq_fp4_scale_bytes": ([st, i64], i64),
        "mq_fp4_quantize": ([vp, st, i64, i64, i64, vp, i64, st, vp, vp, vp, vp], st),
        "mq_fp4_dequantize": ([vp, vp, vp, i64, i64, st, vp, st, i64, vp], st),
        "mq_fp4_pack": ([vp, st, i64, i64, i64, st, vp, ctypes.POINTER(vp)], st),
        "mq_fp4_pack_codes": ([vp, vp, vp, i64, i64, i64, st, vp, ctypes.POINTER(vp)], st),
        "mq_fp4_free": ([vp], None),
        "mq_fp4_get_info": ([vp, ctypes.POINTER(_Fp4Info)], st),
        "mq_fp4_export": ([vp, vp, vp, vp, vp], st),
        "mq_fp4_workspace_bytes": ([vp, i64], i64),
        "mq_fp4_linear": ([vp, vp, st, i64, i64, vp, i64, vp, ctypes.c_size_t, vp], st),
        "mq_fp4_linear_codes": ([vp, vp, vp, vp, i64, vp, st, i64, vp], st),
        "mq_fp4_linear_grouped": ([vp, vp, st, i64, i64, vp, i64, vp, vp, i64, vp, ctypes.c_size_t, vp], st),
        "mq_fp4_linear_grouped_codes": ([vp, vp, vp, vp, i64, vp, vp, st, i64, vp], st),
        "mq_fp4_device_error": ([vp, vp, ctypes.POINTER(ctypes.c_int32)], st),
        "mq_strerror": ([st], ctypes.c_char_p),
        "mq_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _load()


def lib():
    return _lib


def _check(status: int, where: str):
    if status != OK:
        detail = _lib.mq_last_error().decode() or _lib.mq_strerror(status).decode()
        raise MQError(status, where, detail)


def _opts(rho: float, group: int = 128, block_fraction=None, channel_weight=None):
    """Pack options: row mode (rho) unless block_fraction is given, which
    selects block mode. Returns (options, kept) where kept holds the arrays
    the options point at for the duration of the call."""
    if block_fraction is None:
        return _PackOpts(group, float(rho), 0, 0.0, None), None
    h = None
    if channel_weight is not None:
        h = np.ascontiguousarray(channel_weight, dtype=np.float32)
    return _PackOpts(group, 0.0, 1, float(block_fraction), None if h is None else h.ctypes.data), h


def _ptr(a: np.ndarray) -> int:
    return a.ctypes.data if a.size else 0


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def residual_nnz(N: int, K: int, rho: float, group: int = 128, *, block_fraction=None) -> int:
    out = ctypes.c_int64()
    o, _ = _opts(rho, group, block_fraction)
    _check(_lib.mq_residual_nnz(N, K, ctypes.byref(o), ctypes.byref(out)), "mq_residual_nnz")
    return out.value


def _alloc_packed(N: int, K: int, nnz: int):
    arrs = dict(qweight=np.zeros((N, K // 8), np.uint32), sz=np.zeros((N, K // 128), np.uint32),
                row_ptr=np.zeros(N + 1, np.int32), col=np.zeros(nnz, np.uint16),
                val=np.zeros((nnz + 1) // 2, np.uint8), rscale=np.zeros(N, np.uint16))
    hp = _HostPacked(*(_ptr(arrs[k]) for k in
                       ("qweight", "sz", "row_ptr", "col", "val", "rscale")))
    return arrs, hp


def pack_host(W: np.ndarray, rho: float, group: int = 128, *, block_fraction=None,
              channel_weight=None) -> dict:
    """Decompose and pack on the host (no CUDA call). Returns the packed arrays.
    block_fraction selects block mode (see mq_pack_opts)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    nnz = residual_nnz(N, K, rho, group, block_fraction=block_fraction)
    arrs, hp = _alloc_packed(N, K, nnz)
    o, keep = _opts(rho, group, block_fraction, channel_weight)
    _check(_lib.mq_pack_host(_ptr(W), N, K, ctypes.byref(o), ctypes.byref(hp)), "mq_pack_host")
    del keep
    return arrs


def prefill_lists_host(N: int, K: int, packed: dict):
    """The prefill kernel's residual lists of a host pack (pack_host's arrays):
    (ptr int32 [ceil(N/128) * K/64 * 4 + 1], ent uint32 [nnz]); no CUDA call."""
    row_ptr = np.ascontiguousarray(packed["row_ptr"], np.int32)
    col = np.ascontiguousarray(packed["col"], np.uint16)
    val = np.ascontiguousarray(packed["val"], np.uint8)
    nnz = int(row_ptr[-1])
    ptr = np.zeros(((N + 127) // 128) * (K // 64) * 4 + 1, np.int32)
    ent = np.zeros(max(nnz, 1), np.uint32)
    _check(_lib.mq_prefill_lists_host(N, K, _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(ptr), _ptr(ent)),
           "mq_prefill_lists_host")
    return ptr, ent[:nnz]


def wide_lists_host(N: int, K: int, packed: dict):
    """The wide decode kernel's residual lists of a host pack: (ptr int32,
    off uint16 [slices, 136], ent uint16 [nnz], longest slice); no CUDA call."""
    row_ptr = np.ascontiguousarray(packed["row_ptr"], np.int32)
    col = np.ascontiguousarray(packed["col"], np.uint16)
    val = np.ascontiguousarray(packed["val"], np.uint8)
    nnz = int(row_ptr[-1])
    slices = ((N + 127) // 128) * ((K + 255) // 256)
    ptr = np.zeros(slices + 1, np.int32)
    off = np.zeros((slices, 136), np.uint16)
    ent = np.zeros(max(nnz, 1), np.uint16)
    mx = ctypes.c_int64(0)
    _check(_lib.mq_wide_lists_host(N, K, _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(ptr), _ptr(off),
                                   _ptr(ent), ctypes.byref(mx)), "mq_wide_lists_host")
    return ptr, off, ent[:nnz], int(mx.value)


def tile_lists_host(N: int, K: int, packed: dict):
    """The tall-layer decode kernel's residual lists of a host pack: (ptr
    int32 [ceil(N/16) * K/128 + 1], ent uint16 [nnz]); no CUDA call."""
    row_ptr = np.ascontiguousarray(packed["row_ptr"], np.int32)
    col = np.ascontiguousarray(packed["col"], np.uint16)
    val = np.ascontiguousarray(packed["val"], np.uint8)
    nnz = int(row_ptr[-1])
    ptr = np.zeros(((N + 15) // 16) * (K // 128) + 1, np.int32)
    ent = np.zeros(max(nnz, 1), np.uint16)
    _check(_lib.mq_tile_lists_host(N, K, _ptr(row_ptr), _ptr(col), _ptr(val), _ptr(ptr), _ptr(ent)),
           "mq_tile_lists_host")
    return ptr, ent[:nnz]


def selftest_bounded_wait(limit_cycles: int = 1 << 20) -> list:
    """Run the bounded-wait self-test on the current device (synchronous):
    [completed phase seen, stuck wait returned, later wait returned, error
    code]; [1, 0, 0, 2] when the bounded wait works."""
    out = (ctypes.c_int32 * 4)()
    _check(_lib.mq_selftest_bounded_wait(int(limit_cycles), out), "mq_selftest_bounded_wait")
    return list(out)


def _decomp_struct(d: dict, keep: dict) -> "_Decomp":
    return _Decomp(int(d["N"]), int(d["K"]),
                   *(_ptr(keep[k]) for k in ("q", "s", "z", "row_ptr", "col", "qr", "sr")))


def block_tiles_host(d: dict) -> dict:
    """The library's host-side block tiles of a decomposition given as arrays
    (as for Weight.pack_decomposed); MQError with UNSUPPORTED when the
    residual is not made of whole 16 x 64 blocks."""
    keep = dict(
        q=np.ascontiguousarray(d["q"], np.uint8),
        s=np.ascontiguousarray(np.asarray(d["s"], np.float16).view(np.uint16)),
        z=np.ascontiguousarray(np.asarray(d["z"], np.float16).view(np.uint16)),
        row_ptr=np.ascontiguousarray(d["row_ptr"], np.int64),
        col=np.ascontiguousarray(d["col"], np.int32),
        qr=np.ascontiguousarray(d["qr"], np.int8),
        sr=np.ascontiguousarray(np.asarray(d["sr"], np.float16).view(np.uint16)))
    dc = _decomp_struct(d, keep)
    n = ctypes.c_int64()
    _check(_lib.mq_block_tiles_host(ctypes.byref(dc), None, None, None, ctypes.byref(n)),
           "mq_block_tiles_host")
    N = int(d["N"])
    out = dict(blk_ptr=np.zeros(N // 16 + 1, np.int32), blk_col=np.zeros(max(n.value, 1), np.uint16),
               blk_q=np.zeros((max(n.value, 1), 16, 8), np.uint32))
    _check(_lib.mq_block_tiles_host(ctypes.byref(dc), _ptr(out["blk_ptr"]), _ptr(out["blk_col"]),
                                    _ptr(out["blk_q"]), ctypes.byref(n)), "mq_block_tiles_host")
    out["blk_col"] = out["blk_col"][:n.value]
    out["blk_q"] = out["blk_q"][:n.value]
    return out


def read_probe(buf_ptr: int, nbytes: int, sink_ptr: int, *, stream=None) -> None:
    """One launch of the library's streaming-read probe (mq_read_probe) over
    nbytes of device memory at buf_ptr; sink_ptr is a 4-byte device word."""
    _check(_lib.mq_read_probe(ctypes.c_void_p(buf_ptr), int(nbytes), ctypes.c_void_p(sink_ptr),
                              _stream(stream)), "mq_read_probe")


def quantize_activations(X, *, stream=None):
    """Per-token int4 codes (int8 [M, K]) and fp32 scales [M] of bf16 X on
    its device (the W4A4 quantization stage)."""
    import torch
    X = X.contiguous()
    M, K = X.shape
    codes = torch.empty((M, K), dtype=torch.int8, device=X.device)
    scales = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(_lib.mq_quantize_activations(X.data_ptr(), M, K, codes.data_ptr(), scales.data_ptr(),
                                        _stream(stream)), "mq_quantize_activations")
    return codes, scales


class Weight:
    """A packed weight on the current CUDA device (owns its device buffers)."""

    def __init__(self, handle: int):
        self._h = handle

    @classmethod
    def pack(cls, W: np.ndarray, rho: float = 0.0, group: int = 128, stream=None, *,
             block_fraction=None, channel_weight=None) -> "Weight":
        """Decompose, pack and upload fp32 W [N, K]. Row mode keeps k_n =
        floor(rho*K + 0.5) residual entries per row; block_fraction selects
        block mode (16x64 blocks ranked by the channel-weighted squared error,
        channel_weight = K diagonal-Hessian weights or None for all ones)."""
        W = np.ascontiguousarray(W, dtype=np.float32)
        N, K = W.shape
        h = ctypes.c_void_p()
        o, keep = _opts(rho, group, block_fraction, channel_weight)
        _check(_lib.mq_pack(_ptr(W), N, K, ctypes.byref(o), _stream(stream), ctypes.byref(h)),
               "mq_pack")
        del keep
        return cls(h.value)

    @classmethod
    def pack_decomposed(cls, d: dict, stream=None) -> "Weight":
        """Pack a decomposition given as arrays (q u8 [N,K], s/z fp16 [N,G],
        row_ptr, col, qr, sr fp16 [N])."""
        N, K = int(d["N"]), int(d["K"])
        keep = dict(
            q=np.ascontiguousarray(d["q"], np.uint8),
            s=np.ascontiguousarray(np.asarray(d["s"], np.float16).view(np.uint16)),
            z=np.ascontiguousarray(np.asarray(d["z"], np.float16).view(np.uint16)),
            row_ptr=np.ascontiguousarray(d["row_ptr"], np.int64),
            col=np.ascontiguousarray(d["col"], np.int32),
            qr=np.ascontiguousarray(d["qr"], np.int8),
            sr=np.ascontiguousarray(np.asarray(d["sr"], np.float16).view(np.uint16)))
        dc = _decomp_struct(d, keep)
        h = ctypes.c_void_p()
        _check(_lib.mq_pack_decomposed(ctypes.byref(dc), _stream(stream), ctypes.byref(h)),
               "mq_pack_decomposed")
        return cls(h.value)

    @property
    def handle(self) -> int:
        return self._h

    def info(self) -> dict:
        i = _Info()
        _check(_lib.mq_get_info(self._h, ctypes.byref(i)), "mq_get_info")
        return {f: getattr(i, f) for f, _ in _Info._fields_}

    def linear(self, X, Y=None, *, stream=None, path: str = "auto"):
        """Y = X @ W_hat^T for bf16 X [M, K] on the packing device."""
        import torch
        info = self.info()
        if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != info["K"]:
            raise ValueError("X must be a bf16 [M, K] tensor")
        X = X.contiguous()
        if Y is None:
            Y = torch.empty((X.shape[0], info["N"]), dtype=torch.bfloat16, device=X.device)
        self.linear_raw(X.data_ptr(), X.shape[0], Y.data_ptr(), stream=stream, path=path)
        return Y

    def linear_raw(self, x_ptr: int, M: int, y_ptr: int, *, stream=None, path: str = "auto",
                   next_weight: "Weight | None" = None):
        """mq_linear on raw device pointers; with next_weight (decode only),
        mq_linear_prefetch: that weight is brought into L2 meanwhile."""
        if next_weight is not None and path == "auto":
            _check(_lib.mq_linear_prefetch(self._h, x_ptr, M, y_ptr, next_weight._h,
                                           _stream(stream)), "mq_linear_prefetch")
            return
        _check(_lib.mq_linear_path(self._h, x_ptr, M, y_ptr, _stream(stream), _PATHS[path]),
               "mq_linear")

    def linear_unfused(self, X, Y=None, workspace=None, *, stream=None):
        """The split comparison path: dense kernel into an fp32 workspace,
        then a separate residual kernel (caller-owned workspace of M*N fp32)."""
        import torch
        info = self.info()
        X = X.contiguous()
        M = X.shape[0]
        if Y is None:
            Y = torch.empty((M, info["N"]), dtype=torch.bfloat16, device=X.device)
        if workspace is None:
            workspace = torch.empty((M, info["N"]), dtype=torch.float32, device=X.device)
        _check(_lib.mq_linear_unfused(self._h, X.data_ptr(), M, Y.data_ptr(),
                                      workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "mq_linear_unfused")
        return Y

    def linear_w4a4(self, X, Y=None, workspace=None, *, stream=None):
        """The W4A4 variant: per-token int4 activation codes in a
        caller-owned workspace (mq_w4a4_workspace_bytes), then the fused
        int4 x int4 pass (decode kernels for M <= 16, the tcgen05 prefill
        kernel above, which needs K % 256 == 0)."""
        import torch
        info = self.info()
        X = X.contiguous()
        M = X.shape[0]
        if Y is None:
            Y = torch.empty((M, info["N"]), dtype=torch.bfloat16, device=X.device)
        if workspace is None:
            nbytes = max(16, int(_lib.mq_w4a4_workspace_bytes(self._h, M)))
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=X.device)
        _check(_lib.mq_linear_w4a4(self._h, X.data_ptr(), M, Y.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(),
                                   _stream(stream)), "mq_linear_w4a4")
        return Y

    def linear_unfused_noalloc(self, X, Y=None, *, stream=None):
        """The split comparison path with the library's built-in scratch (no
        workspace argument and no device allocation by the library)."""
        import torch
        info = self.info()
        X = X.contiguous()
        if Y is None:
            Y = torch.empty((X.shape[0], info["N"]), dtype=torch.bfloat16, device=X.device)
        _check(_lib.mq_linear_unfused_noalloc(self._h, X.data_ptr(), X.shape[0], Y.data_ptr(),
                                              _stream(stream)), "mq_linear_unfused_noalloc")
        return Y

    def export_blocks(self) -> dict:
        """The device copy of the block tiles (blk_ptr, blk_col, blk_q);
        MQError with UNSUPPORTED when the residual is not block-structured."""
        n = ctypes.c_int64()
        _check(_lib.mq_export_blocks(self._h, None, None, None, ctypes.byref(n)), "mq_export_blocks")
        N = self.info()["N"]
        out = dict(blk_ptr=np.zeros(N // 16 + 1, np.int32), blk_col=np.zeros(max(n.value, 1), np.uint16),
                   blk_q=np.zeros((max(n.value, 1), 16, 8), np.uint32))
        _check(_lib.mq_export_blocks(self._h, _ptr(out["blk_ptr"]), _ptr(out["blk_col"]),
                                     _ptr(out["blk_q"]), ctypes.byref(n)), "mq_export_blocks")
        out["blk_col"] = out["blk_col"][:n.value]
        out["blk_q"] = out["blk_q"][:n.value]
        return out

    def export(self) -> dict:
        info = self.info()
        arrs, hp = _alloc_packed(info["N"], info["K"], info["nnz"])
        _check(_lib.mq_export(self._h, ctypes.byref(hp)), "mq_export")
        return arrs

    def device_error(self, stream=None) -> int:
        code = ctypes.c_int32()
        st = _lib.mq_device_error(self._h, _stream(stream), ctypes.byref(code))
        if st not in (OK, DEVICE_TIMEOUT):
            _check(st, "mq_device_error")
        return code.value

    def free(self):
        if self._h:
            _lib.mq_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


# ---------------------------------------------------------------- fp4
# Microscaled 4-bit floating point (mq_fp4_*). A single token's product takes
# a few microseconds on the device, so the way there is kept short: a call on
# the tensors' own device and its current stream enters no context.

class _Lazy:
    """torch and what the calls need of it, imported when first used."""

    def __getattr__(self, name):
        import torch
        self.torch = torch
        self.empty = torch.empty
        self.bf16, self.fp32, self.u8 = torch.bfloat16, torch.float32, torch.uint8
        self.dtypes = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # mq_dtype
        self.int32 = torch.int32
        self.current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.raw_stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
        return self.__dict__[name]


_t = _Lazy()


def _dtype(t, where: str, fp32: bool = False) -> int:
    d = _t.dtypes.get(t)
    if d is None or (d == 2 and not fp32):
        raise ValueError(f"{where}: unsupported dtype {t}")
    return d


def _fmt(fmt) -> int:
    f = FP4_FORMATS.get(fmt)
    if f is None:
        raise ValueError(f"fp4 format must be one of {sorted(FP4_FORMATS)}, not {fmt!r}")
    return f


def _row_bytes(K: int, fmt: str):
    """mq_fp4_code_bytes and mq_fp4_scale_bytes."""
    cols = 256 if fmt == "nvfp4" else 512
    return (K + 31) // 32 * 16, (K + cols - 1) // cols * 16


def _cuda_index(t) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"a CUDA tensor is needed, not one on {t.device}")
    return index


def _elsewhere(index: int, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    return stream is not None or _t.current_device() != index


class _On:
    """A call's device and stream (None: the device's current stream) made
    current while it runs, so that what the call allocates and converts
    belongs to that stream too."""

    def __init__(self, index: int, stream):
        self.index, self.given = index, stream

    def __enter__(self):
        cuda = _t.torch.cuda
        self.prev = cuda.current_device()
        if self.index != self.prev:
            cuda.set_device(self.index)
        self.was = None
        if self.given is not None:
            current, ptr = cuda.current_stream(), _stream(self.given)
            if ptr != current.cuda_stream:
                self.was = current
                cuda.set_stream(self.given if isinstance(self.given, cuda.Stream) else
                                cuda.ExternalStream(ptr) if ptr else cuda.default_stream())

    def __exit__(self, *exc):
        if self.was is not None:
            _t.torch.cuda.set_stream(self.was)
        if self.index != self.prev:
            _t.torch.cuda.set_device(self.prev)


def _rows_view(X, where: str):
    """A 2-D tensor whose rows are contiguous, its sizes and row stride."""
    shape = X.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{where}: a 2-D tensor with at least one column is needed")
    M, K = shape
    ld, one = X.stride()
    if M > 1 and one == 1 and ld >= K:
        return X, M, K, ld
    if (one != 1 and K > 1) or (ld < K and M > 1):
        X, ld = X.contiguous(), K
    return X, M, K, (ld if M > 1 else K)


def _index(t, index: int, where: str):
    if t.dtype is _t.int32 and t.get_device() == index and t.dim() == 1 and t.is_contiguous():
        return t
    torch = _t.torch
    if t.get_device() != index or t.dim() != 1 or t.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"{where} must be a 1-D int32 or int64 tensor on cuda:{index}")
    if t.dtype == torch.int64:  # what int32 cannot hold is out of range either way
        t = t.clamp(-1, 2**31 - 1).to(torch.int32)
    return t.contiguous()


class Fp4Tensor:
    """A matrix of microscaled 4-bit values: uint8 codes and scales, a row
    each (layout in mosaicq.h), and for nvfp4 the rows' fp32 factors."""

    __slots__ = ("K", "fmt", "rows", "_buffer", "_at", "_codes", "_scales", "_row_scale", "_index")

    def __init__(self, codes, scales, row_scale, K: int, fmt: str):
        f = _fmt(fmt)
        K = int(K)
        want = (_lib.mq_fp4_code_bytes(K), _lib.mq_fp4_scale_bytes(f, K))
        if not want[0]:
            raise ValueError("K must be in [1, 2^24]")
        for t, name, width in ((codes, "codes", want[0]), (scales, "scales", want[1])):
            if t.dtype != _t.u8 or t.dim() < 2 or t.shape[-1] != width or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous uint8 [..., {width}] tensor")
        if codes.shape[:-1] != scales.shape[:-1] or codes.device != scales.device:
            raise ValueError("codes and scales must have the same rows and device")
        if (row_scale is None) != (fmt == "mxfp4"):
            raise ValueError("row_scale belongs to nvfp4, and only to it")
        if row_scale is not None and (row_scale.dtype != _t.fp32 or row_scale.shape != codes.shape[:-1] or
                                      not row_scale.is_contiguous() or row_scale.device != codes.device):
            raise ValueError("row_scale must be a contiguous float32 tensor, one value for each row")
        self.K, self.fmt, self.rows = K, fmt, codes.numel() // codes.shape[-1]
        self._codes, self._scales, self._row_scale = codes, scales, row_scale
        self._buffer, self._index = None, codes.get_device()
        self._at = codes.data_ptr(), scales.data_ptr(), None if row_scale is None else row_scale.data_ptr()

    @classmethod
    def empty(cls, rows: int, K: int, fmt: str, device) -> "Fp4Tensor":
        """Room for a quantised [rows, K] matrix: one buffer, of which codes,
        scales and row_scale are views."""
        q = cls.__new__(cls)
        codes, scales = _row_bytes(K, fmt)
        codes, scales = rows * codes, rows * scales
        q.K, q.fmt, q.rows = K, fmt, rows
        q._codes = q._scales = q._row_scale = None
        if fmt == "nvfp4":
            q._buffer = b = _t.empty(codes + scales + 4 * rows, dtype=_t.u8, device=device)
            at = b.data_ptr()
            q._at = at, at + codes, at + codes + scales
        else:
            q._buffer = b = _t.empty(codes + scales, dtype=_t.u8, device=device)
            at = b.data_ptr()
            q._at = at, at + codes, None
        q._index = b.get_device()
        return q

    def _view(self, which: int):
        codes, scales = _row_bytes(self.K, self.fmt)
        n = self.rows
        if which == 0:
            return self._buffer[:n * codes].view(n, codes)
        if which == 1:
            return self._buffer[n * codes:n * (codes + scales)].view(n, scales)
        return self._buffer[n * (codes + scales):].view(_t.fp32)

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._view(0)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._view(1)
        return self._scales

    @property
    def row_scale(self):
        if self._row_scale is None and self.fmt == "nvfp4":
            self._row_scale = self._view(2)
        return self._row_scale

    @property
    def device(self):
        return (self._buffer if self._codes is None else self._codes).device

    def dequantize(self, dtype=None, *, stream=None):
        """The values as a [rows, K] tensor (fp32 unless a dtype is given)."""
        index = self._index
        if index < 0:
            raise ValueError(f"a CUDA tensor is needed, not one on {self.device}")
        if stream is not None or _t.current_device() != index:
            with _On(index, stream):
                return self.dequantize(dtype)
        if dtype is None:
            dtype = _t.fp32
        d = _t.dtypes.get(dtype)
        if d is None:
            _dtype(dtype, "dequantize", fp32=True)
        rows, K = self.rows, self.K
        Y = _t.empty((rows, K), dtype=dtype, device=self.device)
        codes, scales, row_scale = self._at
        st = _lib.mq_fp4_dequantize(codes, scales, row_scale, rows, K, 1 if row_scale else 0, Y.data_ptr(), d, K,
                                    _t.raw_stream(index))
        if st:
            _check(st, "mq_fp4_dequantize")
        return Y


def fp4_quantize(X, fmt: str = "nvfp4", *, rows=None, stream=None) -> Fp4Tensor:
    """X [M, K] (bf16, fp16 or fp32, any row stride) as microscaled 4-bit
    floating point. With rows (1-D integer tensor) output row r is X[rows[r]],
    and zeros where rows[r] is no row of X."""
    f, d = FP4_FORMATS.get(fmt), _t.dtypes.get(X.dtype)
    if f is None or d is None:
        _fmt(fmt)
        _dtype(X.dtype, "fp4_quantize", fp32=True)
    index = X.get_device()
    if index < 0:
        _cuda_index(X)
    if stream is not None or _t.current_device() != index:
        with _On(index, stream):
            return fp4_quantize(X, fmt, rows=rows)
    X, M, K, ldx = _rows_view(X, "fp4_quantize")
    R, at = M, None
    if rows is not None:
        rows = _index(rows, index, "rows")
        R, at = rows.shape[0], rows.data_ptr()
    q = Fp4Tensor.empty(R, K, fmt, X.device)
    codes, scales, row_scale = q._at
    st = _lib.mq_fp4_quantize(X.data_ptr(), d, R, K, ldx, at, M, f, codes, scales, row_scale, _t.raw_stream(index))
    if st:
        _check(st, "mq_fp4_quantize")
    return q


class Fp4Weight:
    """E packed matrices [N, K] of microscaled 4-bit values on one CUDA device
    (owns its device buffers): a linear layer (E = 1) or a layer's experts."""

    def __init__(self, handle: int):
        self._h = handle
        i = _Fp4Info()
        _check(_lib.mq_fp4_get_info(handle, ctypes.byref(i)), "mq_fp4_get_info")
        self.E, self.N, self.K, self.device_bytes = i.E, i.N, i.K, i.device_bytes
        self.fmt = {v: k for k, v in FP4_FORMATS.items()}[i.format]
        self._index = i.device
        self._workspace_bytes = {}  # rows -> bytes
        self.device = _t.torch.device("cuda", i.device)

    @classmethod
    def pack(cls, W, fmt: str = "nvfp4", *, stream=None) -> "Fp4Weight":
        """Quantise and pack a CUDA tensor W [N, K] or [E, N, K] (bf16, fp16
        or fp32)."""
        f = _fmt(fmt)
        d = _dtype(W.dtype, "Fp4Weight.pack", fp32=True)
        if W.dim() not in (2, 3):
            raise ValueError("W must be [N, K] or [E, N, K]")
        index = _cuda_index(W)
        if _elsewhere(index, stream):
            with _On(index, stream):
                return cls.pack(W, fmt)
        h = ctypes.c_void_p()
        W = W.contiguous()
        E = W.shape[0] if W.dim() == 3 else 1
        _check(_lib.mq_fp4_pack(W.data_ptr(), d, E, W.shape[-2], W.shape[-1], f, _t.raw_stream(index),
                                ctypes.byref(h)), "mq_fp4_pack")
        return cls(h.value)

    @classmethod
    def pack_codes(cls, codes, scales, row_scale, K: int, fmt: str, *, stream=None) -> "Fp4Weight":
        """Pack codes [N, .] or [E, N, .] as they are (CUDA tensors in the
        layout of Fp4Tensor)."""
        q = Fp4Tensor(codes, scales, row_scale, K, fmt)
        if codes.dim() not in (2, 3):
            raise ValueError("codes must be [N, .] or [E, N, .]")
        index = _cuda_index(codes)
        if _elsewhere(index, stream):
            with _On(index, stream):
                return cls.pack_codes(codes, scales, row_scale, K, fmt)
        h = ctypes.c_void_p()
        E = codes.shape[0] if codes.dim() == 3 else 1
        _check(_lib.mq_fp4_pack_codes(*q._at, E, codes.shape[-2], q.K, FP4_FORMATS[fmt], _t.raw_stream(index),
                                      ctypes.byref(h)), "mq_fp4_pack_codes")
        return cls(h.value)

    @property
    def handle(self) -> int:
        return self._h

    def workspace_bytes(self, rows: int) -> int:
        return int(_lib.mq_fp4_workspace_bytes(self._h, rows))

    def export(self, *, stream=None) -> Fp4Tensor:
        """The packed matrices as one quantised [E * N, K] matrix."""
        if _elsewhere(self._index, stream):
            with _On(self._index, stream):
                return self.export()
        q = Fp4Tensor.empty(self.E * self.N, self.K, self.fmt, self.device)
        _check(_lib.mq_fp4_export(self._h, *q._at, _t.raw_stream(self._index)), "mq_fp4_export")
        return q

    def _output(self, Y, rows: int, dtype):
        if Y is None:
            return _t.empty((rows, self.N), dtype=dtype, device=self.device), self.N
        if Y.device != self.device or Y.dtype != dtype or Y.shape != (rows, self.N) or \
                (Y.stride(1) != 1 and self.N > 1) or (Y.stride(0) < self.N and rows > 1):
            raise ValueError(f"Y must be a {dtype} [{rows}, {self.N}] tensor on {self.device} with contiguous rows")
        return Y, (Y.stride(0) if rows > 1 else self.N)

    def _workspace(self, workspace, rows: int):
        if workspace is None:
            n = self._workspace_bytes.get(rows)
            if n is None:
                n = self._workspace_bytes[rows] = self.workspace_bytes(rows)
                if len(self._workspace_bytes) > 4096:
                    self._workspace_bytes = {}
            if not n:
                return None, None, 0
            workspace = _t.empty(n, dtype=_t.u8, device=self.device)
            return workspace, workspace.data_ptr(), n
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"the workspace must be a contiguous tensor on {self.device}")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()

    def _quantized(self, X: Fp4Tensor, dtype, Y):
        if X.fmt != self.fmt or X.K != self.K or X._index != self._index:
            raise ValueError(f"the activations must be {self.fmt} with K = {self.K} on {self.device}")
        if dtype is None:
            dtype = _t.bf16 if Y is None else Y.dtype
        return dtype, _dtype(dtype, "the output")

    def _input(self, X, dtype):
        d = _t.dtypes.get(X.dtype, 2)
        shape = X.shape
        if d == 2 or (dtype is not None and dtype != X.dtype):
            raise ValueError("X must be bf16 or fp16, and Y has its type (dtype is for quantised activations)")
        if len(shape) != 2 or shape[1] != self.K or X.get_device() != self._index:
            raise ValueError(f"X must be a [rows, {self.K}] tensor on {self.device}")
        X, M, _, ld = _rows_view(X, "X")
        return d, X, M, ld

    def linear(self, X, Y=None, workspace=None, *, dtype=None, stream=None):
        """Y = X @ W^T. X: a bf16 or fp16 [M, K] tensor, quantised within the
        call into the workspace (workspace_bytes(M) bytes: a size for M rows
        serves fewer too), with Y of its
        type; or an Fp4Tensor, with Y of `dtype` (Y's own or bf16 unless given)."""
        index = self._index
        if stream is not None or _t.current_device() != index:
            with _On(index, stream):
                return self.linear(X, Y, workspace, dtype=dtype)
        if isinstance(X, Fp4Tensor):
            dtype, d = self._quantized(X, dtype, Y)
            Y, ldy = self._output(Y, X.rows, dtype)
            st = _lib.mq_fp4_linear_codes(self._h, *X._at, X.rows, Y.data_ptr(), d, ldy, _t.raw_stream(index))
            if st:
                _check(st, "mq_fp4_linear_codes")
            return Y
        d, X, M, ldx = self._input(X, dtype)
        Y, ldy = (X.new_empty((M, self.N)), self.N) if Y is None else self._output(Y, M, X.dtype)
        workspace, at_ws, nbytes = self._workspace(workspace, M)
        st = _lib.mq_fp4_linear(self._h, X.data_ptr(), d, M, ldx, Y.data_ptr(), ldy, at_ws, nbytes,
                                _t.raw_stream(index))
        if st:
            _check(st, "mq_fp4_linear")
        return Y

    def linear_grouped(self, X, offsets, Y=None, workspace=None, *, rows=None, dtype=None, stream=None):
        """The experts' products: Y[r] = x[r] @ W[e]^T for offsets[e] <= r <
        offsets[e + 1] (offsets: E + 1 integers on the device). x[r] is
        X[rows[r]], or X[r] without rows; X as for linear. Rows of Y that
        belong to no expert are left as they were (undefined in a Y that the
        call makes)."""
        index = self._index
        if stream is not None or _t.current_device() != index:
            with _On(index, stream):
                return self.linear_grouped(X, offsets, Y, workspace, rows=rows, dtype=dtype)
        offsets = _index(offsets, index, "offsets")
        if offsets.shape[0] != self.E + 1:
            raise ValueError(f"offsets must hold E + 1 = {self.E + 1} values")
        if isinstance(X, Fp4Tensor):
            if rows is not None:
                raise ValueError("rows are taken when X is quantised: fp4_quantize(X, rows=rows)")
            dtype, d = self._quantized(X, dtype, Y)
            Y, ldy = self._output(Y, X.rows, dtype)
            st = _lib.mq_fp4_linear_grouped_codes(self._h, *X._at, X.rows, offsets.data_ptr(), Y.data_ptr(), d,
                                                  ldy, _t.raw_stream(index))
            if st:
                _check(st, "mq_fp4_linear_grouped_codes")
            return Y
        d, X, M, ldx = self._input(X, dtype)
        R, at = M, None
        if rows is not None:
            rows = _index(rows, index, "rows")
            R, at = rows.shape[0], rows.data_ptr()
        Y, ldy = (X.new_empty((R, self.N)), self.N) if Y is None else self._output(Y, R, X.dtype)
        workspace, at_ws, nbytes = self._workspace(workspace, R)
        st = _lib.mq_fp4_linear_grouped(self._h, X.data_ptr(), d, M, ldx, at, R, offsets.data_ptr(), Y.data_ptr(), ldy,
                                        at_ws, nbytes, _t.raw_stream(index))
        if st:
            _check(st, "mq_fp4_linear_grouped")
        return Y

    def device_error(self, stream=None) -> int:
        if _elsewhere(self._index, stream):
            with _On(self._index, stream):
                return self.device_error()
        code = ctypes.c_int32()
        st = _lib.mq_fp4_device_error(self._h, _t.raw_stream(self._index), ctypes.byref(code))
        if st not in (OK, DEVICE_TIMEOUT):
            _check(st, "mq_fp4_device_error")
        return code.value

    def free(self):
        if self._h:
            _lib.mq_fp4_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass

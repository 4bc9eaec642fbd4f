"""Sizes and refusals of the mq_fp4_* calls and their binding, without a GPU:
every refusal comes before any CUDA call."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 20  # stands for a device address: refused calls never follow it


def test_declared_symbols_are_exported(mq):
    src = open(os.path.join(ROOT, "include", "mosaicq.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(mq_fp4_\w+)\s*\(", src)))
    assert len(names) >= 15
    lib = ctypes.CDLL(mq.LIB_PATH)
    assert not [n for n in names if not hasattr(lib, n)]


def test_row_bytes(mq):
    lib = mq.lib()
    for K, codes, mx, nv in ((1, 16, 16, 16), (32, 16, 16, 16), (33, 32, 16, 16), (256, 128, 16, 16),
                             (257, 144, 16, 32), (512, 256, 16, 32), (513, 272, 32, 48), (4096, 2048, 128, 256)):
        assert lib.mq_fp4_code_bytes(K) == codes
        assert lib.mq_fp4_scale_bytes(0, K) == mx
        assert lib.mq_fp4_scale_bytes(1, K) == nv
    for K in (0, -5, (1 << 24) + 1):
        assert lib.mq_fp4_code_bytes(K) == 0 and lib.mq_fp4_scale_bytes(0, K) == 0
    assert lib.mq_fp4_scale_bytes(2, 64) == 0
    assert lib.mq_fp4_workspace_bytes(None, 4) == 0


GOOD = dict(X=BIG, dtype=0, rows=4, K=64, ldx=64, index=None, x_rows=4, fmt=1, codes=BIG, scales=BIG, row_scale=BIG,
            stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(fmt=2), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1),
    (dict(K=0, ldx=0), 1), (dict(K=(1 << 24) + 1, ldx=1 << 25), 1),
    (dict(rows=-1), 1), (dict(x_rows=-1), 1), (dict(x_rows=5), 1),
    (dict(ldx=63), 1), (dict(ldx=(1 << 40) + 1), 1),
    (dict(X=None), 1), (dict(X=BIG + 1), 1), (dict(dtype=2, X=BIG + 2), 1),
    (dict(index=BIG + 2), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(row_scale=None), 1),
    (dict(codes=BIG + 8), 1), (dict(scales=BIG + 8), 1), (dict(row_scale=BIG + 2), 1),
    (dict(rows=(1 << 30) + 1, x_rows=(1 << 30) + 1), 2),
])
def test_quantize_refusals(mq, change, status):
    a = {**GOOD, **change}
    assert mq.lib().mq_fp4_quantize(*a.values()) == status
    assert mq.lib().mq_last_error()


def test_no_rows_is_ok(mq):
    lib = mq.lib()
    assert lib.mq_fp4_quantize(*{**GOOD, "rows": 0, "x_rows": 0, "X": None}.values()) == 0
    assert lib.mq_fp4_quantize(*{**GOOD, "rows": 0, "x_rows": 0, "codes": None}.values()) == 0
    assert lib.mq_fp4_dequantize(BIG, BIG, BIG, 0, 64, 1, BIG, 0, 64, 0) == 0


@pytest.mark.parametrize("args,status", [
    ((None, BIG, BIG, 4, 64, 1, BIG, 0, 64, 0), 1), ((BIG, BIG, None, 4, 64, 1, BIG, 0, 64, 0), 1),
    ((BIG, BIG, BIG, 4, 64, 1, None, 0, 64, 0), 1), ((BIG, BIG, BIG, 4, 64, 1, BIG + 1, 0, 64, 0), 1),
    ((BIG, BIG, BIG, 4, 64, 1, BIG, 0, 63, 0), 1), ((BIG, BIG, BIG, -4, 64, 1, BIG, 0, 64, 0), 1),
    ((BIG, BIG, BIG, 4, 64, 7, BIG, 0, 64, 0), 1), ((BIG, BIG, BIG, 4, 64, 1, BIG, 5, 64, 0), 1),
    ((BIG, BIG, BIG, (1 << 30) + 1, 64, 1, BIG, 0, 64, 0), 2),
])
def test_dequantize_refusals(mq, args, status):
    assert mq.lib().mq_fp4_dequantize(*args) == status


@pytest.mark.parametrize("E,N,K,fmt,status", [
    (0, 8, 64, 0, 1), (1, 0, 64, 0, 1), (1, 8, 0, 0, 1), (1, 8, 64, 3, 1), (65536, 1, 64, 0, 2),
    (1, (1 << 30) + 1, 64, 0, 2), (1024, 1 << 21, 64, 0, 2),
])
def test_pack_refusals(mq, E, N, K, fmt, status):
    h = ctypes.c_void_p(5)
    assert mq.lib().mq_fp4_pack(BIG, 0, E, N, K, fmt, 0, ctypes.byref(h)) == status and not h.value
    h = ctypes.c_void_p(5)
    assert mq.lib().mq_fp4_pack_codes(BIG, BIG, BIG, E, N, K, fmt, 0, ctypes.byref(h)) == status and not h.value


def test_pack_null_refusals(mq):
    lib = mq.lib()
    h = ctypes.c_void_p()
    assert lib.mq_fp4_pack(BIG, 0, 1, 8, 64, 0, 0, None) == 1
    assert lib.mq_fp4_pack(None, 0, 1, 8, 64, 0, 0, ctypes.byref(h)) == 1
    assert lib.mq_fp4_pack(BIG, 4, 1, 8, 64, 0, 0, ctypes.byref(h)) == 1
    assert lib.mq_fp4_pack_codes(BIG, BIG, None, 1, 8, 64, 1, 0, ctypes.byref(h)) == 1
    assert lib.mq_fp4_pack_codes(BIG + 4, BIG, None, 1, 8, 64, 0, 0, ctypes.byref(h)) == 1
    assert lib.mq_fp4_get_info(None, None) == 1
    assert lib.mq_fp4_export(None, BIG, BIG, BIG, 0) == 1
    assert lib.mq_fp4_linear(None, BIG, 0, 1, 64, BIG, 64, BIG, 1 << 20, 0) == 1
    assert lib.mq_fp4_linear_codes(None, BIG, BIG, BIG, 1, BIG, 0, 64, 0) == 1
    assert lib.mq_fp4_linear_grouped(None, BIG, 0, 1, 64, None, 1, BIG, BIG, 64, BIG, 1 << 20, 0) == 1
    assert lib.mq_fp4_linear_grouped_codes(None, BIG, BIG, BIG, 1, BIG, BIG, 0, 64, 0) == 1
    assert lib.mq_fp4_device_error(None, 0, None) == 1
    lib.mq_fp4_free(None)  # NULL-safe


def test_binding_refusals(mq):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mq.fp4_quantize(x)
    with pytest.raises(ValueError, match="format"):
        mq.fp4_quantize(x, "fp4")
    with pytest.raises(ValueError, match="dtype"):
        mq.fp4_quantize(x.double())
    with pytest.raises(ValueError, match="CUDA"):
        mq.Fp4Weight.pack(x)
    with pytest.raises(ValueError, match="N, K"):
        mq.Fp4Weight.pack(x[0])
    codes, scales = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 16, dtype=torch.uint8)
    f = torch.ones(2)
    q = mq.Fp4Tensor(codes, scales, None, 64, "mxfp4")
    assert q.rows == 2
    with pytest.raises(ValueError, match="CUDA"):
        q.dequantize()
    for bad in ((codes[:, :16], scales, None, 64, "mxfp4"), (codes, scales, f, 64, "mxfp4"),
                (codes, scales, None, 64, "nvfp4"), (codes, scales, f[:1], 64, "nvfp4"),
                (codes[:1], scales, None, 64, "mxfp4"), (codes.short(), scales, None, 64, "mxfp4"),
                (codes, scales, None, 0, "mxfp4")):
        with pytest.raises(ValueError):
            mq.Fp4Tensor(*bad)

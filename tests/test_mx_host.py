"""Refusals of the microscaled and norm calls, checked without a GPU: argument checks run before the device is
touched, and pointers of refused calls are never read."""
import ctypes

import pytest
import torch

import binary_factorized_weight_b200 as dbf
from binary_factorized_weight_b200 import build as dbf_build

INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4
P = 1 << 20  # never dereferenced
F16, F32, BF16, I8 = 1, 2, 3, 0


@pytest.fixture(scope="module")
def lib():
    dbf_build.build()
    return dbf.load_library()


def test_sizes(lib):
    assert dbf.dbf_mx_code_bytes(3, 1, dbf.DBF_MX_E2M1) == 3 * 64
    assert dbf.dbf_mx_code_bytes(3, 129, dbf.DBF_MX_E4M3) == 3 * 256
    assert dbf.dbf_mx_scale_bytes(1, 1) == 512
    assert dbf.dbf_mx_scale_bytes(129, 257) == 2 * 3 * 512
    assert dbf.dbf_mx_code_bytes(0, 4, 0) == dbf.dbf_mx_code_bytes(4, 4, 2) == dbf.dbf_mx_scale_bytes(-1, 4) == 0
    assert dbf.dbf_mx_code_bytes((1 << 24) + 1, 4, 0) == 0
    assert dbf.dbf_mx_forward_workspace_bytes(4096, 4096, 1) >= 256
    assert dbf.dbf_mx_forward_workspace_bytes(4096, (1 << 20) + 1, 1) == 0
    assert dbf.dbf_rmsnorm_backward_workspace_bytes(2000, 4096) >= 4096 * 4
    assert dbf.dbf_rmsnorm_backward_workspace_bytes(0, 4096) == 0


@pytest.mark.parametrize("change,status", [
    (dict(src=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(t=I8), INVALID),
    (dict(t=4), INVALID), (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(flags=2), INVALID),
    (dict(rows=0), INVALID), (dict(cols=-3), INVALID), (dict(rows=(1 << 24) + 1), SHAPE),
    (dict(cols=1 << 24, rows=1 << 17), SHAPE), (dict(codes=P + 16), MISALIGNED), (dict(scales=P + 8), MISALIGNED),
    (dict(src=P + 1), MISALIGNED), (dict(src=P + 2, t=F32), MISALIGNED)])
def test_quantize_refusals(lib, change, status):
    a = dict(src=P, t=F16, rows=4, cols=64, fmt=0, flags=0, codes=P, scales=P) | change
    assert lib.dbf_mx_quantize(a["src"], a["t"], a["rows"], a["cols"], a["fmt"], a["flags"], a["codes"], a["scales"],
                               None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dst=None), INVALID), (dict(t=I8), INVALID), (dict(fmt=7), INVALID), (dict(rows=0), INVALID),
    (dict(cols=(1 << 24) + 1), SHAPE), (dict(dst=P + 1), MISALIGNED), (dict(codes=P + 4), MISALIGNED)])
def test_dequantize_refusals(lib, change, status):
    a = dict(dst=P, t=F16, rows=4, cols=64, fmt=1, codes=P, scales=P) | change
    assert lib.dbf_mx_dequantize(a["codes"], a["scales"], a["rows"], a["cols"], a["fmt"], a["dst"], a["t"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(xc=None), INVALID), (dict(xs=None), INVALID), (dict(wc=None), INVALID), (dict(ws=None), INVALID),
    (dict(y=None), INVALID), (dict(yt=I8), INVALID), (dict(xf=2), INVALID), (dict(wf=-1), INVALID), (dict(n=0), INVALID),
    (dict(m=0), INVALID), (dict(b=0), INVALID), (dict(flags=2), INVALID), (dict(m=(1 << 20) + 1), SHAPE),
    (dict(b=(1 << 24) + 1), SHAPE), (dict(xc=P + 16), MISALIGNED), (dict(ws=P + 4), MISALIGNED),
    (dict(y=P + 8), MISALIGNED), (dict(work=None), WORKSPACE), (dict(wb=0), WORKSPACE), (dict(work=P + 4), WORKSPACE)])
def test_forward_refusals(lib, change, status):
    a = dict(xc=P, xs=P, xf=1, wc=P, ws=P, wf=0, n=64, m=64, b=2, y=P, yt=F16, work=P, wb=1 << 20, flags=0) | change
    assert lib.dbf_mx_forward(a["xc"], a["xs"], a["xf"], a["wc"], a["ws"], a["wf"], a["n"], a["m"], a["b"], a["y"],
                              a["yt"], a["work"], a["wb"], a["flags"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(t=I8), INVALID),
    (dict(r=P), INVALID), (dict(h=P), INVALID), (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(cols=(1 << 20) + 1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(x=P + 1), MISALIGNED),
    (dict(y=P + 1), MISALIGNED)])
def test_norm_refusals(lib, change, status):
    a = dict(x=P, r=None, w=P, t=BF16, rows=2, cols=64, eps=1e-5, h=None, y=P) | change
    assert lib.dbf_rmsnorm_forward(a["x"], a["r"], a["w"], a["t"], a["rows"], a["cols"], a["eps"], a["h"], a["y"],
                                   None) == status
    codes = None if a["y"] is None else a["y"] if a["y"] == P else P + 16
    assert lib.dbf_rmsnorm_mx_forward(a["x"], a["r"], a["w"], a["t"], a["rows"], a["cols"], a["eps"], 1, a["h"], codes,
                                      P, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID),
    (dict(t=I8), INVALID), (dict(rows=0), INVALID), (dict(eps=0.0), INVALID), (dict(cols=(1 << 20) + 1), SHAPE),
    (dict(dw=P + 2), MISALIGNED), (dict(dh=P + 1), MISALIGNED), (dict(work=None), WORKSPACE), (dict(wb=64 * 4 - 1), WORKSPACE)])
def test_norm_backward_refusals(lib, change, status):
    a = dict(dy=P, h=P, w=P, dh=None, t=F16, rows=2, cols=64, eps=1e-5, dx=P, dw=P, work=P, wb=64 * 4) | change
    assert lib.dbf_rmsnorm_backward(a["dy"], a["h"], a["w"], a["dh"], a["t"], a["rows"], a["cols"], a["eps"], a["dx"],
                                    a["dw"], a["work"], a["wb"], None) == status


def test_the_binding_refuses_host_tensors(lib):
    x, w, u8 = torch.zeros(2, 64), torch.ones(64), torch.zeros(4096, dtype=torch.uint8)
    for call in (lambda: dbf.dbf_mx_quantize(x, dbf.DBF_MX_E2M1), lambda: dbf.dbf_rmsnorm_forward(x, w, 1e-5),
                 lambda: dbf.dbf_rmsnorm_mx_forward(x, w, 1e-5), lambda: dbf.dbf_rmsnorm_backward(x, x, w, 1e-5),
                 lambda: dbf.dbf_mx_dequantize(u8, u8, 2, 64, 0), lambda: dbf.dbf_mx_forward(u8, u8, u8, u8, 2, 64, 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dbf.dbf_mx_quantize(x.double(), dbf.DBF_MX_E2M1)

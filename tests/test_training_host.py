"""Entry points and argument checks of the training-step operators on the host: exported names,
status codes for bad arguments (found before any launch), and the binding's refusals."""
import ctypes
import os
import re

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from unbiased_nvfp4_gradient_amd import training

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000


def _has_gpu():
    return torch.cuda.device_count() > 0


@pytest.fixture(scope="module")
def L():
    return training._lib()


def test_header_and_exports_agree(L):
    text = open(os.path.join(ROOT, "include", "nvfp4_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert declared == set(training.EXPORTED)
    for name in declared:
        assert getattr(L, name)


def test_layer_norm_refusals(L):
    def f(type=1, p=0, x=FAKE, w=FAKE, b=FAKE, rows=4, n=64, stride=64, eps=1e-5, y=FAKE,
          mean=FAKE, rstd=FAKE):
        return L.layer_norm_forward(type, p, x, w, b, rows, n, stride, eps, y, mean, rstd, None)
    assert f(type=3) == nv.ERR_ARG and f(type=-1) == nv.ERR_ARG
    assert f(p=2) == nv.ERR_ARG and f(type=0, p=1) == nv.ERR_ARG
    assert f(rows=-1) == nv.ERR_SHAPE and f(n=0) == nv.ERR_SHAPE
    assert f(stride=63) == nv.ERR_SHAPE
    assert f(rows=1 << 31) == nv.ERR_ARG and f(rows=1 << 20, n=1 << 20, stride=1 << 20) == nv.ERR_ARG
    assert f(eps=-1.0) == nv.ERR_ARG and f(eps=float("nan")) == nv.ERR_ARG
    for name in ("x", "y", "mean", "rstd"):
        assert f(**{name: None}) == nv.ERR_NULL, name
    assert f(x=FAKE + 1) == nv.ERR_ALIGN and f(w=FAKE + 2) == nv.ERR_ALIGN
    if not _has_gpu():
        assert f() == nv.ERR_HIP and f(w=None, b=None) == nv.ERR_HIP
        assert f(x=FAKE + 2) == nv.ERR_HIP                 # an element's alignment is enough

    need = L.layer_norm_workspace_bytes(1, 4, 64)

    def g(dw=FAKE, db=FAKE, ws=FAKE, bytes=need, dx=FAKE, dy_stride=64):
        return L.layer_norm_backward(1, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 64, dy_stride, 64, dx,
                                     dw, db, ws, bytes, None)
    assert need > 0
    assert g(ws=None) == nv.ERR_WORKSPACE and g(bytes=need - 1) == nv.ERR_WORKSPACE
    assert g(ws=FAKE + 8) == nv.ERR_ALIGN and g(dx=None) == nv.ERR_NULL
    assert g(dy_stride=5) == nv.ERR_SHAPE
    if not _has_gpu():
        assert g() == nv.ERR_HIP and g(dw=None, db=None, ws=None, bytes=0) == nv.ERR_HIP


def test_cross_entropy_refusals(L):
    need = [L.linear_cross_entropy_workspace_bytes(b, 4, 64, 256) for b in (0, 1)]
    assert all(need)

    def f(type=1, h=FAKE, hs=64, w=FAKE, ws_=64, y=FAKE, t=4, d=64, v=256, red=1, loss=FAKE,
          lse=FAKE, ws=FAKE, bytes=None):
        bytes = need[0] if bytes is None else bytes
        return L.linear_cross_entropy_forward(type, h, hs, w, ws_, y, t, d, v, -100, red, loss,
                                              lse, ws, bytes, None)
    assert f(type=0) == nv.ERR_ARG and f(red=3) == nv.ERR_ARG and f(red=-1) == nv.ERR_ARG
    assert f(t=-1) == nv.ERR_SHAPE and f(d=0) == nv.ERR_SHAPE and f(v=0) == nv.ERR_SHAPE
    assert f(hs=63) == nv.ERR_SHAPE and f(ws_=63) == nv.ERR_SHAPE
    assert f(t=1 << 31) == nv.ERR_ARG and f(v=1 << 31) == nv.ERR_ARG
    assert f(t=1 << 20, v=1 << 20) == nv.ERR_ARG
    for name in ("h", "w", "y", "loss", "lse"):
        assert f(**{name: None}) == nv.ERR_NULL, name
    assert f(h=FAKE + 1) == nv.ERR_ALIGN and f(y=FAKE + 4) == nv.ERR_ALIGN
    assert f(ws=None) == nv.ERR_WORKSPACE and f(bytes=need[0] - 1) == nv.ERR_WORKSPACE
    assert f(ws=FAKE + 128) == nv.ERR_ALIGN

    def g(dloss=FAKE, dh=FAKE, dw=FAKE, bytes=None, lse=FAKE):
        bytes = need[1] if bytes is None else bytes
        return L.linear_cross_entropy_backward(1, dloss, FAKE, 64, FAKE, 64, FAKE, lse, 4, 64,
                                               256, -100, 1, dh, dw, FAKE, bytes, None)
    assert g(dloss=None) == nv.ERR_NULL and g(lse=None) == nv.ERR_NULL
    assert g(bytes=need[1] - 1) == nv.ERR_WORKSPACE
    assert g(dh=FAKE + 1) == nv.ERR_ALIGN
    if not _has_gpu():
        assert f() == nv.ERR_HIP and g() == nv.ERR_HIP and g(dh=None) == nv.ERR_HIP


def test_clip_refusals(L):
    def call(ptrs=(FAKE, FAKE + 4096), outs=(FAKE, FAKE + 4096), sizes=(100, 200), types=(0, 1),
             max_norm=1.0, inf=0, norm=FAKE, ws=FAKE, bytes=None, clip=True):
        n = len(sizes)
        p, o = (ctypes.c_void_p * n)(*ptrs), (ctypes.c_void_p * n)(*outs)
        s, k = (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*types)
        bytes = L.grad_norm_workspace_bytes(s, n) if bytes is None else bytes
        if clip:
            return L.clip_grads(p, o, s, k, n, max_norm, inf, norm, ws, bytes, None)
        return L.grad_norm(p, s, k, n, inf, norm, ws, bytes, None)
    for clip in (False, True):
        assert call(clip=clip, types=(0, 3)) == nv.ERR_ARG
        assert call(clip=clip, sizes=(100, -1), bytes=64) == nv.ERR_SHAPE
        assert call(clip=clip, sizes=(100, 1 << 40), bytes=64) == nv.ERR_ARG
        assert call(clip=clip, ptrs=(FAKE, None)) == nv.ERR_NULL
        assert call(clip=clip, ptrs=(FAKE + 2, FAKE + 4096)) == nv.ERR_ALIGN
        assert call(clip=clip, inf=2) == nv.ERR_ARG
        assert call(clip=clip, norm=None) == nv.ERR_NULL
        assert call(clip=clip, ws=None) == nv.ERR_WORKSPACE
        assert call(clip=clip, bytes=8) == nv.ERR_WORKSPACE
        assert call(clip=clip, ws=FAKE + 4) == nv.ERR_ALIGN
    assert call(max_norm=-1.0) == nv.ERR_ARG and call(max_norm=float("nan")) == nv.ERR_ARG
    assert call(outs=(FAKE, None)) == nv.ERR_NULL
    if not _has_gpu():
        assert call() == nv.ERR_HIP and call(clip=False) == nv.ERR_HIP
        assert call(sizes=(0, 0), ptrs=(None, None), outs=(None, None)) == nv.ERR_HIP


def test_clip_refuses_overlap(L):
    def call(ins, outs, sizes, types=None):
        n = len(sizes)
        p, o = (ctypes.c_void_p * n)(*ins), (ctypes.c_void_p * n)(*outs)
        s, k = (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*(types or [0] * n))
        return L.clip_grads(p, o, s, k, n, 1.0, 0, FAKE, FAKE, 1 << 20, None)
    a, b, c, d = (FAKE + i * 4096 for i in range(4))
    bad = [((a, a), (a, a), (10, 10)),                   # listed twice, clipped in place
           ((a, a + 36), (a, a + 36), (10, 10)),         # one element shared, in place
           ((b, a + 4), (b, a + 4), (10, 1024)),         # out of order
           ((a, b), (c, c + 36), (10, 10)),              # outputs overlap
           ((a, b), (b, a), (10, 10)),                   # exchanged
           ((a, b), (a + 4, c), (10, 10)),               # moved by one element
           ((a, d), (c, b), (10, 3000)),                 # a long output reaches another output
           ((a, c, b), (d, c, b), (2049, 5, 5)),         # a read that reaches a tensor clipped
           ]
    for case in bad:
        assert call(*case) == nv.ERR_ARG, case
    assert call((a, a + 18), (a, a + 18), (10, 10), (1, 1)) == nv.ERR_ARG
    if not _has_gpu():
        fine = [((a, a + 40), (a, a + 40), (10, 10)), ((a, a), (b, c), (10, 10)),
                ((b, a), (d, c), (1024, 1024)), ((a, a), (a, a), (0, 10)),
                ((a + 2, a), (a + 2, a), (1, 1))]
        for k, case in enumerate(fine):
            types = (1, 1) if k == 4 else None
            assert call(*case, types) == nv.ERR_HIP, case


def test_binding_refuses_host_tensors_and_bad_arguments():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        nv.layer_norm_forward(x)
    with pytest.raises(ValueError, match="device tensor"):
        nv.linear_cross_entropy_forward(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="on one GPU"):
        nv.clip_grads([x], 1.0)
    with pytest.raises(ValueError, match="at least one"):
        nv.grad_norm([])
    with pytest.raises(ValueError, match="norm_type"):
        nv.grad_norm([x], norm_type=1.0)
    with pytest.raises(ValueError, match="torch tensors"):
        nv.grad_norm([x, None])


@pytest.mark.parametrize("make,what", [
    (lambda: torch.zeros(4, 8)[:, ::2], "contiguous"),
    (lambda: torch.zeros(8).expand(4, 8), "overlap"),
    (lambda: torch.zeros(4, 6, 8)[:, :5], "one distance"),
    (lambda: torch.zeros(4, 0), "at least one"),
    (lambda: torch.zeros(()), "at least one")])
def test_rows_of_other_layouts_are_refused(make, what):
    with pytest.raises(ValueError, match=what):
        training._as_rows(make(), "x")


def test_rows_of_views():
    assert training._as_rows(torch.zeros(4, 16)[:, 3:10], "x") == (4, 7, 16)
    assert training._as_rows(torch.zeros(2, 3, 8), "x") == (6, 8, 8)
    assert training._as_rows(torch.zeros(2, 3, 16)[..., :8], "x") == (6, 8, 16)
    assert training._as_rows(torch.zeros(5, 1)[::2], "x") == (3, 1, 2)
    assert training._as_rows(torch.zeros(1, 8).expand(1, 8), "x") == (1, 8, 8)
    assert training._as_rows(torch.zeros(9), "x") == (1, 9, 9)

"""Entry points and argument checks of the feed-forward block's operators and of AdamW on the
host: exported names, status codes for bad arguments (found before any launch), and the binding's
refusals."""
import ctypes
import os
import re

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from unbiased_nvfp4_gradient_amd import block, optimizer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000000


def _has_gpu():
    return torch.cuda.device_count() > 0


def test_header_and_exports_agree():
    text = open(os.path.join(ROOT, "include", "nvfp4_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"^(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert declared == {*block.EXPORTED, *optimizer.EXPORTED}
    for name in declared:
        assert getattr(nv.lib(), name)


def test_mx_linear_refusals():
    L = block._lib()

    def mx(codes=FAKE, scales=FAKE, k_tiled=0):
        return ctypes.byref(nv._CMx(codes, scales, k_tiled))

    def f(a=(), b=(), M=200, n=64, K=256, rot=0, gated=0, act=2, type=1, bias_type=0, bias=FAKE,
          res=FAKE, rs=64, y=FAKE, z=FAKE):
        a, b = (None if t is None else mx(**dict(t)) for t in (a, b))
        return L.mxfp4_linear_forward(a, b, M, n, K, rot, gated, act, type, bias_type, bias, res,
                                      rs, y, z, None)
    assert f(a=None) == nv.ERR_NULL and f(b=None) == nv.ERR_NULL
    for over in (dict(rot=2), dict(gated=2), dict(act=5), dict(act=-1), dict(type=3),
                 dict(bias_type=2), dict(type=0, bias_type=1), dict(gated=1),
                 dict(a=dict(k_tiled=1)), dict(a=dict(k_tiled=2), b=dict(k_tiled=2)),
                 dict(n=1 << 31, rs=1 << 31), dict(gated=1, res=None, n=1 << 30),
                 dict(M=1 << 31), dict(M=1 << 20, n=1 << 20, rs=1 << 20),
                 dict(n=1 << 20, K=1 << 20, rs=1 << 20), dict(rs=1 << 40)):
        assert f(**over) == nv.ERR_ARG, over
    for over in (dict(M=-1), dict(n=-1), dict(K=-128), dict(K=64), dict(rs=63)):
        assert f(**over) == nv.ERR_SHAPE, over
    for over in (dict(y=None), dict(a=dict(codes=None)), dict(b=dict(scales=None))):
        assert f(**over) == nv.ERR_NULL, over
    for over in (dict(a=dict(codes=FAKE + 8)), dict(b=dict(scales=FAKE + 2)), dict(y=FAKE + 1),
                 dict(z=FAKE + 1), dict(res=FAKE + 1), dict(bias=FAKE + 2)):
        assert f(**over) == nv.ERR_ALIGN, over
    if not _has_gpu():
        assert f() == nv.ERR_HIP and f(bias=None, bias_type=9, res=None, rs=0, z=None) == nv.ERR_HIP
        assert f(M=1, rs=0) == nv.ERR_HIP and f(M=0, y=None) == nv.ERR_HIP
        assert f(K=0, a=dict(codes=None, scales=None), b=dict(codes=None)) == nv.ERR_HIP


def test_mx_linear_binding_refusals():
    a = nv.empty_mx_layout(4, 256, "cpu")
    with pytest.raises(ValueError, match="on a GPU"):
        nv.mxfp4_linear_forward(a, a)
    with pytest.raises(ValueError, match="unknown activation"):
        nv.mxfp4_gated_forward(a, a, activation="swish")
    with pytest.raises(ValueError, match="dtype"):
        nv.mxfp4_gated_forward(a, a, dtype=torch.int8)


def test_activation_backward_refusals():
    L = block._lib()
    need = L.activation_backward_workspace_bytes(1, 1, 4000, 64)
    assert L.activation_backward_workspace_bytes(1, 1, 4, 64) == 0

    def f(type=1, bias_type=0, act=2, gated=1, dy=FAKE, dys=64, z=FAKE, zs=128, rows=4000, n=64,
          dz=FAKE, db=FAKE, ws=FAKE, bytes=need):
        return L.activation_backward(type, bias_type, act, gated, dy, dys, z, zs, rows, n, dz, db,
                                     ws, bytes, None)
    assert need > 0
    assert f(type=3) == nv.ERR_ARG and f(type=-1) == nv.ERR_ARG
    assert f(bias_type=2) == nv.ERR_ARG and f(type=0, bias_type=1) == nv.ERR_ARG
    assert f(act=5) == nv.ERR_ARG and f(act=-1) == nv.ERR_ARG and f(gated=2) == nv.ERR_ARG
    assert f(rows=-1) == nv.ERR_SHAPE and f(n=0) == nv.ERR_SHAPE
    assert f(dys=63) == nv.ERR_SHAPE and f(zs=127) == nv.ERR_SHAPE
    assert f(rows=1 << 31) == nv.ERR_ARG and f(n=1 << 31, dys=1 << 31, zs=1 << 32) == nv.ERR_ARG
    assert f(n=1 << 30, dys=1 << 30, zs=1 << 31, rows=1) == nv.ERR_ARG
    assert f(rows=1 << 20, n=1 << 20, dys=1 << 20, zs=1 << 21) == nv.ERR_ARG
    for name in ("dy", "z", "dz"):
        assert f(**{name: None}) == nv.ERR_NULL, name
        assert f(**{name: FAKE + 1}) == nv.ERR_ALIGN, name
    assert f(db=FAKE + 2) == nv.ERR_ALIGN and f(ws=FAKE + 8) == nv.ERR_ALIGN
    assert f(ws=None) == nv.ERR_WORKSPACE and f(bytes=need - 1) == nv.ERR_WORKSPACE
    if not _has_gpu():
        assert f() == nv.ERR_HIP and f(db=None, ws=None, bytes=0) == nv.ERR_HIP
        assert f(gated=0, act=0, z=None, zs=0) == nv.ERR_HIP
        assert f(gated=0, act=1, z=None) == nv.ERR_NULL
        assert f(rows=1, dys=0, zs=0, ws=None, bytes=0) == nv.ERR_HIP
        assert f(rows=0, dy=None, z=None, dz=None) == nv.ERR_HIP


def test_activation_backward_binding_refusals():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        nv.activation_backward(x, x, "gelu")
    with pytest.raises(ValueError, match="unknown activation"):
        nv.activation_backward(x, x, "tanh")


class CTensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("param", "grad", "m", "v", "m_scale", "v_scale",
                                               "master")] + \
               [("size", ctypes.c_int64), ("type", ctypes.c_int32), ("bits", ctypes.c_int32)]


def spread(k=0, **over):
    """A parameter of 100 bfloat16 elements whose tensors lie apart."""
    at = {name: FAKE + (7 * k + i) * 65536 for i, (name, _) in enumerate(CTensor._fields_[:7])}
    return CTensor(**{**at, **dict(size=100, type=1, bits=8), **over})


def step(*tensors, count=None, table=True, options=True, **over):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1, max_norm=1.0)
    o = optimizer._CAdamWOptions(**{**o, **over})
    rows = (CTensor * max(1, len(tensors)))(*tensors)
    return optimizer._lib().adamw_step(rows if table else None,
                                       len(tensors) if count is None else count,
                                       ctypes.byref(o) if options else None, None)


def test_adamw_refusals():
    for name in ("lr", "eps", "weight_decay"):
        for bad in (-1e-9, float("inf"), float("nan")):
            assert step(spread(), **{name: bad}) == nv.ERR_ARG, (name, bad)
    for name in ("beta1", "beta2"):
        for bad in (-0.1, 1.0, float("nan")):
            assert step(spread(), **{name: bad}) == nv.ERR_ARG, (name, bad)
    assert step(spread(), step=0) == nv.ERR_ARG
    assert step(spread(), norm=FAKE << 4, max_norm=-1.0) == nv.ERR_ARG
    assert step(spread(), norm=FAKE + 2) == nv.ERR_ALIGN
    assert step(spread(), step_device=FAKE + 4, step=0) == nv.ERR_ALIGN
    assert step(spread(), lr_device=FAKE + 2) == nv.ERR_ALIGN
    assert step(spread(), options=False) == nv.ERR_NULL
    assert step(spread(), table=False) == nv.ERR_NULL
    assert step(count=-1) == nv.ERR_SHAPE
    assert step(spread(size=-1)) == nv.ERR_SHAPE
    assert step(spread(size=1 << 40)) == nv.ERR_ARG
    assert step(spread(type=3)) == nv.ERR_ARG and step(spread(bits=16)) == nv.ERR_ARG
    assert step(spread(type=0)) == nv.ERR_ARG                       # float32 with a master
    for name in ("param", "grad", "m", "v", "m_scale", "v_scale"):
        assert step(spread(), spread(1, **{name: None})) == nv.ERR_NULL, name
    for name, by in (("param", 1), ("grad", 1), ("m", 4), ("v", 4), ("master", 2)):
        at = getattr(spread(), name) + by
        assert step(spread(**{name: at})) == nv.ERR_ALIGN, name
    if not _has_gpu():
        assert step(spread(), spread(1)) == nv.ERR_HIP
        assert step(spread(bits=32, m_scale=None, v_scale=None, master=None)) == nv.ERR_HIP
        assert step() == nv.ERR_HIP
        assert step(spread(param=None, size=0)) == nv.ERR_HIP
        assert step(spread(), step=0, step_device=FAKE) == nv.ERR_HIP
        assert step(spread(), lr=-1.0, lr_device=FAKE) == nv.ERR_HIP


def test_adamw_refuses_overlap():
    a, b = spread(), spread(1)
    assert step(a, a) == nv.ERR_ARG                                 # listed twice
    assert step(a, spread(1, param=a.param + 198)) == nv.ERR_ARG    # the last element of another
    assert step(b, spread(grad=b.param + 2)) == nv.ERR_ARG          # a gradient that is written
    assert step(a, spread(1, m=a.v + 120)) == nv.ERR_ARG
    assert step(spread(v_scale=a.m_scale)) == nv.ERR_ARG
    assert step(spread(master=a.m + 124)) == nv.ERR_ARG
    assert step(spread(bits=32, m=a.v - 396)) == nv.ERR_ARG
    if not _has_gpu():
        assert step(b, a) == nv.ERR_HIP                             # any order
        assert step(a, spread(1, param=a.param + 200)) == nv.ERR_HIP
        assert step(a, spread(1, grad=a.grad)) == nv.ERR_HIP        # gradients may be shared
        assert step(a, spread(1, grad=a.grad + 4)) == nv.ERR_HIP
        assert step(spread(master=a.m + 128)) == nv.ERR_HIP         # past one block of codes
        flat = [CTensor(param=FAKE + 200 * k, grad=FAKE + 10 ** 6 + 200 * k,
                        m=FAKE + 2 * 10 ** 6 + 128 * k, v=FAKE + 3 * 10 ** 6 + 128 * k,
                        m_scale=FAKE + 4 * 10 ** 6 + k, v_scale=FAKE + 5 * 10 ** 6 + k, size=100,
                        type=1, bits=8) for k in range(300)]
        assert step(*flat) == nv.ERR_HIP


def test_moment_values_refusals():
    def f(codes=FAKE, scales=FAKE, blocks=4, second=0, out=FAKE):
        return optimizer._lib().adamw_moment_values(codes, scales, blocks, second, out, None)
    assert f(second=2) == nv.ERR_ARG and f(blocks=-1) == nv.ERR_SHAPE
    assert f(blocks=1 << 33) == nv.ERR_ARG
    assert f(codes=None) == nv.ERR_NULL and f(scales=None) == nv.ERR_NULL
    assert f(out=None) == nv.ERR_NULL
    assert f(codes=FAKE + 4) == nv.ERR_ALIGN and f(out=FAKE + 2) == nv.ERR_ALIGN
    if not _has_gpu():
        assert f() == nv.ERR_HIP


def test_adamw_binding_refusals():
    p = torch.zeros(4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on one GPU"):
        nv.adamw_step([p], [p], [nv.adamw_state(p)], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="at least one"):
        nv.adamw_step([], [], [], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="go together"):
        nv.adamw_step([p], [p], [nv.adamw_state(p)], step=1, lr=1e-3, max_norm=1.0)
    with pytest.raises(ValueError, match="one length"):
        nv.adamw_step([p], [p, p], [nv.adamw_state(p)], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="must be a tuple"):
        nv.adamw_step([p], [p], [p], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="bits"):
        nv.adamw_state(p, bits=16)
    with pytest.raises(ValueError, match="bits"):
        nv.AdamW([torch.nn.Parameter(p)], bits=4)
    with pytest.raises(ValueError, match="own master"):
        nv.adamw_state(p.float(), master=True)
    with pytest.raises(ValueError, match="float32, bfloat16"):
        nv.adamw_state(p.double())
    with pytest.raises(ValueError, match="uint8 device tensor"):
        nv.moment_values(p, p)


def test_adamw_state_of_a_parameter():
    p = torch.nn.Parameter(torch.randn(3, 100).to(torch.bfloat16))
    s = nv.adamw_state(p, bits=8, master=True)
    assert s.m.shape == s.v.shape == (3, 128) and s.m_scale.shape == (3,)
    assert not s.m.any() and not s.m_scale.any() and torch.equal(s.master, p.detach().float())
    s = nv.adamw_state(p)
    assert s.m.dtype is torch.float32 and s.m.shape == p.shape and s.master is None


def test_adamw_state_dict_keeps_types():
    # torch's own loading casts every tensor to the parameter's type
    p = torch.nn.Parameter(torch.randn(200).to(torch.bfloat16))
    q = torch.nn.Parameter(torch.randn(5))
    opt = nv.AdamW([{"params": [p], "bits": 8, "master": True}, {"params": [q], "lr": 1.0}])
    for group in opt.param_groups:
        for x in group["params"]:
            opt._state_of(x, group)["step"] = 7
    opt.state[p]["m"].random_(0, 255)
    opt.state[p]["master"].add_(1e-4)
    saved = opt.state_dict()
    new = nv.AdamW([{"params": [p], "bits": 8, "master": True}, {"params": [q]}])
    new.load_state_dict(saved)
    for x in (p, q):
        assert set(new.state[x]) == set(opt.state[x])
        for k, v in opt.state[x].items():
            w = new.state[x][k]
            if isinstance(v, torch.Tensor):
                assert w.dtype is v.dtype and torch.equal(w, v) and w.data_ptr() != v.data_ptr()
            else:
                assert w == v == 7
    assert new.param_groups[1]["lr"] == 1.0

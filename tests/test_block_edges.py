"""Edges of the feed-forward block's operators that need no GPU."""
import ctypes

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from unbiased_nvfp4_gradient_amd import block, linear, optimizer


def act_threads(type, rows, n, sums=1):
    x, y = ctypes.c_int64(), ctypes.c_int64()
    f = nv.lib().nvfp4t_act_threads
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int] + 2 * [ctypes.c_void_p]
    f.restype = None
    f(type, rows, n, sums, ctypes.byref(x), ctypes.byref(y))
    return x.value, y.value


@pytest.mark.parametrize("type", [0, 1, 2])
@pytest.mark.parametrize("n", [1, 1000, (1 << 29) - 32, (1 << 29) - 31, 1 << 29, (1 << 30) - 63,
                               1 << 30, (1 << 31) - 1])
def test_activation_backward_fits_a_launch(type, n):
    """Every width and number of rows that the entry point takes stays within a launch's 2^32 threads in
    a dimension, and 65535 workgroups in the second."""
    block._lib()
    for rows in (0, 1, 2, 300, 511, 512, 513, 5000, (1 << 31) - 1):
        if rows and n > ((1 << 40) - 1) // rows:
            continue
        for sums in (0, 1):
            x, y = act_threads(type, rows, n, sums)
            assert 256 <= x < 1 << 32 and 1 <= y <= 65535, (rows, sums, x, y)


@pytest.mark.parametrize("type,rows,n", [(1, 512, 64), (0, 512, 1000), (0, 257, 1000),
                                         (2, 128, 2048)])
def test_few_rows_without_sums_are_spread(type, rows, n):
    """One workgroup takes all rows of its columns for the sums' sake only."""
    assert act_threads(type, rows, n)[1] == 1 and act_threads(type, rows, n, 0)[1] > 1


def test_adamw_bounded_is_0_or_1():
    for bounded, status in ((2, nv.ERR_ARG), (-1, nv.ERR_ARG), (1, None), (0, None)):
        o = optimizer._CAdamWOptions(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1,
                                     bounded=bounded)
        got = optimizer._lib().adamw_step(None, 0, ctypes.byref(o), None)
        assert got == status if status else got in (nv.OK, nv.ERR_HIP)


def optimizer_with_state():
    p = torch.nn.Parameter(torch.randn(300).to(torch.bfloat16))
    opt = nv.AdamW([p], bits=8, master=True)
    opt._state_of(p, opt.param_groups[0])["step"] = 3
    opt.state[p]["m"].fill_(7)
    return p, opt


def test_load_state_dict_takes_what_its_hooks_return():
    """torch's hooks before loading may return another dictionary, and those after it may change the
    state; moments keep their types all the same."""
    p, opt = optimizer_with_state()
    saved = opt.state_dict()
    calls = []

    def before(optimizer, state_dict):
        calls.append("before")
        state = {k: dict(v, m=v["m"] + 1, step=9) for k, v in state_dict["state"].items()}
        return dict(state_dict, state=state)

    def after(optimizer):
        calls.append("after")
        assert optimizer.state[p]["m"].dtype is torch.uint8
        optimizer.state[p]["master"].fill_(0.25)
    new = nv.AdamW([p], bits=8, master=True)
    new.register_load_state_dict_pre_hook(before)
    new.register_load_state_dict_post_hook(after)
    for k in (1, 2):
        new.load_state_dict(saved)
        assert calls == k * ["before", "after"]
        state = new.state[p]
        assert state["step"] == 9 and state["m"].dtype is torch.uint8
        assert bool((state["m"] == 8).all()) and bool((state["master"] == 0.25).all())
    assert bool((opt.state[p]["m"] == 7).all()) and opt.state[p]["step"] == 3
    # and none that a failed load leaves behind
    with pytest.raises(ValueError):
        new.load_state_dict(dict(saved, param_groups=[]))
    assert len(new._optimizer_load_state_dict_pre_hooks) == 1
    assert len(new._optimizer_load_state_dict_post_hooks) == 1


def test_a_norm_elsewhere_is_refused_before_any_update(monkeypatch):
    """Parameters on two devices and a norm on one of them: nothing is stepped."""
    p = torch.nn.Parameter(torch.ones(8))
    q = torch.nn.Parameter(torch.ones(8, device="meta"))
    opt = nv.AdamW([p, q])
    for x in (p, q):
        x.grad = torch.ones_like(x)
    stepped = []
    monkeypatch.setattr(optimizer, "adamw_step",
                        lambda params, *args, **kw: stepped.extend(params))
    with pytest.raises(ValueError, match="norm must be"):
        opt.step(norm=torch.ones(1), max_norm=1.0)
    assert not stepped and not opt.state
    for norm in (dict(norm=torch.ones(1)), dict(max_norm=1.0)):
        with pytest.raises(ValueError, match="go together"):
            opt.step(**norm)
    assert not stepped and not opt.state
    opt.step()
    assert len(stepped) == 2 and opt.state[p]["step"] == opt.state[q]["step"] == 1


@pytest.mark.parametrize("gated", [False, True])
def test_z_is_kept_for_a_backward_pass_only(gated, monkeypatch):
    """The layer's forward pass where gradients are switched off, and where nobody asks for any."""
    kept = []

    def forward(a, b, *args, keep_z, dtype, **kw):
        kept.append(keep_z)
        y = torch.zeros(128, 128, dtype=dtype)
        return nv.MXLinearForward(y, torch.zeros(128, 128 * (1 + gated)) if keep_z else None)
    quantized = nv.MXQuantized(nv.empty_mx_layout(128, 128, "cpu"), None)
    monkeypatch.setattr(linear, "_quantize", lambda *args: quantized)
    monkeypatch.setattr(linear, "mxfp4_linear_forward", forward)
    monkeypatch.setattr(linear, "mxfp4_gated_forward", forward)
    layer = linear.QuartetLinear(128, 128, scheme="sr", scales="mx", activation="silu", gated=gated,
                                 dtype=torch.bfloat16)
    x = torch.zeros(128, 128, dtype=torch.bfloat16)
    assert layer(x).requires_grad and kept == [True]
    with torch.no_grad():
        assert not layer(x).requires_grad and kept == [True, False]
    with torch.inference_mode():
        layer(x)
    assert kept == [True, False, False]
    layer.requires_grad_(False)
    layer(x)
    assert kept == [True, False, False, False] and layer._seed == 4
    with torch.no_grad(), pytest.raises(ValueError, match="multiple of 128"):
        layer(x[:3])


@pytest.mark.parametrize("bad", [dict(bits=16), dict(lr=-1.0), dict(lr=float("nan")),
                                 dict(eps=-1e-8), dict(weight_decay=float("inf")),
                                 dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9))])
def test_a_refused_group_is_not_added(bad):
    """Else each later step would update the other groups and then be refused."""
    p, q = (torch.nn.Parameter(torch.ones(8)) for _ in range(2))
    opt = nv.AdamW([p])
    with pytest.raises(ValueError, match=next(iter(bad))):
        opt.add_param_group(dict(params=[q], **bad))
    assert len(opt.param_groups) == 1
    opt.add_param_group(dict(params=[q], lr=torch.tensor(0.5), betas=(0.0, 0.0), eps=0))
    with pytest.raises(ValueError, match=next(iter(bad))):
        nv.AdamW([p], **bad)

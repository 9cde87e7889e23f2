"""Host-side refusals of the training-step calls: argument checks that come before any CUDA
call (the pointers are never dereferenced), and the binding's own checks of tensors."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from invariant_selected_token_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAX_ROWS = int(re.search(r"#define RLK_MAX_ROWS (\d+)",
                         open(os.path.join(ROOT, "include", "rlk.h")).read()).group(1))
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


def refused(call, code, **kw):
    assert call(**kw) == code, kw


def test_status_name(L):
    assert L.rlk_status_string(8) == b"RLK_ERR_NONFINITE"
    assert binding.STATUS_NAMES[binding.RLK_ERR_NONFINITE] == "RLK_ERR_NONFINITE"


def test_policy_loss_refusals(L):
    ok = dict(lp=0x1000, old=0x2000, ref=0x3000, adv=0x4000, per_seq=0, act=0x5000, off=0x6000,
              S=2, T=100000, cl=0.2, ch=0.2, dual=0.0, kl=3, klc=0.1, red=1, scale=1.0, loss=0x7000,
              stats=0x8000, grad=0x9000, ws=0x10000, wsb=1 << 20, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_policy_loss(a["lp"], a["old"], a["ref"], a["adv"], a["per_seq"], a["act"],
                                 a["off"], a["S"], a["T"], a["cl"], a["ch"], a["dual"], a["kl"],
                                 a["klc"], a["red"], a["scale"], a["loss"], a["stats"], a["grad"],
                                 a["ws"], a["wsb"], a["status"], None)
    for kw in (dict(lp=None), dict(old=None), dict(adv=None), dict(loss=None), dict(stats=None),
               dict(ws=None), dict(T=-1), dict(T=MAX_ROWS + 1), dict(S=-1), dict(off=None),
               dict(cl=-0.1), dict(ch=-0.1), dict(cl=math.nan), dict(ch=math.inf), dict(dual=0.5),
               dict(dual=1.0), dict(dual=math.inf), dict(klc=math.nan), dict(scale=math.inf),
               dict(ref=None), dict(T=0, adv=None, per_seq=1)):
        refused(call, INVALID, **kw)
    for kw in (dict(kl=0), dict(kl=4), dict(red=3), dict(red=-1)):
        refused(call, UNSUPPORTED, **kw)
    for kw in (dict(lp=0x1002), dict(off=0x6001), dict(ws=0x10010), dict(grad=0x9002),
               dict(status=0x11002)):
        refused(call, ALIGNMENT, **kw)
    refused(call, WORKSPACE, wsb=100)
    assert L.rlk_policy_loss_workspace_size(-1, 1) == 0
    assert L.rlk_policy_loss_workspace_size(10, -1) == 0
    assert L.rlk_policy_loss_workspace_size(32768, 1024) == 0  # one launch, no workspace
    assert L.rlk_policy_loss_workspace_size(32769, 1) > 0
    assert L.rlk_policy_loss_workspace_size(10, 1025) > 1025 * 4
    assert L.rlk_policy_loss_workspace_size(1 << 20, 1 << 14) >= (1 << 14) * 4 + (1 << 10) * 16


def test_preference_loss_refusals(L):
    ok = dict(lp=0x1000, ref=0x2000, act=0x3000, off=0x4000, P=3, T=10, layout=0, kind=0, beta=0.1,
              eps=0.0, margin=0.0, scale=1.0, loss=0x5000, pair=0x6000, rew=0x7000, grad=0x8000, ws=None,
              wsb=0, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_preference_loss(a["lp"], a["ref"], a["act"], a["off"], a["P"], a["T"],
                                     a["layout"], a["kind"], a["beta"], a["eps"], a["margin"], 0,
                                     a["scale"], a["loss"], a["pair"], a["rew"], a["grad"],
                                     a["ws"], a["wsb"], a["status"], None)
    for kw in (dict(lp=None), dict(off=None), dict(loss=None), dict(pair=None), dict(rew=None),
               dict(T=-1), dict(T=MAX_ROWS + 1), dict(P=-1), dict(P=(1 << 30) + 1), dict(beta=0.0),
               dict(beta=-1.0), dict(beta=math.inf), dict(beta=math.nan), dict(eps=-0.1),
               dict(eps=1.5), dict(eps=math.nan), dict(kind=1, eps=0.1), dict(kind=2, eps=0.1),
               dict(kind=2, margin=0.5), dict(margin=math.nan), dict(scale=math.nan)):
        refused(call, INVALID, **kw)
    for kw in (dict(layout=2), dict(kind=3), dict(kind=-1)):
        refused(call, UNSUPPORTED, **kw)
    for kw in (dict(lp=0x1001), dict(off=0x4002), dict(rew=0x7002), dict(ws=0x10010),
               dict(status=0x11001)):
        refused(call, ALIGNMENT, **kw)
    # few pairs of many tokens need a workspace
    refused(call, INVALID, T=200000)
    refused(call, WORKSPACE, T=200000, ws=0x10000, wsb=100)
    assert L.rlk_preference_loss_workspace_size(200000, 3) >= 256 + 12 * (200000 // 256)
    assert L.rlk_preference_loss_workspace_size(10 ** 8, 40) == 0
    assert L.rlk_preference_loss_workspace_size(98000, 3) == 0
    assert L.rlk_preference_loss_workspace_size(-1, 3) == 0


@pytest.mark.parametrize("name,kw", [
    ("scale", {}), ("klc", {}), ("scale", dict(preference=True)), ("beta", dict(preference=True)), ("margin", dict(preference=True))])
def test_loss_parameters_beyond_fp32_are_refused(L, name, kw):
    """The kernels hold them in fp32, where they would be infinite: 0 times such a scale is NaN.
    The largest fp32 number itself passes this check (and the call fails at a later one)."""
    top = float(np.finfo(np.float32).max)

    def call(value):
        if kw.get("preference"):
            a = dict(beta=0.1, margin=0.0, scale=1.0)
            a[name] = value
            return L.rlk_preference_loss(0x1000, 0x2000, 0x3000, 0x4000, 3, 10, 0, 0, a["beta"], 0.0,
                                         a["margin"], 0, a["scale"], 0x5000, 0x6000, 0x7000, 0x8001,
                                         None, 0, None, None)
        a = dict(klc=0.1, scale=1.0)
        a[name] = value
        return L.rlk_policy_loss(0x1000, 0x2000, 0x3000, 0x4000, 0, 0x5000, 0x6000, 2, 100, 0.2,
                                 0.2, 0.0, 3, a["klc"], 1, a["scale"], 0x7000, 0x8000,
                                 0x9001, None, 0, None, None)
    for sign in (1.0, -1.0) if name in ("scale", "klc", "margin") else (1.0,):
        assert call(sign * 1.0001 * top) == INVALID and call(sign * 1e300) == INVALID
        assert call(sign * top) == ALIGNMENT  # of the misplaced grad_logprob
    assert call(0.5) == ALIGNMENT


def test_rmsnorm_backward_refusals(L):
    ok = dict(go=0x10000, god=0, x=0x20000, gamma=0x30000, eps=1e-6, res=None, T=100, H=4096,
              gx=0x40000, gxd=1, gg=0x50000, ws=0x60000, wsb=1 << 20)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_rmsnorm_backward(a["go"], a["god"], a["x"], a["gamma"], a["eps"], a["res"],
                                      a["T"], a["H"], a["gx"], a["gxd"], a["gg"], a["ws"],
                                      a["wsb"], None)
    for kw in (dict(go=None), dict(x=None), dict(gamma=None), dict(gx=None), dict(ws=None),
               dict(T=-1), dict(T=MAX_ROWS + 1), dict(eps=0.0), dict(eps=math.nan),
               dict(gx=0x10000)):  # in place over another type
        refused(call, INVALID, **kw)
    for kw in (dict(H=100), dict(H=0), dict(H=8256), dict(god=2), dict(gxd=2)):
        refused(call, UNSUPPORTED, **kw)
    for kw in (dict(go=0x10008), dict(x=0x20002), dict(res=0x70004), dict(gg=0x50004),
               dict(ws=0x60010)):
        refused(call, ALIGNMENT, **kw)
    refused(call, WORKSPACE, wsb=10)
    refused(call, OK, T=0, gg=None)
    assert L.rlk_rmsnorm_backward_workspace_size(100, 100) == 0
    assert L.rlk_rmsnorm_backward_workspace_size(16, 4096) == 0  # one launch, no workspace
    assert L.rlk_rmsnorm_backward_workspace_size(17, 4096) >= 17 * 4096 * 4


@pytest.mark.parametrize("eps,code", [(2.0 ** -149, INVALID), (2.0 ** -127, INVALID), (-1e-6, INVALID),
                                      (2.0 ** -126, ALIGNMENT), (1e-6, ALIGNMENT)])
def test_rmsnorm_backward_refuses_subnormal_eps(L, eps, code):
    """A row of zeros has rstd^2 = 1 / eps, which would be infinite."""
    assert L.rlk_rmsnorm_backward(0x10008, 0, 0x20000, 0x30000, eps, None, 100, 4096, 0x40000, 1,
                                  0x50000, 0x60000, 1 << 20, None) == code


def _arrays(ptrs, sizes, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes),
            (ctypes.c_int32 * n)(*types), n)


def test_grad_clip_refusals(L):
    def call(ptrs=(0x10000, 0x20000), outs=None, sizes=(16, 16), types=(0, 1), max_norm=1.0,
             norm=0x1000, scale=0x2000, ws=0x100, wsb=1 << 20, norm_only=False, status=None):
        p, s, t, n = _arrays(ptrs, sizes, types)
        o = p if outs is None else (ctypes.c_void_p * n)(*outs)
        if norm_only:
            return L.rlk_grad_norm(p, s, t, n, norm, ws, wsb, status, None)
        return L.rlk_grad_clip(p, o, s, t, n, max_norm, norm, scale, ws, wsb, status, None)
    for kw in (dict(ptrs=(None, 0x20000)), dict(sizes=(-1, 16)), dict(norm=None),
               dict(sizes=(1 << 20, 16), ws=None)):
        refused(call, INVALID, **kw)
        refused(call, INVALID, norm_only=True, **kw)
    for kw in (dict(scale=None), dict(max_norm=-1.0), dict(max_norm=math.nan),
               dict(outs=(0x30000, None)),
               dict(ptrs=(0x10000, 0x10000)),                   # the same gradient twice, in place
               dict(ptrs=(0x10000, 0x10020)),                   # overlapping gradients, in place
               dict(outs=(0x30000, 0x30020)),                   # overlapping outputs
               dict(outs=(0x10010, 0x30000)),                   # an output over its own input, shifted
               dict(outs=(0x20000, 0x30000)),                   # an output over another's input
               dict(outs=(0x30000, 0x1003e))):                  # the input's last bytes
        refused(call, INVALID, **kw)
    for kw in (dict(types=(0, 3)), dict(types=(-1, 0)), dict(sizes=((1 << 38) + 1, 1)), dict(sizes=(1 << 37, (1 << 37) + 1))):
        refused(call, UNSUPPORTED, **kw)
    for kw in (dict(ptrs=(0x10002, 0x20000)), dict(ptrs=(0x10000, 0x20001)),
               dict(outs=(0x30002, 0x40000)), dict(ws=0x110), dict(status=0x3002)):
        refused(call, ALIGNMENT, **kw)
    refused(call, ALIGNMENT, norm_only=True, status=0x3002)
    refused(call, WORKSPACE, sizes=(1 << 20, 16), ptrs=(0x10000, 0x10000000), wsb=4)
    # 16 KB pieces, each tensor counted as if it started at the last byte of a 16-byte line
    types = (ctypes.c_int32 * 2)(0, 1)
    sizes = (ctypes.c_int64 * 2)(95 * 4096 - 4, 8192 - 8)
    assert L.rlk_grad_norm_workspace_size(sizes, types, 2) == 0  # one launch, no workspace
    sizes[1] += 1
    assert L.rlk_grad_norm_workspace_size(sizes, types, 2) >= 97 * 8
    sizes[0] = -1
    assert L.rlk_grad_norm_workspace_size(sizes, types, 2) == 0
    assert L.rlk_grad_norm_workspace_size(None, types, 2) == 0
    assert L.rlk_grad_norm_workspace_size(sizes, None, 2) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    lp = torch.zeros(4)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.policy_loss(lp, lp, lp)
    with pytest.raises(TypeError):
        binding.policy_loss(lp.double(), lp, lp)
    with pytest.raises(TypeError):
        binding.policy_loss([0.0], lp, lp)
    with pytest.raises(ValueError):
        binding.preference_loss(lp, off)
    with pytest.raises(ValueError):
        binding.clip_grads([lp], 1.0)
    with pytest.raises(TypeError):
        binding.clip_grads([lp.double()], 1.0)
    with pytest.raises(TypeError):
        binding.grad_norm([lp.to(torch.int32)])
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.rmsnorm_backward(x, x, x[0])
    with pytest.raises(TypeError):
        binding.rmsnorm_backward(x, x.half(), x[0])

"""Host-side refusals of the block norms, the 8-bit checkpoints and the draft verification: argument
checks that come before any CUDA call (the pointers are never dereferenced), and the binding's own."""
import math
import os
import re

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


@pytest.mark.parametrize("name", ["rlk_act_quantize", "rlk_act_dequantize"])
def test_act_refusals(L, name):
    def call(a=0x10000, b=0x20000, s=0x30001, fmt=1, T=10, H=4096):
        if name == "rlk_act_quantize":
            return L.rlk_act_quantize(a, fmt, T, H, b, s, None)
        return L.rlk_act_dequantize(a, s, fmt, T, H, b, None)
    for kw in (dict(a=None), dict(b=None), dict(s=None), dict(T=-1), dict(T=MAX_ROWS + 1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(fmt=0), dict(fmt=3), dict(H=0), dict(H=96), dict(H=(1 << 20) + 64)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(a=0x10008), dict(b=0x20004)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(T=0, a=None, b=None, s=None) == OK


def test_block_norm_refusals(L):
    ok = dict(b=0x10000, post=0x20000, g=0x30000, kind=2, r=0x40000, rs=1.0, bs=1.0, pre=0x50000, eps=1e-6,
              T=10, H=4096, out=0x60000, ro=0x70000, fmt=1, sx=0x80000, sxs=0x90001, sb=0xa0000,
              sbs=0xb0001, sg=0xc0000, sgs=0xd0001)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_block_norm(a["b"], a["post"], a["g"], a["kind"], a["r"], a["rs"], a["bs"], a["pre"],
                                a["eps"], a["T"], a["H"], a["out"], a["ro"], a["fmt"], a["sx"], a["sxs"],
                                a["sb"], a["sbs"], a["sg"], a["sgs"], None)
    for kw in (dict(b=None), dict(r=None), dict(pre=None), dict(out=None), dict(ro=None), dict(T=-1),
               dict(T=MAX_ROWS + 1), dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf),
               dict(rs=math.inf), dict(bs=math.nan), dict(sx=None), dict(sxs=None), dict(sbs=None),
               dict(sb=None), dict(sgs=None), dict(g=None),      # a checkpoint of no gate
               dict(fmt=0),                                      # checkpoints without a format
               dict(out=0x70000), dict(out=0x40000), dict(ro=0x10000)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=100), dict(H=0), dict(H=8256), dict(kind=0), dict(kind=3), dict(fmt=3)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(b=0x10008), dict(post=0x20002), dict(g=0x30001), dict(out=0x60008), dict(sx=0x80004),
               dict(sg=0xc0008)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(T=0) == OK


def test_block_norm_backward_refusals(L):
    ok = dict(go=0x10000, god=1, res=0x20000, fmt=1, x=0x30000, xs=0x31001, b=0x40000, bs=0x41001, g=0x50000,
              gs=0x51001, kind=2, post=0x60000, pre=0x70000, rs=1.0, sc=1.0, eps=1e-6, T=100, H=4096,
              gr=0x80000, gb=0x90000, gg=0xa0000, gxd=1, gpre=0xb0000, gpost=0xc0000, ws=0xd0000, wsb=1 << 24)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_block_norm_backward(
            a["go"], a["god"], a["res"], a["fmt"], a["x"], a["xs"], a["b"], a["bs"], a["g"], a["gs"],
            a["kind"], a["post"], a["pre"], a["rs"], a["sc"], a["eps"], a["T"], a["H"], a["gr"], a["gb"],
            a["gg"], a["gxd"], a["gpre"], a["gpost"], a["ws"], a["wsb"], None)
    none = dict(gr=None, gb=None, gg=None, gpre=None, gpost=None)
    for kw in (dict(go=None), dict(x=None), dict(pre=None), dict(b=None, bs=None), dict(xs=None), dict(bs=None),
               dict(gs=None), dict(fmt=0), dict(ws=None), none, dict(T=-1), dict(T=MAX_ROWS + 1),
               dict(eps=0.0), dict(eps=2.0 ** -127), dict(eps=math.nan), dict(rs=math.nan), dict(sc=math.inf),
               dict(post=None),                       # grad_gamma_post without gamma_post
               dict(g=None, gs=None),                 # grad_gate without a gate
               dict(gr=0x10000, god=0),               # in place over another type
               dict(gb=0x20000), dict(gg=0x20000),    # only grad_residual may be grad_residual_out
               dict(gb=0x80000), dict(gg=0x90000), dict(gg=0x80000)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(H=100), dict(H=8256), dict(god=2), dict(gxd=2), dict(kind=0), dict(fmt=5), dict(fmt=-1)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(go=0x10008), dict(x=0x30008), dict(post=0x60002), dict(gr=0x80008), dict(gpre=0xb0004),
               dict(ws=0xd0010)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(wsb=100) == WORKSPACE
    assert call(T=0, **none) == OK
    size = L.rlk_block_norm_backward_workspace_size
    assert size(100, 4096) >= 100 * 2 * 4096 * 4 and size(10 ** 6, 4096) == size(152, 4096)
    assert size(-1, 4096) == 0 and size(10, 100) == 0


def test_rmsnorm_backward_q8_refusals(L):
    def call(go=0x10000, god=0, fmt=2, x=0x20000, xs=0x21001, gamma=0x30000, eps=1e-6, res=None, T=100, H=4096,
             gx=0x40000, gxd=1, gg=0x50000, ws=0x60000, wsb=1 << 24):
        return L.rlk_rmsnorm_backward_q8(go, god, fmt, x, xs, gamma, eps, res, T, H, gx, gxd, gg, ws, wsb, None)
    for kw in (dict(go=None), dict(x=None), dict(xs=None), dict(gamma=None), dict(gx=None), dict(ws=None),
               dict(T=-1), dict(eps=0.0), dict(gx=0x10000)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(fmt=0), dict(fmt=3), dict(H=100), dict(god=2), dict(gxd=3)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(x=0x20008), dict(gx=0x40008), dict(res=0x70002)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(wsb=8) == WORKSPACE
    assert call(T=0, gg=None, gx=None) == OK


def test_draft_verify_refusals(L):
    ok = dict(t=0x10000, td=0, ldt=1000, tok=0x20000, d=0x30000, dd=1, ldd=1000, lse=0x40000, u=0x50000, n=0x60000,
              ldn=1000, off=0x70000, act=None, D=8, S=2, V=1000, acc=0x80000, out=0x90000, lp=0xa0000,
              ws=0xb0000, wsb=1 << 20, status=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.rlk_draft_verify(a["t"], a["td"], a["ldt"], a["tok"], a["d"], a["dd"], a["ldd"], a["lse"], a["u"],
                                  a["n"], a["ldn"], a["off"], a["act"], a["D"], a["S"], a["V"], a["acc"],
                                  a["out"], a["lp"], a["ws"], a["wsb"], a["status"], None)
    for kw in (dict(t=None), dict(tok=None), dict(u=None), dict(n=None), dict(off=None), dict(acc=None),
               dict(out=None), dict(lp=None), dict(ws=None), dict(D=-1), dict(S=-1), dict(D=MAX_ROWS),
               dict(S=0), dict(ldt=999), dict(ldd=999), dict(ldn=999), dict(V=0),
               dict(d=None)):                          # a draft's lse without its logits
        assert call(**kw) == INVALID, kw
    for kw in (dict(td=2), dict(dd=2), dict(V=262145, ldt=262145, ldd=262145, ldn=262145)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(t=0x10002), dict(td=1, t=0x10001), dict(d=0x30001), dict(tok=0x20002), dict(n=0x60002),
               dict(off=0x70001), dict(ws=0xb0010), dict(status=0xc0002)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(wsb=100) == WORKSPACE
    assert call(D=0, S=0, t=None, d=None, lse=None) == OK
    size = L.rlk_draft_verify_workspace_size
    assert size(8, 2, 1000) >= 10 * 8 * 8
    assert size(-1, 2, 1000) == 0 and size(8, 2, 0) == 0 and size(MAX_ROWS, 1, 1000) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    g = x[0]
    saved = binding.Saved(torch.zeros((2, 64), dtype=torch.int8), torch.zeros((2, 2), dtype=torch.uint8))
    for call in (lambda: binding.act_quantize(x), lambda: binding.act_dequantize(saved),
                 lambda: binding.block_norm(x, x, g), lambda: binding.block_norm_backward(x, x, g),
                 lambda: binding.rmsnorm_backward_q8(x, saved, g),
                 lambda: binding.draft_verify(x, x, x, x, x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: binding.act_quantize(x.float()), lambda: binding.act_dequantize(x),
                 lambda: binding.block_norm(x, x.half(), g), lambda: binding.block_norm_backward([0.0], x, g)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        binding.act_quantize(x, "fp4")

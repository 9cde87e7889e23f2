"""A sigmoid gate on a block whose output is not normed: forward and all gradients against the fp64
definition.  In the backward the block itself stands where its norm would, and grad_block is the gated
gradient with no second reduction.  Tolerances as in test_gpu_block_norm.py, where they are derived."""
import numpy as np
import pytest
import torch
from test_gpu_block_norm import CASES, U, half_step, held, make, n64, tolerances

from oracle import block as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
RS, BS = 1.25, float(np.float32(-0.7))


@pytest.mark.parametrize("T,H", CASES)
def test_forward(rlk, cuda_device, T, H):
    a = make(T, H, cuda_device, T * H + 40, False, "sigmoid")
    out, x, _ = rlk.block_norm(**a, residual_scale=RS, block_scale=BS, eps=1e-5)
    want, t = B.block_stream(n64(a["block"]), n64(a["residual"]), None, n64(a["gate"]), "sigmoid", RS, BS, 1e-5)
    assert np.all(np.abs(n64(x) - want) <= 20 * U * np.abs(t) + U * np.abs(want) + half_step(x) * np.abs(want))
    assert torch.equal(out, rlk.rmsnorm(x, a["gamma_pre"], 1e-5)[0])
    for fmt in ("int8", "e4m3"):
        _, _, saved = rlk.block_norm(**a, residual_scale=RS, block_scale=BS, eps=1e-5, save=fmt)
        for s, of in zip(saved, (x, a["block"], a["gate"])):
            q = rlk.act_quantize(of, fmt)
            assert torch.equal(s.scales, q.scales) and torch.equal(s.codes.view(torch.uint8), q.codes.view(torch.uint8))


@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("go,gx,res", [(F32, F32, True), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, False)])
def test_backward(rlk, cuda_device, T, H, fmt, go, gx, res):
    a = make(T, H, cuda_device, T * H + 41, False, "sigmoid")
    a["gate"][0, :32] *= 30  # gates that are wide open and shut
    x = (a["residual"].float() + 0.3).to(BF16)
    kept, plain = held(rlk, a, x, fmt)
    g = torch.Generator(device=cuda_device)
    g.manual_seed(T + H)
    grad_out = (torch.randn(T, H, device=cuda_device, generator=g) * 0.01).to(go)
    grad_res = (torch.randn(T, H, device=cuda_device, generator=g) * 0.01).to(gx) if res else None
    kw = dict(gamma_pre=a["gamma_pre"], gate_kind="sigmoid", residual_scale=RS, block_scale=BS, eps=1e-5,
              grad_residual_out=grad_res, grad_dtype=gx)
    got = rlk.block_norm_backward(grad_out, **kept, **kw)
    want = B.block_backward(n64(grad_out), n64(plain["x"]), n64(a["gamma_pre"]), n64(plain["block"]), None, n64(plain["gate"]),
                            "sigmoid", RS, BS, 1e-5, n64(grad_res))
    tol = tolerances(a, plain, want, RS, BS, 1e-5, grad_out, grad_res)
    assert got.grad_gamma_post is None
    for name in ("grad_block", "grad_residual", "grad_gate", "grad_gamma_pre"):
        v = getattr(got, name)
        step = 0 if name == "grad_gamma_pre" else half_step(v) * np.abs(want[name])
        # a gate below -87 counts as -87, where gate and slope are e^-87 < 2^-125 and the true ones lie between that
        # and 0; above 86 e^-z < 2^-124, all of the slope, counts as 0; 2^-133 is the smallest step of bf16
        floor = 2.0 ** -133
        if name in ("grad_block", "grad_gate"):
            floor = floor + 2.0 ** -124 * np.abs(want["d"]) * (np.abs(want["n"]) if name == "grad_gate" else 1)
        assert np.all(np.abs(n64(v) - want[name]) <= tol[name] + step + floor), name
    if fmt != "bf16":
        for p, q in zip(got, rlk.block_norm_backward(grad_out, **plain, **kw)):
            assert (p is None and q is None) or torch.equal(p, q)

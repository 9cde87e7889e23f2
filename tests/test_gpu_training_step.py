"""The training-step operators together: norm, head logprob, loss, head backward, norm backward,
clipping -- one optimiser step's gradients against the fp64 chain, and captured in a graph."""
import numpy as np
import pytest
import torch

from invariant_selected_token_gb300 import workloads as WL
from oracle import linear_logprob as O
from oracle import rmsnorm as R
from oracle import training as TR

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def make(device, seed, T=96, H=256, V=1500):
    w = WL.small_case(T, H, V, seed=seed, w_std=0.05, inactive_frac=0.2)
    dw = WL.to_device(w, device)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return dict(w=w, W=dw.W, targets=dw.targets, active=dw.active,
                x=(r(T, H) * 2).to(torch.bfloat16), res=r(T, H).to(torch.bfloat16),
                gamma=(1 + 0.1 * r(H)).to(torch.bfloat16),
                grad_res=(r(T, H) * 0.01).to(torch.bfloat16), adv=r(8), noise=r(T) * 0.1,
                offsets=torch.tensor([0, 10, 24, 24, 40, 55, 70, 80, T], dtype=torch.int32, device=device))


def step(rlk, a, loss_kind, status, max_norm=0.05, saved=False):
    hidden, x_res = rlk.rmsnorm(a["x"], a["gamma"], 1e-6, a["res"], want_residual_out=True)
    if saved:
        lp, lse, logits = rlk.linear_logprob_save_logits(hidden, a["W"], a["targets"], a["active"], status=status)
    else:
        lp, lse = rlk.linear_logprob(hidden, a["W"], a["targets"], a["active"], status=status)
    if loss_kind == "policy":
        loss, _, g = rlk.policy_loss(lp, a["old"], a["adv"], ref_logprob=a["ref"], active=a["active"],
                                     seq_offsets=a["offsets"], advantages_per_seq=True, kl_coef=0.05,
                                     reduction="seq_mean", status=status)
    else:
        loss, _, _, g = rlk.preference_loss(lp, a["offsets"], ref_logprob=a["ref"], active=a["active"],
                                            status=status)
    if saved:
        dh, dW = rlk.linear_logprob_backward_from_logits(logits, hidden, a["W"], a["targets"], g, lse,
                                                         a["active"], status=status)
    else:
        dh, dW = rlk.linear_logprob_backward(hidden, a["W"], a["targets"], g, lse, a["active"], status=status)
    dx, dgamma = rlk.rmsnorm_backward(dh, x_res, a["gamma"], 1e-6, grad_residual=a["grad_res"],
                                      grad_dtype=torch.bfloat16)
    norm, scale = rlk.clip_grads([dW, dgamma], max_norm, status=status)
    return dict(hidden=hidden, x_res=x_res, lp=lp, loss=loss, g=g, dh=dh, dx=dx, norm=norm, scale=scale,
                dW=dW, dgamma=dgamma)


def with_rollout(rlk, a):
    """The rollout's and the reference model's logprobs: this model's with noise."""
    hidden, _ = rlk.rmsnorm(a["x"], a["gamma"], 1e-6, a["res"], want_residual_out=True)
    lp, _ = rlk.linear_logprob(hidden, a["W"], a["targets"], a["active"])
    a["old"], a["ref"] = lp + a["noise"], lp - 0.5 * a["noise"]
    return a


@pytest.mark.parametrize("loss_kind", ["policy", "preference"])
@pytest.mark.parametrize("saved", [False, True])
def test_one_step_against_the_fp64_chain(rlk, cuda_device, loss_kind, saved):
    a = with_rollout(rlk, make(cuda_device, 21))
    status = rlk.new_status(cuda_device)
    got = step(rlk, a, loss_kind, status, saved=saved)
    rlk.raise_on_device_status(status)
    lp64, _ = O.selected_logprob(bits(got["hidden"]), a["w"].W, a["w"].targets, a["w"].active)
    old, ref = a["old"].cpu().numpy(), a["ref"].cpu().numpy()
    off = a["offsets"].tolist()
    if loss_kind == "policy":
        loss, _, g, _ = TR.policy_loss(lp64, old, a["adv"].cpu().numpy(), ref, a["w"].active, off, True,
                                       kl_coef=0.05, reduction="seq_mean")
    else:
        loss, _, _, g, _ = TR.preference_loss(lp64, off, ref, a["w"].active)
    # the logprobs are within 1e-4 of fp64 (the forward's bound), which moves a ratio and with it
    # a gradient by at most that much of itself, and the loss by the sum of the gradients
    assert abs(float(got["loss"]) - loss) <= 1e-4 * np.abs(g).sum() + 1e-5 * abs(loss)
    assert np.abs(got["g"].cpu().numpy() - g).max() <= 2e-4 * np.abs(g).max()
    # the head's backward rounds G to bf16: 2^-9 of each entry, and p's own error
    dh, dW = O.backward(bits(got["hidden"]), a["w"].W, a["w"].targets, g, a["w"].active)
    assert np.abs(got["dh"].cpu().numpy() - dh).max() <= 2.0 ** -8 * np.abs(dh).max()
    x64, gam = R.decode_bf16(bits(got["x_res"])), R.decode_bf16(bits(a["gamma"]))
    dx, dgamma = TR.rmsnorm_backward(dh, x64, gam, 1e-6, R.decode_bf16(bits(a["grad_res"])))
    assert np.abs(R.decode_bf16(bits(got["dx"])) - dx).max() <= 2.0 ** -7 * np.abs(dx).max()
    norm, scale = TR.clip_scale([dW, dgamma], 0.05)
    assert scale < 1 and abs(float(got["norm"]) - norm) <= 2.0 ** -8 * norm
    assert np.abs(got["dW"].cpu().numpy() - dW * scale).max() <= 2.0 ** -7 * np.abs(dW * scale).max()
    assert np.abs(got["dgamma"].cpu().numpy() - dgamma * scale).max() <= 2.0 ** -7 * np.abs(dgamma * scale).max()


@pytest.mark.parametrize("loss_kind", ["policy", "preference"])
def test_the_step_in_a_graph(rlk, cuda_device, loss_kind):
    sets = [with_rollout(rlk, make(cuda_device, s)) for s in (22, 23)]
    status = rlk.new_status(cuda_device)
    eager = [step(rlk, a, loss_kind, status) for a in sets]
    held = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in sets[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(rlk, held, loss_kind, status)
    for a, e in zip(sets, eager):
        for k, v in a.items():
            if isinstance(v, torch.Tensor):
                held[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for k in e:
            assert torch.equal(out[k], e[k]), k
    rlk.raise_on_device_status(status)


def test_calls_at_once_on_two_streams(rlk, cuda_device):
    """Every operator on two streams at a time, small and large sizes mixed, each with its own
    buffers: the bits of the calls made one after the other."""
    g = torch.Generator(device=cuda_device)
    g.manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_device)  # noqa: E731

    def calls(T, H):
        lp, old, adv = -r(T).abs(), -r(T).abs(), r(T)
        off = torch.tensor([0, T // 5, T // 2, T // 2 + 1, T], dtype=torch.int32, device=cuda_device)
        act = (r(T) < 1).to(torch.uint8)
        x, dy = r(T % 977 + 3, H).to(torch.bfloat16), r(T % 977 + 3, H)
        gamma = r(H).to(torch.bfloat16)
        grads = [r(T), r(3 * T + 1).to(torch.bfloat16), r(7)]
        return [lambda: rlk.policy_loss(lp, old, adv, ref_logprob=old, active=act, seq_offsets=off, kl_coef=0.1,
                                        reduction="seq_mean"),
                lambda: rlk.preference_loss(lp, off, ref_logprob=old, active=act),
                lambda: rlk.rmsnorm_backward(dy, x, gamma),
                lambda: (*rlk.clip_grads(grads, 1.0, out=[torch.empty_like(t) for t in grads]), )]
    work = [calls(T, H) for T, H in ((700, 256), (9000, 1024), (300000, 4096))]
    want = [[f() for f in fs] for fs in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    got = []
    for rep in range(4):
        for fs in work:
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got.append([f() for f in (fs if k else fs[::-1])][::1 if k else -1])
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i // 2 % 3]):
            assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)

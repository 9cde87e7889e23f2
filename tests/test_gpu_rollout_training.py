"""The operators together, as they are used: a rollout verifies drafted tokens and keeps their strict
logprobs; the training step runs its trunk's last block norms with 8-bit checkpoints, finds the same
logprobs bit for bit, and takes the gradients back through the head, the norms and the gate."""
import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import linear_logprob as O

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(rlk, device, seed, H=256, V=1500, lens=(3, 0, 5, 2)):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    D, S = sum(lens), len(lens)
    T = D + S
    a = dict(lens=lens, offsets=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device),
             block=r(T, H).to(BF16), gate=r(T, H).to(BF16), residual=(2 * r(T, H)).to(BF16),
             gamma_post=(1 + 0.1 * r(H)).to(BF16), gamma_pre=(1 + 0.1 * r(H)).to(BF16), W=(0.15 * r(V, H)).to(BF16),
             uniforms=torch.rand(D, generator=g, device=device),
             noise=torch.rand(S, V, generator=g, device=device).clamp(min=1e-9).log().neg().clamp(min=1e-9),
             advantages=r(T), grad_res=(r(T, H) * 0.01).to(BF16))
    # a draft model that is the target with noise, and its sampled tokens
    hidden, _, _ = rlk.block_norm(a["block"], a["residual"], a["gamma_pre"], gamma_post=a["gamma_post"], gate=a["gate"])
    rows = torch.arange(D, device=device) + torch.repeat_interleave(torch.arange(S), torch.tensor(lens)).to(device)
    a["draft_logits"] = rlk.debug_logits(hidden, a["W"])[rows] + 0.5 * r(D, V)
    race = torch.rand(D, V, generator=g, device=device).clamp(min=1e-9).log().neg()
    a["draft_tokens"] = (torch.softmax(a["draft_logits"], 1) / race).argmax(1).to(torch.int32)
    _, a["draft_lse"] = rlk.logits_logprob(a["draft_logits"], a["draft_tokens"])
    return a


def rollout(rlk, a, status):
    hidden, _, _ = rlk.block_norm(a["block"], a["residual"], a["gamma_pre"], gamma_post=a["gamma_post"], gate=a["gate"])
    logits = rlk.debug_logits(hidden, a["W"])
    return rlk.draft_verify(logits, a["draft_tokens"], a["uniforms"], a["noise"], a["offsets"],
                            draft_logits=a["draft_logits"], draft_lse=a["draft_lse"], status=status)


def train(rlk, a, tokens, old, status, fmt="int8"):
    hidden, x, saved = rlk.block_norm(a["block"], a["residual"], a["gamma_pre"], gamma_post=a["gamma_post"],
                                      gate=a["gate"], save=fmt)
    active = (tokens >= 0).to(torch.uint8)
    targets = tokens.clamp(min=0)
    lp, lse = rlk.linear_logprob(hidden, a["W"], targets, active, status=status)
    loss, stats, g = rlk.policy_loss(lp, old, a["advantages"], active=active, status=status)
    dh, dW = rlk.linear_logprob_backward(hidden, a["W"], targets, g, lse, active, status=status)
    grads = rlk.block_norm_backward(dh, saved.x, a["gamma_pre"], block=saved.block, gamma_post=a["gamma_post"],
                                    gate=saved.gate, grad_residual_out=a["grad_res"], grad_dtype=BF16)
    return dict(lp=lp, loss=loss, stats=stats, g=g, dh=dh, dW=dW, saved=saved, active=active, targets=targets,
                hidden=hidden, **grads._asdict())


def test_the_trainer_finds_the_rollouts_logprobs(rlk, cuda_device):
    a = make(rlk, cuda_device, 41)
    status = rlk.new_status(cuda_device)
    accepted, tokens, old = rollout(rlk, a, status)
    got = train(rlk, a, tokens, old, status)
    rlk.raise_on_device_status(status)
    on = got["active"].bool()
    assert int(on.sum()) == int(accepted.sum()) + len(a["lens"])
    # the same bits: every ratio is exactly 1, nothing is clipped, and the loss is -mean(advantage)
    assert torch.equal(got["lp"].view(torch.int32)[on], old.view(torch.int32)[on])
    assert float(got["stats"][2]) == 0 and float(got["stats"][3]) == 0
    want = -a["advantages"][on].double().mean()
    assert abs(float(got["loss"]) - float(want)) <= 2.0 ** -20 * float(a["advantages"].abs().max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gradients_against_the_fp64_chain(rlk, cuda_device, fmt):
    a = make(rlk, cuda_device, 42)
    status = rlk.new_status(cuda_device)
    _, tokens, old = rollout(rlk, a, status)
    got = train(rlk, a, tokens, old, status, fmt)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    on = got["active"].cpu().numpy()
    g = np.where(on != 0, -n(a["advantages"]) / on.sum(), 0.0)
    dh, dW = O.backward(bits(got["hidden"]), bits(a["W"]), got["targets"].cpu().numpy(), g, on)
    # the head's backward rounds G to bf16: 2^-9 of each entry, and p's own error
    assert np.abs(n(got["dh"]) - dh).max() <= 2.0 ** -8 * np.abs(dh).max()
    assert np.abs(n(got["dW"]) - dW).max() <= 2.0 ** -8 * np.abs(dW).max()
    held = {k: n(rlk.act_dequantize(v)) for k, v in got["saved"]._asdict().items()}
    want = B.block_backward(dh, held["x"], n(a["gamma_pre"]), held["block"], n(a["gamma_post"]), held["gate"],
                            grad_res=n(a["grad_res"]))
    for name in ("grad_block", "grad_residual", "grad_gate", "grad_gamma_pre", "grad_gamma_post"):
        # dh's error passes through linear maps of a row, whose gain in the largest norm the rows of
        # a few hundred features keep below 8, and half a step of bf16
        assert np.abs(n(got[name]) - want[name]).max() <= 2.0 ** -5 * np.abs(want[name]).max(), name


def test_checkpoints_cost_little_gradient(rlk, cuda_device):
    """Against the backward from the bf16 tensors themselves: an int8 code is off by at most 2^-7 of the
    block's largest power of two, an e4m3 one by 2^-4 of the feature, and a gradient of the norms is
    linear in dy and smooth in x, block and gate."""
    a = make(rlk, cuda_device, 43)
    hidden, x, _ = rlk.block_norm(a["block"], a["residual"], a["gamma_pre"], gamma_post=a["gamma_post"], gate=a["gate"])
    dy = torch.randn(x.shape, device=cuda_device)
    kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], grad_dtype=torch.float32)
    exact = rlk.block_norm_backward(dy, x, block=a["block"], gate=a["gate"], **kw)
    for fmt, share in (("int8", 2.0 ** -5), ("e4m3", 2.0 ** -3)):
        got = rlk.block_norm_backward(dy, rlk.act_quantize(x, fmt), block=rlk.act_quantize(a["block"], fmt),
                                      gate=rlk.act_quantize(a["gate"], fmt), **kw)
        for p, q in zip(got, exact):
            assert float((p - q).norm()) <= share * float(q.norm())


def test_the_step_in_a_graph(rlk, cuda_device):
    sets = [make(rlk, cuda_device, s) for s in (44, 45)]
    status = rlk.new_status(cuda_device)

    def step(a):
        accepted, tokens, old = rollout(rlk, a, status)
        out = train(rlk, a, tokens, old, status)
        return [accepted, tokens, old, *(out[k] for k in ("lp", "loss", "dW", "grad_block", "grad_residual", "grad_gate",
                                                          "grad_gamma_pre", "grad_gamma_post"))]
    eager = [step(a) for a in sets]
    held = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in sets[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for a, e in zip(sets, eager):
        for k, v in a.items():
            if isinstance(v, torch.Tensor):
                held[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, e))
    rlk.raise_on_device_status(status)

"""Draft verification where the draft's row is masked: -infinity and NaN in some or all of its places.

A token whose q is 0 keeps its p; one whose q is NaN is never drawn, also where the token is drawn from
the target itself because p exceeds q nowhere.  Margins as in the parity tests: 2^-17 covers the
kernel's error of p and of a weight (2^-18)."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
MARGIN = 2.0 ** -17
F32, BF16 = torch.float32, torch.bfloat16
NAN, INF = float("nan"), float("inf")


def make(device, lens, V, seed, target=F32, draft=F32):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    exp = lambda *s: torch.rand(*s, generator=g, device=device).clamp(min=1e-9).log().neg().clamp(min=1e-9)  # noqa: E731
    S, D = len(lens), sum(lens)
    logits = (2 * r(D + S, V)).to(target)
    rows = torch.arange(D) + torch.repeat_interleave(torch.arange(S), torch.tensor(lens))
    q = (logits[rows.to(device)].float() + 0.7 * r(D, V)).to(draft)
    return dict(target_logits=logits, draft_tokens=q.float().argmax(1).to(torch.int32), uniforms=torch.rand(D, generator=g, device=device),
                noise=exp(S, V), draft_offsets=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device),
                draft_logits=q, draft_lse=torch.logsumexp(q.float(), 1))


def num(t):
    return None if t is None else t.double().cpu().numpy()


def check(rlk, a, status, least=0.9):
    acc, tok, lp = rlk.draft_verify(**a, status=status)
    want_acc, want_tok, want_lp, margin = B.draft_verify(
        num(a["target_logits"]), a["draft_tokens"].cpu().numpy(), num(a["uniforms"]), num(a["noise"]),
        a["draft_offsets"].cpu().numpy(), num(a["draft_logits"]), num(a["draft_lse"]))
    off, sure = a["draft_offsets"].cpu().numpy(), margin > MARGIN
    assert sure.mean() >= least
    for s in np.nonzero(sure)[0]:
        rows = slice(off[s] + s, off[s + 1] + s + 1)
        assert int(acc[s]) == want_acc[s] and tok[rows].tolist() == want_tok[rows].tolist(), s
    return acc, tok, lp


@pytest.mark.parametrize("V", [515, 5000, 100000])
@pytest.mark.parametrize("target,draft", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_minus_infinity_in_the_draft(rlk, cuda_device, V, target, draft):
    """A draft of a smaller vocabulary: the rest of its row is -infinity, and keeps the target's p."""
    a = make(cuda_device, [3, 0, 5, 1] * 5, V, 31, target, draft)
    gone = torch.rand(V, device=cuda_device) < 0.6
    gone[V * 3 // 4:] = True
    a["draft_logits"] = a["draft_logits"].masked_fill(gone, -INF)
    a["draft_lse"] = torch.logsumexp(a["draft_logits"].float(), 1)
    status = rlk.new_status(cuda_device)
    check(rlk, a, status)
    # drafts that their own row masks have q = 0 and are accepted, the others are refused: drawn from p - q,
    # of which most is where the draft has nothing
    a["uniforms"].fill_(1e30)
    off = a["draft_offsets"].tolist()
    masked = gone[a["draft_tokens"].long()].tolist()
    acc, tok, _ = check(rlk, a, status)
    assert acc.tolist() == [(masked[b:e] + [False]).index(False) for b, e in zip(off, off[1:])]
    assert gone[tok[tok >= 0].long()].any()
    # all of them masked
    a["draft_tokens"].fill_(V - 1)
    acc, tok, _ = check(rlk, a, status)
    assert acc.tolist() == [3, 0, 5, 1] * 5
    rlk.raise_on_device_status(status)


@pytest.mark.parametrize("V", [515, 50000])
@pytest.mark.parametrize("where", ["row", "lse"])
def test_a_draft_that_is_no_number_anywhere(rlk, cuda_device, V, where):
    a = make(cuda_device, [2, 1, 0, 3], V, 32)
    status = rlk.new_status(cuda_device)
    want = rlk.draft_verify(**dict(a, uniforms=torch.full_like(a["uniforms"], 1e30)), status=status)
    rlk.raise_on_device_status(status)
    if where == "row":
        a["draft_logits"][3] = NAN  # the last sequence's first draft
    else:
        a["draft_lse"][3] = NAN
    a["uniforms"].fill_(1e30)
    acc, tok, lp = rlk.draft_verify(**a, status=status)
    assert int(status) == 1 << rlk.RLK_ERR_NONFINITE
    assert acc.tolist() == [0] * 4 and tok[6:].tolist() == [-1] * 4 and torch.isnan(lp[6]) and not lp[7:].any()
    assert torch.equal(tok[:6], want[1][:6]) and torch.equal(lp[:6], want[2][:6])


@pytest.mark.parametrize("V", [515, 4099, 50000, 100000])
@pytest.mark.parametrize("target,draft", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_drawn_from_the_target_where_the_draft_is_a_number(rlk, cuda_device, V, target, draft):
    """q above p in every place that is a number (its lse is a good 1 too small), NaN in the rest, the
    likeliest places among them."""
    lens = [2, 1, 3, 1]
    a = make(cuda_device, lens, V, 33, target, draft)
    rows = torch.tensor([0, 1, 3, 5, 6, 7, 9], device=cuda_device)
    q = a["target_logits"][rows].float()
    a["draft_lse"] = torch.logsumexp(q, 1) - 1.25
    bad = torch.rand(V, device=cuda_device) < 0.7
    bad[a["target_logits"][rows].float().amax(0) > 3.0] = True
    bad[V // 2] = False
    a["draft_logits"] = q.to(draft).masked_fill(bad, NAN)
    a["uniforms"].fill_(1e30)
    status = rlk.new_status(cuda_device)
    acc, tok, lp = check(rlk, a, status)
    rlk.raise_on_device_status(status)
    first = torch.tensor([0, 3, 5, 9], device=cuda_device)
    assert not acc.any() and not bad[tok[first].long()].any()
    # the same tokens as with infinite noise in those places and a draft of numbers
    b = dict(a, draft_logits=q.to(draft), noise=a["noise"].masked_fill(bad[None], INF))
    assert torch.equal(rlk.draft_verify(**b)[1][first], tok[first])
    # one place left
    keep = V // 2
    a["draft_logits"].fill_(NAN)
    a["draft_logits"][:, keep] = 30.0
    assert torch.all(rlk.draft_verify(**a, status=status)[1][first] == keep)
    rlk.raise_on_device_status(status)


@pytest.mark.parametrize("V", [16, 3001, 100000])
def test_ties_of_the_target_alone_go_to_the_lowest_token(rlk, cuda_device, V):
    a = make(cuda_device, [1, 1], V, 34)
    a["target_logits"].fill_(1.5)
    a["draft_logits"].fill_(1.5)
    a["draft_lse"].fill_(0.0)
    a["noise"].fill_(2.0)
    a["uniforms"].fill_(1e30)
    a["draft_logits"][1, :V // 3] = NAN
    assert rlk.draft_verify(**a)[1].tolist() == [0, -1, V // 3, -1]

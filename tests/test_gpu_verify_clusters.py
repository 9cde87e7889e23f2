"""Draft verification with every number of CTAs a sequence (8, 4, 2 and 1, by how many sequences there
are) and sequences of more rows than one group of the cluster finishes at a time (8 rows a CTA).

Decisions against the fp64 definition where its own margin is above 2^-17 (the kernel's error of a weight
is 2^-18 of p), and bit for bit against each sequence alone, which eight CTAs work on."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
MARGIN = 2.0 ** -17


def make(device, lens, V, seed):
    """Uniform numbers that refuse a draft in the first, second or a later group of rows, or nowhere."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    S, D = len(lens), int(sum(lens))
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    target = 2 * torch.randn(D + S, V, generator=g, device=device)
    rows = np.arange(D) + np.repeat(np.arange(S), lens)
    q = target[torch.from_numpy(rows).to(device)] + 0.7 * torch.randn(D, V, generator=g, device=device)
    u = np.full(D, 1e-6, np.float32)
    for s in range(S):
        stop = rng.integers(0, lens[s] + 2)  # some nowhere
        if stop < lens[s]:
            u[off[s] + stop] = 1e30
            u[off[s] + stop + 1:off[s + 1]] = rng.random(lens[s] - stop - 1)
    noise = torch.rand(S, V, generator=g, device=device).clamp(min=1e-9).log().neg().clamp(min=1e-9)
    return dict(target_logits=target, draft_tokens=q.argmax(1).to(torch.int32), uniforms=torch.from_numpy(u).to(device), noise=noise,
                draft_offsets=torch.from_numpy(off).to(device), draft_logits=q, draft_lse=torch.logsumexp(q, 1))


def num(t):
    return None if t is None else t.double().cpu().numpy()


# sequences, and the CTAs that each has on 152 SMs
@pytest.mark.parametrize("seqs,ctas", [(3, 8), (70, 8), (77, 4), (150, 4), (153, 2), (200, 2), (304, 2), (305, 1), (420, 1)])
@pytest.mark.parametrize("V,certain", [(517, False), (4099, False), (300, True)])
def test_long_sequences(rlk, cuda_device, seqs, ctas, V, certain):
    rng = np.random.default_rng(seqs + V)
    lens = rng.integers(0, 5, seqs)
    lens[rng.permutation(seqs)[:max(3, seqs // 8)]] = rng.integers(9, 42, max(3, seqs // 8))
    lens[0], lens[-1] = 8 * ctas, 8 * ctas + 1  # the row behind the last draft opens a group of its own
    a = make(cuda_device, lens, V, seqs * 7 + V)
    if certain:
        a["draft_logits"] = a["draft_lse"] = None
    status = rlk.new_status(cuda_device)
    acc, tok, lp = rlk.draft_verify(**a, status=status)
    rlk.raise_on_device_status(status)
    off = a["draft_offsets"].cpu().numpy()
    want_acc, want_tok, _, margin = B.draft_verify(num(a["target_logits"]), a["draft_tokens"].cpu().numpy(), num(a["uniforms"]),
                                                   num(a["noise"]), off, num(a["draft_logits"]), num(a["draft_lse"]))
    sure = margin > MARGIN
    assert sure.mean() >= 0.95
    got_acc, got_tok = acc.cpu().numpy(), tok.cpu().numpy()
    for s in np.nonzero(sure)[0]:
        rows = slice(off[s] + s, off[s + 1] + s + 1)
        assert got_acc[s] == want_acc[s] and np.array_equal(got_tok[rows], want_tok[rows]), s
    if ctas <= 2 and not certain:  # decided in the first group of rows and behind it
        assert (got_acc[lens > 8 * ctas] < 8 * ctas).any() and (got_acc >= 8 * ctas).any()
    on = tok >= 0
    strict, _ = rlk.logits_logprob(a["target_logits"], tok.clamp(min=0))
    assert torch.equal(lp.view(torch.int32)[on], strict.view(torch.int32)[on]) and not lp[~on].any()
    # alone: the same bits
    for s in sorted({0, seqs - 1, *np.argsort(-lens)[:4].tolist(), *rng.integers(0, seqs, 4).tolist()}):
        b, e = int(off[s]), int(off[s + 1])
        one = rlk.draft_verify(a["target_logits"][b + s:e + s + 1], a["draft_tokens"][b:e], a["uniforms"][b:e], a["noise"][s:s + 1],
                               torch.tensor([0, e - b], dtype=torch.int32, device=cuda_device),
                               draft_logits=None if certain else a["draft_logits"][b:e], draft_lse=None if certain else a["draft_lse"][b:e])
        assert int(one[0]) == int(acc[s]) and torch.equal(one[1], tok[b + s:e + s + 1])
        assert torch.equal(one[2].view(torch.int32), lp[b + s:e + s + 1].view(torch.int32))


@pytest.mark.parametrize("seqs,ctas", [(5, 8), (100, 4), (200, 2), (400, 1)])
@pytest.mark.parametrize("V", [517, 2049])
def test_refusals_around_the_end_of_a_group_of_rows(rlk, cuda_device, seqs, ctas, V):
    """Certain drafts of the likeliest token: u = 0 accepts, u = 2 refuses.  One place refuses in each sequence, the
    last sequence accepts all of its own."""
    group = 8 * ctas
    places = [group - 1, group, group + 1, 2 * group]
    lens = np.full(seqs, 2, np.int64)
    lens[:4] = 2 * group + 3
    lens[-1] = 2 * group + ctas + 1
    a = make(cuda_device, lens, V, seqs)
    off = a["draft_offsets"].cpu().numpy()
    rows = torch.from_numpy(np.arange(off[-1]) + np.repeat(np.arange(seqs), lens)).to(cuda_device)
    a.update(draft_logits=None, draft_lse=None, draft_tokens=a["target_logits"][rows].argmax(1).to(torch.int32))
    u = np.zeros(off[-1], np.float32)
    stops = [int(lens[s]) for s in range(seqs)]
    for s in range(4):
        stops[s] = places[s]
        u[off[s] + places[s]] = 2.0
    a["uniforms"] = torch.from_numpy(u).to(cuda_device)
    acc, tok, lp = rlk.draft_verify(**a)
    assert acc.tolist() == stops
    on = torch.zeros(len(tok), dtype=torch.bool)
    for s in range(seqs):
        b = off[s] + s
        on[b:b + stops[s] + 1] = True
        assert torch.equal(tok[b:b + stops[s]], a["draft_tokens"][off[s]:off[s] + stops[s]])
    assert torch.equal((tok >= 0).cpu(), on)
    strict, _ = rlk.logits_logprob(a["target_logits"], tok.clamp(min=0))
    assert torch.equal(lp[on], strict[on]) and not lp[~on].any()
    for s in range(4):  # the refused token is not drawn
        assert int(tok[off[s] + s + stops[s]]) != int(a["draft_tokens"][off[s] + stops[s]])


@pytest.mark.parametrize("target,draft", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("V", [1000, 50257, 100000, 151936])
def test_types_of_target_and_draft_apart(rlk, cuda_device, target, draft, V):
    lens = [3, 0, 5, 2, 1, 4] * 2
    a = make(cuda_device, lens, V, V + 1)
    a["target_logits"] = a["target_logits"].to(target)
    a["draft_logits"] = a["draft_logits"].to(draft)
    a["uniforms"] = torch.rand(sum(lens), device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(V))
    a["draft_lse"] = torch.logsumexp(a["draft_logits"].float(), 1)
    off = a["draft_offsets"].cpu().numpy()
    acc, tok, lp = rlk.draft_verify(**a)
    want_acc, want_tok, _, margin = B.draft_verify(num(a["target_logits"]), a["draft_tokens"].cpu().numpy(), num(a["uniforms"]),
                                                   num(a["noise"]), off, num(a["draft_logits"]), num(a["draft_lse"]))
    sure = margin > MARGIN
    assert sure.mean() >= 0.9
    for s in np.nonzero(sure)[0]:
        rows = slice(off[s] + s, off[s + 1] + s + 1)
        assert int(acc[s]) == want_acc[s] and tok[rows].tolist() == want_tok[rows].tolist(), s
    on = tok >= 0
    strict, _ = rlk.logits_logprob(a["target_logits"], tok.clamp(min=0))
    assert torch.equal(lp.view(torch.int32)[on], strict.view(torch.int32)[on])

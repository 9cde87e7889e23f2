"""Draft verification on the GPU against the fp64 definition.

Decisions are compared where the definition's own are not within the kernel's error of the border:
p errs by less than 2^-19 relatively (the row's sum: 7 levels in a tile and at most 11 above, each with a
rounding and an exponential of 1.5 u, u = 2^-24; exponential and quotient 4 u), q and the product with u by
6 u, a weight by 2^-18 of p (and the quotient by e by u of itself).  The inputs are such that nearly every
sequence is further than that from going the other way; how many are is asserted too.  Logprobs have
logits_logprob's bits."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
MARGIN = 2.0 ** -17
F32, BF16 = torch.float32, torch.bfloat16


def make(device, lens, V, seed, dtype=F32, draft="logits", noise=0.7, scale=2.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    S, D = len(lens), sum(lens)
    target = (scale * r(D + S, V)).to(dtype)
    ids = torch.repeat_interleave(torch.arange(S), torch.tensor(lens))
    rows = torch.arange(D) + ids
    q = (target[rows.to(device)].float() + noise * r(D, V)).to(dtype)
    lse = torch.logsumexp(q.float(), 1)
    race = torch.rand(D, V, generator=g, device=device).clamp(min=1e-9).log().neg()
    tokens = (torch.softmax(q.float(), 1) / race).argmax(1).to(torch.int32) if D else torch.zeros(0, dtype=torch.int32, device=device)
    a = dict(target_logits=target, draft_tokens=tokens, uniforms=torch.rand(D, generator=g, device=device),
             noise=torch.rand(S, V, generator=g, device=device).clamp(min=1e-9).log().neg().clamp(min=1e-9),
             draft_offsets=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=device),
             draft_logits=q, draft_lse=lse)
    if draft == "logp":
        a["draft_logits"], a["draft_lse"] = q.float() - lse[:, None], None
    if draft == "none":
        a["draft_logits"] = a["draft_lse"] = None
        a["draft_tokens"] = torch.where(torch.rand(D, generator=g, device=device) < 0.6,
                                        target[rows.to(device)].float().argmax(1).to(torch.int32), tokens) if D else tokens
    return a


def num(t):
    return None if t is None else t.double().cpu().numpy()


def check(rlk, a, status, least=0.95):
    acc, tok, lp = rlk.draft_verify(**a, status=status)
    want_acc, want_tok, want_lp, margin = B.draft_verify(
        num(a["target_logits"]), a["draft_tokens"].cpu().numpy(), num(a["uniforms"]), num(a["noise"]),
        a["draft_offsets"].cpu().numpy(), num(a["draft_logits"]), num(a["draft_lse"]),
        None if a.get("active") is None else a["active"].cpu().numpy())
    off = a["draft_offsets"].cpu().numpy()
    sure = margin > MARGIN
    assert sure.mean() >= least
    got_acc, got_tok = acc.cpu().numpy(), tok.cpu().numpy()
    for s in np.nonzero(sure)[0]:
        rows = slice(off[s] + s, off[s + 1] + s + 1)
        assert got_acc[s] == want_acc[s] and np.array_equal(got_tok[rows], want_tok[rows]), s
    # every emitted token's logprob has the strict path's bits
    on = tok >= 0
    strict, _ = rlk.logits_logprob(a["target_logits"], tok.clamp(min=0))
    assert torch.equal(lp.view(torch.int32)[on], strict.view(torch.int32)[on]) and not lp[~on].any()
    return acc, tok, lp


@pytest.mark.parametrize("lens,V", [([0], 1000), ([4], 50257), ([3, 0, 1, 5, 2], 1), ([2, 2, 2], 2), ([1] * 40, 127),
                                    ([0, 7, 0, 3], 128), ([5, 4], 129), ([2, 3, 1, 0, 8] * 8, 4099), ([600], 1000),
                                    ([1] * 200 + [0] * 200, 515), ([8, 3, 6], 151936)])
@pytest.mark.parametrize("dtype,draft", [(F32, "logits"), (BF16, "logits"), (F32, "none"), (BF16, "logp")])
def test_parity(rlk, cuda_device, lens, V, dtype, draft):
    status = rlk.new_status(cuda_device)
    a = make(cuda_device, lens, V, len(lens) + V, dtype, draft)
    # bf16 logits of few tokens tie: p = q, and a margin of nothing
    check(rlk, a, status, 0.95 if V > 2 else 0.0)
    rlk.raise_on_device_status(status)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padded_and_misaligned_rows(rlk, cuda_device, dtype):
    V = 1003
    a = make(cuda_device, [3, 1, 4], V, 5, dtype)
    want = rlk.draft_verify(**a)
    for pad, shift in ((1, 1), (29, 4), (5, 8)):
        moved = dict(a)
        for name in ("target_logits", "draft_logits", "noise"):
            t = a[name]
            buf = torch.full((t.shape[0], V + pad + shift), float("nan"), dtype=t.dtype, device=cuda_device)
            moved[name] = buf[:, shift:shift + V]
            moved[name].copy_(t)
        for p, q in zip(rlk.draft_verify(**moved), want):
            assert torch.equal(p.view(torch.int32), q.view(torch.int32))


@pytest.mark.parametrize("V", [130, 40000])
def test_all_accepted_and_none(rlk, cuda_device, V):
    status = rlk.new_status(cuda_device)
    lens = [4, 0, 2, 7]
    a = make(cuda_device, lens, V, 6)
    a["uniforms"].zero_()
    acc, tok, _ = check(rlk, a, status)
    assert acc.tolist() == lens and torch.all(tok >= 0)
    a["uniforms"].fill_(1e30)  # beyond any ratio
    acc, tok, _ = check(rlk, a, status)
    assert not acc.any() and int((tok >= 0).sum()) == len(lens)
    rlk.raise_on_device_status(status)


def test_masked_logits(rlk, cuda_device):
    """-inf (and the type's lowest value) in most places of target and draft: such tokens are never
    drawn, and a draft of one is refused."""
    status = rlk.new_status(cuda_device)
    for dtype, low in ((F32, -float("inf")), (BF16, -float("inf")), (F32, torch.finfo(F32).min), (BF16, torch.finfo(BF16).min)):
        V = 5000
        a = make(cuda_device, [3, 0, 5, 1] * 5, V, 8, dtype)
        allowed = torch.rand(a["target_logits"].shape, device=cuda_device) < 0.01
        allowed[:, 17] = True
        a["target_logits"] = a["target_logits"].masked_fill(~allowed, low)
        acc, tok, _ = check(rlk, a, status)
        on = tok >= 0
        rows = torch.nonzero(on)[:, 0]
        assert torch.all(allowed[rows, tok[on].long()])
    rlk.raise_on_device_status(status)


def test_one_token_left(rlk, cuda_device):
    a = make(cuda_device, [1, 0], 1000, 9)
    a["target_logits"].fill_(-float("inf"))
    a["target_logits"][:, 777] = -5.0
    acc, tok, lp = rlk.draft_verify(**a)
    hit = int(a["draft_tokens"][0]) == 777
    assert tok.tolist() == ([777, 777, 777] if hit else [777, -1, 777]) and not lp.any()


def test_no_token_where_the_target_exceeds_the_draft(rlk, cuda_device):
    """Draft "probabilities" above the target's everywhere: drawn from the target itself."""
    status = rlk.new_status(cuda_device)
    a = make(cuda_device, [2, 1, 3], 700, 10)
    a["draft_logits"] = a["target_logits"][torch.tensor([0, 1, 3, 5, 6, 7], device=cuda_device)].clone()
    a["draft_lse"] = torch.logsumexp(a["draft_logits"], 1) - 1.0
    a["uniforms"].fill_(0.9)
    acc, tok, _ = check(rlk, a, status)
    assert not acc.any()
    rlk.raise_on_device_status(status)


@pytest.mark.parametrize("V", [16, 3000, 100000])
def test_ties_go_to_the_lowest_token(rlk, cuda_device, V):
    a = make(cuda_device, [0, 0], V, 11)
    a["target_logits"].fill_(1.5)
    a["noise"].fill_(2.0)
    assert rlk.draft_verify(**a)[1].tolist() == [0, 0]
    a["noise"][1, :V // 2] = 3.0
    assert rlk.draft_verify(**a)[1].tolist() == [0, V // 2]


def test_rows_that_are_not_distributions(rlk, cuda_device):
    V = 2000
    for value, where in ((float("nan"), 5), (float("inf"), 5), (-float("inf"), slice(None))):
        a = make(cuda_device, [2, 2, 0], V, 12)
        a["uniforms"].zero_()
        clean = rlk.draft_verify(**a)
        status = rlk.new_status(cuda_device)
        a["target_logits"][4, where] = value  # the second sequence's second row
        acc, tok, lp = rlk.draft_verify(**a, status=status)
        with pytest.raises(rlk.RlkError) as e:
            rlk.raise_on_device_status(status)
        assert e.value.code == rlk.RLK_ERR_NONFINITE
        assert acc.tolist() == [2, 1, 0] and tok[4:6].tolist() == [-1, -1]
        assert torch.isnan(lp[4]) and lp[5] == 0
        for p, q in zip((tok, lp), clean[1:]):
            assert torch.equal(p[:4], q[:4]) and torch.equal(p[6:], q[6:])
    # behind the first refusal nothing is looked at
    a = make(cuda_device, [3], V, 13)
    a["uniforms"].fill_(1e30)
    status = rlk.new_status(cuda_device)
    want = rlk.draft_verify(**a)
    a["target_logits"][1:] = float("nan")
    a["draft_logits"][1:] = float("nan")
    a["draft_tokens"][1:] = -5
    for p, q in zip(rlk.draft_verify(**a, status=status), want):
        assert torch.equal(p, q)
    rlk.raise_on_device_status(status)


def test_noise_of_any_positive_size(rlk, cuda_device):
    """The race is run over the whole fp32 range of weights and noise: the smallest normal noise on an
    unlikely token, the largest on the others."""
    a = make(cuda_device, [0] * 4, 3001, 14, scale=0.1)
    a["noise"].fill_(3.0e38)
    a["target_logits"][0, 1234] = -80.0
    a["noise"][0, 1234] = 2.0 ** -126
    a["target_logits"][1, 2345] = -30.0
    a["noise"][1, 2345] = 1.0
    a["noise"][2] = 1.0
    a["noise"][2, 77] = 2.0 ** -126
    a["target_logits"][3, 9] = 5.0
    assert rlk.draft_verify(**a)[1].tolist() == [1234, 2345, 77, 9]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [3001, 50000])
def test_subnormal_noise_on_subnormal_probabilities(rlk, cuda_device, V, dtype):
    """p = e^-94 is a subnormal number and so is the token's noise: their quotient, 1.1, is the largest weight
    by far, by p alone and from a draft that gives the token less."""
    a = make(cuda_device, [0, 1, 1], V, 26, dtype)
    a["target_logits"].fill_(-94.0)
    a["target_logits"][:, 11] = 0.0
    a["noise"].fill_(1.0)
    a["noise"][:, 11] = 1.0e4
    a["draft_logits"].fill_(-100.0)
    a["draft_logits"][:, 11] = 0.0
    a["draft_lse"].zero_()
    a["draft_tokens"].fill_(11)
    a["uniforms"].copy_(torch.tensor([0.0, 1e30], device=cuda_device))
    for at in (0, 1000, V - 1):
        noise = a["noise"].clone()
        noise[:, at] = 1.4e-41
        acc, tok, _ = rlk.draft_verify(**dict(a, noise=noise))
        assert acc.tolist() == [0, 1, 0] and tok.tolist() == [at, 11, at, at, -1]


@pytest.mark.parametrize("V", [3001, 50000])
def test_tokens_without_a_noise_or_a_draft_are_never_drawn(rlk, cuda_device, V):
    """NaN in the noise, or in the refused draft's row, takes those tokens out; where all are, none is
    drawn."""
    a = make(cuda_device, [2, 1, 0, 3], V, 25)
    a["uniforms"].fill_(1e30)
    bad = torch.rand(V, device=cuda_device) < 0.7
    for name, rows in (("noise", 4), ("draft_logits", 6)):
        b = dict(a, **{name: a[name].clone()})
        b[name][:, bad] = float("nan")
        status = rlk.new_status(cuda_device)
        acc, tok, _ = rlk.draft_verify(**b, status=status)
        rlk.raise_on_device_status(status)
        drawn = tok[tok >= 0].long()
        drawn = drawn if name == "noise" else tok[[0, 3, 6]].long()
        assert not acc.any() and not bad[drawn].any()
        # the same as with those tokens' noise beyond all others
        c = dict(a, noise=a["noise"].masked_fill(bad[None], float("inf")))
        same = rlk.draft_verify(**c)[1]
        assert torch.equal(tok, same) if name == "noise" else torch.equal(tok[[0, 3, 6]], same[[0, 3, 6]])
    b = dict(a, noise=torch.full_like(a["noise"], float("nan")))
    status = rlk.new_status(cuda_device)
    acc, tok, lp = rlk.draft_verify(**b, status=status)
    assert int(status) == 1 << rlk.RLK_ERR_NONFINITE and torch.all(tok == -1)


def test_tokens_and_offsets_out_of_range(rlk, cuda_device):
    V = 900
    a = make(cuda_device, [2, 3, 1], V, 15)
    a["uniforms"].zero_()
    want = rlk.draft_verify(**a)
    for bad in (V, -1, 2 ** 31 - 1, -2 ** 31):
        b = dict(a, draft_tokens=a["draft_tokens"].clone())
        b["draft_tokens"][3] = bad
        status = rlk.new_status(cuda_device)
        acc, tok, lp = rlk.draft_verify(**b, status=status)
        assert int(status) == 1 << rlk.RLK_ERR_TARGET_RANGE
        assert acc.tolist() == [2, 1, 1] and 0 <= int(tok[4]) < V and tok[5:7].tolist() == [-1, -1]
        assert torch.equal(tok[:4], want[1][:4]) and torch.equal(tok[7:], want[1][7:])
    for off, lost in (([0, 2, 1, 6], [1]), ([-1, 2, 5, 6], [0]), ([0, 2, 5, 7], [2]), ([0, 2 ** 31 - 1, 5, 6], [0, 1])):
        status = rlk.new_status(cuda_device)
        out = dict(accepted=torch.full((3,), 99, dtype=torch.int32, device=cuda_device),
                   tokens=torch.full((11,), 99, dtype=torch.int32, device=cuda_device)[1:10],
                   logprob=torch.full((9,), 99.0, device=cuda_device))
        b = dict(a, draft_offsets=torch.tensor(off, dtype=torch.int32, device=cuda_device))
        acc, tok, lp = rlk.draft_verify(**b, **out, status=status)
        assert int(status) & (1 << rlk.RLK_ERR_INVALID_ARG)
        assert [s for s in range(3) if int(acc[s]) == -1] == lost


def test_rows_of_no_sequence_are_left_alone(rlk, cuda_device):
    V = 800
    a = make(cuda_device, [2, 3, 2], V, 16)
    a["draft_offsets"] = torch.tensor([1, 3, 3, 5], dtype=torch.int32, device=cuda_device)
    out = dict(tokens=torch.full((10,), 99, dtype=torch.int32, device=cuda_device), logprob=torch.full((10,), 99.0, device=cuda_device))
    status = rlk.new_status(cuda_device)
    acc, tok, lp = rlk.draft_verify(**a, **out, status=status)
    rlk.raise_on_device_status(status)
    written = torch.zeros(10, dtype=torch.bool)
    for s, (b, e) in enumerate(((1, 3), (3, 3), (3, 5))):
        written[b + s:e + s + 1] = True
    assert torch.equal((tok != 99).cpu(), written) and torch.equal((lp != 99).cpu(), written)


def test_inactive_sequences(rlk, cuda_device):
    V = 3000
    a = make(cuda_device, [2, 3, 0, 4], V, 17)
    want = rlk.draft_verify(**a)
    a["active"] = torch.tensor([1, 0, 0, 7], dtype=torch.uint8, device=cuda_device)
    a["target_logits"][3:8] = float("nan")
    a["draft_logits"][2:5] = float("nan")
    a["draft_tokens"][2:5] = -9
    status = rlk.new_status(cuda_device)
    acc, tok, lp = rlk.draft_verify(**a, status=status)
    rlk.raise_on_device_status(status)
    assert torch.all(tok[3:8] == -1) and not lp[3:8].any() and acc[1:3].tolist() == [0, 0]
    for p, q in zip((tok, lp), want[1:]):
        assert torch.equal(p[:3], q[:3]) and torch.equal(p[8:], q[8:])


@pytest.mark.parametrize("V", [515, 50257])
def test_a_sequence_does_not_depend_on_the_batch(rlk, cuda_device, V):
    """One sequence alone (eight CTAs) and among hundreds (one or two): the same bits."""
    lens = [3, 1, 0, 5] * 80 if V < 1000 else [3, 1, 0, 5] * 20
    a = make(cuda_device, lens, V, 18)
    acc, tok, lp = rlk.draft_verify(**a)
    for s in (0, 1, 2, 3, len(lens) - 1):
        b, e = int(a["draft_offsets"][s]), int(a["draft_offsets"][s + 1])
        one = rlk.draft_verify(a["target_logits"][b + s:e + s + 1], a["draft_tokens"][b:e], a["uniforms"][b:e],
                               a["noise"][s:s + 1], torch.tensor([0, e - b], dtype=torch.int32, device=cuda_device),
                               draft_logits=a["draft_logits"][b:e], draft_lse=a["draft_lse"][b:e])
        assert int(one[0]) == int(acc[s]) and torch.equal(one[1], tok[b + s:e + s + 1])
        assert torch.equal(one[2].view(torch.int32), lp[b + s:e + s + 1].view(torch.int32))


def test_emitted_tokens_follow_the_target(rlk, cuda_device):
    """40000 sequences with the same two distributions: the first emitted token is distributed as the
    target's, whatever the draft's (each count within 5 standard deviations of a binomial's)."""
    V, S = 7, 40000
    g = torch.Generator(device=cuda_device)
    g.manual_seed(19)
    p, q = torch.randn(2, V, generator=g, device=cuda_device)
    tokens = torch.multinomial(torch.softmax(q, 0), S, replacement=True, generator=g).to(torch.int32)
    exp = lambda *s: torch.rand(*s, generator=g, device=cuda_device).clamp(min=1e-9).log().neg().clamp(min=1e-9)  # noqa: E731
    off = torch.arange(S + 1, dtype=torch.int32, device=cuda_device)
    for draft in (q, None):
        acc, tok, _ = rlk.draft_verify(p.expand(2 * S, V).contiguous(), tokens, torch.rand(S, generator=g, device=cuda_device),
                                       exp(S, V), off,
                                       draft_logits=None if draft is None else draft.expand(S, V).contiguous(),
                                       draft_lse=None if draft is None else torch.logsumexp(draft, 0).expand(S).contiguous())
        first = tok.view(S, 2)[:, 0].long()
        want = num(torch.softmax(p.double(), 0))
        if draft is None:  # certain drafts: kept with p(x), else drawn from the rest
            assert abs(float(acc.float().mean()) - float(num(torch.softmax(p, 0))[tokens.cpu().numpy()].mean())) < 0.02
        count = np.bincount(first.cpu().numpy(), minlength=V)
        assert np.all(np.abs(count - S * want) <= 5 * np.sqrt(S * want * (1 - want)))
        second = tok.view(S, 2)[:, 1]
        assert torch.equal(second >= 0, acc == 1)


def test_graph_replay_streams_and_two_at_once(rlk, cuda_device):
    sets = [make(cuda_device, [3, 0, 2, 6], 20011, s) for s in (20, 21)]
    eager = [rlk.draft_verify(**a) for a in sets]
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(cuda_device))
    got = [[rlk.draft_verify(**sets[k], stream=streams[k]) for k in range(2)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for k in range(2):
            assert all(torch.equal(p, q) for p, q in zip(pair[k], eager[k]))
    held = {k: (None if v is None else v.clone()) for k, v in sets[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rlk.draft_verify(**held)
    for a, e in zip(sets, eager):
        for k, v in a.items():
            held[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, e))


def test_rows_past_2_31_elements(rlk, cuda_device):
    """The last sequence of a batch whose target and draft pass 2^31 elements."""
    V, S = 262144, 4100
    a = make(cuda_device, [3], V, 22, BF16)
    n = 2 * S
    target = torch.zeros((n + 4, V), dtype=BF16, device=cuda_device)
    target[-4:] = a["target_logits"]
    draft = torch.zeros((S * 2 + 3, V), dtype=BF16, device=cuda_device)[S:]
    draft[-3:] = a["draft_logits"]
    tokens = torch.zeros(S + 3, dtype=torch.int32, device=cuda_device)
    tokens[-3:] = a["draft_tokens"]
    u = torch.zeros(S + 3, device=cuda_device)
    u[-3:] = a["uniforms"]
    noise = torch.ones((S + 1, V), device=cuda_device)
    noise[-1:] = a["noise"]
    off = torch.cat([torch.arange(S + 1, device=cuda_device), torch.tensor([S + 3], device=cuda_device)]).to(torch.int32)
    lse = torch.full((S + 3,), float(np.log(V)), device=cuda_device)
    lse[-3:] = a["draft_lse"]
    acc, tok, lp = rlk.draft_verify(target, tokens, u, noise, off, draft_logits=draft, draft_lse=lse)
    want = rlk.draft_verify(**a)
    assert int(acc[-1]) == int(want[0][0]) and torch.equal(tok[-4:], want[1]) and torch.equal(lp[-4:], want[2])
    assert torch.all(acc[:-1] == 1) and torch.all(tok[:-4] == 0)


def test_binding_checks(rlk, cuda_device):
    a = make(cuda_device, [2, 1], 500, 23)
    call = lambda **kw: rlk.draft_verify(**dict(a, **kw))  # noqa: E731
    for kw in (dict(target_logits=a["target_logits"].half()), dict(noise=a["noise"].to(BF16)),
               dict(draft_tokens=a["draft_tokens"].long()), dict(draft_logits=a["draft_logits"].double())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(target_logits=a["target_logits"][:4]), dict(noise=a["noise"][:, :400]),
               dict(draft_logits=a["draft_logits"][:2]), dict(uniforms=a["uniforms"][:2]),
               dict(target_logits=a["target_logits"].t().contiguous().t()), dict(draft_lse=a["draft_lse"][:1]),
               dict(active=torch.ones(3, dtype=torch.uint8, device=cuda_device)),
               dict(tokens=torch.zeros(4, dtype=torch.int32, device=cuda_device))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(draft_logits=None), dict(noise=a["noise"][:1].expand(2, 500)),
               dict(workspace=torch.empty(255, dtype=torch.uint8, device=cuda_device))):
        with pytest.raises(rlk.RlkError):
            call(**kw)
    none = make(cuda_device, [0, 0, 0], 500, 24)
    acc, tok, _ = rlk.draft_verify(**none)
    assert not acc.any() and torch.all(tok >= 0)
    empty = rlk.draft_verify(none["target_logits"][:0], none["draft_tokens"], none["uniforms"], none["noise"][:0],
                             torch.zeros(1, dtype=torch.int32, device=cuda_device))
    assert [t.numel() for t in empty] == [0, 0, 0]

"""Preference loss on the GPU against the fp64 definition.

Tolerances (u = 2^-24): a log ratio is held exactly as two floats and its sum compensated, so m
errs by far less than u (sum |d|) 2^-10 + n 2^-46 sum |d|; rewards are rounded once (u |beta m|).
z is rounded once: u |z|.  e^-|z| then errs by (2 + |z|) u of itself, log(1 + e) and the
sigmoids by 8 u of themselves more: the loss is within u (|z| + 12 l) and dl/dz within
u (12 + |z|) of the sum of its two absolute parts.  IPO's square doubles the relative error of
its root, whose own is 2^-50: three roundings.  Grads are rounded once."""
import numpy as np
import pytest
import torch

from oracle import training as TR

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def batch(T, offsets, seed, mask=0.8, ref=True):
    rng = np.random.default_rng(seed)
    base = -np.abs(rng.standard_normal(T)) ** 2
    lp = (base + 0.2 * rng.standard_normal(T)).astype(np.float32)
    return dict(lp=lp, ref=base.astype(np.float32) if ref else None, offsets=offsets,
                active=(rng.random(T) < mask).astype(np.uint8) if mask < 1 else None)


def dev(a, device, dtype=None):
    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).to(device)


def run(rlk, device, b, **kw):
    status = rlk.new_status(device)
    out = rlk.preference_loss(dev(b["lp"], device), dev(b["offsets"], device, np.int32),
                              ref_logprob=dev(b["ref"], device), active=dev(b["active"], device),
                              status=status, **kw)
    rlk.raise_on_device_status(status)
    return [x.cpu().numpy() for x in out]


def check(out, b, **kw):
    loss, pair, rewards, grad = out
    r_loss, r_pair, r_rew, r_grad, z = TR.preference_loss(b["lp"], b["offsets"], b["ref"], b["active"], **kw)
    beta, scale, kind = kw.get("beta", 0.1), kw.get("scale", 1.0), kw.get("kind", "sigmoid")
    total = np.abs(b["lp"] if b["ref"] is None else b["lp"].astype(np.float64) - b["ref"]).sum()
    m_err = total * (2.0 ** -34 + len(b["lp"]) * 2.0 ** -46)
    assert np.all(np.abs(rewards - r_rew) <= U * np.abs(r_rew) + beta * m_err)
    z_err = U * np.abs(z) + 2 * beta * m_err
    if kind == "ipo":
        pair_tol = 4 * U * r_pair + 4 * m_err * np.sqrt(r_pair)
    else:
        pair_tol = z_err + 12 * U * r_pair
    assert np.all(np.abs(pair - r_pair) <= pair_tol)
    assert abs(loss - r_loss) <= scale * pair_tol.mean() + U * abs(r_loss) if len(r_pair) else loss == 0
    big = np.abs(z).max() if len(z) else 0.0
    slope = {"sigmoid": beta, "hinge": beta, "ipo": 2 * np.sqrt(r_pair.max()) if len(r_pair) else 0}[kind]
    tol = (12 + big) * U * np.abs(r_grad) if kind != "sigmoid" else \
        scale / max(1, len(r_pair)) * slope * (12 + big) * U * np.ones_like(r_grad)
    tol = np.where(r_grad == 0, 0, tol + scale * 4 * m_err)
    assert np.all(np.abs(grad - r_grad) <= tol)


CASES = [
    (2, [0, 1, 2]),
    (11, [0, 4, 4, 4, 11]),                                   # sides without any token
    (700, [3, 40, 296, 297, 553, 553, 690]),                  # 256-token chunks met exactly
    (9001, [0, 4096, 8999]),
    (30000, [0] + list(range(101, 29990, 467))[:63] + [30000]),
    (3000, [0] + list(range(20, 2990, 3))[:599] + [3000]),     # hundreds of tiny pairs
    (600001, [0, 262144 + 1, 300000, 300001, 600000]),        # more than 1024 chunks in one
    (400003, [7, 7, 200000, 200000, 400000]),                 # long pairs with empty sides
    (300000, [9, 9, 9, 9, 9]),
]


@pytest.mark.parametrize("T,offsets", CASES)
@pytest.mark.parametrize("kw", [
    dict(), dict(label_smoothing=0.2, margin=0.3, layout="halves"),
    dict(kind="hinge", margin=-0.1, beta=0.02), dict(kind="ipo", length_normalize=True, layout="halves"),
    dict(length_normalize=True, beta=2.0, scale=0.25)])
@pytest.mark.parametrize("mask,ref", [(0.7, True), (1.0, False)])
def test_preference_loss_parity(rlk, cuda_device, T, offsets, kw, mask, ref):
    b = batch(T, offsets, seed=T, mask=mask, ref=ref)
    check(run(rlk, cuda_device, b, **kw), b, **kw)


@pytest.mark.parametrize("beta,h", [(0.1, 10), (0.2, 5), (0.05, 20), (0.3, 4), (0.1, 9), (0.7, 2)])
def test_hinge_of_whole_numbers(rlk, cuda_device, beta, h):
    """Sums that are whole numbers may meet the border z = 1 exactly: the decision is that of beta
    itself, not of its value in fp32."""
    margin = round(beta * h - 1.0, 6)
    lp = np.array([-1.0] * h + [-2.0] * h, np.float32)
    b = dict(lp=lp, ref=np.full(2 * h, -1.5, np.float32), active=None, offsets=[0, h, 2 * h])
    kw = dict(kind="hinge", beta=beta, margin=margin)
    out = run(rlk, cuda_device, b, **kw)
    z = beta * h - margin
    assert out[3].any() == (z < 1.0)
    check(out, b, **kw)


@pytest.mark.parametrize("T,offsets", [CASES[2], CASES[4], CASES[6], CASES[7]])
@pytest.mark.parametrize("layout", ["adjacent", "halves"])
def test_the_loss_alone(rlk, cuda_device, T, offsets, layout):
    b = batch(T, offsets, seed=T)
    args = (dev(b["lp"], cuda_device), dev(b["offsets"], cuda_device, np.int32))
    kw = dict(ref_logprob=dev(b["ref"], cuda_device), active=dev(b["active"], cuda_device), layout=layout)
    full = rlk.preference_loss(*args, **kw)
    alone = rlk.preference_loss(*args, want_grad=False, **kw)
    assert alone[3] is None and all(torch.equal(x, y) for x, y in zip(full[:3], alone[:3]))


def test_gradient_against_differences(rlk, cuda_device):
    """Central differences of the loss in steps of 2^-4: the sigmoid loss's third derivative in
    one token is below 0.1 beta^3, so the quotient errs by h^2 / 6 of it plus two roundings of
    the loss over h."""
    b = batch(24, [0, 6, 11, 17, 24], seed=3)
    grad = run(rlk, cuda_device, b)[3]
    h = 2.0 ** -4
    for t in range(24):
        v = []
        for s in (h, -h):
            c = dict(b, lp=b["lp"].copy())
            c["lp"][t] += np.float32(s)
            v.append((float(run(rlk, cuda_device, c)[0]), float(c["lp"][t])))
        num = (v[0][0] - v[1][0]) / (v[0][1] - v[1][1])
        assert abs(num - grad[t]) <= h * h / 6 * 1e-4 + 16 * U / h


@pytest.mark.parametrize("lengths", [(40, 3000, 700, 1), (70000, 9, 300, 5000), (130000, 9, 300, 5000),
                                     (70000, 270000, 9, 0)])
def test_a_pairs_bits_do_not_depend_on_its_place(rlk, cuda_device, lengths):
    """The same sequences alone, shifted, among others and with the other layout."""
    n = sum(lengths)
    at = np.concatenate([[0], np.cumsum(lengths)])
    b = batch(n, list(at), seed=4)
    loss, pair, rew, grad = run(rlk, cuda_device, b, layout="adjacent")
    for shift in (1, 2, 77):
        pad = batch(n + shift + 50, list(at + shift), seed=5)
        for k in ("lp", "ref", "active"):
            pad[k][shift:shift + n] = b[k]
        l2, p2, r2, g2 = run(rlk, cuda_device, pad, layout="adjacent")
        assert l2 == loss and np.array_equal(p2, pair) and np.array_equal(r2, rew)
        assert np.array_equal(g2[shift:shift + n], grad)
        assert not g2[:shift].any() and not g2[shift + n:].any()
    # one pair alone: the same loss, and the gradient without the mean over two
    one = {k: (None if v is None else v[:at[2]]) for k, v in b.items() if k != "offsets"}
    one["offsets"] = list(at[:3])
    _, p1, r1, _ = run(rlk, cuda_device, one)
    assert np.array_equal(p1, pair[:1]) and np.array_equal(r1, rew[:2])
    # halves: chosen ones first
    order = [0, 2, 1, 3]
    h = {k: np.concatenate([b[k][at[i]:at[i + 1]] for i in order]) for k in ("lp", "ref", "active")}
    h["offsets"] = [0] + list(np.cumsum([lengths[i] for i in order]))
    l3, p3, r3, g3 = run(rlk, cuda_device, h, layout="halves")
    assert l3 == loss and np.array_equal(p3, pair) and np.array_equal(r3, rew[order])


def test_masked_tokens_may_hold_anything(rlk, cuda_device):
    b = batch(3000, [100, 900, 2900], seed=6, mask=0.6)
    clean = run(rlk, cuda_device, b)
    on = b["active"].astype(bool).copy()
    on[:100] = on[2900:] = False
    for bad in (np.nan, np.inf, -np.inf, np.finfo(np.float32).min):
        d = dict(b, lp=np.where(on, b["lp"], np.float32(bad)).astype(np.float32),
                 ref=np.where(on, b["ref"], np.float32(bad)).astype(np.float32))
        for x, y in zip(clean, run(rlk, cuda_device, d)):
            assert np.array_equal(x, y)


def test_far_margins_do_not_overflow(rlk, cuda_device):
    b = dict(lp=np.array([0.0, -5000.0, -5000.0, 0.0], np.float32), ref=None, active=None,
             offsets=[0, 1, 2, 3, 4])
    loss, pair, _, grad = run(rlk, cuda_device, b, beta=1.0)
    assert pair.tolist() == [0.0, 5000.0] and float(loss) == 2500.0
    assert grad.tolist() == [0.0, 0.0, -0.5, 0.5]


def test_infinite_margins(rlk, cuda_device):
    """A token of probability 0 on either side: the loss is 0 or infinite, its slope 0 or beta."""
    inf = np.inf
    b = dict(lp=np.array([-1.0, -inf, -inf, -1.0], np.float32), ref=None, active=None,
             offsets=[0, 1, 2, 3, 4])
    _, pair, rew, grad = run(rlk, cuda_device, b, beta=1.0)
    assert pair.tolist() == [0.0, inf] and rew.tolist() == [-1.0, -inf, -inf, -1.0]
    assert grad.tolist() == [0.0, 0.0, -0.5, 0.5]
    _, pair, _, _ = run(rlk, cuda_device, b, beta=1.0, label_smoothing=1.0)
    assert pair.tolist() == [inf, 0.0]


def test_one_sided_nan_stays_in_its_pair(rlk, cuda_device):
    b = batch(400, [0, 100, 200, 300, 400], seed=7, mask=1.0)
    b["lp"][150] = np.nan
    loss, pair, rew, grad = run(rlk, cuda_device, b)
    assert np.isnan(loss) and np.isnan(pair[0]) and np.isfinite(pair[1]) and np.isfinite(grad[200:]).all()
    assert np.isfinite(rew[[0, 2, 3]]).all() and np.isnan(rew[1])


@pytest.mark.parametrize("T", [1000, 70000, 300000])
@pytest.mark.parametrize("offsets", [[0, 700, 600, 800, 1000], [-1, 5, 5, 5, 5], [0, 1, 2, 3, 1001],
                                     [9, 2 ** 31 - 1, -2 ** 31, 5, 10], [0, 2 ** 31 - 1, 0, 2 ** 31 - 1, 0],
                                     [300400, 300400, 300400, 300400, 300400],
                                     [2 ** 31 - 1, 2 ** 31 - 1, 9, 9, 9], [0, 0, 0, -2 ** 31, -2 ** 31]])
def test_bad_offsets_are_reported(rlk, cuda_device, T, offsets):
    if offsets == [0, 1, 2, 3, 1001]:
        offsets = [0, 1, 2, 3, T + 1]
    b = batch(T, [0] * 5, seed=8)
    status = rlk.new_status(cuda_device)
    guard = torch.full((T + 512,), 7.0, device=cuda_device)
    loss = rlk.preference_loss(dev(b["lp"], cuda_device), dev(offsets, cuda_device, np.int32),
                               ref_logprob=dev(b["ref"], cuda_device), status=status,
                               grad_logprob=guard[256:256 + T])[0]
    with pytest.raises(rlk.RlkError) as e:
        rlk.raise_on_device_status(status)
    assert e.value.code == rlk.RLK_ERR_INVALID_ARG and torch.isnan(loss)
    assert torch.all(guard[:256] == 7) and torch.all(guard[256 + T:] == 7)


def test_more_than_2_31_bytes(rlk, cuda_device):
    """Positions whose byte offsets pass 32 bits: two sequences over 2^29 + 9 tokens."""
    T = 2 ** 29 + 9
    lp = torch.full((T,), -1.0, device=cuda_device)
    ref = torch.full((T,), -1.5, device=cuda_device)
    half = T // 2
    off = torch.tensor([0, half, T], dtype=torch.int32, device=cuda_device)
    loss, pair, rew, grad = rlk.preference_loss(lp, off, ref_logprob=ref, beta=1.0, margin=0.5)
    # m = half / 2 and (half + 1) / 2: h = -0.5, z = -1
    want = np.log1p(np.exp(1.0))
    assert rew.tolist() == [float(np.float32(half / 2)), float(np.float32((T - half) / 2))]
    assert abs(float(loss) - want) <= 16 * U
    slope = -1 / (1 + np.exp(-1.0))
    for t, s in ((0, 1), (half - 1, 1), (half, -1), (T - 1, -1)):
        assert abs(float(grad[t]) - s * slope) <= 16 * U


def test_no_pairs(rlk, cuda_device):
    x = torch.full((9,), -1.0, device=cuda_device)
    off = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    loss, pair, rew, grad = rlk.preference_loss(x, off)
    assert float(loss) == 0.0 and pair.numel() == 0 and rew.numel() == 0 and not grad.any()
    loss, pair, _, grad = rlk.preference_loss(x[:0], torch.zeros(3, dtype=torch.int32, device=cuda_device))
    assert abs(float(loss) - np.log(2)) <= 2 * U and grad.numel() == 0


@pytest.mark.parametrize("T,P", [(500, 3), (200000, 2)])
def test_graph_replay_and_streams(rlk, cuda_device, T, P):
    off = list(np.linspace(0, T, 2 * P + 1).astype(int))
    bs = [batch(T, off, seed=s) for s in (11, 12)]
    eager = [run(rlk, cuda_device, b) for b in bs]
    lp, ref, act = (dev(bs[0][k], cuda_device) for k in ("lp", "ref", "active"))
    o = dev(off, cuda_device, np.int32)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    other = rlk.preference_loss(lp, o, ref_logprob=ref, active=act, stream=s)
    s.synchronize()
    for x, y in zip(other, eager[0]):
        assert np.array_equal(x.cpu().numpy(), y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = rlk.preference_loss(lp, o, ref_logprob=ref, active=act)
    for b, e in zip(bs, eager):
        for t, k in ((lp, "lp"), (ref, "ref"), (act, "active")):
            t.copy_(dev(b[k], cuda_device))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, e):
            assert np.array_equal(x.cpu().numpy(), y)


def test_binding_shape_checks(rlk, cuda_device):
    x = torch.zeros(8, device=cuda_device)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=cuda_device)
    for call in (lambda: rlk.preference_loss(x, off[:2]), lambda: rlk.preference_loss(x, off, ref_logprob=x[:4]),
                 lambda: rlk.preference_loss(x, off, kind="kto"), lambda: rlk.preference_loss(x, off, layout="x"),
                 lambda: rlk.preference_loss(x, off[:0]),
                 lambda: rlk.preference_loss(x, off, grad_logprob=x[:3])):
        with pytest.raises(ValueError):
            call()

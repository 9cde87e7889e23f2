"""Clipped policy loss with a KL term on the GPU against the fp64 definition.

Tolerances, from the operations of one token (u = 2^-24, half a step of fp32).  The ratio r:
exp within 2u of e^d' for the rounded d', corrected by the rest of d to first order, 3u together.
r A, w (two conversions, a product and a division: 4u), scale w and the last product: the policy
term and its gradient are within 12 u |w r A|.  The KL terms: u' = ref - lp is rounded (u |u'|,
which moves e^u' by |u'| u e^u'), the series or e^u' - 1 - u' then errs by at most
4 u (e^u' + 1 + |u'|); the coefficient's rounding, w and the products add 8 u of the value.  A sum
of n positive-weight terms by the kernel's tree adds at most 16 roundings in fp32 (the product with
w, 2 over a lane's tokens, 5 over the lanes, 8 over the spans) of its absolute sum, then sums as
pairs of floats and one rounding."""
import numpy as np
import pytest
import torch

from oracle import training as TR

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def batch(T, offsets, seed, mask=0.8, spread=0.25):
    rng = np.random.default_rng(seed)
    old = (-np.abs(rng.standard_normal(T)) ** 2).astype(np.float32)
    lp = (old + spread * rng.standard_normal(T)).astype(np.float32)
    ref = (old + spread * rng.standard_normal(T)).astype(np.float32)
    active = (rng.random(T) < mask).astype(np.uint8) if mask < 1 else None
    return dict(lp=lp, old=old, ref=ref, active=active, offsets=offsets,
                adv_t=rng.standard_normal(T).astype(np.float32),
                adv_s=rng.standard_normal(len(offsets) - 1).astype(np.float32))


def dev(a, device, dtype=None):
    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))).to(device)


def run(rlk, device, b, per_seq=False, use_ref=True, **kw):
    status = rlk.new_status(device)
    out = rlk.policy_loss(dev(b["lp"], device), dev(b["old"], device),
                          dev(b["adv_s"] if per_seq else b["adv_t"], device),
                          ref_logprob=dev(b["ref"], device) if use_ref else None,
                          active=dev(b["active"], device),
                          seq_offsets=dev(b["offsets"], device, np.int32),
                          advantages_per_seq=per_seq, status=status, **kw)
    rlk.raise_on_device_status(status)
    return out


def bounds(b, ref_out, per_seq, use_ref, kl, kl_coef, scale):
    """Largest error of each grad and of the four stats, as the module comment derives them."""
    w = ref_out[3]
    T = w.shape[0]
    lp, old, ref = (b[k].astype(np.float64) for k in ("lp", "old", "ref"))
    A = np.zeros(T)
    o = b["offsets"]
    for s in range(len(o) - 1):
        A[o[s]:o[s + 1]] = b["adv_s"][s] if per_seq else b["adv_t"][o[s]:o[s + 1]]
    with np.errstate(over="ignore"):
        pol = np.where(w > 0, np.maximum(np.exp(np.minimum(lp - old, 80)), 4) * np.abs(A), 0)
        u = ref - lp
        e = np.exp(u)
        size = {"k1": 1 + np.abs(u), "k2": 1 + np.abs(u) + u * u,
                "k3": (4 + np.abs(u)) * (e + 1 + np.abs(u))}[kl]
    klb = np.where(w > 0, 12 * U * size, 0) if use_ref else np.zeros(T)
    grad = abs(scale) * w * (12 * U * pol + abs(kl_coef) * klb)
    n_u = 34 * U
    stats = np.array([(w * pol).sum() * n_u,
                      (w * (klb + 22 * U * np.where(w > 0, size, 0))).sum() if use_ref else 0.0,
                      w.sum() * n_u, (w * np.abs(lp - old)).sum() * n_u])
    return grad, stats + 1e-30


CASES = [
    # T, offsets
    (1, [0, 1]),
    (7, [0, 3, 3, 7]),                       # an empty sequence
    (300, [5, 40, 41, 41, 41, 200, 290]),    # tokens before the first and behind the last
    (1023, [0, 1023]),
    (1025, [0, 1000, 1025]),
    (5000, [0] + sorted(set(range(3, 4990, 37))) + [5000]),
    (40001, [0, 1, 20000, 39999, 40001]),
    (300001, [7, 120001, 120001, 299990]),
]


@pytest.mark.parametrize("T,offsets", CASES)
@pytest.mark.parametrize("per_seq,reduction,kl,dual,mask", [
    (True, "token_mean", "k3", 0.0, 0.8), (False, "seq_mean", "k3", 3.0, 0.8),
    (True, "seq_mean", "k1", 1.5, 1.0), (False, "sum", "k2", 0.0, 1.0),
    (False, "token_mean", "k1", 1.2, 1.0), (True, "sum", "k3", 0.0, 0.5)])
def test_policy_loss_parity(rlk, cuda_device, T, offsets, per_seq, reduction, kl, dual, mask):
    b = batch(T, offsets, seed=T + 1, mask=mask)
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=dual, kl=kl, kl_coef=0.05,
              reduction=reduction, scale=0.5)
    loss, stats, grad = run(rlk, cuda_device, b, per_seq, **kw)
    ref = TR.policy_loss(b["lp"], b["old"], b["adv_s"] if per_seq else b["adv_t"], b["ref"],
                         b["active"], offsets, per_seq, **kw)
    g_tol, s_tol = bounds(b, ref, per_seq, True, kl, 0.05, 0.5)
    assert np.all(np.abs(grad.cpu().numpy() - ref[2]) <= g_tol)
    assert np.all(np.abs(stats.cpu().numpy() - ref[1]) <= s_tol + U * np.abs(ref[1]))
    assert abs(float(loss) - ref[0]) <= 0.5 * (s_tol[0] + 0.05 * s_tol[1]) + U * abs(ref[0])


def test_policy_loss_without_reference_mask_or_offsets(rlk, cuda_device):
    b = batch(777, [0, 777], seed=3, mask=1.0)
    lp, old, adv = (dev(b[k], cuda_device) for k in ("lp", "old", "adv_t"))
    loss, stats, grad = rlk.policy_loss(lp, old, adv)
    ref = TR.policy_loss(b["lp"], b["old"], b["adv_t"])
    g_tol, s_tol = bounds(b, ref, False, False, "k3", 0.0, 1.0)
    assert np.all(np.abs(grad.cpu().numpy() - ref[2]) <= g_tol)
    assert abs(float(loss) - ref[0]) <= s_tol[0] + U * abs(ref[0]) and float(stats[1]) == 0.0
    only, _, none = rlk.policy_loss(lp, old, adv, want_grad=False)
    assert none is None and torch.equal(only, loss)


def test_gradient_against_differences(rlk, cuda_device):
    """The loss's own central differences, in steps of 2^-6 away from the clip's borders: a
    term's third derivative is at most 3 |A| r, so the difference quotient errs by
    h^2 / 6 * 3 |A| r + (two roundings of the loss) / h."""
    T, h = 12, 2.0 ** -6
    rng = np.random.default_rng(5)
    lp = rng.uniform(-2, -1, T).astype(np.float32)
    ratio = np.tile([0.5, 1.0, 2.0], 4)
    adv = np.repeat([1.0, -1.0], 6).astype(np.float32)
    old = (lp - np.log(ratio)).astype(np.float32)
    ref = (lp + 0.3).astype(np.float32)
    kw = dict(reduction="sum", kl_coef=0.1)

    def loss_of(v):
        return float(rlk.policy_loss(dev(v, cuda_device), dev(old, cuda_device),
                                     dev(adv, cuda_device), ref_logprob=dev(ref, cuda_device),
                                     want_grad=False, **kw)[0])
    _, _, grad = rlk.policy_loss(dev(lp, cuda_device), dev(old, cuda_device),
                                 dev(adv, cuda_device), ref_logprob=dev(ref, cuda_device), **kw)
    grad = grad.cpu().numpy()
    for t in range(T):
        a, b = lp.copy(), lp.copy()
        a[t] += np.float32(h)
        b[t] -= np.float32(h)
        num = (loss_of(a) - loss_of(b)) / (float(a[t]) - float(b[t]))
        assert abs(num - grad[t]) <= h * h / 6 * 3 * 2.2 + 40 * U * 20 / h, t


def test_clip_decision_is_exact_next_to_the_border(rlk, cuda_device):
    """d one float step either side of log(1.2) and log(0.8): the decision is that of exact
    arithmetic on the given floats, where a comparison of rounded ratios could go either way."""
    hi, lo = np.float32(np.log1p(0.2)), np.float32(np.log1p(-0.2))
    ds = []
    for c in (hi, lo):
        x = c
        for _ in range(4):
            x = np.nextafter(x, np.float32(-10))
        for _ in range(9):
            ds.append(x)
            x = np.nextafter(x, np.float32(10))
    d = np.array(ds, np.float32)
    adv = np.concatenate([np.ones(9), -np.ones(9)]).astype(np.float32)
    zero = np.zeros_like(d)  # lp - old = d exactly
    _, _, grad = rlk.policy_loss(dev(d, cuda_device), dev(zero, cuda_device), dev(adv, cuda_device),
                                 reduction="sum")
    shut = grad.cpu().numpy() == 0
    d64 = d.astype(np.float64)
    want = np.where(adv > 0, d64 > np.log1p(0.2), d64 < np.log1p(-0.2))
    assert np.array_equal(shut, want)


def test_masked_tokens_may_hold_anything(rlk, cuda_device):
    b = batch(3000, [100, 900, 2900], seed=6, mask=0.6)
    clean = run(rlk, cuda_device, b, kl_coef=0.1)
    on = b["active"].astype(bool).copy()
    on[:100] = False
    on[2900:] = False
    for bad in (np.nan, np.inf, -np.inf, np.finfo(np.float32).min):
        dirty = {k: v for k, v in b.items()}
        for k in ("lp", "old", "ref", "adv_t"):
            dirty[k] = np.where(on, b[k], np.float32(bad)).astype(np.float32)
        out = run(rlk, cuda_device, dirty, kl_coef=0.1)
        for x, y in zip(clean, out):
            assert torch.equal(x, y)
    assert torch.all(clean[2][torch.from_numpy(~on).to(cuda_device)] == 0)


@pytest.mark.parametrize("reduction", ["sum", "token_mean", "seq_mean"])
def test_nothing_active(rlk, cuda_device, reduction):
    b = batch(2500, [0, 1000, 2500], seed=7, mask=1.0)
    b["active"] = np.zeros(2500, np.uint8)
    loss, stats, grad = run(rlk, cuda_device, b, kl_coef=0.1, reduction=reduction)
    assert float(loss) == 0.0 and not stats.any() and not grad.any()


@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean"])
def test_more_than_2_31_bytes(rlk, cuda_device, reduction):
    """Positions whose byte offsets pass 32 bits: one sequence of 2^29 + 9 tokens, half of them
    active, ratio 1 and advantage 1 but for the last token."""
    T = 2 ** 29 + 9
    lp = torch.full((T,), -1.0, device=cuda_device)
    adv = torch.ones(T, device=cuda_device)
    adv[-1] = -3.0
    act = torch.ones(T, dtype=torch.uint8, device=cuda_device)
    act[:T // 2] = 0
    n = T - T // 2
    loss, stats, grad = rlk.policy_loss(lp, lp, adv, active=act, reduction=reduction)
    assert abs(float(loss) + (n - 4) / n) <= 40 * U and float(stats[2]) == 0.0
    assert float(grad[T // 2 - 1]) == 0.0
    for t, want in ((T // 2, -1 / n), (T - 2, -1 / n), (T - 1, 3 / n)):
        assert abs(float(grad[t]) - want) <= 8 * U * abs(want)


def test_no_tokens_and_no_sequences(rlk, cuda_device):
    e = torch.zeros(0, device=cuda_device)
    loss, stats, grad = rlk.policy_loss(e, e, e)
    assert float(loss) == 0.0 and not stats.any() and grad.numel() == 0
    for T in (9, 9000, 40000):
        for reduction in ("sum", "token_mean", "seq_mean"):
            x = torch.full((T,), -1.0, device=cuda_device)
            loss, stats, grad = rlk.policy_loss(x, x, e, advantages_per_seq=True, reduction=reduction,
                                                seq_offsets=torch.zeros(1, dtype=torch.int32, device=cuda_device))
            assert float(loss) == 0.0 and not stats.any() and not grad.any()
    # no tokens in more sequences than one launch takes
    loss, stats, _ = rlk.policy_loss(e, e, torch.ones(2000, device=cuda_device), advantages_per_seq=True,
                                     seq_offsets=torch.zeros(2001, dtype=torch.int32, device=cuda_device))
    assert float(loss) == 0.0 and not stats.any()


def test_extreme_ratios(rlk, cuda_device):
    """Ratios beyond fp32: clipped where the clip says so, infinite where the formula is."""
    lp = torch.tensor([0.0, 0.0, 0.0, -200.0, -200.0, 0.0], device=cuda_device)
    old = torch.tensor([-200.0, -200.0, -200.0, 0.0, 0.0, -200.0], device=cuda_device)
    adv = torch.tensor([1.0, -1.0, 0.0, 1.0, -1.0, -1.0], device=cuda_device)
    _, _, g = rlk.policy_loss(lp, old, adv, reduction="sum")
    assert g.tolist() == [0.0, float("inf"), 0.0, 0.0, 0.0, float("inf")]
    loss, stats, g = rlk.policy_loss(lp, old, adv, reduction="sum", dual_clip=3.0)
    # -1.2 + 3 + 0 - e^-200 + 0.8 + 3
    assert abs(float(loss) - 5.6) <= 8 * U * 8 and not g[:3].any() and float(stats[2]) == 4.0


@pytest.mark.parametrize("T", [6, 9000, 40000])  # every launch shape
@pytest.mark.parametrize("per_seq", [False, True])
def test_an_advantage_that_is_nan_reaches_its_own_gradient(rlk, cuda_device, T, per_seq):
    """Whether the ratio lies below, within or above the clip's range; a NaN advantage is clipped
    by neither side.  Nothing else of the batch changes but the sum."""
    d = np.zeros(T, np.float32)
    d[:6] = [-1.0, 0.0, 1.0, -1.0, 0.0, 1.0]
    adv = np.ones(T, np.float32)
    offsets = [0, 1, 2, 3, 4, 5, T]
    kw = dict(reduction="sum", dual_clip=3.0, advantages_per_seq=per_seq,
              seq_offsets=dev(offsets, cuda_device, np.int32))
    lp, old = dev(d, cuda_device), dev(np.zeros(T, np.float32), cuda_device)
    held = adv[:6] if per_seq else adv
    _, clean_stats, clean = rlk.policy_loss(lp, old, dev(held, cuda_device), **kw)
    for t in range(5):
        bad = held.copy()
        bad[t] = np.nan
        loss, stats, grad = rlk.policy_loss(lp, old, dev(bad, cuda_device), **kw)
        assert torch.isnan(loss) and torch.isnan(stats[0]) and torch.isnan(grad[t])
        assert float(stats[2]) == float(clean_stats[2]) - (d[t] > 0) and stats[3] == clean_stats[3]
        grad[t] = clean[t]
        assert torch.equal(grad, clean)


@pytest.mark.parametrize("T", [6, 9000, 40000])  # every launch shape
def test_zero_advantages(rlk, cuda_device, T):
    """A ratio that is finite but beyond fp32 makes nothing of an advantage of 0, and no token with
    one is clipped; an old_logprob of -inf gives NaN as infinity times 0 does."""
    lp, old = np.zeros(T, np.float32), np.zeros(T, np.float32)
    old[:5] = [-200.0, 200.0, -1.0, 1.0, -2.0e38]
    for adv in (0.0, -0.0):
        a = np.full(T, adv, np.float32)
        kw = dict(reduction="sum", dual_clip=3.0)
        loss, stats, grad = rlk.policy_loss(dev(lp, cuda_device), dev(old, cuda_device), dev(a, cuda_device), **kw)
        want = TR.policy_loss(lp[:4], old[:4], a[:4], **kw)  # beyond that e^d leaves fp64 too
        assert float(loss) == want[0] == 0.0 and float(stats[2]) == want[1][2] == 0.0 and not grad.any()
        # the largest finite values: the difference is beyond fp32, and still finite
        far_lp, far = lp.copy(), old.copy()
        far_lp[4], far[4] = 3.0e38, -3.0e38
        loss, stats, grad = rlk.policy_loss(dev(far_lp, cuda_device), dev(far, cuda_device), dev(a, cuda_device), **kw)
        assert float(loss) == 0.0 and float(stats[2]) == 0.0 and not grad.any()
        for t in (0, 5):
            inf = old.copy()
            inf[t] = -np.inf
            loss, stats, grad = rlk.policy_loss(dev(lp, cuda_device), dev(inf, cuda_device), dev(a, cuda_device), **kw)
            assert torch.isnan(loss) and torch.isnan(grad[t]) and float(stats[2]) == 0.0
            grad[t] = 0.0
            assert not grad.any()


@pytest.mark.parametrize("T", [6, 9000, 40000])  # every launch shape
def test_ratios_next_to_the_largest_number(rlk, cuda_device, T):
    """d = 88.62 .. 88.72, a large part of whose last bits lies in its second float: the ratio is as
    exact as any other's, up to the largest fp32 number."""
    n = 64
    lp, old, adv = (np.zeros(T, np.float32) for _ in range(3))
    k = min(T, n)
    lp[:k] = np.linspace(88.62, 88.72, n)[:k]
    old[:k] = (np.random.default_rng(15).random(n) * 2.0 ** -17)[:k]
    adv[:k] = -1e-10
    want = 1e-10 * np.exp(lp[:k].astype(np.float64) - old[:k])
    _, _, grad = rlk.policy_loss(dev(lp, cuda_device), dev(old, cuda_device), dev(adv, cuda_device),
                                 reduction="sum")
    adv32 = float(np.float32(1e-10)) / 1e-10
    assert np.all(np.abs(grad.cpu().numpy()[:k] - want * adv32) <= 12 * U * want)


@pytest.mark.parametrize("T", [6, 9000, 40000])  # every launch shape
def test_clip_limits_beyond_fp32_clip_nothing(rlk, cuda_device, T):
    b = batch(T, [0, T], seed=16, mask=1.0, spread=2.0)
    args = [dev(b[k], cuda_device) for k in ("lp", "old", "adv_t")]
    for big in (1e39, 1e308):
        loss, stats, grad = rlk.policy_loss(*args, clip_low=big, clip_high=big, dual_clip=big, reduction="sum")
        ref = TR.policy_loss(b["lp"], b["old"], b["adv_t"], clip_low=1e30, clip_high=1e30, reduction="sum")
        g_tol, s_tol = bounds(b, ref, False, False, "k3", 0.0, 1.0)
        assert float(stats[2]) == 0.0 and np.all(np.abs(grad.cpu().numpy() - ref[2]) <= g_tol)
        assert abs(float(loss) - ref[0]) <= s_tol[0] + U * abs(ref[0])


@pytest.mark.parametrize("offsets", [[0, 700, 600, 1000], [-1, 500, 1000, 1000], [0, 500, 900, 1001],
                                     [5, 2 ** 31 - 1, -2 ** 31, 1000]])
@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean"])
def test_bad_offsets_are_reported(rlk, cuda_device, offsets, reduction):
    b = batch(1000, [0, 300, 600, 1000], seed=8)
    status = rlk.new_status(cuda_device)
    guard = torch.full((1000 + 512,), 7.0, device=cuda_device)
    loss, stats, _ = rlk.policy_loss(dev(b["lp"], cuda_device), dev(b["old"], cuda_device),
                                     dev(b["adv_s"], cuda_device), active=dev(b["active"], cuda_device),
                                     seq_offsets=torch.tensor(offsets, dtype=torch.int32, device=cuda_device),
                                     advantages_per_seq=True, reduction=reduction, status=status,
                                     grad_logprob=guard[256:1256])
    with pytest.raises(rlk.RlkError) as e:
        rlk.raise_on_device_status(status)
    assert e.value.code == rlk.RLK_ERR_INVALID_ARG
    assert torch.isnan(loss) and torch.isnan(stats).all()
    assert torch.all(guard[:256] == 7) and torch.all(guard[1256:] == 7)


@pytest.mark.parametrize("T", [0, 50000, 300000])
@pytest.mark.parametrize("place", [0, 1, 777, 1999, 2000])
def test_one_bad_offset_among_many_is_reported(rlk, cuda_device, T, place):
    """2001 offsets, of which one leaves [0, T] or descends; without tokens too."""
    off = torch.linspace(0, T, 2001, device=cuda_device).to(torch.int32)
    off[-1] = T
    x = torch.full((T,), -1.0, device=cuda_device)
    adv = torch.ones(2000, device=cuda_device)
    good = rlk.policy_loss(x, x, adv, seq_offsets=off, advantages_per_seq=True, reduction="seq_mean")
    assert torch.isfinite(good[0])
    for value in (-1, T + 1, 2 ** 31 - 1):
        bad = off.clone()
        bad[place] = value
        status = rlk.new_status(cuda_device)
        loss, stats, _ = rlk.policy_loss(x, x, adv, seq_offsets=bad, advantages_per_seq=True,
                                         reduction="seq_mean", status=status)
        with pytest.raises(rlk.RlkError) as e:
            rlk.raise_on_device_status(status)
        assert e.value.code == rlk.RLK_ERR_INVALID_ARG
        assert torch.isnan(loss) and torch.isnan(stats).all()


@pytest.mark.parametrize("T", [801, 9001, 60001])
def test_repeats_views_and_streams_give_the_same_bits(rlk, cuda_device, T):
    b = batch(T, [0, 10, 400, T], seed=9)
    first = run(rlk, cuda_device, b, kl_coef=0.1, reduction="seq_mean")
    again = run(rlk, cuda_device, b, kl_coef=0.1, reduction="seq_mean")
    # inputs at odd places of larger buffers, on another stream
    held = {}
    for k in ("lp", "old", "ref", "adv_t"):
        held[k] = torch.cat([torch.zeros(1, device=cuda_device), dev(b[k], cuda_device)])[1:]
    act = torch.cat([torch.zeros(3, dtype=torch.uint8, device=cuda_device), dev(b["active"], cuda_device)])[3:]
    off = dev(b["offsets"], cuda_device, np.int32)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    other = rlk.policy_loss(held["lp"], held["old"], held["adv_t"], ref_logprob=held["ref"], active=act,
                            seq_offsets=off, kl_coef=0.1, reduction="seq_mean", stream=s)
    s.synchronize()
    for x, y, z in zip(first, again, other):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_a_tokens_gradient_does_not_depend_on_the_batch(rlk, cuda_device):
    b = batch(5000, [0, 2100, 5000], seed=10, mask=1.0)
    full = run(rlk, cuda_device, b, kl_coef=0.1, reduction="sum")[2]
    for lo, hi in ((0, 1), (17, 1500), (2500, 5000)):
        part = {k: (v[lo:hi] if k in ("lp", "old", "ref", "adv_t") else v) for k, v in b.items()}
        part["offsets"] = [0, hi - lo]
        assert torch.equal(run(rlk, cuda_device, part, kl_coef=0.1, reduction="sum")[2], full[lo:hi])


@pytest.mark.parametrize("T", [600, 5000, 20000, 50000])
def test_graph_replay(rlk, cuda_device, T):
    bs = [batch(T, [0, T // 3, T], seed=s) for s in (11, 12)]
    eager = [run(rlk, cuda_device, b, kl_coef=0.1) for b in bs]
    lp, old, ref, adv, act = (dev(bs[0][k], cuda_device) for k in ("lp", "old", "ref", "adv_t", "active"))
    off = dev(bs[0]["offsets"], cuda_device, np.int32)
    grad = torch.empty(T, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, stats, _ = rlk.policy_loss(lp, old, adv, ref_logprob=ref, active=act, seq_offsets=off,
                                         kl_coef=0.1, grad_logprob=grad)
    for b, e in zip(bs, eager):
        for t, k in ((lp, "lp"), (old, "old"), (ref, "ref"), (adv, "adv_t"), (act, "active")):
            t.copy_(dev(b[k], cuda_device))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, e[0]) and torch.equal(stats, e[1]) and torch.equal(grad, e[2])


def test_a_reported_kl_may_overflow(rlk, cuda_device):
    """ref - lp = 200: k3 is beyond fp32, and with kl_coef 0 only the report is."""
    lp = torch.tensor([-200.0, -1.0], device=cuda_device)
    ref = torch.tensor([0.0, -1.0], device=cuda_device)
    for T in (2, 9000, 40000):  # every launch shape
        pad = torch.zeros(T - 2, device=cuda_device)
        x, r = torch.cat([lp, pad]), torch.cat([ref, pad])
        loss, stats, g = rlk.policy_loss(x, x, torch.ones_like(x), ref_logprob=r, reduction="sum")
        assert float(loss) == -T and torch.all(g == -1) and torch.isinf(stats[1])


def test_binding_shape_checks(rlk, cuda_device):
    x = torch.zeros(8, device=cuda_device)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=cuda_device)
    for call in (lambda: rlk.policy_loss(x, x[:4], x), lambda: rlk.policy_loss(x, x, x, seq_offsets=off, advantages_per_seq=True),
                 lambda: rlk.policy_loss(x, x, x, kl="k4"), lambda: rlk.policy_loss(x, x, x, reduction="mean"),
                 lambda: rlk.policy_loss(x[::2], x[::2], x[::2]),
                 lambda: rlk.policy_loss(x, x, x, grad_logprob=x[:3])):
        with pytest.raises(ValueError):
            call()
    class Elsewhere:  # a stream of another device
        device = torch.device("cuda", x.get_device() + 1)
    with pytest.raises(ValueError):
        rlk.policy_loss(x, x, x, stream=Elsewhere())
    with pytest.raises(TypeError):
        rlk.policy_loss(x, x, x, seq_offsets=off.long())
    with pytest.raises(rlk.RlkError):
        rlk.policy_loss(x, x, x, kl_coef=0.1)


@pytest.mark.parametrize("reduction", ["sum", "token_mean", "seq_mean"])
def test_every_launch_shape_gives_the_same_bits(rlk, cuda_device, reduction):
    """The same sequences in batches of 1024 to 200000 tokens (the others behind the last
    sequence), which one CTA, one cluster with one and with four tokens a thread and two launches
    take; and among 2000 empty sequences."""
    n, offsets = 1000, [3, 300, 300, 700, 990]
    b = batch(200000, offsets, seed=14, mask=0.7)
    results = []
    for T in (1000, 1024, 1025, 8192, 8193, 32768, 32769, 200000):
        part = {k: (v[:T] if k in ("lp", "old", "ref", "adv_t", "active") else v) for k, v in b.items()}
        loss, stats, grad = run(rlk, cuda_device, part, True, kl_coef=0.1, reduction=reduction)
        assert not grad[n:].any()
        results.append((loss, stats, grad[:n]))
    for r in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, results[0]))
    if reduction != "seq_mean":  # where the number of sequences does not count
        many = {k: (v[:n] if k in ("lp", "old", "ref", "adv_t", "active") else v) for k, v in b.items()}
        many["offsets"] = offsets + [990] * 2000
        many["adv_s"] = np.concatenate([b["adv_s"], np.full(2000, np.nan, np.float32)])
        r = run(rlk, cuda_device, many, True, kl_coef=0.1, reduction=reduction)
        assert all(torch.equal(x, y) for x, y in zip(r, results[0]))

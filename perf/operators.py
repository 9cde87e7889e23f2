"""Timed cases of the training-step operators around the selected-token logprob.

The operators take a training step from the per-token log-probabilities to
clipped gradients: the clipped policy loss with a KL term, the preference loss
on paired log ratios, the backward of the strict RMSNorm, and the global
gradient norm with clipping.  ``run`` computes one pass either in plain form
(elementary torch operations) or, with ``own`` set, through
``invariant_selected_token_gb300.binding``.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a micro-batch of eight short answers, as in a debugging run or the last ragged
        # micro-batch of an epoch: latency is all that counts
        dict(name="policy_micro", op="policy", T=512, seqs=8, mask="prompt", per_seq=True, ref=False,
             reduction="token_mean", kl="k3", kl_coef=0.0, clip_low=0.2, clip_high=0.2, dual=0.0),
        # one 8192-row call of a long-response batch, each sequence weighted alike, with the
        # KL term against the reference model
        dict(name="policy_chunk", op="policy", T=8192, seqs=8, mask="prompt", per_seq=True, ref=True,
             reduction="seq_mean", kl="k3", kl_coef=0.02, clip_low=0.2, clip_high=0.28, dual=0.0),
        # a whole step of 512 long responses at once, per-token advantages, dual clip
        dict(name="policy_step", op="policy", T=1769477, seqs=512, mask="prompt", per_seq=False,
             ref=True, reduction="token_mean", kl="k3", kl_coef=0.001, clip_low=0.2, clip_high=0.2,
             dual=3.0),
        # four short preference pairs
        dict(name="pref_micro", op="pref", T=1021, pairs=4, mask="prompt", ref=True, kind="sigmoid",
             beta=0.1, smoothing=0.0, margin=0.0, mean=False, layout="halves"),
        # a usual batch of 64 pairs, smoothed labels, chosen and rejected side by side
        dict(name="pref_batch", op="pref", T=131073, pairs=64, mask="prompt", ref=True,
             kind="sigmoid", beta=0.1, smoothing=0.1, margin=0.0, mean=False, layout="adjacent"),
        # few very long answers: four pairs over a million tokens, length-normalised
        dict(name="pref_long", op="pref", T=1048583, pairs=4, mask="prompt", ref=True, kind="ipo",
             beta=0.1, smoothing=0.0, margin=0.0, mean=True, layout="halves"),
        # a handful of small tensors (norm weights, adapters)
        dict(name="clip_small", op="clip", n=12, total=40001, dtypes="f32", mode="clip"),
        # the gradients of a trunk: many ragged tensors back to back in buckets, so that most
        # of them start at an odd place
        dict(name="clip_buckets", op="clip", n=290, total=200000003, dtypes="bf16+f32",
             mode="clip"),
        # the gradients that the head's backward gives: grad_W [151936, 4096] and the norm
        # weight's [4096]
        dict(name="clip_head", op="clip", n=2, total=151936 * 4096 + 4096, dtypes="f32",
             mode="clip"),
        # the norm before the head for a 64-row micro-batch, from the fp32 grad_hidden
        dict(name="rms_micro", op="rms", T=64, H=4096, grad="f32", out="f32", residual=False),
        # the same for the packed batch, into a bf16 residual stream
        dict(name="rms_packed", op="rms", T=4096, H=4096, grad="f32", out="bf16", residual=True),
        # a wide trunk's norm, bf16 throughout, a ragged row count
        dict(name="rms_wide", op="rms", T=8191, H=8192, grad="bf16", out="bf16", residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "pref", "clip", "rms"])
    if op == "policy":
        T = _log_int(rng, 300, 1769477)
        seqs = max(1, min(T // 8, _log_int(rng, 1, 1024)))
        ref = rng.random() < 0.6
        return dict(op=op, T=T, seqs=seqs, mask=rng.choice(["prompt", "prompt", "none"]),
                    per_seq=rng.random() < 0.5, ref=ref,
                    reduction=rng.choice(["token_mean", "seq_mean", "sum"]),
                    kl=rng.choice(["k1", "k2", "k3"]),
                    kl_coef=rng.choice([0.001, 0.02, 0.1]) if ref else 0.0,
                    clip_low=rng.choice([0.1, 0.2]), clip_high=rng.choice([0.2, 0.28]),
                    dual=rng.choice([0.0, 3.0]))
    if op == "pref":
        T = _log_int(rng, 300, 1048583)
        pairs = max(1, min(T // 32, _log_int(rng, 1, 512)))
        kind = rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"])
        return dict(op=op, T=T, pairs=pairs, mask=rng.choice(["prompt", "prompt", "none"]),
                    ref=rng.random() < 0.8, kind=kind, beta=rng.choice([0.05, 0.1, 0.5]),
                    smoothing=rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0,
                    margin=rng.choice([0.0, 0.25]) if kind != "ipo" else 0.0,
                    mean=kind == "ipo" or rng.random() < 0.3,
                    layout=rng.choice(["halves", "adjacent"]))
    if op == "clip":
        n = _log_int(rng, 1, 400)
        return dict(op=op, n=n, total=max(n, _log_int(rng, 30000, 200000003)),
                    dtypes=rng.choice(["f32", "bf16", "f16", "bf16+f32"]),
                    mode=rng.choice(["clip", "clip", "norm"]))
    return dict(op=op, T=_log_int(rng, 16, 8192), H=64 * _log_int(rng, 4, 128),
                grad=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]),
                residual=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """The element counts of a clip case's tensors, by dtype: [(dtype name, count)]."""
    if case["n"] == 2 and case["total"] == 151936 * 4096 + 4096:
        return [("f32", 151936 * 4096), ("f32", 4096)]
    n, total, names = case["n"], case["total"], case["dtypes"].split("+")
    r = random.Random(n * 1000003 + total)
    w = [math.exp(r.uniform(0.0, 6.0)) for _ in range(n)]
    cut, at = [0], 0.0
    for x in w:
        at += x
        cut.append(int(round(total * at / sum(w))))
    cut[-1] = total
    # one tensor in four of a mixed set is held in the second type
    return [(names[-1] if i % 4 == 3 else names[0], cut[i + 1] - cut[i]) for i in range(n)]


def _tokens(case, n_seqs, g, dev):
    """Offsets [n_seqs + 1], the activity mask (or None) and each token's sequence."""
    T = case["T"]
    w = torch.rand(n_seqs, generator=g, device=dev, dtype=torch.float64) + 0.25
    cut = torch.round(torch.cumsum(w, 0) / w.sum() * T).to(torch.int32)
    cut[-1] = T
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device=dev), cut])
    ids = torch.bucketize(torch.arange(T, device=dev, dtype=torch.int32), offsets[1:], right=True)
    active = None
    if case["mask"] == "prompt":
        start, length = offsets[:-1].double(), (offsets[1:] - offsets[:-1]).double()
        first = start + torch.floor((0.05 + 0.3 * torch.rand(n_seqs, generator=g, device=dev)) * length)
        if n_seqs >= 16:  # an answer that a filter has taken out
            first[n_seqs // 3] = T
        active = (torch.arange(T, device=dev) >= first[ids]).to(torch.uint8)
    return offsets, active, ids


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": case}
    if case["op"] in ("policy", "pref"):
        n_seqs = case["seqs"] if case["op"] == "policy" else 2 * case["pairs"]
        T = case["T"]
        offsets, active, ids = _tokens(case, n_seqs, g, dev)
        # most tokens are nearly certain, some are not; the models differ by small noise
        old = -(rand(T).abs() ** 3) * 0.7
        live = 1.0 if active is None else active.float()
        s["offsets"], s["active"] = offsets, active
        s["ref"] = torch.clamp(old + 0.15 * rand(T), max=0.0) * live if case["ref"] else None
        if case["op"] == "policy":
            s["old"] = old * live
            s["lp"] = torch.clamp(old + 0.12 * rand(T), max=0.0) * live
            s["adv"] = rand(n_seqs) if case["per_seq"] else rand(n_seqs)[ids] * 0.5 + rand(T)
        else:
            s["lp"] = torch.clamp(old + 0.08 * rand(T) + 0.01, max=0.0) * live
    elif case["op"] == "clip":
        sizes = _sizes(case)
        std = 5.0 / math.sqrt(case["total"])
        s["grads"], s["outs"], s["buckets"] = [None] * len(sizes), [None] * len(sizes), []
        for name in sorted(set(d for d, _ in sizes)):
            held = [(i, k) for i, (d, k) in enumerate(sizes) if d == name]
            flat = (rand(sum(k for _, k in held)) * std).to(DTYPES[name])
            out = torch.empty_like(flat) if case["mode"] == "clip" else flat
            s["buckets"].append(out)
            at = 0
            for i, k in held:
                s["grads"][i], s["outs"][i] = flat[at:at + k], out[at:at + k]
                at += k
    else:
        T, H = case["T"], case["H"]
        s["x"] = (rand(T, H) * 2.0).to(torch.bfloat16)
        s["gamma"] = (1.0 + 0.1 * rand(H)).to(torch.bfloat16)
        s["grad_out"] = (rand(T, H) * 1e-2).to(DTYPES[case["grad"]])
        s["residual"] = (rand(T, H) * 1e-2).to(DTYPES[case["out"]]) if case["residual"] else None
    return s


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from invariant_selected_token_gb300 import binding
    case = s["case"]
    if case["op"] == "policy":
        loss, stats, grad = binding.policy_loss(
            s["lp"], s["old"], s["adv"], ref_logprob=s["ref"], active=s["active"],
            seq_offsets=s["offsets"], advantages_per_seq=case["per_seq"],
            clip_low=case["clip_low"], clip_high=case["clip_high"], dual_clip=case["dual"],
            kl=case["kl"], kl_coef=case["kl_coef"], reduction=case["reduction"])
        return {"loss": loss, "stats": stats, "grad": grad}
    if case["op"] == "pref":
        loss, pair_loss, rewards, grad = binding.preference_loss(
            s["lp"], s["offsets"], ref_logprob=s["ref"], active=s["active"], kind=case["kind"],
            beta=case["beta"], label_smoothing=case["smoothing"], margin=case["margin"],
            length_normalize=case["mean"], layout=case["layout"])
        return {"loss": loss, "pair_loss": pair_loss, "rewards": rewards, "grad": grad}
    if case["op"] == "clip":
        if case["mode"] == "norm":
            return {"norm": binding.grad_norm(s["grads"])}
        norm, scale = binding.clip_grads(s["grads"], 1.0, out=s["outs"])
        return {"norm": norm, "scale": scale, "grads": s["buckets"]}
    grad_x, grad_gamma = binding.rmsnorm_backward(
        s["grad_out"], s["x"], s["gamma"], 1e-6, grad_residual=s["residual"],
        grad_dtype=DTYPES[case["out"]])
    return {"grad_x": grad_x, "grad_gamma": grad_gamma}


# ------------------------------------------------------------------ the plain forms
def _plain_policy(s):
    case, lp, old, ref, offsets = s["case"], s["lp"], s["old"], s["ref"], s["offsets"]
    T, S = lp.numel(), offsets.numel() - 1
    act = torch.ones_like(lp, dtype=torch.bool) if s["active"] is None else s["active"] != 0
    ids = torch.bucketize(torch.arange(T, device=lp.device, dtype=torch.int32), offsets[1:], right=True)
    adv = s["adv"][ids] if case["per_seq"] else s["adv"]
    d = lp.double() - old.double()  # in 64 bits: it is compared with the clip's borders
    ratio = d.exp().float()
    shut = torch.where(adv > 0, d > math.log1p(case["clip_high"]),
                       (adv < 0) & (d < math.log1p(-case["clip_low"])))
    held = torch.where(shut, torch.where(adv > 0, 1.0 + case["clip_high"], 1.0 - case["clip_low"]), ratio)
    if case["dual"] > 0:
        cap = (adv < 0) & (d > math.log(case["dual"]))
        held, shut = torch.where(cap, case["dual"], held), shut | cap
    policy = -held * adv
    slope = torch.where(shut, 0.0, -ratio * adv)
    kl = torch.zeros_like(lp)
    if ref is not None:
        u = ref.double() - lp.double()  # in 64 bits: expm1(u) - u loses all of 32 near 0
        if case["kl"] == "k1":
            kl, dkl = (-u).float(), torch.ones_like(lp)
        elif case["kl"] == "k2":
            kl, dkl = (0.5 * u * u).float(), (-u).float()
        else:
            kl, dkl = (u.expm1() - u).float(), (-u.expm1()).float()
        slope = slope + case["kl_coef"] * dkl
    if case["reduction"] == "token_mean":
        w = 1.0 / act.sum().clamp(min=1).float()
    elif case["reduction"] == "seq_mean":
        at = torch.cat([torch.zeros(1, device=lp.device, dtype=torch.int64), act.cumsum(0)])[offsets.long()]
        w = 1.0 / (S * (at[1:] - at[:-1]).clamp(min=1).float())[ids]
    else:
        w = 1.0
    parts = torch.stack([policy, kl, shut.float(), -d.float()])
    stats = torch.where(act, w * parts, 0.0).sum(1, dtype=torch.float64)
    loss = stats[0] + case["kl_coef"] * stats[1]
    return {"loss": loss.float(), "stats": stats.float(), "grad": torch.where(act, w * slope, 0.0)}


def _plain_pref(s):
    case, lp, ref, offsets = s["case"], s["lp"], s["ref"], s["offsets"].long()
    T, P, beta, eps = lp.numel(), case["pairs"], case["beta"], case["smoothing"]
    act = torch.ones_like(lp, dtype=torch.bool) if s["active"] is None else s["active"] != 0
    ids = torch.bucketize(torch.arange(T, device=lp.device), offsets[1:], right=True)
    one = torch.zeros(1, device=lp.device, dtype=torch.float64)
    d = torch.where(act, lp.double() if ref is None else lp.double() - ref.double(), 0.0)
    at = torch.cat([one, d.cumsum(0)])[offsets]  # long sums that cancel in pairs: 64 bits
    count = torch.cat([one, act.double().cumsum(0)])[offsets]
    m = at[1:] - at[:-1]
    n = (count[1:] - count[:-1]).clamp(min=1) if case["mean"] else torch.ones_like(m)
    m = m / n
    pair = m.view(2, P) if case["layout"] == "halves" else m.view(P, 2).t()
    h = pair[0] - pair[1]
    z = beta * h - case["margin"]
    if case["kind"] == "sigmoid":
        soft = torch.log1p(torch.exp(-z.abs()))
        each = (1 - eps) * (soft + (-z).clamp(min=0)) + eps * (soft + z.clamp(min=0))
        slope = beta * ((1.0 / (1.0 + torch.exp(-z))) - (1 - eps))
    elif case["kind"] == "hinge":
        each, slope = (1 - z).clamp(min=0), torch.where(z < 1, -beta, 0.0)
    else:
        each, slope = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
    slope = torch.stack([slope, -slope]) / P
    slope = (slope if case["layout"] == "halves" else slope.t()).reshape(-1) / n
    return {"loss": each.mean().float(), "pair_loss": each.float(), "rewards": (beta * m).float(),
            "grad": torch.where(act, slope.float()[ids], 0.0)}


def _plain_clip(s):
    each = [g.float().square().sum() for g in s["grads"]]
    norm = torch.stack(each).double().sum().sqrt()
    if s["case"]["mode"] == "norm":
        return {"norm": norm.float()}
    scale = torch.where(torch.isfinite(norm) & (norm > 1.0), 1.0 / norm, 1.0).float()
    [o.copy_(g.float() * scale) for g, o in zip(s["grads"], s["outs"])]
    return {"norm": norm.float(), "scale": scale, "grads": s["buckets"]}


def _plain_rms(s):
    x, dy = s["x"].float(), s["grad_out"].float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    n = x * rstd
    up = dy * s["gamma"].float()
    dx = rstd * (up - n * (up * n).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"grad_x": dx.to(DTYPES[s["case"]["out"]]), "grad_gamma": (dy * n).sum(0)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return (_plain_policy(state) if op == "policy" else _plain_pref(state) if op == "pref"
            else _plain_clip(state) if op == "clip" else _plain_rms(state))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "policy":
        T, S = case["T"], case["seqs"]
        per = 12 + (4 if case["ref"] else 0) + (1 if case["mask"] != "none" else 0)
        per += 0 if case["per_seq"] else 4
        return {"bytes": T * per + S * (8 if case["per_seq"] else 4) + 24, "flops": 40 * T}
    if case["op"] == "pref":
        T, P = case["T"], case["pairs"]
        per = 8 + (4 if case["ref"] else 0) + (1 if case["mask"] != "none" else 0)
        return {"bytes": T * per + P * 20 + 4, "flops": 4 * T}
    if case["op"] == "clip":
        size = {"f32": 4, "bf16": 2, "f16": 2}
        held = sum(size[d] * k for d, k in _sizes(case))
        return {"bytes": held * (2 if case["mode"] == "clip" else 1),
                "flops": case["total"] * (3 if case["mode"] == "clip" else 2)}
    T, H = case["T"], case["H"]
    per = 2 + (4 if case["grad"] == "f32" else 2)
    per += (4 if case["out"] == "f32" else 2) * (2 if case["residual"] else 1)
    return {"bytes": T * H * per + 6 * H, "flops": 12 * T * H}


# ------------------------------------------------------------------ the definitions in 64 bits
def _spans(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def _exact_policy(s):
    case = s["case"]
    lp, old = s["lp"].double(), s["old"].double()
    on = torch.ones_like(lp) if s["active"] is None else (s["active"] != 0).double()
    spans = _spans(s["offsets"])
    adv = s["adv"].double()
    if case["per_seq"]:
        adv = torch.repeat_interleave(adv, torch.tensor([e - b for b, e in spans], device=lp.device))
    w = torch.ones_like(lp)
    if case["reduction"] == "token_mean":
        w = w / max(1.0, float(on.sum()))
    if case["reduction"] == "seq_mean":
        for b, e in spans:
            w[b:e] = 1.0 / (len(spans) * max(1.0, float(on[b:e].sum())))
    x = lp.clone().requires_grad_(True)
    r = torch.exp(x - old)
    surrogate = torch.minimum(r * adv, r.clamp(1 - case["clip_low"], 1 + case["clip_high"]) * adv)
    if case["dual"] > 0:
        surrogate = torch.where(adv < 0, torch.maximum(surrogate, case["dual"] * adv), surrogate)
    free = (surrogate == r * adv) & ((r - r.clamp(1 - case["clip_low"], 1 + case["clip_high"]) == 0)
                                     | (adv * (r - 1) < 0)) & ~((case["dual"] > 0) & (adv < 0) & (r > max(case["dual"], 1.0)))
    kl = torch.zeros_like(x)
    if s["ref"] is not None:
        u = s["ref"].double() - x
        kl = -u if case["kl"] == "k1" else u * u / 2 if case["kl"] == "k2" else torch.expm1(u) - u
    total = (w * on * (-surrogate + case["kl_coef"] * kl)).sum()
    total.backward()
    stats = [(w * on * v).sum() for v in (-surrogate, kl, (~free).double(), old - lp)]
    return {"loss": total.detach(), "stats": torch.stack(stats).detach(), "grad": x.grad}


def _exact_pref(s):
    case, P = s["case"], s["case"]["pairs"]
    on = torch.ones_like(s["lp"], dtype=torch.float64) if s["active"] is None else (s["active"] != 0).double()
    x = s["lp"].double().clone().requires_grad_(True)
    v = (x if s["ref"] is None else x - s["ref"].double()) * on
    m = []
    for b, e in _spans(s["offsets"]):
        m.append(v[b:e].sum() / (max(1.0, float(on[b:e].sum())) if case["mean"] else 1.0))
    each = []
    for i in range(P):
        c, r = (m[i], m[P + i]) if case["layout"] == "halves" else (m[2 * i], m[2 * i + 1])
        z = case["beta"] * (c - r) - case["margin"]
        if case["kind"] == "sigmoid":
            each.append((1 - case["smoothing"]) * torch.logaddexp(-z, z * 0)
                        + case["smoothing"] * torch.logaddexp(z, z * 0))
        elif case["kind"] == "hinge":
            each.append(torch.relu(1 - z))
        else:
            each.append((c - r - 1 / (2 * case["beta"])) ** 2)
    each = torch.stack(each)
    each.mean().backward()
    return {"loss": each.mean().detach(), "pair_loss": each.detach(),
            "rewards": case["beta"] * torch.stack(m).detach(), "grad": x.grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "policy":
        return _exact_policy(s)
    if case["op"] == "pref":
        return _exact_pref(s)
    if case["op"] == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2
                                   for g in s["grads"]))
        out = {"norm": torch.tensor(norm, dtype=torch.float64)}
        if case["mode"] == "clip":
            scale = 1.0 / norm if norm > 1.0 else 1.0
            for g, o in zip(s["grads"], s["outs"]):
                o.copy_(g)
            out["scale"] = torch.tensor(scale, dtype=torch.float64)
            out["grads"] = [o.double() * scale for o in s["buckets"]]
        return out
    x = s["x"].double().requires_grad_(True)
    gamma = s["gamma"].double().requires_grad_(True)
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * gamma
    y.backward(s["grad_out"].double())
    more = 0.0 if s["residual"] is None else s["residual"].double()
    return {"grad_x": x.grad + more, "grad_gamma": gamma.grad}

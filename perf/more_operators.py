"""Timed cases of the operators around the selected-token logprob's trunk and rollout.

Three families: the norms before and after a block fused with its gate and the residual stream's
scales (forward and backward); activation checkpoints in 8 bits, saved, restored and used by the
norms' backward; and the verification of drafted tokens against the target's probabilities.
``run`` computes one pass either in plain form (elementary torch operations) or, with ``own`` set,
through ``invariant_selected_token_gb300.binding``.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's decoding step: four drafted tokens, nothing but latency
        dict(name="verify_one", op="verify", seqs=1, most=4, ragged=False, V=151936, dtype="bf16", draft="logits"),
        # a batch whose drafts were looked up in the prompt (no draft distribution), an odd vocabulary
        dict(name="verify_lookup", op="verify", seqs=64, most=7, ragged=True, V=50257, dtype="f32", draft="none"),
        # a rollout engine's full batch with drafts of 0 to 8 tokens, fp32 logits of the strict head
        dict(name="verify_batch", op="verify", seqs=256, most=8, ragged=True, V=151936, dtype="f32", draft="logits"),
        # decoding: eight tokens through a block's two norms, nothing saved
        dict(name="norms_decode", op="norms", T=8, H=4096, post=True, gate="none", rs=1.0, bs=1.0, save="none"),
        # a packed batch through a gated block, with everything its backward needs saved in 8 bits
        dict(name="norms_packed", op="norms", T=4096, H=4096, post=True, gate="sigmoid", rs=1.0, bs=0.5, save="int8"),
        # a 64-row micro-batch, the last block's norms below the head's fp32 gradient
        dict(name="norms_bwd_micro", op="norms_bwd", T=64, H=4096, post=True, gate="none", rs=1.0, bs=1.0,
             saved="bf16", grad="f32", out="bf16", res=False),
        # the packed batch's backward from int8 checkpoints, gate and all
        dict(name="norms_bwd_packed", op="norms_bwd", T=4096, H=4096, post=True, gate="sigmoid", rs=1.0, bs=0.5,
             saved="int8", grad="bf16", out="bf16", res=True),
        # a wide trunk, ungated, a ragged row count, inputs kept in bf16
        dict(name="norms_bwd_wide", op="norms_bwd", T=8191, H=8192, post=True, gate="none", rs=1.0, bs=1.0,
             saved="bf16", grad="bf16", out="bf16", res=True),
        # a micro-batch's residual stream into a checkpoint and back
        dict(name="ckpt_micro", op="ckpt", T=256, H=4096, fmt="int8"),
        # a long packed batch's, where outliers share blocks with small values
        dict(name="ckpt_packed", op="ckpt", T=16385, H=4096, fmt="e4m3"),
        # the head's norm backward from an int8 checkpoint, fp32 grad_hidden
        dict(name="rms_q8_packed", op="rms_q8", T=4096, H=4096, saved="int8", grad="f32", out="bf16", res=True),
        # a narrow model's norm, many rows, e4m3
        dict(name="rms_q8_narrow", op="rms_q8", T=32771, H=1024, saved="e4m3", grad="bf16", out="bf16", res=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["verify", "norms", "norms_bwd", "ckpt", "rms_q8"])
    if op == "verify":
        seqs = _log_int(rng, 1, 256)
        most = rng.randint(1, 8)
        V = _log_int(rng, 1000, 151936)
        return dict(op=op, seqs=seqs, most=most, ragged=rng.random() < 0.7, V=V,
                    dtype=rng.choice(["f32", "bf16"]) if most < 5 or seqs < 128 else "bf16",
                    draft=rng.choice(["logits", "logp", "none"]))
    H = 64 * _log_int(rng, 2, 128)
    T = _log_int(rng, 1, max(16, min(32768, 67000000 // H)))
    if op == "ckpt":
        return dict(op=op, T=T, H=H, fmt=rng.choice(["int8", "e4m3"]))
    if op == "rms_q8":
        return dict(op=op, T=T, H=H, saved=rng.choice(["int8", "e4m3"]), grad=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["f32", "bf16"]), res=rng.random() < 0.6)
    T = max(1, T // 2)
    case = dict(op=op, T=T, H=H, post=rng.random() < 0.7, gate=rng.choice(["none", "identity", "sigmoid"]),
                rs=rng.choice([1.0, 1.0, 2.5]), bs=rng.choice([1.0, 0.5, 0.22]))
    if op == "norms":
        return dict(case, save=rng.choice(["none", "int8", "e4m3"]))
    return dict(case, saved=rng.choice(["bf16", "int8", "e4m3"]), grad=rng.choice(["f32", "bf16"]),
                out=rng.choice(["f32", "bf16"]), res=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """Drafted tokens of each sequence."""
    S, most = case["seqs"], case["most"]
    if not case["ragged"]:
        return [most] * S
    r = random.Random(S * 1000003 + most * 1009 + case["V"])
    return [r.randint(0, most) for _ in range(S)]


def _two_to(k):
    """2^k in 64 bits, exactly: a rounding next to a tie goes by it."""
    return (k.long() + 1023).bitwise_left_shift(52).view(torch.float64)


def _codes(x, fmt):
    """A bf16 tensor's checkpoint: codes [T, H] (int8 or e4m3) and a scale byte per 32 features.
    int8 codes stand for code * 2^(scale - 133), e4m3 ones for code * 2^(scale - 127)."""
    T, H = x.shape
    v = x.double().view(T, H // 32, 32)
    mant, expo = torch.frexp(v.abs().amax(2, keepdim=True))  # the largest is mant * 2^expo, mant in [1/2, 1)
    if fmt == "int8":
        scale = torch.where(mant > 0, expo + 126, 0).clamp(min=0)
        codes = torch.round(v * _two_to(133 - scale)).clamp(-127, 127).to(torch.int8)
    else:
        scale = torch.where(mant > 0, expo + 118 + (mant > 0.875), 0).clamp(min=0)
        codes = (v * _two_to(127 - scale)).float().to(torch.float8_e4m3fn)
    return codes.view(T, H), scale.to(torch.uint8).view(T, H // 32)


def _values(codes, scales):
    """What a checkpoint's codes stand for, as bf16."""
    T, H = codes.shape
    bias = 133 if codes.dtype == torch.int8 else 127
    v = codes.float().view(T, H // 32, 32)
    return (v * _two_to(scales.view(T, H // 32, 1).long() - bias).float()).view(T, H).to(torch.bfloat16)


def _verify_inputs(case, rand, g, dev):
    S, V, dtype = case["seqs"], case["V"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    D = sum(lens)
    R = D + S
    s = {"offsets": torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32, device=dev)}
    target = rand(R, V) * 1.5
    # a few likely tokens in each row, as a trained model has them
    start = torch.randint(V, (R, 1), generator=g, device=dev)
    likely = (start + 7 * torch.arange(24, device=dev)) % V
    target.scatter_(1, likely, 9.0 + 7.0 * torch.rand(R, 24, generator=g, device=dev))
    ids = torch.repeat_interleave(torch.arange(S, device=dev), torch.tensor(lens, device=dev))
    rows = torch.arange(D, device=dev) + ids
    s["target"] = target.to(dtype)
    draft = target[rows] + 0.6 * rand(D, V)
    del target
    if case["draft"] == "none":  # looked up: often, not always, what the target finds likely
        pick = torch.randint(24, (D, 1), generator=g, device=dev)
        s["tokens"] = likely[rows].gather(1, pick).view(-1).to(torch.int32)
        best = s["target"][rows].float().argmax(1).to(torch.int32)
        s["tokens"] = torch.where(torch.rand(D, generator=g, device=dev) < 0.7, best, s["tokens"])
        s["draft"] = s["draft_lse"] = None
    else:
        draft = draft.to(dtype)
        lse = torch.logsumexp(draft.float(), 1) if D else torch.zeros(0, device=dev)
        if case["draft"] == "logp":
            draft, lse = draft.float() - lse[:, None], None
        s["draft"], s["draft_lse"] = draft, lse
        race = torch.empty(D, V, device=dev).exponential_(generator=g).log_()
        s["tokens"] = (draft.float() - race).argmax(1).to(torch.int32) if D else torch.zeros(0, dtype=torch.int32, device=dev)
    s["uniforms"] = torch.rand(D, generator=g, device=dev)
    s["noise"] = torch.empty(S, V, device=dev).exponential_(generator=g).clamp_(min=1e-30)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "verify":
        return dict(_verify_inputs(case, rand, g, dev), case=case)
    s, T, H = {"case": case}, case["T"], case["H"]

    def stream():
        """A residual stream: a few features far larger than the others."""
        x = rand(T, H) * 2.0
        x[:, torch.randint(H, (max(1, H // 512),), generator=g, device=dev)] *= 40.0
        return x.to(torch.bfloat16)

    def gamma():
        return (1.0 + 0.1 * rand(H)).to(torch.bfloat16)

    if case["op"] == "ckpt":
        return dict(s, x=stream())
    if case["op"] == "rms_q8":
        s["x"], s["gamma"] = _codes(stream(), case["saved"]), gamma()
    else:
        s["pre"], s["post"] = gamma(), gamma() if case["post"] else None
        block = (rand(T, H) * 0.7).to(torch.bfloat16)
        gate = None if case["gate"] == "none" else (1.0 + rand(T, H)).to(torch.bfloat16)
        if case["op"] == "norms":
            return dict(s, block=block, gate=gate, residual=stream())
        needed = {"x": stream(), "gate": gate, "block": block if case["post"] or gate is not None else None}
        for name, t in needed.items():
            s[name] = t if t is None or case["saved"] == "bf16" else _codes(t, case["saved"])
    s["grad_out"] = (rand(T, H) * 1e-2).to(DTYPES[case["grad"]])
    s["grad_res"] = (rand(T, H) * 1e-2).to(DTYPES[case["out"]]) if case["res"] else None
    return s


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from invariant_selected_token_gb300 import binding
    case = s["case"]
    if case["op"] == "verify":
        accepted, tokens, logprob = binding.draft_verify(
            s["target"], s["tokens"], s["uniforms"], s["noise"], s["offsets"], draft_logits=s["draft"],
            draft_lse=s["draft_lse"])
        return {"accepted": accepted, "tokens": tokens, "logprob": logprob}
    if case["op"] == "ckpt":
        return {"values": binding.act_dequantize(binding.act_quantize(s["x"], case["fmt"]))}
    if case["op"] == "rms_q8":
        grad_x, grad_gamma = binding.rmsnorm_backward_q8(
            s["grad_out"], binding.Saved(*s["x"]), s["gamma"], EPS, grad_residual=s["grad_res"],
            grad_dtype=DTYPES[case["out"]])
        return {"grad_x": grad_x, "grad_gamma": grad_gamma}
    if case["op"] == "norms":
        out, residual, saved = binding.block_norm(
            s["block"], s["residual"], s["pre"], gamma_post=s["post"], gate=s["gate"], gate_kind=case["gate"],
            residual_scale=case["rs"], block_scale=case["bs"], eps=EPS,
            save=None if case["save"] == "none" else case["save"])
        held = [None if v is None else binding.act_dequantize(v) for v in saved] if saved else [None] * 3
        return {"out": out, "residual": residual, "x": held[0], "block": held[1], "gate": held[2]}
    held = {n: s[n] if case["saved"] == "bf16" or s[n] is None else binding.Saved(*s[n]) for n in ("x", "block", "gate")}
    g = binding.block_norm_backward(
        s["grad_out"], held["x"], s["pre"], block=held["block"], gamma_post=s["post"], gate=held["gate"],
        gate_kind=case["gate"], residual_scale=case["rs"], block_scale=case["bs"], eps=EPS,
        grad_residual_out=s["grad_res"], grad_dtype=DTYPES[case["out"]])
    return g._asdict()


# ------------------------------------------------------------------ the plain forms
def _plain_verify(s):
    target, off, tok = s["target"], s["offsets"].long(), s["tokens"].long()
    (R, V), D, S = target.shape, tok.numel(), s["offsets"].numel() - 1
    lens = off[1:] - off[:-1]
    draft_at = torch.arange(D, device=off.device)
    ids = torch.bucketize(draft_at, off[1:], right=True)
    top = target.amax(1).float()
    sums = torch.exp(target.float() - top[:, None]).sum(1, dtype=torch.float64)
    lse = top.double() + torch.log(sums)  # in 64 bits: it decides next to a border
    log_p = target[draft_at + ids, tok].double() - lse[draft_at + ids]
    q = torch.ones_like(log_p)
    if s["draft"] is not None:
        q = torch.exp(s["draft"][draft_at, tok].double() - (0.0 if s["draft_lse"] is None else s["draft_lse"].double()))
    ok = s["uniforms"].double() * q < torch.exp(log_p)
    upto = torch.where(ok, lens[ids], draft_at - off[ids])
    accepted = lens.scatter_reduce(0, ids, upto, "amin")
    row, refused = off[:-1] + torch.arange(S, device=off.device) + accepted, accepted < lens
    p = torch.exp(target[row].double() - lse[row, None])
    weight = p
    if D:
        at = (off[:-1] + accepted).clamp(max=D - 1)
        if s["draft"] is None:
            q_row = torch.zeros_like(p).scatter_(1, tok[at, None], 1.0)
        else:
            q_row = s["draft"][at].double()
            q_row = torch.exp(q_row if s["draft_lse"] is None else q_row - s["draft_lse"][at, None].double())
        left = torch.where(refused[:, None], (p - q_row).clamp(min=0), p)
        weight = torch.where(left.amax(1, keepdim=True) > 0, left, p)
    new = (weight / s["noise"]).argmax(1)
    seq = torch.repeat_interleave(torch.arange(S, device=off.device), lens + 1, output_size=R)
    place = torch.arange(R, device=off.device) - off[seq] - seq
    given = torch.cat([tok, tok.new_zeros(S)])[(off[seq] + place).clamp(max=D + S - 1)]
    out = torch.where(place < accepted[seq], given, torch.where(place == accepted[seq], new[seq], -1))
    logprob = target.gather(1, out.clamp(min=0)[:, None])[:, 0].double() - lse
    return {"accepted": accepted.int(), "tokens": out.int(), "logprob": torch.where(out >= 0, logprob, 0.0).float()}


def _plain_gate(case, gate):
    return torch.sigmoid(gate.float()) if case["gate"] == "sigmoid" else gate.float()


def _plain_norm(x):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)


def _plain_norms(s):
    case, branch = s["case"], s["block"].float()
    if s["post"] is not None:
        branch = _plain_norm(branch) * s["post"].float()
    if s["gate"] is not None:
        branch = branch * _plain_gate(case, s["gate"])
    x = (case["rs"] * s["residual"].float() + case["bs"] * branch).to(torch.bfloat16)
    out = (_plain_norm(x.float()) * s["pre"].float()).to(torch.bfloat16)
    held = {"x": None, "block": None, "gate": None}
    if case["save"] != "none":
        needed = s["block"] if case["post"] or s["gate"] is not None else None
        held = {n: None if t is None else _plain_round(t, case["save"])
                for n, t in (("x", x), ("block", needed), ("gate", s["gate"]))}
    return dict(held, out=out, residual=x)


def _plain_round(x, fmt):
    """The values that an 8-bit checkpoint of a bf16 tensor holds."""
    v = x.float().view(x.shape[0], -1, 32)
    mant, expo = torch.frexp(v.abs().amax(2, keepdim=True))
    expo = expo - 7 if fmt == "int8" else expo - 9 + (mant > 0.875).int()
    down, up = _two_to(-expo).float(), _two_to(expo).float()
    codes = torch.round(v * down).clamp(-127, 127) if fmt == "int8" else (v * down).to(torch.float8_e4m3fn).float()
    return (codes * up).view_as(x).to(torch.bfloat16)


def _plain_rms_backward(up, x, gamma):
    """(grad_x, grad_gamma) of x / rms(x) * gamma, in 32 bits."""
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    n, scaled = x * rstd, up * gamma
    return rstd * (scaled - n * (scaled * n).mean(1, keepdim=True)), (up * n).sum(0)


def _held(t):
    return t if t is None or isinstance(t, torch.Tensor) else _values(*t)


def _plain_norms_bwd(s):
    case, dtype = s["case"], DTYPES[s["case"]["out"]]
    x, block, gate = (_held(s[n]) for n in ("x", "block", "gate"))
    dx, d_pre = _plain_rms_backward(s["grad_out"].float(), x.float(), s["pre"].float())
    if s["grad_res"] is not None:
        dx = dx + s["grad_res"].float()
    got = {"grad_residual": (case["rs"] * dx).to(dtype), "grad_gamma_pre": d_pre, "grad_gate": None, "grad_gamma_post": None}
    branch = None if block is None else block.float()
    if s["post"] is not None:
        branch = _plain_norm(branch) * s["post"].float()
    d_branch = case["bs"] * dx
    if gate is not None:
        open_ = _plain_gate(case, gate)
        slope = open_ * (1 - open_) if case["gate"] == "sigmoid" else 1.0
        got["grad_gate"] = (d_branch * branch * slope).to(dtype)
        d_branch = d_branch * open_
    if s["post"] is not None:
        d_branch, got["grad_gamma_post"] = _plain_rms_backward(d_branch, block.float(), s["post"].float())
    return dict(got, grad_block=d_branch.to(dtype))


def _plain_rms_q8(s):
    dx, d_gamma = _plain_rms_backward(s["grad_out"].float(), _values(*s["x"]).float(), s["gamma"].float())
    if s["grad_res"] is not None:
        dx = dx + s["grad_res"].float()
    return {"grad_x": dx.to(DTYPES[s["case"]["out"]]), "grad_gamma": d_gamma}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "ckpt":
        return {"values": _plain_round(state["x"], state["case"]["fmt"])}
    return (_plain_verify(state) if op == "verify" else _plain_norms(state) if op == "norms"
            else _plain_norms_bwd(state) if op == "norms_bwd" else _plain_rms_q8(state))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "verify":
        S, V, D = case["seqs"], case["V"], sum(_lengths(case))
        row = V * size[case["dtype"]]
        # every target row; a sequence's noise, and the draft's row where a sequence can refuse one
        draft = {"none": 0, "logits": row, "logp": 4 * V}[case["draft"]]
        can = sum(n > 0 for n in _lengths(case))
        return {"bytes": (D + S) * row + S * 4 * V + can * draft + D * 12 + S * 12 + (D + S) * 8, "flops": 4 * (D + S) * V}
    T, H = case["T"], case["H"]
    q8 = 1 + 1 / 32
    if case["op"] == "ckpt":  # saved and read back
        return {"bytes": T * H * (4 + 2 * q8), "flops": 4 * T * H}
    if case["op"] == "rms_q8":
        per = q8 + size[case["grad"]] + size[case["out"]] * (2 if case["res"] else 1)
        return {"bytes": T * H * per + 6 * H, "flops": 12 * T * H}
    gated, post = case["gate"] != "none", case["post"]
    if case["op"] == "norms":
        per = 8 + (2 if gated else 0)
        if case["save"] != "none":  # written, and read back by the pass that returns them
            per += (1 + (1 if post or gated else 0) + (1 if gated else 0)) * (2 * q8 + 2)
        return {"bytes": T * H * per + 4 * H, "flops": 12 * T * H}
    held = 2 if case["saved"] == "bf16" else q8
    per = size[case["grad"]] + held * (1 + (1 if post or gated else 0) + (1 if gated else 0))
    per += size[case["out"]] * ((1 if case["res"] else 0) + 2 + (1 if gated else 0))
    return {"bytes": T * H * per + 12 * H, "flops": 30 * T * H}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_verify(s):
    off, S = s["offsets"].tolist(), s["offsets"].numel() - 1
    accepted, logprob = [], []
    for i in range(S):
        b, e = off[i], off[i + 1]
        logp = torch.log_softmax(s["target"][b + i:e + i + 1].double(), 1)
        n = e - b
        tok = s["tokens"][b:e].long()
        if n:
            log_ratio = logp[:n].gather(1, tok[:, None])[:, 0]
            if s["draft"] is not None:
                log_ratio = log_ratio - s["draft"][b:e].gather(1, tok[:, None])[:, 0].double()
                if s["draft_lse"] is not None:
                    log_ratio = log_ratio + s["draft_lse"][b:e].double()
            keep = s["uniforms"][b:e].double() < log_ratio.exp()
            n = int(torch.cumprod(keep.long(), 0).sum())
        w = logp[n].exp()
        if n < e - b:
            if s["draft"] is None:
                w[tok[n]] -= 1.0
            else:
                w = w - (s["draft"][b + n].double() - (0.0 if s["draft_lse"] is None else s["draft_lse"][b + n].double())).exp()
        if not bool((w > 0).any()):
            w = logp[n].exp()
        new = torch.argmax(w / s["noise"][i].double())
        said = torch.cat([tok[:n], new[None]])
        accepted.append(n)
        logprob.append(logp[:n + 1].gather(1, said[:, None])[:, 0])
        logprob.append(torch.zeros(e - b - n, dtype=torch.float64, device=logp.device))
    return {"accepted": torch.tensor(accepted), "tokens": None, "logprob": torch.cat(logprob)}


def _exact_round(x, fmt):
    """The nearest values that the blocks of 32 can hold, ties to the even code."""
    v = x.double().view(x.shape[0], -1, 32)
    big = torch.frexp(v.abs().amax(2, keepdim=True).clamp(min=2.0 ** -126))[1] - 1
    if fmt == "int8":
        step = _two_to(big - 6)
        return (torch.round(v / step) * step).clamp(-127 * step, 127 * step).view_as(x)
    scale = _two_to(big - 8)
    scale = torch.where(v.abs().amax(2, keepdim=True) > 448 * scale, 2 * scale, scale)
    u = v / scale
    step = _two_to(torch.frexp(u.abs().clamp(min=2.0 ** -6))[1] - 4)
    return (torch.round(u / step) * step * scale).view_as(x)


def _exact_norm(x, gamma):
    return x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * gamma


def _exact_branch(case, block, post, gate):
    v = block if post is None else _exact_norm(block, post)
    if gate is not None:
        v = v * (1 / (1 + torch.exp(-gate)) if case["gate"] == "sigmoid" else gate)
    return case["bs"] * v


def _wide(t, leaf=True):
    return None if t is None else _held(t).double().requires_grad_(leaf)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    if case["op"] == "ckpt":
        return {"values": _exact_round(s["x"], case["fmt"])}
    if case["op"] == "norms":
        block, post, gate = (_wide(s[n], False) for n in ("block", "post", "gate"))
        x = case["rs"] * s["residual"].double() + _exact_branch(case, block, post, gate)
        # the norm's input is the stream as it is stored
        return {"out": _exact_norm(x.to(torch.bfloat16).double(), s["pre"].double()), "residual": x, "x": None,
                "block": None, "gate": None}
    if case["op"] == "rms_q8":
        x, gamma = _wide(s["x"]), _wide(s["gamma"])
        _exact_norm(x, gamma).backward(s["grad_out"].double())
        more = 0.0 if s["grad_res"] is None else s["grad_res"].double()
        return {"grad_x": x.grad + more, "grad_gamma": gamma.grad}
    x, pre = _wide(s["x"]), _wide(s["pre"])
    _exact_norm(x, pre).backward(s["grad_out"].double())
    dx = x.grad if s["grad_res"] is None else x.grad + s["grad_res"].double()
    block, post, gate = (_wide(s[n]) for n in ("block", "post", "gate"))
    if block is None:
        return {"grad_residual": case["rs"] * dx, "grad_gamma_pre": pre.grad, "grad_gate": None,
                "grad_gamma_post": None, "grad_block": case["bs"] * dx}
    _exact_branch(case, block, post, gate).backward(dx)
    return {"grad_residual": case["rs"] * dx, "grad_gamma_pre": pre.grad, "grad_gate": None if gate is None else gate.grad,
            "grad_gamma_post": None if post is None else post.grad, "grad_block": block.grad}

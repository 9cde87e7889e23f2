"""The block norms and their backward on the GPU against the fp64 definition.

Tolerances (u = 2^-24).  rstd errs by 10 u (tests of the RMSNorm backward).  Forward: n = b rstd
gamma 12 u; the sigmoid 1 / (1 + e^-z): e^-z 2 u, of which the sum keeps at most that and adds u, the
reciprocal 1.02 u: 4.02 u, within the 6 u counted; products with gate and scale 1 u each: t = bs n
gate 20 u; the fma rounds once, the store by half a step of bf16 (eps / 2).  out is compared with
rlk_rmsnorm's bits on the stored x'.
Backward: dx errs by E = u [14 rstd |up| + 56 rstd^3 |x| sum|up x| / H] + u (|res| + |dx|), as the
RMSNorm's; a product passes its operands' errors on and adds u of itself; sigmoid' = e r r errs by 10 u
at most (8.04: e's 2 u once, since e and r r move against each other, 2.02 for each r, two products); a dot of
H terms adds 18 u of the sum of their magnitudes (8 in a lane's chain, at most 10 levels above);
rstd^2 / H 24 u; stores half a step.  grad_gammas: chains of 64 rows, one sum per chain, at most 16
teams, 152 ranges in 5 + 5 levels."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def n64(t):
    return None if t is None else t.double().cpu().numpy()


def half_step(t):
    return torch.finfo(t.dtype).eps / 2 * (1 + 2.0 ** -7)


def make(T, H, device, seed, post=True, gate="sigmoid", std=2.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return dict(block=r(T, H).to(BF16), residual=(r(T, H) * std).to(BF16),
                gamma_pre=(1 + 0.2 * r(H)).to(BF16), gamma_post=(1 + 0.2 * r(H)).to(BF16) if post else None,
                gate=None if gate == "none" else (1.5 * r(T, H)).to(BF16), gate_kind=gate)


CASES = [(1, 64), (3, 128), (7, 192), (5, 320), (33, 512), (9, 576), (20, 1024), (11, 1088), (6, 2048),
         (13, 2560), (17, 4096), (4, 4160), (3, 8128), (5, 8192), (700, 256), (310, 4096)]
FORMS = [(True, "none", 1.0, 1.0), (True, "sigmoid", 1.0, 0.5), (False, "identity", 2.5, 0.22),
         (False, "none", 0.75, 1.0), (True, "identity", 0.0, -1.5)]


@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("post,gate,rs,bs", FORMS)
def test_forward_parity(rlk, cuda_device, T, H, post, gate, rs, bs):
    a = make(T, H, cuda_device, T * H + 1, post, gate)
    rs, bs = float(np.float32(rs)), float(np.float32(bs))
    out, x, saved = rlk.block_norm(**a, residual_scale=rs, block_scale=bs, eps=1e-5)
    assert saved is None
    want, t = B.block_stream(n64(a["block"]), n64(a["residual"]), n64(a["gamma_post"]), n64(a["gate"]), gate, rs, bs, 1e-5)
    err = np.abs(n64(x) - want)
    assert np.all(err <= 20 * U * np.abs(t) + U * np.abs(want) + half_step(x) * np.abs(want))
    y, _ = rlk.rmsnorm(x, a["gamma_pre"], 1e-5)
    assert torch.equal(out, y)
    for fmt in ("int8", "e4m3"):
        out2, x2, saved = rlk.block_norm(**a, residual_scale=rs, block_scale=bs, eps=1e-5, save=fmt)
        assert torch.equal(out2, out) and torch.equal(x2, x)
        assert (saved.block is None) == (not post and gate == "none") and (saved.gate is None) == (gate == "none")
        for s, of in zip(saved, (x, a["block"], a["gate"])):
            if s is not None:
                q = rlk.act_quantize(of, fmt)
                assert torch.equal(s.scales, q.scales)
                assert torch.equal(s.codes.view(torch.uint8), q.codes.view(torch.uint8))


@pytest.mark.parametrize("T,H", [(1, 64), (40, 256), (33, 4096), (9, 8192)])
def test_plain_residual_add_is_the_rmsnorm(rlk, cuda_device, T, H):
    a = make(T, H, cuda_device, 3, False, "none")
    y, x = rlk.rmsnorm(a["block"], a["gamma_pre"], 1e-6, a["residual"], want_residual_out=True)
    out, got, _ = rlk.block_norm(**a)
    assert torch.equal(got, x) and torch.equal(out, y)


def tolerances(a, s, want, rs, bs, eps, grad_out, grad_res):
    """The bounds of the module's docstring, per gradient."""
    dy, x, gp, b, gq = n64(grad_out), n64(s["x"]), n64(a["gamma_pre"]), n64(s["block"]), n64(a["gamma_post"])
    T, H = x.shape
    up, rstd = np.abs(dy * gp), B._rms(x, eps)
    e_dx = U * (14 * rstd * up + 56 * rstd ** 3 * np.abs(x) * (up * np.abs(x)).mean(1, keepdims=True))
    e_dx = e_dx + U * np.abs(want["dx"]) + (0 if grad_res is None else U * np.abs(n64(grad_res)))
    e_d = abs(bs) * e_dx + U * np.abs(want["d"])
    tol = dict(grad_residual=abs(rs) * e_dx + U * np.abs(want["grad_residual"]))
    g = np.abs(want.get("gate", 1.0))
    if want["grad_gate"] is not None:
        tol["grad_gate"] = e_d * np.abs(want["n"] * want["slope"]) + 24 * U * np.abs(want["grad_gate"])
    e_w = e_d * g + 7 * U * np.abs(want["w"])
    rounds = 64 + -(-T // (152 * 64)) + 1 + 16 + 10
    tol["grad_gamma_pre"] = (rounds + 12) * U * np.abs(dy * x * rstd).sum(0)
    tol["grad_block"] = e_w
    if gq is not None:
        rb = B._rms(b, eps)
        v = np.abs(want["w"] * gq)
        e_v = e_w * np.abs(gq) + U * v
        k = rb ** 2 * (v * np.abs(b)).mean(1, keepdims=True)
        e_k = rb ** 2 * ((e_v * np.abs(b)).mean(1, keepdims=True) + 18 * U * (v * np.abs(b)).mean(1, keepdims=True)) + 24 * U * k
        tol["grad_block"] = rb * (e_v + np.abs(b) * e_k + 12 * U * (v + np.abs(b) * k))
        tol["grad_gamma_post"] = (e_w * np.abs(b) * rb).sum(0) + (rounds + 12) * U * np.abs(want["w"] * b * rb).sum(0)
    return tol


def held(rlk, a, x, fmt):
    """(what the backward gets, the same as bf16 tensors)"""
    t = dict(x=x, block=a["block"] if a["gamma_post"] is not None or a["gate"] is not None else None, gate=a["gate"])
    if fmt == "bf16":
        return t, t
    q = {k: None if v is None else rlk.act_quantize(v, fmt) for k, v in t.items()}
    return q, {k: None if v is None else rlk.act_dequantize(v) for k, v in q.items()}


@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("go,gx,res", [(F32, F32, True), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, False)])
def test_backward_parity(rlk, cuda_device, T, H, fmt, go, gx, res):
    for n, (post, gate, rs, bs) in enumerate(FORMS):
        rs, bs = float(np.float32(rs)), float(np.float32(bs))
        a = make(T, H, cuda_device, T * H + n, post, gate)
        x = (a["residual"].float() + 0.3).to(BF16)
        kept, plain = held(rlk, a, x, fmt)
        grad_out = (torch.randn(T, H, device=cuda_device) * 0.01).to(go)
        grad_res = (torch.randn(T, H, device=cuda_device) * 0.01).to(gx) if res else None
        kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], gate_kind=gate, residual_scale=rs,
                  block_scale=bs, eps=1e-5, grad_residual_out=grad_res, grad_dtype=gx)
        got = rlk.block_norm_backward(grad_out, **kept, **kw)
        want = B.block_backward(n64(grad_out), n64(plain["x"]), n64(a["gamma_pre"]), n64(plain["block"]),
                                n64(a["gamma_post"]), n64(plain["gate"]), gate, rs, bs, 1e-5, n64(grad_res))
        tol = tolerances(a, plain, want, rs, bs, 1e-5, grad_out, grad_res)
        for name, g in got._asdict().items():
            if want[name] is None:
                assert g is None
                continue
            assert g.dtype == (F32 if "gamma" in name else gx)
            step = 0 if "gamma" in name else half_step(g) * np.abs(want[name])
            assert np.all(np.abs(n64(g) - want[name]) <= tol[name] + step), (name, post, gate)
        if fmt != "bf16":  # a checkpoint's gradients have the bits of the restored tensors'
            same = rlk.block_norm_backward(grad_out, **plain, **kw)
            for p, q in zip(got, same):
                assert (p is None and q is None) or torch.equal(p, q)
        if n == 1:  # each output alone has the same bits
            for want_one in ("want_block", "want_residual", "want_gate", "want_gammas"):
                flags = {w: w == want_one for w in ("want_block", "want_residual", "want_gate", "want_gammas")}
                for p, q in zip(rlk.block_norm_backward(grad_out, **kept, **kw, **flags), got):
                    assert p is None or torch.equal(p, q)


@pytest.mark.parametrize("T,H", [(1, 64), (64, 4096), (300, 1024), (7, 8192), (500, 320)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("go,gx,res", [(F32, F32, False), (F32, BF16, True), (BF16, BF16, True), (BF16, F32, True)])
def test_rmsnorm_backward_q8(rlk, cuda_device, T, H, fmt, go, gx, res):
    a = make(T, H, cuda_device, T + H)
    saved = rlk.act_quantize(a["residual"], fmt)
    grad_out = (torch.randn(T, H, device=cuda_device) * 0.01).to(go)
    grad_res = (torch.randn(T, H, device=cuda_device) * 0.01).to(gx) if res else None
    kw = dict(eps=1e-6, grad_residual=grad_res, grad_dtype=gx)
    got, gg = rlk.rmsnorm_backward_q8(grad_out, saved, a["gamma_pre"], **kw)
    want, want_gg = rlk.rmsnorm_backward(grad_out, rlk.act_dequantize(saved), a["gamma_pre"], **kw)
    assert torch.equal(got, want)
    x, dy = n64(rlk.act_dequantize(saved)), n64(grad_out)
    # both sums err by at most 12 + 64 + 1 + 1 + 16 + 10 roundings, or for one cluster fewer
    assert np.all(np.abs(n64(gg) - n64(want_gg)) <= 2 * 104 * U * np.abs(dy * x * B._rms(x, 1e-6)).sum(0))
    only, none = rlk.rmsnorm_backward_q8(grad_out, saved, a["gamma_pre"], want_gamma=False, **kw)
    assert none is None and torch.equal(only, got)


def test_gradients_against_differences(rlk, cuda_device):
    """The loss sum(dy out) + sum(up x') moved along a direction, from the kernels' own forward in
    steps that bf16 holds exactly: x' and out round to bf16, so a difference of two losses errs by half
    a step of each summand, and by the third-order term of the definition."""
    T, H, h = 4, 64, 0.25
    a = make(T, H, cuda_device, 9, True, "identity")
    dy, up = torch.randn(2, T, H, device=cuda_device).to(BF16)
    kw = dict(gate_kind="identity", residual_scale=1.0, block_scale=0.5, eps=1e-3)
    out, x, _ = rlk.block_norm(a["block"], a["residual"], a["gamma_pre"], gamma_post=a["gamma_post"], gate=a["gate"], **kw)
    g = rlk.block_norm_backward(dy.float(), x, a["gamma_pre"], block=a["block"], gamma_post=a["gamma_post"],
                                gate=a["gate"], grad_residual_out=up.float(), **kw)
    for name in ("block", "residual", "gate"):
        sign = torch.sign(torch.randn(T, H, device=cuda_device))
        ends, grads64 = [], []
        for s in (1, -1):
            moved = dict(a)
            moved[name] = (a[name].float() + s * h * sign).to(BF16)
            o, xx, _ = rlk.block_norm(moved["block"], moved["residual"], a["gamma_pre"], gamma_post=a["gamma_post"],
                                      gate=moved["gate"], **kw)
            ends.append(((n64(dy) * n64(o)).sum() + (n64(up) * n64(xx)).sum(),
                         ((np.abs(n64(dy)) * np.abs(n64(o))).sum() + (np.abs(n64(up)) * np.abs(n64(xx))).sum()) * 2.0 ** -8,
                         n64(moved[name])))
        num = (ends[0][0] - ends[1][0]) / 2
        step = (ends[0][2] - ends[1][2]) / 2

        def f(s):
            m = {k: n64(a[k]) for k in ("block", "residual", "gate")}
            m[name] = m[name] + s * step
            xx, _ = B.block_stream(m["block"], m["residual"], n64(a["gamma_post"]), m["gate"], "identity", 1.0, 0.5, 1e-3)
            return (n64(dy) * xx * B._rms(xx, 1e-3) * n64(a["gamma_pre"])).sum() + (n64(up) * xx).sum()
        got = (n64(getattr(g, "grad_" + name)) * step).sum()
        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        third = abs((f(1.0) - f(-1.0)) / 2 - slope)
        middle = np.abs((ends[0][2] + ends[1][2]) / 2 - n64(a[name]))  # the midpoint's own rounding
        size = np.abs(n64(getattr(g, "grad_" + name)))
        # x', where the backward is taken, is a rounding away from the definition's
        rounding = (ends[0][1] + ends[1][1]) / 2 + 2 * third + (size * middle).sum() * 4 + 2.0 ** -7 * (size * np.abs(step)).sum()
        assert abs(num - got) <= rounding, name
        assert abs(slope - got) <= 2.0 ** -5 * (size * np.abs(step)).sum(), name


@pytest.mark.parametrize("H", [64, 576, 4096, 8192])
def test_rows_do_not_depend_on_the_batch(rlk, cuda_device, H):
    a = make(400, H, cuda_device, 10)
    out, x, saved = rlk.block_norm(**a, save="int8")
    dy = torch.randn(400, H, device=cuda_device).to(BF16)
    kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"])
    g = rlk.block_norm_backward(dy, **saved._asdict(), **kw, grad_residual_out=dy)
    for lo, hi in ((0, 1), (13, 200), (399, 400)):
        part = dict(a, **{k: a[k][lo:hi] for k in ("block", "residual", "gate")})
        o2, x2, s2 = rlk.block_norm(**part, save="int8")
        assert torch.equal(o2, out[lo:hi]) and torch.equal(x2, x[lo:hi])
        g2 = rlk.block_norm_backward(dy[lo:hi], **s2._asdict(), **kw, grad_residual_out=dy[lo:hi])
        for k in range(3):
            assert torch.equal(g2[k], g[k][lo:hi])


def test_not_a_number_stays_in_its_row(rlk, cuda_device):
    for H in (192, 1024, 8192):
        a = make(20, H, cuda_device, 11)
        clean = rlk.block_norm(**a)
        dy = torch.randn(20, H, device=cuda_device)
        kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], grad_dtype=BF16)
        g = rlk.block_norm_backward(dy, clean[1], block=a["block"], gate=a["gate"], **kw)
        keep = torch.arange(20, device=cuda_device) != 7
        for name, value in (("block", float("nan")), ("residual", float("inf")), ("gate", -float("inf")), ("gate", float("nan"))):
            bad = dict(a, **{name: a[name].clone()})
            bad[name][7, 100] = value
            got = rlk.block_norm(**bad)
            assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])
            if name == "gate" and value < 0:  # a gate that is shut
                assert torch.isfinite(got[0]).all()
            else:
                assert not torch.isfinite(got[0][7]).all()
            b = rlk.block_norm_backward(dy, got[1], block=bad["block"], gate=bad["gate"], **kw)
            for k in range(3):
                assert torch.equal(b[k][keep], g[k][keep])


def test_zero_rows_and_extreme_gates(rlk, cuda_device):
    a = make(8, 256, cuda_device, 12)
    a["block"][::2] = 0
    a["residual"][::4] = 0
    a["gate"][1] = 300.0
    a["gate"][3] = -300.0
    out, x, _ = rlk.block_norm(**a)
    assert torch.isfinite(out.float()).all() and not out[0].any()
    assert torch.equal(x[3], a["residual"][3])
    dy = torch.randn(8, 256, device=cuda_device)
    for eps in (1e-6, 2.0 ** -126):
        g = rlk.block_norm_backward(dy * 1e-3, x, a["gamma_pre"], block=a["block"], gamma_post=a["gamma_post"],
                                    gate=a["gate"], eps=eps)
        want = B.block_backward(n64(dy * 1e-3), n64(x), n64(a["gamma_pre"]), n64(a["block"]), n64(a["gamma_post"]),
                                n64(a["gate"]), "sigmoid", eps=eps)
        tol = tolerances(a, dict(x=x, block=a["block"]), want, 1.0, 1.0, eps, dy * 1e-3, None)
        for name in ("grad_residual", "grad_block", "grad_gate"):
            # a sigmoid below 2^-126 has lost digits of its own
            assert np.all(np.abs(n64(getattr(g, name)) - want[name]) <= tol[name] + 2 * U * np.abs(want[name]) + 2.0 ** -120), (name, eps)


@pytest.mark.parametrize("H", [64, 1024, 8192])
@pytest.mark.parametrize("gx", [BF16, F32])
def test_in_place_and_canaries(rlk, cuda_device, H, gx):
    T = 131
    a = make(T, H, cuda_device, 13)
    want = rlk.block_norm(**a, save="e4m3")
    buf = {k: a[k].clone() for k in ("block", "residual")}
    got = rlk.block_norm(**dict(a, **buf), out=buf["block"], residual_out=buf["residual"], save="e4m3")
    assert got[0].data_ptr() == buf["block"].data_ptr() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for s, w in zip(got[2], want[2]):
        assert torch.equal(s.codes.view(torch.uint8), w.codes.view(torch.uint8)) and torch.equal(s.scales, w.scales)
    guard = [torch.full((T + 2, H), 7.0, dtype=BF16, device=cuda_device) for _ in range(2)]
    rlk.block_norm(**a, out=guard[0][1:-1], residual_out=guard[1][1:-1])
    for t, w in zip(guard, want):
        assert torch.equal(t[1:-1], w) and torch.all(t[0] == 7) and torch.all(t[-1] == 7)
    dy, res = torch.randn(2, T, H, device=cuda_device).to(gx)
    kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], **want[2]._asdict())
    g = rlk.block_norm_backward(dy, **kw, grad_residual_out=res)
    n = rlk.block_norm_backward_workspace_size(T, H)
    ws = torch.full((n + 1024,), 9, dtype=torch.uint8, device=cuda_device)
    mine = res.clone()
    g2 = rlk.block_norm_backward(dy, **kw, grad_residual_out=mine, grad_residual=mine, workspace=ws[:n])
    assert g2.grad_residual.data_ptr() == mine.data_ptr() and torch.all(ws[n:] == 9)
    for p, q in zip(g, g2):
        assert torch.equal(p, q)
    over = dy.clone()
    g3 = rlk.block_norm_backward(over, **kw, grad_residual_out=res, grad_residual=over)
    assert torch.equal(g3.grad_residual, g.grad_residual) and torch.equal(g3.grad_block, g.grad_block)


@pytest.mark.parametrize("H", [320, 4096])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("go", [BF16, F32])
@pytest.mark.parametrize("gx", [BF16, F32])
def test_the_residuals_gradient_in_place(rlk, cuda_device, H, fmt, go, gx):
    """Every way in which the residual's gradient is read, from more rows than are under way at once."""
    T = 152 * 40 + 11
    a = make(T, H, cuda_device, 29)
    x = a["residual"]
    kept = dict(x=x, block=a["block"], gate=a["gate"])
    if fmt != "bf16":
        kept = {k: rlk.act_quantize(t, fmt) for k, t in kept.items()}
    dy, res = torch.randn(T, H, device=cuda_device).to(go), torch.randn(T, H, device=cuda_device).to(gx)
    kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], **kept)
    want = rlk.block_norm_backward(dy, **kw, grad_residual_out=res, grad_dtype=gx)
    for k in range(2):
        mine = res.clone()
        got = rlk.block_norm_backward(dy, **kw, grad_residual_out=mine, grad_residual=mine)
        assert got.grad_residual.data_ptr() == mine.data_ptr()
        for p, q in zip(got, want):
            assert torch.equal(p, q)


def test_no_rows(rlk, cuda_device):
    x = torch.zeros((0, 128), dtype=BF16, device=cuda_device)
    gamma = torch.ones(128, dtype=BF16, device=cuda_device)
    out, xx, saved = rlk.block_norm(x, x, gamma, gamma, save="int8")
    assert out.shape == xx.shape == saved.x.codes.shape == (0, 128)
    g = rlk.block_norm_backward(x, x, gamma, block=x, gamma_post=gamma)
    assert g.grad_block.shape == (0, 128) and not g.grad_gamma_pre.any() and not g.grad_gamma_post.any()
    g = rlk.block_norm_backward(x, saved.x, gamma, want_gammas=False)
    assert g.grad_residual.shape == (0, 128)
    gx, gg = rlk.rmsnorm_backward_q8(x, saved.x, gamma)
    assert gx.shape == (0, 128) and not gg.any()


@pytest.mark.parametrize("T,H,fmt", [(200003, 512, "int8"), (2 ** 20 + 3, 64, "bf16"), (30011, 4096, "e4m3"), (20001, 8192, "bf16")])
def test_grad_gammas_of_many_rows(rlk, cuda_device, T, H, fmt):
    """The same row of positive terms T times: a long chain of additions would drift."""
    g = torch.Generator(device=cuda_device)
    g.manual_seed(18)
    row = lambda: torch.rand(1, H, generator=g, device=cuda_device) + 0.5  # noqa: E731
    x1, b1, dy1 = row().to(BF16), row().to(BF16), row().to(BF16)
    ones = torch.ones(H, dtype=BF16, device=cuda_device)
    wide = lambda t: t.expand(T, H).contiguous()  # noqa: E731
    kept = dict(x=wide(x1), block=wide(b1))
    if fmt != "bf16":
        kept = {k: rlk.act_quantize(v, fmt) for k, v in kept.items()}
        x1, b1 = (rlk.act_dequantize(rlk.act_quantize(v, fmt)) for v in (x1, b1))
    got = rlk.block_norm_backward(wide(dy1), gamma_pre=ones, gamma_post=ones, grad_residual_out=wide(10 * dy1), **kept,
                                  want_block=False, want_residual=False)
    want = B.block_backward(n64(dy1), n64(x1), n64(ones), n64(b1), n64(ones), grad_res=n64(10 * dy1))
    a = dict(gamma_pre=ones, gamma_post=ones)
    tol = tolerances(a, dict(x=x1, block=b1), want, 1.0, 1.0, 1e-6, dy1, 10 * dy1)
    extra = -(-T // (152 * 64)) * U  # sums of chains
    for name in ("grad_gamma_pre", "grad_gamma_post"):
        assert np.all(np.abs(n64(getattr(got, name)) - T * want[name]) <= T * (tol[name] + extra * np.abs(want[name])))


def test_more_than_2_31_elements(rlk, cuda_device):
    """Row offsets past 32 bits: the last rows of a 2.1 G-element batch have their alone-bits."""
    T, H = 262147, 8192
    a = make(5, H, cuda_device, 16, gate="none")
    block, residual = (torch.zeros((T, H), dtype=BF16, device=cuda_device) for _ in range(2))
    block[-5:], residual[-5:] = a["block"], a["residual"]
    kw = dict(gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"])
    out, x, saved = rlk.block_norm(block, residual, save="int8", **kw)
    want = rlk.block_norm(a["block"], a["residual"], save="int8", **kw)
    assert torch.equal(out[-5:], want[0]) and torch.equal(x[-5:], want[1]) and not out[:-5].any()
    for s, w in zip(saved[:2], want[2][:2]):
        assert torch.equal(s.codes[-5:], w.codes) and torch.equal(s.scales[-5:], w.scales)
    block.zero_()
    block[-5:] = a["residual"]
    g = rlk.block_norm_backward(block, x=saved.x, block=saved.block, want_gammas=False, grad_residual=block, **kw)
    w = rlk.block_norm_backward(a["residual"], x=want[2].x, block=want[2].block, want_gammas=False, **kw)
    assert torch.equal(g.grad_block[-5:], w.grad_block) and torch.equal(g.grad_residual[-5:], w.grad_residual)
    assert not g.grad_residual[:-5].any()


@pytest.mark.parametrize("T,H", [(5, 256), (700, 4096)])
def test_graph_replay_streams_and_two_at_once(rlk, cuda_device, T, H):
    def step(a, dy, **kw):
        out, x, saved = rlk.block_norm(**a, save="int8", **kw)
        g = rlk.block_norm_backward(dy, **saved._asdict(), gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"],
                                    grad_residual_out=dy, **kw)
        return [out, x, *g]
    sets = [(make(T, H, cuda_device, s), torch.randn(T, H, device=cuda_device).to(BF16)) for s in (21, 22)]
    eager = [step(*s) for s in sets]
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(cuda_device))
    got = [[step(*sets[k], stream=streams[k]) for k in range(2)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        for k in range(2):
            assert all(torch.equal(p, q) for p, q in zip(pair[k], eager[k]))
    held_a = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in sets[0][0].items()}
    held_dy = sets[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held_a, held_dy)
    for (a, dy), e in zip(sets, eager):
        for k, v in a.items():
            if isinstance(v, torch.Tensor):
                held_a[k].copy_(v)
        held_dy.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, e))


def test_binding_checks(rlk, cuda_device):
    a = make(4, 128, cuda_device, 30)
    out, x, saved = rlk.block_norm(**a, save="int8")
    bwd = lambda dy=x, **kw: rlk.block_norm_backward(  # noqa: E731
        dy, **dict(dict(x=x, gamma_pre=a["gamma_pre"], gamma_post=a["gamma_post"], block=a["block"]), **kw))
    bwd()
    for bad in (lambda: rlk.block_norm(**dict(a, block=a["block"].half())), lambda: bwd(dy=x.half()),
                lambda: bwd(grad_dtype=torch.float16), lambda: bwd(x=saved.x),    # a bf16 block beside it
                lambda: bwd(x=saved.x, block=rlk.act_quantize(a["block"], "e4m3")),
                lambda: bwd(x=(saved.x.codes, saved.x.scales)), lambda: bwd(grad_residual_out=x.float()),
                lambda: rlk.rmsnorm_backward_q8(x, x, a["gamma_pre"])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: rlk.block_norm(**dict(a, gate_kind="tanh")), lambda: rlk.block_norm(**a, save="fp4"),
                lambda: rlk.block_norm(**dict(a, gate=a["gate"][:2])), lambda: bwd(block=None),
                lambda: bwd(gamma_post=a["gamma_post"][:64]), lambda: bwd(dy=x[:2]),
                lambda: rlk.block_norm(**a, stream=torch.cuda.Stream(cuda_device), out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: rlk.block_norm(**a, eps=0.0), lambda: rlk.block_norm(**a, out=a["residual"]),
                lambda: bwd(eps=2.0 ** -130), lambda: rlk.block_norm(**a, block_scale=float("inf"))):
        with pytest.raises(rlk.RlkError):
            bad()

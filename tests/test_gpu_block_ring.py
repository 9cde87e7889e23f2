"""The block norms over many different rows a CTA: every stage of the backward's ring is filled again and
again, sums over the rows go past their first chain, and the forward's CTAs take several rows each.

Per-row results are compared, bit for bit, with those of the same rows in calls small enough that no
stage of the ring is used twice (a row a team), whose parity with the definition other tests check; the
grad_gammas with the fp64 definition over all rows, formed here by torch in fp64.

Tolerances of the grad_gammas (u = 2^-24): a summand of grad_gamma_pre, dy x rstd, errs by 12 u (rstd 10, two
products), the sum by one u of the magnitudes for each of at most 64 (chain) + T / (152 * 64) + 1 (sums of chains)
+ 16 (teams) + 10 (ranges) additions.  A summand of grad_gamma_post is w b rstd_b with w = d gate(z): dx errs by u [14
rstd |up| + 56 rstd^3 |x| sum |up x| / H] + u (|res| + |dx|), d by the scale's share of that and u, w by 7 u
more (gate 6, product 1)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-5
WIDTHS = [512, 1024, 4096, 8192]  # 1, 2, 8 and 16 warps a row
FORMS = [("none", False), ("none", True), ("identity", True), ("sigmoid", True), ("identity", False), ("sigmoid", False)]


def teams(H):
    warps = 1
    while warps * 512 < H:
        warps *= 2
    return 16 // warps


def make(T, H, device, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return dict(x=(2 * r(T, H)).to(BF16), block=r(T, H).to(BF16), gate=(1.5 * r(T, H)).to(BF16)), \
        (1 + 0.2 * r(H)).to(BF16), (1 + 0.2 * r(H)).to(BF16), 0.01 * r(T, H), 0.01 * r(T, H)


def cut(v, lo, hi):
    return None if v is None else type(v)(*(t[lo:hi] for t in v)) if isinstance(v, tuple) else v[lo:hi]


def norms64(t, x, pre, post, dy, res, kind, bs):
    """(grad_gamma_pre, its tolerance, grad_gamma_post, its tolerance) in fp64."""
    T, H = x.shape
    x, dy, gp = x.double(), dy.double(), pre.double()
    rounds = 64 + -(-T // (152 * 64)) + 1 + 16 + 10
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    n = dy * x * rstd
    out = [n.sum(0), (rounds + 12) * U * n.abs().sum(0)]
    if post is None:
        return out + [None, None]
    b, up = t["block"].double(), dy * gp
    dx = rstd * (up - x * rstd ** 2 * (up * x).mean(1, keepdim=True))
    e = U * (14 * rstd * up.abs() + 56 * rstd ** 3 * x.abs() * (up * x).abs().mean(1, keepdim=True))
    if res is not None:
        dx += res.double()
        e += U * res.double().abs()
    e += U * dx.abs()
    d = bs * dx
    e = abs(bs) * e + U * d.abs()
    if t["gate"] is not None:
        z = t["gate"].double()
        z = torch.sigmoid(z) if kind == "sigmoid" else z
        d = d * z
        e = e * z.abs() + 7 * U * d.abs()
    rb = torch.rsqrt(b.square().mean(1, keepdim=True) + EPS)
    n = d * b * rb
    return out + [n.sum(0), (e * b.abs() * rb).sum(0) + (rounds + 12) * U * n.abs().sum(0)]


def run(rlk, T, H, device, seed, kind, post, fmt, go, gx, res, plain=False, step=None):
    """A call over T rows against the same rows in calls of `step` rows, and the grad_gammas' definition.
    plain: the RMSNorm's backward from a checkpoint, which has no branch."""
    t, g_pre, g_post, dy, up = make(T, H, device, seed)
    dy, up = dy.to(go), up.to(gx) if res else None
    g_post = g_post if post else None
    if kind == "none":
        t["gate"] = None
    if plain or (kind == "none" and not post):
        t["block"] = None
    kept, held = t, t
    if fmt != "bf16":
        kept = {k: None if v is None else rlk.act_quantize(v, fmt) for k, v in t.items()}
        held = {k: None if v is None else rlk.act_dequantize(v) for k, v in kept.items()}
    del t

    def call(lo, hi, gammas):
        if plain:
            return list(rlk.rmsnorm_backward_q8(dy[lo:hi], cut(kept["x"], lo, hi), g_pre, EPS, grad_residual=cut(up, lo, hi),
                                                want_gamma=gammas, grad_dtype=gx))
        g = rlk.block_norm_backward(dy[lo:hi], cut(kept["x"], lo, hi), g_pre, block=cut(kept["block"], lo, hi), gamma_post=g_post,
                                    gate=cut(kept["gate"], lo, hi), gate_kind=kind, residual_scale=1.5, block_scale=-0.5, eps=EPS,
                                    grad_residual_out=cut(up, lo, hi), grad_dtype=gx, want_gammas=gammas)
        return [g.grad_residual, g.grad_block, g.grad_gate, g.grad_gamma_pre, g.grad_gamma_post]
    got = call(0, T, True)
    rows = got[:1] if plain else [v for v in got[:3] if v is not None]
    step = step or 152 * teams(H)
    for lo in range(0, T, step):
        part = call(lo, min(T, lo + step), False)
        for a, b in zip(rows, part[:1] if plain else [v for v in part[:3] if v is not None]):
            assert torch.equal(a[lo:lo + step], b), lo
    want = norms64(held, held["x"], g_pre, None if plain else g_post, dy, up, kind, -0.5)
    for name, value, w, tol in (("pre", got[1] if plain else got[3], *want[:2]), ("post", None if plain else got[4], *want[2:])):
        if w is not None:
            assert torch.all((value.double() - w).abs() <= tol), name


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("go,gx,res", [(F32, F32, True), (F32, BF16, False), (BF16, BF16, True), (BF16, F32, True)])
def test_backward_of_rows_that_follow_each_other(rlk, cuda_device, H, fmt, go, gx, res):
    T = 152 * teams(H) * 9 + 5
    for n, (kind, post) in enumerate(FORMS):
        run(rlk, T, H, cuda_device, H + n, kind, post, fmt, go, gx, res)
    if fmt != "bf16":
        run(rlk, T, H, cuda_device, H + 9, "none", False, fmt, go, gx, res, plain=True)


@pytest.mark.parametrize("H", [320, 960, 1920, 4032, 7744])
def test_backward_of_rows_that_end_inside_a_warp(rlk, cuda_device, H):
    T = 152 * teams(H) * 6 + 77
    run(rlk, T, H, cuda_device, H, "sigmoid", True, "int8", F32, F32, True)
    run(rlk, T, H, cuda_device, H + 1, "identity", True, "bf16", F32, BF16, True)
    run(rlk, T, H, cuda_device, H + 2, "none", False, "e4m3", F32, BF16, True, plain=True)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("kind,post,fmt,go,gx,plain", [
    ("sigmoid", True, "int8", BF16, BF16, False), ("sigmoid", True, "bf16", F32, F32, False), ("identity", True, "e4m3", F32, BF16, False),
    ("none", True, "bf16", BF16, BF16, False), ("none", False, "int8", F32, BF16, True), ("none", False, "e4m3", BF16, F32, True)])
def test_backward_of_several_chains(rlk, cuda_device, H, kind, post, fmt, go, gx, plain):
    """More than 64 rows a team: the sums so far move to shared memory, which shortens the ring, twice in the
    last team."""
    T = 152 * teams(H) * 130 + 11
    run(rlk, T, H, cuda_device, H, kind, post, fmt, go, gx, True, plain, step=152 * teams(H) * 2)


@pytest.mark.parametrize("H", WIDTHS + [64, 7744])
@pytest.mark.parametrize("kind,post,save", [("sigmoid", True, "int8"), ("identity", True, "e4m3"), ("sigmoid", False, None), ("none", True, None)])
def test_forward_of_several_rows_a_team(rlk, cuda_device, H, kind, post, save):
    """Beyond 64 CTAs an SM a CTA goes on with further rows."""
    a_cta = max(1, teams(H) // 2) if H <= 1024 else 1  # of 256 threads where a row takes one or two warps
    T = 152 * 64 * a_cta + 1001
    t, g_pre, g_post, _, _ = make(T, H, cuda_device, H + 5)
    call = lambda lo, hi: rlk.block_norm(t["block"][lo:hi], t["x"][lo:hi], g_pre, g_post if post else None,  # noqa: E731
                                         t["gate"][lo:hi] if kind != "none" else None, kind, 1.5, -0.5, EPS, save=save)
    out, x, saved = call(0, T)
    for lo in range(0, T, 9000):
        o, y, s = call(lo, min(T, lo + 9000))
        assert torch.equal(o, out[lo:lo + 9000]) and torch.equal(y, x[lo:lo + 9000])
        for p, q in zip(saved or (), s or ()):
            if p is not None:
                assert torch.equal(p.codes[lo:lo + 9000].view(torch.uint8), q.codes.view(torch.uint8))
                assert torch.equal(p.scales[lo:lo + 9000], q.scales)


@pytest.mark.parametrize("H", [64, 960, 8192])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_a_gradient_in_the_place_of_grad_out(rlk, cuda_device, H, dtype, fmt):
    """The C entry lets any one of the three gradients take grad_out's place."""
    T = 152 * teams(H) * 5 + 3
    t, g_pre, g_post, dy, up = make(T, H, cuda_device, H + 6)
    dy, up, code = dy.to(dtype), up.to(dtype), 0 if dtype is F32 else 1
    kept = t if fmt == "bf16" else {k: rlk.act_quantize(v, fmt) for k, v in t.items()}
    want = rlk.block_norm_backward(dy, kept["x"], g_pre, block=kept["block"], gamma_post=g_post, gate=kept["gate"], eps=EPS,
                                   grad_residual_out=up)
    ptr = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    both = [(v.codes, v.scales) if isinstance(v, tuple) else (v, None) for v in (kept["x"], kept["block"], kept["gate"])]
    ws = torch.empty(rlk.block_norm_backward_workspace_size(T, H), dtype=torch.uint8, device=cuda_device)
    for k in range(3):
        over = dy.clone()
        grads = [over if n == k else torch.empty_like(dy) for n in range(3)]  # residual, block, gate
        gam = [torch.empty(H, device=cuda_device) for _ in range(2)]
        code_ = rlk.lib().rlk_block_norm_backward(
            ptr(over), code, ptr(up), 0 if fmt == "bf16" else 1, *(ptr(v) for pair in both for v in pair), 2, ptr(g_post),
            ptr(g_pre), 1.0, 1.0, EPS, T, H, *(ptr(g) for g in grads), code, ptr(gam[0]), ptr(gam[1]), ptr(ws), ws.numel(),
            torch.cuda.current_stream(cuda_device).cuda_stream)
        assert code_ == 0
        for got, w in zip(grads + gam, (want.grad_residual, want.grad_block, want.grad_gate, want.grad_gamma_pre, want.grad_gamma_post)):
            assert torch.equal(got, w), k

"""Backward of the strict RMSNorm on the GPU against the fp64 definition.

Tolerances (u = 2^-24).  rstd: the mean square's 13 tree levels, division and eps add 15 u, the
root halves that, rlk_rsqrt errs by 2 u: 10 u.  The dot product sum up_i x_i: each product rounds
twice, 8 terms in a thread and at most 10 tree levels: 20 u of sum |up_i x_i|.  So
rstd (up - x c) errs by at most u [14 rstd |up| + 56 rstd^3 |x| sum |up x| / H] (c takes the dot's
20 u, twice rstd's 10 u and 4 roundings; the product with rstd 12 u more), the residual's sum by u
of itself, and the store by half a step of its type.  grad_gamma: dy x rstd errs by 12 u, a range
of ceil(T / 152) rows at most is summed in order (15 more where several teams share it) and the
ranges by at most 10 + 5 more roundings."""
import numpy as np
import pytest
import torch

from invariant_selected_token_gb300 import workloads as WL
from oracle import training as TR

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def make(T, H, device, seed, go=F32, res=None, x_std=2.0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    return dict(grad_out=(r(T, H) * 0.01).to(go), x=(r(T, H) * x_std).to(BF16),
                gamma=(1 + 0.2 * r(H)).to(BF16),
                grad_residual=None if res is None else (r(T, H) * 0.01).to(res))


def n64(t):
    return None if t is None else t.double().cpu().numpy()


def check(a, eps, grad_x, grad_gamma):
    dy, x, gam, res = (n64(a[k]) for k in ("grad_out", "x", "gamma", "grad_residual"))
    T, H = x.shape
    want_x, want_g = TR.rmsnorm_backward(dy, x, gam, eps, res)
    rstd = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    up = np.abs(dy * gam)
    tol = U * (14 * rstd * up + 56 * rstd ** 3 * np.abs(x) * (up * np.abs(x)).sum(1, keepdims=True) / H)
    if res is not None:
        tol = tol + U * (np.abs(res) + np.abs(want_x))
    tol = tol + np.abs(want_x) * (torch.finfo(grad_x.dtype).eps / 2) * (1 + 2.0 ** -8)
    assert np.all(np.abs(n64(grad_x) - want_x) <= tol)
    if grad_gamma is not None:
        rounds = 12 + (-(-T // 152) if T > 16 else 2) + 23 + 15
        assert np.all(np.abs(n64(grad_gamma) - want_g) <= rounds * U * np.abs(dy * x * rstd).sum(0))


CASES = [(1, 64), (3, 128), (7, 192), (64, 4096), (16, 4096), (17, 4096), (16, 320), (9, 2048),
         (16, 8192), (13, 1024), (33, 2560), (305, 320), (5, 8192), (130, 8128),
         (700, 1024), (911, 576), (2, 4160)]


@pytest.mark.parametrize("T,H", CASES)
@pytest.mark.parametrize("go,gx,res", [(F32, F32, False), (F32, BF16, True), (BF16, BF16, True),
                                       (BF16, F32, True), (BF16, BF16, False)])
def test_rmsnorm_backward_parity(rlk, cuda_device, T, H, go, gx, res):
    a = make(T, H, cuda_device, T * H, go, gx if res else None)
    grad_x, grad_gamma = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], 1e-6,
                                              grad_residual=a["grad_residual"], grad_dtype=gx)
    assert grad_x.dtype == gx
    check(a, 1e-6, grad_x, grad_gamma)
    only, none = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], 1e-6, want_gamma=False,
                                      grad_residual=a["grad_residual"], grad_dtype=gx)
    assert none is None and torch.equal(only, grad_x)


@pytest.mark.parametrize("go,gx", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("H", [4160, 8192])
def test_wide_rows_in_one_cluster_keep_their_bits(rlk, cuda_device, H, go, gx):
    """Up to 16 rows wider than 4096 features: the sums for grad_gamma lie where the rows' inputs
    did, and no warp may put its own there before the slowest one has read its row.  grad_x has the
    bits of the call that forms no such sums, and grad_gamma the same ones each time."""
    for T in range(1, 17):
        a = make(T, H, cuda_device, 100 * T + 1, go, gx)
        call = lambda **kw: rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"],  # noqa: E731
                                                 grad_residual=a["grad_residual"], grad_dtype=gx, **kw)
        want, _ = call(want_gamma=False)
        outs = [call() for _ in range(20)]
        check(a, 1e-6, *outs[0])
        for grad_x, grad_gamma in outs:
            assert torch.equal(grad_x, want) and torch.equal(grad_gamma, outs[0][1])


@pytest.mark.parametrize("eps,x_std", [(1e-5, 1e-4), (1.0, 0.1), (1e-6, 300.0)])
def test_eps_and_scale(rlk, cuda_device, eps, x_std):
    a = make(40, 512, cuda_device, 5, x_std=x_std)
    check(a, eps, *rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], eps))


def test_zero_rows(rlk, cuda_device):
    """Rows of zeros (padding): rstd = 1 / sqrt(eps), no division by zero."""
    a = make(9, 256, cuda_device, 6)
    a["x"][::2] = 0
    grad_x, grad_gamma = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], 1e-4)
    check(a, 1e-4, grad_x, grad_gamma)
    assert torch.isfinite(grad_x).all()


def test_zero_rows_with_the_smallest_eps(rlk, cuda_device):
    a = make(9, 256, cuda_device, 17)
    a["x"][::2] = 0
    grad_x, grad_gamma = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], 2.0 ** -126)
    check(a, 2.0 ** -126, grad_x, grad_gamma)
    assert torch.isfinite(grad_x).all()


def test_gradient_against_differences_of_the_forward(rlk, cuda_device):
    """Directional difference of sum dy * rmsnorm(x) along v.  The forward rounds y to bf16, so a
    difference of outputs errs by up to 2 * 2^-9 * |y| per element over 2h; with 64 rows of one
    direction the bound is the sum of those."""
    T, H, h = 4, 64, 0.25
    a = make(T, H, cuda_device, 7)
    grad_x, grad_gamma = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], 1e-6)
    v = torch.sign(torch.randn(T, H, generator=torch.Generator().manual_seed(1))).to(cuda_device)
    plus, minus = (a["x"].float() + h * v).to(BF16), (a["x"].float() - h * v).to(BF16)
    yp, _ = rlk.rmsnorm(plus, a["gamma"])
    ym, _ = rlk.rmsnorm(minus, a["gamma"])
    dy = n64(a["grad_out"])
    num = (dy * (n64(yp) - n64(ym))).sum() / 2
    step = (n64(plus) - n64(minus)) / 2
    got = (n64(grad_x) * step).sum()
    rounding = (np.abs(dy) * (np.abs(n64(yp)) + np.abs(n64(ym))) * 2.0 ** -9).sum() / 2
    # the third-order term of y along the step, from the fp64 definition's own differences
    def f(s):
        xx = n64(a["x"]) + s * step
        return (dy * xx / np.sqrt((xx * xx).mean(1, keepdims=True) + 1e-6) * n64(a["gamma"])).sum()
    third = abs((f(1.0) - f(-1.0)) / 2 - (f(1e-4) - f(-1e-4)) / 2e-4)
    first = abs(n64(a["x"]) - (n64(plus) + n64(minus)) / 2).max()  # the midpoint's own rounding
    assert abs(num - got) <= rounding + 2 * third + np.abs(dy).sum() * first * 2
    dg = n64(grad_gamma)
    y, _ = rlk.rmsnorm(a["x"], torch.ones_like(a["gamma"]))
    want = (dy * n64(y)).sum(0)  # y is linear in gamma
    assert np.all(np.abs(dg - want) <= (np.abs(dy * n64(y)) * 2.0 ** -8).sum(0) + 1e-12)


def test_rows_do_not_depend_on_the_batch(rlk, cuda_device):
    a = make(700, 2048, cuda_device, 8, BF16, BF16)
    full, _ = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], grad_residual=a["grad_residual"])
    for lo, hi in ((0, 1), (13, 400), (699, 700)):
        part, _ = rlk.rmsnorm_backward(a["grad_out"][lo:hi], a["x"][lo:hi], a["gamma"],
                                       grad_residual=a["grad_residual"][lo:hi])
        assert torch.equal(part, full[lo:hi])


@pytest.mark.parametrize("H", [64, 1024, 8192])
def test_in_place_and_canaries(rlk, cuda_device, H):
    T = 131
    a = make(T, H, cuda_device, 9, BF16, BF16)
    kw = dict(x=a["x"], gamma=a["gamma"])
    want, want_g = rlk.rmsnorm_backward(a["grad_out"], grad_residual=a["grad_residual"], **kw)
    for name in ("grad_residual", "grad_out"):
        buf = {k: a[k].clone() for k in ("grad_residual", "grad_out")}
        got, _ = rlk.rmsnorm_backward(buf["grad_out"], grad_residual=buf["grad_residual"],
                                      grad_x=buf[name], **kw)
        assert got.data_ptr() == buf[name].data_ptr() and torch.equal(got, want)
    guard = torch.full((T + 16, H), 7.0, dtype=BF16, device=cuda_device)
    gg = torch.full((H + 128,), 7.0, device=cuda_device)
    ws_n = rlk.lib().rlk_rmsnorm_backward_workspace_size(T, H)
    ws = torch.full((ws_n + 1024,), 9, dtype=torch.uint8, device=cuda_device)
    rlk.rmsnorm_backward(a["grad_out"], grad_residual=a["grad_residual"], grad_x=guard[8:8 + T],
                         grad_gamma=gg[64:64 + H], workspace=ws[:ws_n], **kw)
    assert torch.equal(guard[8:8 + T], want) and torch.equal(gg[64:64 + H], want_g)
    assert torch.all(guard[:8] == 7) and torch.all(guard[8 + T:] == 7)
    assert torch.all(gg[:64] == 7) and torch.all(gg[64 + H:] == 7) and torch.all(ws[ws_n:] == 9)


def test_in_place_fp32(rlk, cuda_device):
    a = make(700, 4096, cuda_device, 15, F32, F32)
    kw = dict(x=a["x"], gamma=a["gamma"])
    want, _ = rlk.rmsnorm_backward(a["grad_out"], grad_residual=a["grad_residual"], **kw)
    for name in ("grad_residual", "grad_out"):
        buf = {k: a[k].clone() for k in ("grad_residual", "grad_out")}
        got, _ = rlk.rmsnorm_backward(buf["grad_out"], grad_residual=buf["grad_residual"],
                                      grad_x=buf[name], **kw)
        assert torch.equal(got, want)


def test_more_than_2_31_bytes(rlk, cuda_device):
    """Row offsets past 32 bits: the last rows of a 2.5 G-element batch have their alone-bits."""
    T, H = 300007, 8192
    x = torch.zeros((T, H), dtype=BF16, device=cuda_device)
    dy = torch.zeros((T, H), dtype=BF16, device=cuda_device)
    a = make(5, H, cuda_device, 16, BF16)
    x[-5:], dy[-5:] = a["x"], a["grad_out"]
    gx, gg = rlk.rmsnorm_backward(dy, x, a["gamma"], grad_x=dy)
    want, want_g = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"])
    assert torch.equal(gx[-5:], want) and not gx[:-5].any()
    tol = 64 * U * n64((a["grad_out"].float() * a["x"].float()).abs().sum(0))
    assert np.all(np.abs(n64(gg) - n64(want_g)) <= tol)


@pytest.mark.parametrize("T,H,go", [(304003, 4160, BF16), (2 ** 21 + 3, 64, F32), (400000, 2048, BF16)])
def test_grad_gamma_of_many_rows(rlk, cuda_device, T, H, go):
    """The same row of positive products T times, so that a long chain of additions would round the
    same way each time and drift.  A chain has at most 64 rows (64 roundings), a team adds up one
    sum per chain, at most 16 teams share a range, and 152 ranges follow."""
    g = torch.Generator(device=cuda_device)
    g.manual_seed(18)
    row = lambda: torch.rand(1, H, generator=g, device=cuda_device) + 0.5  # noqa: E731
    x1, dy1 = row().to(BF16), row().to(go)
    x, dy = x1.expand(T, H).contiguous(), dy1.expand(T, H).contiguous()
    _, gg = rlk.rmsnorm_backward(dy, x, torch.ones(H, dtype=BF16, device=cuda_device), grad_dtype=BF16)
    teams = max(1, 16 // max(1, 1 << ((H - 1) // 512).bit_length()))
    chains = -(-T // (152 * teams * 64))
    want = T * (n64(dy1) * n64(x1) / np.sqrt((n64(x1) ** 2).mean() + 1e-6))[0]
    assert np.all(np.abs(n64(gg) - want) <= (12 + 64 + chains + 1 + teams + 10) * U * want)


def test_no_rows(rlk, cuda_device):
    x = torch.zeros((0, 128), dtype=BF16, device=cuda_device)
    gx, gg = rlk.rmsnorm_backward(x, x, torch.ones(128, dtype=BF16, device=cuda_device))
    assert gx.shape == (0, 128) and not gg.any()


def test_nan_stays_in_its_row(rlk, cuda_device):
    a = make(20, 512, cuda_device, 10)
    clean, _ = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"])
    a["grad_out"][7, 100] = float("nan")
    got, gg = rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"])
    keep = torch.arange(20, device=cuda_device) != 7
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[7]).all()
    assert torch.isnan(gg[100]) and int(torch.isnan(gg).sum()) == 1


@pytest.mark.parametrize("T,H", [(5, 256), (700, 4096)])
def test_graph_replay_and_streams(rlk, cuda_device, T, H):
    sets = [make(T, H, cuda_device, s, F32, BF16) for s in (11, 12)]
    call = lambda a, **kw: rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"],  # noqa: E731
                                                grad_residual=a["grad_residual"], grad_dtype=BF16, **kw)
    eager = [call(a) for a in sets]
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    other = call(sets[0], stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(other, eager[0]))
    held = {k: v.clone() for k, v in sets[0].items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(held)
    for a, e in zip(sets, eager):
        for k, v in a.items():
            held[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, e))


def test_binding_checks(rlk, cuda_device):
    a = make(4, 128, cuda_device, 13)
    with pytest.raises(TypeError):
        rlk.rmsnorm_backward(a["grad_out"].half(), a["x"], a["gamma"])
    with pytest.raises(TypeError):
        rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], grad_dtype=torch.float16)
    with pytest.raises(TypeError):  # the residual's gradient has grad_x's type
        rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], grad_residual=a["x"])
    with pytest.raises(ValueError):
        rlk.rmsnorm_backward(a["grad_out"][:2], a["x"], a["gamma"])
    with pytest.raises(ValueError):
        rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"][:64])
    with pytest.raises(rlk.RlkError):
        rlk.rmsnorm_backward(a["grad_out"], a["x"], a["gamma"], eps=0.0)


def test_rstd_is_the_forwards(rlk, cuda_device):
    """With grad_out = 0 but for the residual, grad_x is the residual; and with gamma = 1 and a
    one-hot grad_out, grad_gamma is the forward's x * rstd before its rounding to bf16."""
    a = make(1, 1024, cuda_device, 14)
    ones = torch.ones(1024, dtype=BF16, device=cuda_device)
    y, _ = rlk.rmsnorm(a["x"], ones)
    _, gg = rlk.rmsnorm_backward(torch.ones(1, 1024, device=cuda_device), a["x"], ones)
    assert torch.equal(gg.to(BF16), y[0])
    assert np.abs(WL.bf16_bits_to_f32(WL.bf16_tensor_bits(y))).max() > 1

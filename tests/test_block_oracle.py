"""The fp64 definitions of the block norms, the checkpoints and the draft verification, against
central differences, closed forms and enumeration."""
import numpy as np
import pytest

from oracle import block as B


@pytest.mark.parametrize("post,gate,kind", [(False, False, "identity"), (True, False, "identity"),
                                            (True, True, "sigmoid"), (False, True, "identity"),
                                            (True, True, "identity")])
def test_block_gradients_against_differences(post, gate, kind):
    rng = np.random.default_rng(1)
    T, H, rs, bs, eps = 3, 64, 1.5, 0.5, 1e-3
    b, r, dy = rng.standard_normal((3, T, H))
    gp, gq = 1 + 0.1 * rng.standard_normal((2, H))
    z = rng.standard_normal((T, H)) if gate else None
    up = rng.standard_normal((T, H))
    gq = gq if post else None

    def f(b, r, z, gp, gq):  # no rounding of x' here
        x, _ = B.block_stream(b, r, gq, z, kind, rs, bs, eps)
        return (dy * x * B._rms(x, eps) * gp).sum() + (up * x).sum()
    x, _ = B.block_stream(b, r, gq, z, kind, rs, bs, eps)
    got = B.block_backward(dy, x, gp, b, gq, z, kind, rs, bs, eps, up)
    args = [b, r, z, gp, gq]
    for k, name in enumerate(("grad_block", "grad_residual", "grad_gate", "grad_gamma_pre", "grad_gamma_post")):
        if args[k] is None:
            assert got[name] is None
            continue
        step = rng.standard_normal(args[k].shape)
        lo, hi = list(args), list(args)
        lo[k], hi[k] = args[k] - 1e-6 * step, args[k] + 1e-6 * step
        num = (f(*hi) - f(*lo)) / 2e-6
        assert abs(num - (got[name] * step).sum()) <= 1e-6 * np.abs(got[name] * step).sum()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_code_is_the_nearest_one(fmt):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((8, 64)) * 2.0 ** rng.integers(-60, 60, (8, 1))
    x = (np.float32(x).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    x[3, :32] = 0
    codes, scales = B.quantize(x, fmt)
    back = B.dequantize(codes, scales, fmt)
    grid = np.arange(-127, 128) * 1.0 if fmt == "int8" else np.delete(B.E4M3, [0x7F, 0xFF])
    for t in range(8):
        for k in range(2):
            sl = slice(32 * k, 32 * k + 32)
            step = 2.0 ** (int(scales[t, k]) - (133 if fmt == "int8" else 127))
            nearest = np.abs(grid[None] * step - x[t, sl, None]).min(1)
            assert np.array_equal(np.abs(back[t, sl] - x[t, sl]), nearest)
    assert np.all(back[3, :32] == 0)
    again = B.quantize(back, fmt)
    assert np.array_equal(B.dequantize(*again, fmt), back)  # a value that fits stays


def test_e4m3_numbers():
    assert B.E4M3[0x7E] == 448 and B.E4M3[0x01] == 2.0 ** -9 and B.E4M3[0x08] == 2.0 ** -6 and B.E4M3[0xB8] == -1


def test_verified_tokens_follow_the_target():
    """Every outcome of one drafted token, weighted: sum over drafts and acceptance of its
    probability is the target's own distribution."""
    rng = np.random.default_rng(3)
    V = 6
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    left = np.maximum(p - q, 0)
    total = np.zeros(V)
    for x in range(V):
        keep = min(1.0, p[x] / q[x])
        total[x] += q[x] * keep
        total += q[x] * (1 - keep) * left / left.sum()
    assert np.allclose(total, p, rtol=0, atol=1e-12)
    # and the oracle's decisions are those: accepted just below the ratio, refused at it
    x = int(np.argmax(q / p))
    ratio = p[x] / q[x]
    for u, want in ((ratio * (1 - 1e-9), 1), (ratio * (1 + 1e-9), 0)):
        acc, tok, lp, _ = B.draft_verify(np.log(np.stack([p, p])), [x], [u], np.ones((1, V)), [0, 1],
                                         np.log(q)[None])
        assert acc[0] == want
        assert tok[0] == (x if want else int(np.argmax(left)))
        assert abs(lp[0] - np.log(p[tok[0]])) < 1e-12

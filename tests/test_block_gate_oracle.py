"""The fp64 definition of a sigmoid gate on a block that is not normed, against central differences."""
import numpy as np
import pytest

from oracle import block as B


@pytest.mark.parametrize("rs,bs", [(1.0, 1.0), (1.5, -0.5)])
def test_gradients_against_differences(rs, bs):
    rng = np.random.default_rng(11)
    T, H, eps = 3, 64, 1e-3
    b, r, z, dy, up = rng.standard_normal((5, T, H))
    gp = 1 + 0.1 * rng.standard_normal(H)

    def f(b, r, z, gp):
        x, _ = B.block_stream(b, r, None, z, "sigmoid", rs, bs, eps)
        return (dy * x * B._rms(x, eps) * gp).sum() + (up * x).sum()
    x, _ = B.block_stream(b, r, None, z, "sigmoid", rs, bs, eps)
    got = B.block_backward(dy, x, gp, b, None, z, "sigmoid", rs, bs, eps, up)
    assert got["grad_gamma_post"] is None
    args = [b, r, z, gp]
    for k, name in enumerate(("grad_block", "grad_residual", "grad_gate", "grad_gamma_pre")):
        step = rng.standard_normal(args[k].shape)
        lo, hi = list(args), list(args)
        lo[k], hi[k] = args[k] - 1e-6 * step, args[k] + 1e-6 * step
        num = (f(*hi) - f(*lo)) / 2e-6
        assert abs(num - (got[name] * step).sum()) <= 1e-6 * np.abs(got[name] * step).sum()

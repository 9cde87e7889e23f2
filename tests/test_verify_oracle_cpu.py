"""The fp64 definition of the draft verification where q is not a number in some places."""
import numpy as np

from oracle import block as B


def verify(p, q, tokens=(0,), noise=None):
    V = len(p)
    return B.draft_verify(np.log(np.stack([p, p])), list(tokens), [1e30], np.ones((1, V)) if noise is None else noise, [0, 1],
                          np.asarray(q)[None])


def test_a_token_without_a_q_is_not_drawn():
    p = np.array([0.5, 0.3, 0.15, 0.05])
    with np.errstate(invalid="ignore"):
        # of p - q only token 0 has a weight, and its q is no number: p itself, without that token
        acc, tok, lp, _ = verify(p, [np.nan, 0.0, 0.0, 0.0])
        assert acc[0] == 0 and tok[0] == 1 and abs(lp[0] - np.log(0.3)) < 1e-12
        # where p exceeds q elsewhere it is drawn there
        assert verify(p, [np.nan, 0.0, 0.0, -9.0])[1][0] == 3
        # nothing is left
        acc, tok, lp, _ = verify(p, [np.nan] * 4)
        assert acc[0] == 0 and tok.tolist() == [-1, -1] and np.isnan(lp[0]) and lp[1] == 0

"""Selected logprob and log_softmax on rows of logits that start off 16-byte boundaries, over several slices of a
row: every output bit against the C emulator's, from the same values.

fp32 rows are staged word by word; bf16 rows word by word where they start at a word and by halves of
two words where they do not (an odd V or an odd first column makes both kinds)."""
import numpy as np
import pytest
import torch

from invariant_selected_token_gb300 import workloads as WL
from oracle import emulator as E

pytestmark = pytest.mark.gpu


def same_bits(got, want, what):
    got, want = got.cpu().numpy().view(np.uint32).ravel(), np.ascontiguousarray(want, np.float32).view(np.uint32).ravel()
    wrong = np.flatnonzero(got != want)
    assert wrong.size == 0, "%s: %d differ, the first at %d" % (what, wrong.size, wrong[0])


# a slice of a row is 4096 columns
WIDTHS = [1, 2, 3, 127, 129, 131, 4095, 4097, 4098, 4099, 8193, 12289, 20481, 50257, 151937]


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (1, 2), (2, 1), (3, 8), (7, 4)])
def test_bits(rlk, cuda_device, V, dtype, shift, pad):
    """Rows V + pad apart, the first `shift` elements behind a 16-byte boundary, NaN in every place beside them."""
    rng = np.random.default_rng(V * 64 + shift * 8 + pad)
    T = 7 if V < 20000 else 4
    L = (3 * rng.standard_normal((T, V))).astype(np.float32)
    tg = rng.integers(0, V, T).astype(np.int32)
    tg[0], tg[1] = 0, V - 1
    act = (rng.random(T) > 0.2).astype(np.uint8)
    if dtype == "bf16":
        L = WL.bf16_bits_to_f32(WL.f32_to_bf16_bits(L))
    kind = torch.float32 if dtype == "fp32" else torch.bfloat16
    buf = torch.full((shift + T * (V + pad) + 16,), float("nan"), dtype=kind, device=cuda_device)
    rows = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    rows.copy_(torch.from_numpy(L))
    assert rows.data_ptr() == buf.data_ptr() + shift * buf.element_size()
    targets, active = torch.from_numpy(tg).to(cuda_device), torch.from_numpy(act).to(cuda_device)
    tiles = (V + 127) // 128
    for n in (1, 4):
        if n > tiles:
            continue
        want = E.linear_logprob(L, tg, act, n_shards=n)
        lp, lse = rlk.logits_logprob(rows, targets, active, n)
        same_bits(lp, want["logprob"], "logprob")
        same_bits(lse, want["lse"], "lse")
    out, lse = rlk.log_softmax(rows)
    want, want_lse = E.log_softmax(L)
    same_bits(out, want, "log_softmax")
    same_bits(lse, want_lse, "its lse")

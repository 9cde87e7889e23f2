"""Global gradient norm and clipping on the GPU against the fp64 definition.

Tolerances (u = 2^-24): squares and their sums are positive, so every rounding on the way of a
sum adds at most u of it.  A thread adds at most 64 squares to a sum before that is added to a
second one, itself the sum of a sixteenth as many pieces as the CTA has (one at these sizes), and
trees of 8 levels follow: 64 + 1 + 8 = 73 roundings, and the root halves the relative error: 37 u,
for the norm with its own roundings 40 u (the rest are pairs of floats).  The scale adds one
rounding, the product another, and the store half a step of the type (or of its smallest
subnormal)."""
import numpy as np
import pytest
import torch

from oracle import training as TR

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def tensors(sizes, dtypes, device, seed, std=1.0, odd=False):
    """Gradients cut out of one buffer per type, `odd`ly placed where asked."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    out = []
    for i, (n, dt) in enumerate(zip(sizes, dtypes)):
        lead = i % 8 if odd else 0
        flat = (torch.randn(n + lead, generator=g, device=device) * std).to(dt)
        out.append(flat[lead:])
    return out


def f64(t):
    return t.double().cpu().numpy()


SETS = [
    ([1], [torch.float32]),
    ([0, 5, 0], [torch.float32, torch.bfloat16, torch.float16]),
    ([7, 4095, 4096, 4097, 16383, 33001], [torch.float32] * 6),
    ([7, 8191, 8192, 8193, 100003], [torch.bfloat16] * 5),
    ([95 * 4096 - 4, 8192 - 8], [torch.float32, torch.bfloat16]),  # the last that one cluster takes
    ([95 * 4096 - 4, 8192 - 7], [torch.float32, torch.bfloat16]),
    ([64, 16391, 65, 40000], [torch.float16, torch.bfloat16, torch.float32, torch.float16]),
    ([3, 1000, 17, 257] * 400, [torch.bfloat16, torch.float32, torch.float16, torch.bfloat16] * 400),
    ([5000011, 12, 3000017], [torch.bfloat16, torch.float32, torch.float32]),
]


@pytest.mark.parametrize("sizes,dtypes", SETS)
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_parity(rlk, cuda_device, sizes, dtypes, odd, in_place):
    std = 7.0 / max(1, sum(sizes)) ** 0.5
    grads = tensors(sizes, dtypes, cuda_device, len(sizes), std, odd)
    want_norm, _ = TR.clip_scale([f64(g) for g in grads], 1.0)
    max_norm = want_norm / 3
    _, want_scale = TR.clip_scale([f64(g) for g in grads], max_norm)
    before = [f64(g) for g in grads]
    assert abs(float(rlk.grad_norm(grads)) - want_norm) <= 40 * U * want_norm
    out = None if in_place else [torch.empty_like(g) for g in grads]
    status = rlk.new_status(cuda_device)
    norm, scale = rlk.clip_grads(grads, max_norm, out=out, status=status)
    rlk.raise_on_device_status(status)
    assert abs(float(norm) - want_norm) <= 40 * U * want_norm
    assert abs(float(scale) - want_scale) <= 41 * U * want_scale
    for g, b, o in zip(grads, before, grads if in_place else out):
        want = b * want_scale
        tol = np.abs(want) * (42 * U + torch.finfo(g.dtype).eps / 2) + TINY[g.dtype] / 2
        assert np.all(np.abs(f64(o) - want) <= tol * (1 + 2.0 ** -8))
        if not in_place:
            assert np.array_equal(f64(g), b)


def test_below_the_limit_nothing_changes(rlk, cuda_device):
    grads = tensors([1000, 20001], [torch.float32, torch.bfloat16], cuda_device, 1, odd=True)
    before = [g.clone() for g in grads]
    out = [torch.empty_like(g) for g in grads]
    norm = rlk.grad_norm(grads)
    for limit in (float(norm), float(norm) * 2, float("inf")):
        _, scale = rlk.clip_grads(grads, limit, out=out)
        assert float(scale) == 1.0
        assert all(torch.equal(a, b) for a, b in zip(out, before))
        rlk.clip_grads(grads, limit)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    _, scale = rlk.clip_grads(grads, 0.0)
    assert float(scale) == 0.0 and not any(g.any() for g in grads)


@pytest.mark.parametrize("sizes", [[5], [300000, 300000]])  # one launch and two
def test_limits_next_to_the_norm(rlk, cuda_device, sizes):
    """The norm, an fp32 number, is compared with max_norm itself, not with its rounded value."""
    g = [torch.zeros(n, device=cuda_device) for n in sizes]
    g[0][:2] = torch.tensor([3.0, 4.0])  # norm 5 exactly
    for limit, shrinks in ((5.0, False), (5.0 - 1e-12, True), (5.0 + 1e-12, False), (1e300, False),
                           (float("inf"), False), (0.0, True), (1e-60, True)):
        out = [torch.empty_like(t) for t in g]
        norm, scale = rlk.clip_grads(g, limit, out=out)
        assert float(norm) == 5.0
        # a limit that rounds to the norm gives a scale of 1 either way
        assert float(scale) == (np.float32(limit) / np.float32(5.0) if shrinks else 1.0)
        assert torch.equal(out[0], g[0] * scale)
    big = [t * 1e25 for t in g]  # squares beyond fp32
    assert float(rlk.grad_norm(big)) == float("inf")


def test_zero_gradients(rlk, cuda_device):
    grads = [torch.zeros(100, device=cuda_device)]
    norm, scale = rlk.clip_grads(grads, 0.0)
    assert float(norm) == 0.0 and float(scale) == 1.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_a_norm_that_is_not_finite_leaves_the_gradients(rlk, cuda_device, bad, dtype):
    grads = tensors([100, 40000], [dtype, torch.float32], cuda_device, 2)
    grads[0][99] = bad
    before = [g.clone() for g in grads]
    status = rlk.new_status(cuda_device)
    norm, scale = rlk.clip_grads(grads, 1.0, status=status)
    with pytest.raises(rlk.RlkError) as e:
        rlk.raise_on_device_status(status)
    assert e.value.code == rlk.RLK_ERR_NONFINITE
    assert not np.isfinite(float(norm)) and float(scale) == 1.0
    assert all(torch.equal(a.nan_to_num(9.0, 8.0, 7.0), b.nan_to_num(9.0, 8.0, 7.0))
               for a, b in zip(grads, before))
    status.zero_()
    rlk.grad_norm(grads, status=status)
    with pytest.raises(rlk.RlkError):
        rlk.raise_on_device_status(status)


def test_repeats_and_other_addresses_give_the_same_bits(rlk, cuda_device):
    """The same places within 16 bytes: the same bits, wherever the buffers are, whatever the
    outputs' places, on any stream.  Other places: the same norm within its bound."""
    sizes, dtypes = [70001, 33, 16400], [torch.bfloat16, torch.float16, torch.float32]
    even = tensors(sizes, dtypes, cuda_device, 3)
    seen = {}
    for lead in range(18):
        moved = []
        for t in even:
            buf = torch.empty(t.numel() + 24, dtype=t.dtype, device=cuda_device)
            buf[lead:lead + t.numel()] = t
            moved.append(buf[lead:lead + t.numel()])
        out = [torch.empty_like(t) for t in even]  # aligned otherwise than its input
        norm, scale = rlk.clip_grads(moved, 3.0, out=out)
        got = [norm, scale] + out
        for x, t in zip(out, even):
            assert torch.equal(x, (t.float() * scale).to(t.dtype))
        ref = seen.setdefault(lead % 8, got)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert abs(float(norm) - float(seen[0][0])) <= 80 * U * float(norm)
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    norm, scale = rlk.clip_grads(even, 3.0, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([norm, scale] + even, seen[0]))


def test_neighbours_are_left_alone(rlk, cuda_device):
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for lead, n in ((1, 1), (3, 8192), (4, 8190), (5, 16390), (7, 50001)):
            buf = torch.full((n + 64,), 3.0, dtype=dtype, device=cuda_device)
            rlk.clip_grads([buf[lead:lead + n]], 1.0)
            assert torch.all(buf[:lead] == 3) and torch.all(buf[lead + n:] == 3)
            assert torch.all(buf[lead:lead + n] < 3)


def test_empty_list_and_checks(rlk, cuda_device):
    assert float(rlk.grad_norm([], device=cuda_device)) == 0.0
    norm, scale = rlk.clip_grads([], 1.0, device=cuda_device)
    assert float(norm) == 0.0 and float(scale) == 1.0
    x = torch.ones(64, device=cuda_device)
    with pytest.raises(ValueError):
        rlk.clip_grads([x.view(8, 8).t()], 1.0)
    with pytest.raises(ValueError):
        rlk.clip_grads([x], 1.0, out=[x.bfloat16()])
    with pytest.raises(ValueError):
        rlk.clip_grads([x], 1.0, out=[])
    for grads, out in (([x, x], None), ([x[:40], x[30:]], None), ([x[:32], x[32:]], [x[32:], x[:32]]),
                       ([x[:32]], [x[1:33]])):
        with pytest.raises(rlk.RlkError) as e:
            rlk.clip_grads(grads, 1.0, out=out)
        assert e.value.code == rlk.RLK_ERR_INVALID_ARG
    assert torch.all(x == 1)
    # the same tensor twice is counted twice where nothing is written over it
    assert float(rlk.grad_norm([x, x])) == pytest.approx(128 ** 0.5, rel=1e-6)


@pytest.mark.parametrize("sizes", [[100, 300], [300000, 17, 90001]])
def test_graph_replay(rlk, cuda_device, sizes):
    dtypes = [torch.float32, torch.bfloat16, torch.float32][:len(sizes)]
    sets = [tensors(sizes, dtypes, cuda_device, s) for s in (4, 5)]
    eager = []
    for grads in sets:
        out = [torch.empty_like(t) for t in grads]
        eager.append(list(rlk.clip_grads(grads, 1.0, out=out)) + out)
    held = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm, scale = rlk.clip_grads(held, 1.0)
    for grads, want in zip(sets, eager):
        for h, t in zip(held, grads):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([norm, scale] + held, want))


def test_more_than_2_31_bytes_in_one_tensor(rlk, cuda_device):
    """Offsets past 32 bits: 2^31 + 9 bf16 elements, all zero but a few at the far end."""
    n = 2 ** 31 + 9
    t = torch.zeros(n, dtype=torch.bfloat16, device=cuda_device)
    t[-3:] = 2.0
    t[2 ** 30] = 2.0
    norm, scale = rlk.clip_grads([t], 1.0)
    assert float(norm) == 4.0 and float(scale) == 0.25
    assert t[-4:].tolist() == [0.0, 0.5, 0.5, 0.5] and float(t[2 ** 30]) == 0.5

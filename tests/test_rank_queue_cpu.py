"""What a rank puts into a queue is there for its parent after the rank has gone: tensors travel by
value (tests/rank_queue.py), not as storage that the receiver has to fetch from the sender."""
import torch
import torch.multiprocessing as mp


def _leave_at_once(out_q):
    out_q.put((7, [torch.arange(6, dtype=torch.int32).view(2, 3), torch.ones(2, dtype=torch.bfloat16)]))


def test_tensors_outlive_the_rank_that_sent_them():
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    p = ctx.Process(target=_leave_at_once, args=(q,), daemon=True)
    p.start()
    p.join(timeout=120)
    assert p.exitcode == 0
    rank, (a, b) = q.get(timeout=60)
    assert rank == 7 and torch.equal(a, torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32))
    assert b.dtype == torch.bfloat16 and torch.equal(b.float(), torch.ones(2))

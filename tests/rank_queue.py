"""The queue by which the ranks of the multi-process CPU tests hand results to their parent.

torch.multiprocessing sends a tensor as a handle that the receiver redeems with the sending process, which
fails where that one has left by then.  Here an object is pickled by value before it goes into the queue."""
import pickle
from multiprocessing.context import BaseContext


class ValueQueue:
    def __init__(self, queue):
        self.queue = queue

    def put(self, obj, *args, **kwargs):
        self.queue.put(pickle.dumps(obj), *args, **kwargs)

    def get(self, *args, **kwargs):
        return pickle.loads(self.queue.get(*args, **kwargs))

    def __getattr__(self, name):
        if name == "queue":  # not there yet while an instance is unpickled
            raise AttributeError(name)
        return getattr(self.queue, name)


def new_queue(ctx, maxsize=0):
    return ValueQueue(BaseContext.Queue(ctx, maxsize))

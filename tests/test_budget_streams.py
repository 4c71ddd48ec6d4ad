"""Where the cache-budget operators take their memory from when they run on a stream of
their own (host logic, with stand-ins for the allocator and the streams)."""
import contextlib

import torch

from paged_latent_attention_gb300 import api


def _stand_ins(monkeypatch):
    current, made = ["caller"], []

    class Block:
        def __init__(self, stream):
            self.stream, self.recorded = stream, []

        def record_stream(self, stream):
            self.recorded.append(stream)

    @contextlib.contextmanager
    def stream(s):
        before = current[0]
        current[0] = before if s is None else s
        yield
        current[0] = before

    def empty(*args, **kw):
        made.append(Block(current[0]))
        return made[-1]

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch, "empty", empty)
    return made


def test_memory_comes_from_the_launch_stream(monkeypatch):
    """A block of the caller's stream can be free for that stream while work queued on it
    still uses it, so a call on another stream must not get it; and what is returned to
    the caller stays until the caller's stream has passed."""
    _stand_ins(monkeypatch)
    block = api._empty((3, 4), torch.float32, "cuda", "side")
    assert block.stream == "side" and block.recorded == ["caller"]
    block = api._empty((3, 4), torch.float32, "cuda", None)
    assert block.stream == "caller" and block.recorded == []

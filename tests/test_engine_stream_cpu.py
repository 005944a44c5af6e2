"""FocusEngine with a stream of its own, on the CPU: every call sits between what the current stream holds and what it
will do, and what a call allocates is allocated on the engine's stream.  Streams and the context are fakes that record."""
import contextlib

import pytest
import torch

from decodability_aware_token_b200 import StepParams
from decodability_aware_token_b200.scheduler import FocusEngine


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.device = name, log, torch.device("cpu")

    def wait_stream(self, other):
        self.log.append((self.name, "waits for", other.name))


class Context:
    def __init__(self, log, current, fail):
        self.log, self.current, self.fail = log, current, fail

    def _note(self, what, stream):
        self.log.append((what, self.current[-1].name, stream.name))
        if self.fail:
            raise RuntimeError("refused")

    def alloc_outputs(self, n, block, importance=True, hidden=True):
        from decodability_aware_token_b200 import StepOutputs
        self.log.append(("allocates on", self.current[-1].name))
        return StepOutputs.alloc(n, block, block, 4, "cpu", importance, hidden)

    def step(self, view, params, out=None, stream=None):
        self._note("step", stream)

    def commit_block(self, view, stream=None):
        self._note("commit", stream)

    def prefill(self, chunk, tokens, new_len, batch, pages, head, *, mask_block, stream=None, **kw):
        self._note("prefill", stream)


@pytest.mark.parametrize("fail", [False, True])
@pytest.mark.parametrize("same", [False, True])
def test_calls_are_ordered_with_the_current_stream(monkeypatch, fail, same):
    log = []
    here, own = Stream("here", log), Stream("own", log)
    current = [own if same else here]

    @contextlib.contextmanager
    def under(s):
        current.append(s)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", under)
    eng = FocusEngine(Context(log, current, fail), StepParams(), stream=own, chunk=object())
    i32 = dict(dtype=torch.int32)
    view = {"block_tokens": torch.zeros(2, 8, **i32), "prefix_len": torch.zeros(2, **i32)}
    for what, call in (("step", lambda: eng.step(view, True)), ("commit", lambda: eng.commit(view)),
                       ("prefill", lambda: eng.prefill(view, torch.zeros(2, 3, **i32), torch.ones(2, **i32), torch.zeros(1, **i32)))):
        del log[:]
        with pytest.raises(RuntimeError) if fail else contextlib.nullcontext():
            call()
        want = [(what, "own", "own")]
        if what == "step":
            want = [("allocates on", "own")] + want
        if not same:
            want = [("own", "waits for", "here")] + want + [("here", "waits for", "own")]
        assert log == want
        current[1:] = []

"""Refusals of the calls around the top-k that need no device."""
import pytest
import torch

from drafter_vocab_top_amd import topk_cols as T


@pytest.mark.parametrize("index", [False, True])
def test_adjust_refuses_a_mask_without_rows(index):
    """An empty tensor has no address: it must not turn into no mask at all."""
    with pytest.raises(ValueError, match="at least one row"):
        T.AdjustRules(100, 14, lanes=2, mask=torch.zeros((0, 4), dtype=torch.int32),
                      mask_index=torch.zeros(14, dtype=torch.int32) if index else None)


def test_outputs_are_allocated_on_the_stream_that_writes_them(monkeypatch):
    """Memory of the current stream may still be in use there, and goes back
    to it when the tensor is dropped."""
    import contextlib
    entered, made = [], []

    @contextlib.contextmanager
    def stream_context(stream):
        entered.append(stream)
        yield
        entered.pop()

    def recording(function):
        def call(*args, **kw):
            made.append(entered[-1] if entered else None)
            return function(*args, **kw)
        return call
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    x, values, ids, out = torch.zeros(14, 100, dtype=torch.bfloat16), torch.zeros(16, 8), i32(16, 8), i32(2)
    rules = T.AdjustRules(100, 14, lanes=2)
    calls = {
        1: lambda s: rules.apply(x, stream=s),
        2: lambda s: T.verify(values, ids, None, i32(14), None, lanes=2, max_tokens=8, stream=s),
        7: lambda s: T.plan(i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 8, stream=s),
    }
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(T, "_launch", lambda *a: None)
    monkeypatch.setattr(T, "_raw_stream", lambda *a: 0)
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, recording(getattr(torch, name)))
    for n, call in calls.items():
        for stream in ("side", None):
            made.clear()
            call(stream)
            assert made == [stream] * n
    # one output given: only the other is made
    made.clear()
    T.verify(values, ids, None, i32(14), None, lanes=2, max_tokens=8, out_count=out, stream="side")
    assert made == ["side"]

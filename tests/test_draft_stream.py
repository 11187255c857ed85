"""DraftTreeDecoder's own copies go to the stream that its calls are given (no GPU: the library's entry
points and torch's stream context are stand-ins that keep a record)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from serving_ls_beam_gb300 import draft  # noqa: E402


class Recorded(torch.Tensor):
    """A buffer whose copies are kept in the record."""
    record: list = []

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.Tensor.copy_:
            cls.record.append("copy")
        return super().__torch_function__(func, types, args, kwargs or {})


class Stream:
    cuda_stream = 77


@pytest.mark.parametrize("given", ["none", "object", "handle"])
def test_copies_follow_the_stream(monkeypatch, given):
    record = []
    monkeypatch.setattr(Recorded, "record", record)
    monkeypatch.setattr(draft, "ls_workspace_init", lambda *a: 0)
    monkeypatch.setattr(draft, "ls_tree_attention_workspace_size", lambda *a: 256)
    monkeypatch.setattr(draft, "ls_cross_attention_workspace_size", lambda *a: 256)
    monkeypatch.setattr(draft, "ls_sample_workspace_size", lambda *a: 256)
    monkeypatch.setattr(draft, "ls_tree_attention", lambda *a, stream=None: record.append(("attention", stream)) or 0)

    @contextlib.contextmanager
    def on(stream):
        record.append(("enter", stream.cuda_stream))
        yield
        record.append(("leave", stream.cuda_stream))

    class External:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    dec = draft.DraftTreeDecoder(1, 2, 3, 2, 1, 8, 5, 10, 2, device="cpu")
    dec.draft_key, dec.draft_value = dec.draft_key.as_subclass(Recorded), dec.draft_value.as_subclass(Recorded)
    q, kv = torch.zeros(2, 3, 2, 8).half(), torch.ones(2, 3, 1, 8).half()
    stream = {"none": None, "object": Stream(), "handle": 77}[given]
    dec.self_attention(0, q, kv, kv, torch.zeros(2, 3, dtype=torch.int32), stream=stream)
    assert (dec.draft_key == 1).all() and (dec.draft_value == 1).all()
    calls = [r for r in record if r == "copy" or r[0] in ("enter", "leave", "attention")]
    if given == "none":
        assert calls == ["copy", "copy", ("attention", None)]
    else:
        assert calls == [("enter", 77), "copy", "copy", ("leave", 77), ("attention", stream)]

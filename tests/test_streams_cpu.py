"""What a call on an explicit stream makes itself, outputs and their fills, is made on that
stream: a fill on another one could land behind the call's kernels.  Host side, with the stream
calls and the library replaced by recorders (no GPU)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import atomic_expert_routing_b200 as omni

BF, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
HERE, OTHER = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=22)


@pytest.fixture
def made(monkeypatch):
    """Records (maker, size, the stream it ran on) of every tensor that a call makes, and the
    streams that tensors are kept for."""
    log = SimpleNamespace(made=[], kept=[], at=HERE.cuda_stream)

    @contextlib.contextmanager
    def on(stream):
        before, log.at = log.at, stream.cuda_stream
        yield
        log.at = before

    def recorded(name):
        make = getattr(torch, name)

        def call(*a, **k):
            t = make(*a, **k)
            log.made.append((name, tuple(t.shape), log.at))
            return t
        return call

    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, recorded(name))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: HERE)
    monkeypatch.setattr(torch.cuda, "ExternalStream",
                        lambda ptr, device=None: SimpleNamespace(cuda_stream=ptr))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.kept.append((tuple(t.shape), s.cuda_stream)))
    monkeypatch.setattr(omni, "_index", lambda t: 0)
    monkeypatch.setattr(omni, "_addresses", lambda index, names, tensors: [None] * len(tensors))
    monkeypatch.setattr(omni, "_run", lambda *a: None)
    return log


def _z(*shape, dtype=BF):
    return torch.ones(shape, dtype=dtype)


def _linear_calls(stream):
    x, W, dy = _z(8, 64), _z(2, 16, 64), _z(8, 16)
    xq, Wq = _z(8, 64, dtype=I8), _z(2, 16, 64, dtype=I8)
    xs, Ws = _z(8, dtype=F32), _z(2, 16, dtype=F32)
    off, one = torch.tensor([0, 3, 8], dtype=I32), _z(1, dtype=I32)
    kw = {"stream": stream}
    return {
        "product": (lambda: omni.grouped_linear(x, W, off, **kw), ["empty"]),
        "gradients": (lambda: omni.grouped_linear_backward(x, W, dy, off, n_groups=one, **kw),
                      ["empty", "zeros"]),
        "every group": (lambda: omni.grouped_linear_backward(x, W, dy, off, **kw),
                        ["empty", "empty"]),
        "quantisation": (lambda: omni.quantize_rows(x, **kw), ["empty", "empty"]),
        "one row": (lambda: omni.quantize_rows(x[0], **kw), ["empty", "empty"]),
        "8 bits": (lambda: omni.quantized_linear(xq, xs, Wq, Ws, off, **kw), ["empty"]),
    }


@pytest.mark.parametrize("name", list(_linear_calls(None)))
def test_outputs_are_made_on_the_calls_stream(made, name):
    call, makers = _linear_calls(OTHER)[name]
    call()
    assert [m for m, *_ in made.made] == makers
    assert {at for *_, at in made.made} == {OTHER.cuda_stream}
    # and kept for the stream the caller is on
    assert made.kept == [(size, HERE.cuda_stream) for _, size, _ in made.made]


@pytest.mark.parametrize("stream", [None, HERE], ids=["default", "the current one"])
@pytest.mark.parametrize("name", list(_linear_calls(None)))
def test_on_the_current_stream_nothing_is_recorded(made, name, stream):
    call, makers = _linear_calls(stream)[name]
    call()
    assert [m for m, *_ in made.made] == makers and not made.kept
    assert {at for *_, at in made.made} == {HERE.cuda_stream}

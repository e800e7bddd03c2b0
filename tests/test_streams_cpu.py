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
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: HERE.cuda_stream,
                        raising=False)
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


def _layer_calls(stream):
    D = omni.LayerDims(L=6, d=64, Nr=4, Nc=4, k=2, K=2, B=2)
    x, R, W = _z(6, 64), _z(4, 64), _z(16, 64)
    W1, W2 = _z(32, 64), _z(64, 32)
    idx, gate = _z(6, 2, dtype=I32), _z(6, 2, dtype=F32)
    sched = {k: _z(12, dtype=F32 if k == "task_gate" else I32)
             for k in ("task_token", "task_expert", "task_gate", "uniq", "group_off", "counts")}
    kw = {"stream": stream}
    return {
        "route": lambda: omni.route(D, x, R, R, **kw),
        "router_logits": lambda: omni.router_logits(D, x, R, R, **kw),
        "route_select": lambda: omni.route_select(D, _z(6, 8, dtype=F32), **kw),
        "schedule": lambda: omni.schedule(D, idx, gate, **kw),
        "expert_forward": lambda: omni.expert_forward(D, x, W, W, sched, **kw),
        "moe_forward": lambda: omni.moe_forward(D, x, R, R, W, W, **kw),
        "moe_forward_shard": lambda: omni.moe_forward_shard(D, x, R, R, W, W, 0, 16, **kw),
        "moe_forward_shard_routed":
            lambda: omni.moe_forward_shard_routed(D, x, W, W, 0, 16, idx, gate, **kw),
        "cast_output": lambda: omni.cast_output(D, _z(6, 64, dtype=F32), **kw),
        "moe_backward": lambda: omni.moe_backward(D, x, R, R, W, W, idx, gate, x, **kw),
        "shared_mlp": lambda: omni.shared_mlp(D, x, W1, W2, **kw),
        "moe_mlp_forward": lambda: omni.moe_mlp_forward(D, x, R, R, W, W, W1, W2, **kw),
        "token_centric_forward": lambda: omni.token_centric_forward(D, x, W, W, idx, gate, **kw),
    }


@pytest.fixture
def no_library(monkeypatch):
    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(omni._lib, "load", lambda: Library())
    monkeypatch.setattr(omni, "_ptr", lambda t: None)
    monkeypatch.setattr(omni, "workspace_size", lambda D, which: 64)
    monkeypatch.setattr(omni, "mlp_workspace_size", lambda D, F, routed: 64)


@pytest.mark.parametrize("name", list(_layer_calls(None)))
def test_layer_calls_make_everything_on_their_stream(made, no_library, name):
    """Outputs, zeroed gradients and counters, and the workspace of a call that is given none."""
    _layer_calls(OTHER)[name]()
    assert made.made and {at for *_, at in made.made} == {OTHER.cuda_stream}
    for _, size, _ in made.made:
        assert (size, HERE.cuda_stream) in made.kept
    made.made.clear()
    _layer_calls(None)[name]()
    assert {at for *_, at in made.made} == {HERE.cuda_stream}


def test_a_workspace_is_kept_for_every_stream_that_uses_it(made):
    ws, third = omni.Workspace(), SimpleNamespace(cuda_stream=33)
    dev = torch.device("meta")
    a = ws.get(64, dev, OTHER)
    assert [at for *_, at in made.made] == [OTHER.cuda_stream]
    assert {s for _, s in made.kept} == {OTHER.cuda_stream, HERE.cuda_stream}
    made.kept.clear()
    assert ws.get(32, dev, OTHER) is a and not made.kept
    assert ws.get(32, dev, third) is a and made.kept == [((64,), 33)]
    assert ws.get(32, dev) is a and ws.get(32, dev) is a
    made.kept.clear()
    b = ws.get(128, dev)  # grown: another buffer, its own streams
    assert b is not a and made.made[-1][2] == HERE.cuda_stream
    ws.get(128, dev, third)
    assert ((128,), 33) in made.kept

"""Calls on an explicit stream while the current one is busy: what a call makes itself is neither
filled behind its kernels nor taken from memory that the current stream still uses.  Results are
compared bit for bit with the same call made alone."""
import pytest
import torch

import atomic_expert_routing_b200 as omni

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LONG = 400_000_000  # cycles the current stream is busy for: 0.2 s and more


def _case():
    g = torch.Generator(device="cuda")
    g.manual_seed(60)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF)

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    x, W, dy = normal(300, 256), normal(6, 136, 256), normal(300, 136)
    where = {"ids": i32(0, 2, 3, 5), "n_groups": i32(4)}
    off = i32(0, 40, 41, 200, 300)
    xq, xs = omni.quantize_rows(x)
    Wq, Ws = omni.quantize_rows(W)
    return {
        "product": lambda st: [omni.grouped_linear(x, W, off, stream=st, **where)],
        "gradients": lambda st: list(omni.grouped_linear_backward(
            x, W, dy, off, out_dtype=F32, stream=st, **where).values()),
        "quantisation": lambda st: list(omni.quantize_rows(W, stream=st)),
        "8 bits": lambda st: [omni.quantized_linear(xq, xs, Wq, Ws, off, out_dtype=F32,
                                                    stream=st, **where)],
    }


NAMES = ["product", "gradients", "quantisation", "8 bits"]


@pytest.mark.parametrize("name", NAMES)
def test_nothing_lands_behind_the_call(name):
    call = _case()[name]
    ref = call(None)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    got = call(other)
    other.synchronize()
    torch.cuda.synchronize()  # whatever the current stream had queued is done too
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("name", NAMES)
def test_memory_in_use_by_the_current_stream_is_left_alone(name):
    call = _case()[name]
    ref = call(None)
    other = torch.cuda.Stream()
    held = [torch.full_like(t, 3) for t in ref]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in held]
    del held  # free for this stream's next tensors, not for another stream's writes
    got = call(other)
    other.synchronize()
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_in_use_by_the_current_stream_are_kept(name):
    call = _case()[name]
    ref = call(None)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = call(other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(LONG)
    copies = [t.clone() for t in first]
    del first
    with torch.cuda.stream(other):
        later = [torch.zeros_like(t) for t in ref]  # the next tensors of that stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, ref))
    assert not any(bool(t.float().any()) for t in later)

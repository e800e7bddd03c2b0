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


def _layer():
    g = torch.Generator(device="cuda")
    g.manual_seed(61)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)

    D = omni.LayerDims(L=64, d=256, Nr=8, Nc=8, k=4, K=4, B=1)
    return D, dict(x=normal(64, 256), Wr=normal(8, 256, std=0.06), Wc=normal(8, 256, std=0.06),
                   W=normal(64, 256, std=0.06), V=normal(64, 256), dy=normal(64, 256))


def test_schedule_and_backward_behind_a_busy_stream():
    """The counters and the parameter gradients that a call zeroes itself.  The counts are exact;
    the gradients are compared with the same call on the current stream."""
    D, p = _layer()
    rt = (p["x"], p["Wr"], p["Wc"], p["W"], p["V"])
    idx, gate, _ = omni.route(D, *rt[:3])
    s0 = omni.schedule(D, idx, gate)
    g0 = omni.moe_backward(D, *rt, idx, gate, p["dy"])
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    s1 = omni.schedule(D, idx, gate, stream=other)
    g1 = omni.moe_backward(D, *rt, idx, gate, p["dy"], stream=other)
    other.synchronize()
    torch.cuda.synchronize()
    n, groups = (int(v) for v in s0["counts"][:2])
    assert torch.equal(s0["counts"], s1["counts"]) and n > 0
    for k, m in (("task_token", D.M), ("task_expert", D.M), ("uniq", n), ("group_off", groups + 1)):
        assert torch.equal(s0[k][:m], s1[k][:m])
    for k, a in g0.items():
        # atomics add in any order (2^-23 a term, 256 terms), and a term that is rounded to bf16
        # next may then fall on the other side of a border (two half steps, 2^-7 of it); a term
        # is taken as up to twice the largest result
        tol = 2 * (2.0 ** -7 + 256 * 2.0 ** -23) * float(a.abs().max())
        assert bool(a.any()) and float((a - g1[k]).abs().max()) <= tol


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_forked_inside_a_capture(name):
    """A call on a second stream of a capture: its outputs and fills are part of the graph, and
    replays give the same again."""
    call = _case()[name]
    ref = call(None)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(main):
        call(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        first = call(side)
        call(side)  # outputs that nobody keeps
        got = call(side)
        main.wait_stream(side)
    for _ in range(2):
        for t in got + first:
            t.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for out in (first, got):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    del graph

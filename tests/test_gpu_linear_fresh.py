"""Gradient calls one after another on arrays that are rewritten in between, with nothing waited
for on the host: dx and dW of a call run side by side, and both see what was written last."""
import numpy as np
import pytest
import torch

import atomic_expert_routing_b200 as omni

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _sets(g, E, M, T, n_in, n_out, count):
    """Batches of small integers (every sum is exact): x, dy, off, ids, n, rows and dW."""
    out = []
    for k in range(count):
        rng = np.random.default_rng(100 + k)
        n = int(rng.integers(1, E + 1))
        ids = np.sort(rng.choice(E, n, replace=False))
        ends = np.sort(rng.integers(0, M + 1, n - 1))
        off = np.concatenate(([0], ends, [M], np.full(E - n, M)))
        x = torch.randint(-2, 3, (T, n_in), generator=g, device="cuda").to(BF)
        dy = torch.randint(-2, 3, (M, n_out), generator=g, device="cuda").to(BF)
        rows = torch.randint(0, T, (M,), generator=g, device="cuda", dtype=I32)
        dW = torch.zeros((E, n_out, n_in), device="cuda")
        for q in range(n):
            a, b = int(off[q]), int(off[q + 1])
            dW[ids[q]] = (dy[a:b].double().T @ x[rows[a:b].long()].double()).float()
        arrays = [torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")
                  for v in (off, np.concatenate((ids, np.zeros(E - n))), [n])]
        out.append((x, dy, *arrays, rows, dW))
    return out


@pytest.mark.parametrize("E,M,T,n_in,n_out", [(4, 70, 40, 64, 72), (40, 500, 300, 264, 136),
                                              (16, 3000, 900, 256, 512)])
def test_rewritten_arrays(E, M, T, n_in, n_out):
    g = torch.Generator(device="cuda")
    g.manual_seed(70)
    sets = _sets(g, E, M, T, n_in, n_out, 5)
    live = [t.clone() for t in sets[0][:6]]
    W = torch.randint(-2, 3, (E, n_out, n_in), generator=g, device="cuda").to(BF)
    off_by = torch.zeros((), device="cuda")
    counts = omni.new_counts("cuda")
    for k in range(200):
        s = sets[k % len(sets)]
        for t, v in zip(live, s):
            t.copy_(v)
        x, dy, off, ids, n, rows = live
        r = omni.grouped_linear_backward(x, W, dy, off, ids=ids, n_groups=n, rows=rows,
                                         out_dtype=F32, counts=counts)
        off_by = torch.maximum(off_by, (r["dW"] - s[6]).abs().max())
    assert float(off_by) == 0.0 and counts.tolist() == [0, 0, 0, 0]

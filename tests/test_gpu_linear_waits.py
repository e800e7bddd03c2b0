"""dW where one CTA sums for longer than a wait's limit between two blocks with rows to zero."""
import pytest
import torch

import atomic_expert_routing_b200 as omni

pytestmark = pytest.mark.gpu


def test_a_tail_behind_a_sum_of_more_than_a_second():
    """A first group of 400 million rows, which ends with a whole block, and the group whose ten
    rows are the same CTA's next: 6.3 million blocks of 64 rows one after another, 1.5 s and more.
    x is zero but for a few rows, so every sum is a small integer and exact."""
    R, E, n = 400_000_000, 149, 8
    M = R + 147 * 16 + 10
    off = torch.cat([torch.tensor([0]), R + 16 * torch.arange(148), torch.tensor([M])])
    off = off.to(torch.int32).cuda()
    x = torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
    dy = torch.ones((M, n), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, R // 2, R - 1, R, R + 17, M - 10, M - 3, M - 1], device="cuda")
    x[at] = torch.arange(1, 10, device="cuda").to(torch.bfloat16)[:, None]
    W = torch.zeros((E, n, n), dtype=torch.bfloat16, device="cuda")
    counts = omni.new_counts("cuda")
    dW = omni.grouped_linear_backward(x, W, dy, off, need_dx=False, counts=counts)["dW"]
    group = torch.searchsorted(off[1:].contiguous(), at.int(), right=True)
    ref = torch.zeros(E, device="cuda").index_add_(0, group, torch.arange(1, 10, device="cuda").float())
    assert counts.tolist() == [0, 0, 0, 0]
    assert torch.equal(dW, ref[:, None, None].expand(E, n, n))

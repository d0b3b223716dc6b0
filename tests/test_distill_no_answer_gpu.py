"""Rows of the distillation loss that have no answer: not a number in the loss and in every column of the gradient, and in
no other row."""
import pytest
import torch

import zero_gradient_reduction_gb300 as zr
from test_distill_gpu import BF16, F16, F32, case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T,V,dtype", [(12, 7, F32), (12, 130, BF16), (12, 50_000, F32), (12, 50_001, F16), (400, 2000, BF16), (160, 58_001, BF16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_whole_rows(T, V, dtype, in_place):
    """By a block's row, a cluster's, one that shared memory holds a part of: logits that are not numbers, an id past the
    vocabulary, and a kept teacher's entry of NaN or +inf."""
    z, ids, teacher, weight = case(T, V, 5, dtype, seed=V)
    weight[:] = 1.0
    ids = ids.clamp(min=0)
    nan, inf = float("nan"), float("inf")
    z[0, V - 1], z[1, 3], z[2] = nan, inf, -inf
    ids[3, 2] = V
    teacher[4, 0], teacher[5, 4] = nan, inf
    teacher[6, 1], ids[6, 1] = nan, -1   # not kept: the row has an answer
    teacher[7, 2], weight[7] = nan, 0.0  # no weight: zeros
    teacher[8, 3] = -inf                 # not kept
    loss, grad = torch.empty(T, device="cuda"), z if in_place else torch.empty_like(z)
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight)
    want = (torch.arange(T) < 6).cuda()
    assert torch.equal(torch.isnan(loss), want)
    assert torch.equal(torch.isnan(grad).all(1), want)
    assert torch.equal(torch.isnan(grad).any(1), want)
    assert float(loss[7]) == 0 and bool((grad[7] == 0).all())
    alone = torch.empty(T, device="cuda")
    if not in_place:
        zr.distill_topk(z, ids, teacher, alone, weight=weight)
        assert torch.equal(torch.isnan(alone), want)


def test_an_id_past_the_vocabulary_counts_without_being_kept():
    """An entry of -inf is not kept, but its id has to be one; in a row with nothing kept no id is looked at."""
    z, ids, teacher, weight = case(4, 130, 5, F32, seed=3)
    weight[:] = 1.0
    ids = ids.clamp(min=0)
    ids[1, 2], teacher[1, 2] = 130, -float("inf")
    ids[2, 2], teacher[2] = 130, -float("inf")
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(z)
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight)
    assert torch.equal(torch.isnan(loss).cpu(), torch.arange(4) == 1)
    assert torch.equal(torch.isnan(grad).all(1).cpu(), torch.arange(4) == 1)
    assert float(loss[2]) == 0 and bool((grad[2] == 0).all())

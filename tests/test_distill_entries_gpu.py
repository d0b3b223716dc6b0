"""The teacher's entries at the end of their array: rows of odd and even lengths, in each type, with what is no number
behind the last one."""
import pytest
import torch

from test_distill_gpu import BF16, F16, F32, case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("T,K", [(1, 1), (1, 2), (1, 3), (2, 33), (3, 5), (5, 1023)])
@pytest.mark.parametrize("tdt", [F32, F16, BF16])
def test_last_entries(T, K, tdt):
    z, ids, teacher, weight = case(T, 1100, K, BF16, seed=T * K, ids_type=(torch.int32, torch.int64)[K % 2], tdt=tdt)
    ids, weight = ids.clamp(min=0), torch.ones_like(weight)
    room = torch.full((T * K + 9,), float("nan"), dtype=tdt, device="cuda")
    room[:T * K] = teacher.flatten()
    check(z, ids, room[:T * K].view(T, K), weight, tau=1.5)

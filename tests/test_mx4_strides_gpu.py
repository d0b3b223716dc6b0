"""Operands whose rows lie apart: random bytes, and a teacher's entries that are the first of longer rows."""
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr
from test_distill_gpu import case, check
from test_mx4_gpu import BF16, F16, F32, matrix, on_host, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("rows,cols", [(1, 40), (70, 1), (131, 301), (200, 256)])
@pytest.mark.parametrize("apart", [1, 3, 4, 8, 16])
def test_random_bytes_of_wider_rows(rows, cols, apart):
    ld = cols + apart
    x = matrix(rows, cols, BF16, seed=ld)
    rand = torch.randint(0, 256, (rows, ld), dtype=torch.uint8, generator=torch.Generator().manual_seed(ld)).cuda()[:, :cols]
    q, qt = zr.Mx4(rows, cols), zr.Mx4(cols, rows)
    zr.mx4_quantize(x, q, qt, rand=rand)
    h, r = on_host(x), rand.cpu().numpy()
    same(q, ref.quantise(h, r), cols)
    same(qt, ref.quantise(h.T, r.T), rows)


@pytest.mark.parametrize("T,K,ld", [(1, 5, 9), (7, 1, 4), (9, 16, 33), (40, 33, 64)])
@pytest.mark.parametrize("tdt,ids_type", [(F32, torch.int32), (F16, torch.int64), (BF16, torch.int32)])
def test_the_first_of_a_teachers_entries(T, K, ld, tdt, ids_type):
    z, ids, teacher, weight = case(T, 2000, ld, BF16, seed=ld, ids_type=ids_type, tdt=tdt)
    check(z, ids[:, :K], teacher[:, :K], weight)


def test_strides_that_the_library_cannot_take():
    x, q = torch.zeros(8, 64, device="cuda"), zr.Mx4(8, 64)
    bytes_ = torch.zeros(64, 8, dtype=torch.uint8, device="cuda")
    z, ids, teacher, weight = case(6, 50, 8, F32, seed=1)
    loss = torch.empty(6, device="cuda")
    for call in (lambda: zr.mx4_quantize(x, q, rand=bytes_.t()), lambda: zr.mx4_quantize(x, q, rand=bytes_.t().contiguous()[:1].expand(8, 64)),
                 lambda: zr.distill_topk(z, ids[:, :4], teacher[:, :4].contiguous(), loss),
                 lambda: zr.distill_topk(z, ids[:, :4].contiguous(), teacher[:, :4], loss),
                 lambda: zr.distill_topk(z, ids[:, ::2], teacher[:, :4], loss),
                 lambda: zr.distill_topk(z, ids[:1].expand(6, 8), teacher[:1].expand(6, 8), loss)):
        with pytest.raises(zr.ZrError) as e:
            call()
        assert e.value.status == 1

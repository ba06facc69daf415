"""The weight's gradient of one expert with more than 2^29 gathered rows: the
ids of its routes are 2 GB and more."""
import pytest
import torch

import mixture_experts_grouped_amd as M
from tests import harness as Hn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()
    yield
    torch.cuda.empty_cache()


def test_ids_past_a_descriptor():
    """Whole numbers, zero but for a few rows: the sums are exact.  (One workgroup walks 8.4 million stages, 10 to 20
    seconds.)"""
    rows, topk, W = 2 ** 29 + 200, 8, 8
    dev = dict(device="cuda")
    pool = {"counts": torch.tensor([rows], dtype=torch.int32, **dev), "offsets": torch.tensor([0, rows], dtype=torch.int32, **dev),
            "row_to_route": torch.arange(rows, dtype=torch.int32, **dev)}
    a = torch.arange(-(-rows // topk), dtype=torch.int32, **dev).remainder(251).to(torch.bfloat16)[:, None].repeat(1, W)
    a *= torch.tensor([1, -1, 1, -1, 1, -1, 1, -1], dtype=torch.bfloat16, **dev)
    grad = torch.zeros(rows, W, dtype=torch.bfloat16, **dev)
    at = torch.tensor([0, 1, 63, 64, 130, 2 ** 28, 2 ** 29 - 129, 2 ** 29 - 5, 2 ** 29, 2 ** 29 + 7, 2 ** 29 + 64, rows - 1], **dev)
    grad[at] = (1 + torch.arange(at.numel(), **dev)).to(torch.bfloat16)[:, None].expand(-1, W)
    got = M.expert_weight_grad(pool, grad, a, topk=topk, dtype=torch.float32)
    want = grad[at].double().t().cpu() @ a[at // topk].double().cpu()
    assert torch.equal(got[0].double().cpu(), want)

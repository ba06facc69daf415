"""The orthogonalising optimiser step on matrices of nearly 2^31 elements, the
most that are allowed: the workspace asked for, and a step of one row."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import muon as OMU
from tests import harness as Hn
from tests.test_gpu_muon import BF, HYPER

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()
    yield
    torch.cuda.empty_cache()


def workspace(*shapes):
    d = B.MoeMuonDesc(B.MOE_TYPE_BF16, B.MOE_TYPE_BF16, 1, 5, 0.02, 0.95, 0.01, 0.2, 1e-7, 1.0, *OMU.QUINTIC, None)
    ts = (B.MoeMuonTensor * len(shapes))(*[B.MoeMuonTensor(None, None, None, None, *s) for s in shapes])
    v = ctypes.c_size_t()
    assert B.library().moe_muon_workspace_size(ctypes.byref(d), ts, len(shapes), ctypes.byref(v)) == B.MOE_OK
    return v.value


@pytest.mark.parametrize("shape", [(1, MOST), (MOST, 1), (16, MOST // 16), (129, MOST // 129), (256, MOST // 256)])
def test_workspace(shape):
    """One part of the long side at least and about 1,024 at most; more matrices take more."""
    r = -(-min(shape) // 16)
    tile = r * (r + 1) // 2 * 256 * 8
    rest = (256 * r * r + 4) * 4 + (6 * 256 * r * r + 2) * 8  # Q, and the rounds' matrices of long short sides
    one, two = workspace((1, *shape)), workspace((2, *shape))
    assert tile <= one <= 1100 * tile + rest
    assert one < two <= 2 * one
    assert one < workspace((1, *shape), (3, 8, 100)) <= one + 64 * 2 ** 20


def test_step_of_the_longest_row():
    n = MOST - 2
    g = torch.Generator(device="cuda").manual_seed(41)
    p = torch.randn(1, n, generator=g, device="cuda", dtype=BF).mul_(0.05)
    d = torch.randn(1, n, generator=g, device="cuda", dtype=BF).mul_(0.01)
    before = p.clone()
    opt = M.MoeMuon([p], [d], **HYPER)
    opt.step()
    f = lambda v: float(np.float32(v))  # noqa: E731
    pieces = range(0, n, 1 << 27)
    at = [slice(i, min(i + (1 << 27), n)) for i in pieces]
    norm = np.sqrt(sum(float(d[0, s].double().mul_(1 + f(0.9)).square_().sum()) for s in at))
    a, b, c = OMU.QUINTIC
    x = norm / (norm + 1e-7)
    for _ in range(5):
        x = a * x + b * x ** 3 + c * x ** 5
    mom = opt.states["momentum"][0]
    for s in at:
        u = d[0, s].double().mul_(1 + f(0.9))
        p0 = before[0, s].double()
        change = f(0.05) * (f(0.2) * np.sqrt(n) * x / norm * u + f(0.1) * p0)
        want = p0 - change
        # a dozen fp32 roundings of the change and one of p, then p's to bf16
        tol = 12 * 2.0 ** -24 * (change.abs() + 0.005 * p0.abs()) + 2.0 ** -24 * want.abs()
        tol += 2.0 ** -8 * (want.abs() + tol)
        assert bool(((p[0, s].double() - want).abs() <= tol).all()), s
        assert torch.equal(mom[0, s], d[0, s].float()), s

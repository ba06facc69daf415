"""The orthogonalising optimiser step at the ends of what fp32 holds: matrices
of zeros and of the smallest values beside a small eps, and norms past fp32's
largest number, over short sides of each kernel of the rounds."""
import numpy as np
import pytest
import torch

from oracle import muon as OMU
from tests import harness as Hn
from tests.test_gpu_muon import BF, F32, HYPER, SLOPE, f64, make, optimiser, update_tolerance

pytestmark = pytest.mark.gpu
SMALLEST = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def decayed(p0):
    """What the decay alone makes of fp32 values."""
    return p0 * (1 - float(np.float32(np.float32(HYPER["lr"]) * np.float32(HYPER["weight_decay"]))))


@pytest.mark.parametrize("rounds,abc", [(5, OMU.QUINTIC), (16, OMU.QUINTIC), (3, (1e30, -1.0, 1.0))])
@pytest.mark.parametrize("eps", [1e-7, 1e-38, SMALLEST])
@pytest.mark.parametrize("shape", [(3, 8, 90), (3, 64, 40), (3, 30, 100), (2, 200, 210)])
def test_zeros_move_by_their_decay_alone(shape, eps, rounds, abc):
    """A factor of an expert that has seen no token yet."""
    for ptype, masters in ((F32, False), (BF, True)):
        t = make(torch.Generator().manual_seed(31), shape, ptype, F32, masters)
        for n in ("grad", "momentum"):
            t[n][0] = 0
        x = t["master"] if masters else t["param"]
        p0 = f64(x)
        optimiser([t], eps=eps, rounds=rounds, coefficients=abc).step()
        got = f64(x)
        assert np.all(np.abs(got[0] - decayed(p0[0])) <= 2.0 ** -23 * np.abs(p0[0]))
        assert not t["momentum"][0].any()
        if abc is OMU.QUINTIC:
            assert np.isfinite(got).all()


def check_scaled(shape, scale, eps, seed=32):
    t = make(torch.Generator().manual_seed(seed), shape, F32, F32, False, momentum=0.0)
    t["param"].zero_()
    t["grad"] *= 100
    t["grad"] *= scale
    g = f64(t["grad"])
    opt = optimiser([t], eps=eps, weight_decay=0.0)
    opt.step()
    f = lambda v: float(np.float32(v))  # noqa: E731
    got, m = f64(t["param"]), f64(t["momentum"])
    assert np.array_equal(m, g)  # from zeros: nothing is rounded
    for i in range(shape[0]):
        q, mm, x = OMU.step(0 * g[i], g[i], 0 * g[i], lr=f(HYPER["lr"]), mu=f(HYPER["momentum"]), nesterov=True,
                            weight_decay=0.0, rms=f(HYPER["rms"]), eps=eps, grad_scale=1.0)
        u = g[i] + f(HYPER["momentum"]) * mm
        n = np.sqrt((u * u).sum()) + eps
        # U's rounding is at least half of fp32's smallest step, whatever its value
        tol = update_tolerance(u, x, eps) + SLOPE * np.sqrt(u.size) * 0.5 * SMALLEST / n
        tol *= HYPER["lr"] * HYPER["rms"] * np.sqrt(max(shape[1:]))
        assert np.isfinite(got[i]).all()
        assert np.linalg.norm(got[i] - q) <= tol + 4 * 2.0 ** -24 * np.linalg.norm(q), (i, np.linalg.norm(got[i] - q), tol)


@pytest.mark.parametrize("scale,eps", [(1e-36, 1e-38), (1e-39, 1e-38), (1e-38, SMALLEST), (1e-42, 1e-30), (1e-40, 1e-44),
                                       (1e-42, SMALLEST)])
@pytest.mark.parametrize("shape", [(2, 8, 90), (2, 64, 40), (2, 300, 30), (1, 200, 210)])
def test_smallest_values(shape, scale, eps):
    check_scaled(shape, scale, eps)


@pytest.mark.parametrize("shape", [(2, 8, 400000), (1, 100000, 16), (1, 100, 20000), (1, 200, 4000), (1, 4001, 250)])
def test_norms_past_the_largest_number(shape):
    check_scaled(shape, 2e37, 1e-7)

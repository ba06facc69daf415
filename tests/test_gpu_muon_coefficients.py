"""The orthogonalising optimiser step with other polynomials than the usual
quintic, a term of it left out among them, over short sides of each kernel of
the rounds, against float64."""
import numpy as np
import pytest
import torch

from oracle import muon as OMU
from tests import harness as Hn
from tests.test_gpu_muon import F32, HYPER, SLOPE, f64, make, optimiser, update_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def check_rounds(shape, abc, rounds, seed):
    """p after a step from p = 0, without decay: the update alone."""
    t = make(torch.Generator().manual_seed(seed), shape, F32, F32, False)
    t["param"].zero_()
    f = lambda v: float(np.float32(v))  # noqa: E731
    g, m = f64(t["grad"]), f64(t["momentum"])
    opt = optimiser([t], weight_decay=0.0, coefficients=abc, rounds=rounds)
    opt.step()
    got = f64(t["param"])
    # what the rounds make of U's roundings: their own slope in place of the usual quintic's
    slope = OMU.slope(rounds, abc)
    for i in range(shape[0]):
        q, mm, x = OMU.step(0 * g[i], g[i], m[i], lr=f(HYPER["lr"]), mu=f(HYPER["momentum"]), nesterov=True, weight_decay=0.0,
                            rms=f(HYPER["rms"]), eps=HYPER["eps"], grad_scale=1.0, rounds=rounds, abc=abc)
        u = g[i] + f(HYPER["momentum"]) * mm
        tol = update_tolerance(u, x, HYPER["eps"]) + 2.0 ** -23 * (slope - SLOPE)
        tol *= HYPER["lr"] * HYPER["rms"] * np.sqrt(max(shape[1:]))
        assert np.linalg.norm(got[i] - q) <= tol + 4 * 2.0 ** -24 * np.linalg.norm(q), (i, np.linalg.norm(got[i] - q), tol)


SHORT = [(2, 8, 300), (2, 300, 20), (2, 100, 300), (1, 200, 310), (1, 300, 250)]


@pytest.mark.parametrize("abc", [(1.0, 0.0, 0.0), (1.25, 0.0, -0.25), (1.5, -0.5, 0.0), (0.0, 0.0, 1.0), (0.0, 1.0, 0.0)])
@pytest.mark.parametrize("shape", SHORT)
def test_coefficients(shape, abc):
    """The update itself, Newton's iteration, and each term alone."""
    check_rounds(shape, abc, 2, 21)


@pytest.mark.parametrize("rounds", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("shape", SHORT)
def test_numbers_of_rounds(shape, rounds):
    """First, last, even and odd rounds of each kernel."""
    check_rounds(shape, OMU.QUINTIC, rounds, 22)

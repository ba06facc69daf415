"""Pins of the oracles of the expert products, the 4-bit quantiser and the
orthogonalising optimiser step: closed forms, autograd, differences, and each
rule turned the wrong way."""
import numpy as np
import pytest
import torch

from mixture_experts_grouped_amd import inputs as I
from oracle import mxfp4 as OMX
from oracle import muon as OMU
from oracle import products as OP


def test_product_and_its_gradients_against_autograd_and_differences():
    r = np.random.default_rng(0)
    a, w, g = r.standard_normal((5, 7)), r.standard_normal((4, 7)), r.standard_normal((5, 4))
    ta, tw = torch.tensor(a, requires_grad=True), torch.tensor(w, requires_grad=True)
    (ta @ tw.T * torch.tensor(g)).sum().backward()
    assert np.allclose(OP.product(g, w.T)[0], ta.grad.numpy(), rtol=1e-14)  # the data gradient: the transposed weight
    dw = OP.weight_grad(g, a)[0]
    assert np.allclose(dw, tw.grad.numpy(), rtol=1e-14)
    h = 1e-4
    for n, k in ((0, 0), (3, 6), (2, 4)):
        d = np.zeros_like(w)
        d[n, k] = h
        diff = ((OP.product(a, w + d)[0] - OP.product(a, w - d)[0]) * g).sum() / (2 * h)
        assert abs(diff - dw[n, k]) < 1e-9
    assert not OP.weight_grad(g[:0], a[:0])[0].any()


def test_bound_of_fp32_sums_holds_for_sums_in_fp32():
    r = np.random.default_rng(1)
    a, w = r.standard_normal((3, 500)).astype(np.float32), r.standard_normal((2, 500)).astype(np.float32)
    ref, tol = OP.product(a.astype(np.float64), w.astype(np.float64))
    s = np.zeros((3, 2), np.float32)
    for k in range(500):
        s = s + a[:, k:k + 1] * w[None, :, k]
    assert np.all(np.abs(s - ref) <= tol)


def test_mxfp4_quantiser_against_the_packing_of_the_base():
    r = np.random.default_rng(2)
    x = r.standard_normal((6, 128)) * np.exp(3 * r.standard_normal((6, 128)))
    x[0, :32] = 0
    x[1, 40] = -0.0
    x = x.astype(np.float32).astype(np.float64)
    codes, exps = OMX.quantize(x)
    c, e = I.mxfp4_quantize(x)
    assert np.array_equal(codes, c) and np.array_equal(exps, e)
    v = OMX.dequantize(codes, exps)
    scale = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 32, -1)
    # nearest: half a step of the binade, or what the largest code cuts off (below 8)
    m = np.abs(x) / scale
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    assert np.all(np.abs(np.abs(v) / scale - np.minimum(m, 6)) <= step / 2) and np.all(m < 8)


def test_mxfp4_ties_and_edges():
    x = np.zeros((1, 32))
    x[0, :9] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5, -0.25]  # exponent 0: the middles of all neighbours
    codes, exps = OMX.quantize(x)
    assert exps[0, 0] == 127
    assert OMX.dequantize(codes, exps)[0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, -4, 0]
    assert codes[0, 4] == 0  # -0.25 becomes +0
    for bad in (np.nan, np.inf):
        x[0, 3] = bad
        assert OMX.quantize(x)[1][0, 0] == 255
    x[:] = 2.0 ** -126
    assert OMX.quantize(x)[1][0, 0] == 0 and OMX.quantize(x * 4)[1][0, 0] == 1


@pytest.mark.parametrize("m,n", [(4, 9), (9, 4), (5, 5), (1, 6), (6, 1)])
def test_rounds_against_singular_values(m, n):
    U = np.random.default_rng(m * n).standard_normal((m, n))
    for rounds in (1, 3, 5):
        x = OMU.orthogonalise(U, 1e-7, rounds)
        assert np.allclose(x, OMU.by_singular_values(U, 1e-7, rounds), atol=1e-12)
    s = np.linalg.svd(x, compute_uv=False)
    assert m == n or np.all((s > 0.6) & (s < 1.3))
    # the update's direction: positive along U's own singular directions
    u, _, v = np.linalg.svd(U, full_matrices=False)
    assert np.all(np.diag(u.T @ x @ v.T) > 0)


def test_slope_against_differences():
    d = OMU.slope(5)
    a, b, c = OMU.QUINTIC

    def f(s):
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        return s
    s = np.linspace(0, 1, 5001)
    assert abs(np.abs(np.diff(f(s)) / np.diff(s)).max() / d - 1) < 0.05
    assert d >= a ** 5 * (1 - 1e-12)


def test_step_closed_forms():
    kw = dict(lr=0.1, mu=0.9, weight_decay=0.5, rms=0.2, eps=1e-7, grad_scale=2.0)
    p, g = np.full((1, 4), 3.0), np.array([[1.0, 2.0, 2.0, 4.0]])
    # one row: X is the unit row times the quintic's value through the rounds
    q, M, X = OMU.step(p, g, np.ones((1, 4)), nesterov=False, **kw)
    assert np.allclose(M, 0.9 + 2 * g)
    unit = M / np.sqrt((M * M).sum())
    s = 1.0
    a, b, c = OMU.QUINTIC
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(X, s * unit, rtol=1e-6)
    assert np.allclose(q, p - 0.1 * (0.2 * 2.0 * X + 0.5 * p))
    assert not np.allclose(OMU.step(p, g, np.ones((1, 4)), nesterov=True, **kw)[0], q)
    z = OMU.step(p, 0 * g, 0 * g, nesterov=True, **kw)
    assert np.allclose(z[0], 0.95 * p) and not z[2].any()

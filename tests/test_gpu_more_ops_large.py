"""Expert products, their gradients, 4-bit rows and the orthogonalising
optimiser past 2^31 elements: of activations, weights, results, codes and
parameters, at the places where 32-bit offsets would wrap, against float64."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import muon as OMU
from oracle import mxfp4 as OMX
from oracle import products as OP
from tests import harness as Hn
from tests.test_gpu_muon import HYPER, update_tolerance
from tests.test_gpu_product import build, extents, f64, half_step, routing

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()
    yield
    torch.cuda.empty_cache()


def noise(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=BF).mul_(std)


def some(pool, n=3):
    """A few rows of each expert's ends: (expert, rows, routes)."""
    return [(e, r[np.r_[:n, -n:0]], t[np.r_[:n, -n:0]]) for e, r, t in extents(pool) if len(r) >= 2 * n]


@pytest.mark.parametrize("K,N", [(64, 4104), (4104, 64)])
def test_rows_past_32_bits(K, N):
    """Pool rows in and out: capacity times the wider side over 2^31."""
    idx = torch.arange(530000, dtype=torch.int32).remainder(3)[:, None].contiguous()
    pool = build(idx, 3)
    cap = pool["row_to_route"].numel()
    assert cap * max(N, K) > 2 ** 31
    a, w = noise(1, cap, K), noise(2, 3, N, K, std=K ** -0.5)
    out = M.expert_product(pool, a, w)
    for e, rows, _ in some(pool):
        ref, tol = OP.product(f64(a[rows]), f64(w[e]))
        assert np.all(np.abs(f64(out[rows]) - ref) <= half_step(ref, tol)), e
    back = M.expert_product(pool, out, w, transposed=True)
    for e, rows, _ in some(pool):
        ref, tol = OP.product(f64(out[rows]), f64(w[e]).T)
        assert np.all(np.abs(f64(back[rows]) - ref) <= half_step(ref, tol)), e
    dw = M.expert_weight_grad(pool, out[:, :8].contiguous(), a, dtype=F32)
    for e, rows, _ in extents(pool):
        ref, tol = OP.weight_grad(f64(out[rows][:, :8]), f64(a[rows][:, :64]))
        assert np.all(np.abs(f64(dw[e][:, :64]) - ref) <= tol), e


@pytest.mark.parametrize("transposed", [False, True])
def test_weights_past_32_bits(transposed):
    E, N, K = 136, 4096, 4104
    assert E * N * K > 2 ** 31
    idx = routing(60, E, 4, 1)
    idx[:4, 0] = torch.tensor([0, E - 1, E - 2, E // 2], dtype=torch.int32)
    idx[:4, 1:] = -1
    pool = build(idx, E)
    w, a = noise(3, E, N, K, std=K ** -0.5), noise(4, 60, N if transposed else K)
    out = M.expert_product(pool, a, w, topk=4, transposed=transposed)
    for e, rows, routes in extents(pool):
        if len(rows) and (e < 2 or e > E - 12):
            m = f64(w[e])
            ref, tol = OP.product(f64(a)[routes // 4], m.T if transposed else m)
            assert np.all(np.abs(f64(out[rows]) - ref) <= half_step(ref, tol)), e


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradient_past_32_bits(dtype):
    E, N, K = 136, 4096, 4104
    idx = routing(60, E, 4, 2)
    pool = build(idx, E)
    a, d = noise(5, 60, K), noise(6, pool["row_to_route"].numel(), N)
    out = torch.ones(E, N, K, dtype=dtype, device="cuda")
    M.expert_weight_grad(pool, d, a, topk=4, out=out, accumulate=True)
    for e, rows, routes in extents(pool):
        if e < 2 or e > E - 4:
            ref, tol = OP.weight_grad(f64(d[rows]), f64(a)[routes // 4])
            ref, tol = ref + 1, tol + 2.0 ** -24 * (np.abs(ref + 1) + tol)
            assert np.all(np.abs(f64(out[e]) - ref) <= (half_step(ref, tol) if dtype == BF else tol)), e


def test_rows_and_weights_in_4_bits_past_32_bits():
    """4-bit rows of more than 2^32 elements in and out, the product of pool rows over 2^31 codes."""
    R, K = 1060000, 4096
    x = noise(7, R, K)
    assert x.numel() > 2 ** 32
    c, e = M.mxfp4_quantize_rows(x)
    v = M.mxfp4_dequantize(c, e)
    at = [0, 1, 2 ** 31 // K - 1, 2 ** 31 // K, 2 ** 32 // K - 1, 2 ** 32 // K, R - 1]
    want_c, want_e = OMX.quantize(f64(x[at]))
    assert np.array_equal(c[at].cpu().numpy(), want_c) and np.array_equal(e[at].cpu().numpy(), want_e)
    assert np.array_equal(f64(v[at]), OMX.dequantize(want_c, want_e))
    del x, v
    E = 5
    idx = torch.arange(R - E * 16, dtype=torch.int32).remainder(E)[:, None].contiguous()
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    assert cap <= R and cap * K > 2 ** 32
    w, ew = M.mxfp4_quantize_weight(noise(8, E, 128, K, std=K ** -0.5))
    out = M.mxfp4_product(pool, c[:cap], e[:cap], w, ew)
    for ex, rows, _ in some(pool):
        a = OMX.dequantize(c[rows].cpu().numpy(), e[rows].cpu().numpy())
        ref, tol = OP.product(a, OMX.dequantize(w[ex].cpu().numpy(), ew[ex].cpu().numpy()))
        assert np.all(np.abs(f64(out[rows]) - ref) <= half_step(ref, tol)), ex


def test_weights_in_4_bits_past_32_bits():
    E, N, K = 264, 4096, 4096
    assert E * N * K > 2 ** 32
    W = noise(9, E, N, K, std=K ** -0.5)
    w, ew, wt, ewt = M.mxfp4_quantize_weight(W, transposed=True)
    ends = (0, 127, 128, E - 1)
    for e in ends:
        for got, gote, m in ((w, ew, W[e]), (wt, ewt, W[e].t())):
            c, x = OMX.quantize(f64(m[-64:]))
            assert np.array_equal(got[e, -64:].cpu().numpy(), c) and np.array_equal(gote[e, -64:].cpu().numpy(), x), e
    del W
    idx = torch.tensor(ends, dtype=torch.int32)[:, None].contiguous()
    pool = build(idx, E)
    a, ea = M.mxfp4_quantize_rows(noise(10, 4, K))
    out = M.mxfp4_product(pool, a, ea, w, ew, topk=1)
    back = M.mxfp4_product(pool, a, ea, wt, ewt, topk=1)
    for e, rows, routes in extents(pool):
        if len(rows):
            av = OMX.dequantize(a.cpu().numpy(), ea.cpu().numpy())[routes]
            for got, q, s in ((out, w, ew), (back, wt, ewt)):
                ref, tol = OP.product(av, OMX.dequantize(q[e].cpu().numpy(), s[e].cpu().numpy()))
                assert np.all(np.abs(f64(got[rows]) - ref) <= half_step(ref, tol)), e


@pytest.mark.parametrize("shape", [(17000, 32, 4096), (20, 110000000, 1)])
def test_parameters_past_32_bits(shape):
    """Stacks past 2^31 elements: of many matrices, and of a few with one very long side."""
    batch, m, n = shape
    assert batch * m * n > 2 ** 31
    p, g = noise(11, *shape), noise(12, *shape, std=0.01)
    first = {b: (f64(p[b]), f64(g[b])) for b in (0, 2 ** 31 // (m * n), batch - 1)}
    opt = M.MoeMuon([p], [g], **HYPER)
    opt.step()
    f = lambda v: float(np.float32(v))  # noqa: E731
    for b, (p0, g0) in first.items():
        q, mm, x = OMU.step(p0, g0, 0 * g0, lr=f(0.05), mu=f(0.9), nesterov=True, weight_decay=f(0.1), rms=f(0.2), eps=1e-7,
                            grad_scale=1.0)
        assert np.all(np.abs(f64(opt.states["momentum"][0][b]) - mm) <= 2.0 ** -23 * np.abs(mm))
        # one column: Q is a number, and |Q| |U| the norm of x
        tol = update_tolerance(g0 * (1 + f(0.9)), x, 1e-7) if n > 1 else 2.0 ** -23 * (OMU.slope(5) + 2 * np.linalg.norm(x))
        tol *= 0.05 * 0.2 * np.sqrt(max(m, n))
        each = 4 * 2.0 ** -24 * (np.abs(q - p0) + 0.005 * np.abs(p0)) + 2.0 ** -24 * np.abs(q) + 2.0 ** -8 * (np.abs(q) + tol)
        assert np.linalg.norm(np.maximum(np.abs(f64(p[b]) - q) - each, 0)) <= tol, b

"""4-bit rows, weights and expert products against float64, the layer's own
4-bit base, non-finite blocks, other streams and replayed graphs."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import mxfp4 as OMX
from oracle import products as OP
from tests import harness as Hn
from tests.test_gpu_product import Kernels, build, extents, f64, half_step, routing

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def values(codes, exps):
    return OMX.dequantize(codes.cpu().numpy(), exps.cpu().numpy())


def spread(g, *shape):
    return (torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(1, shape[-1], generator=g))).to(BF)


@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (17, 640), (130, 2048)])
def test_rows(rows, K):
    """Every code and exponent: scaling by powers of two rounds nothing."""
    x = spread(torch.Generator().manual_seed(rows), rows, K)
    x[0, :32] = torch.tensor([4, .25, .75, 1.25, 1.75, 2.5, 3.5, -5, -.25, 5] + [0] * 22).to(BF)  # ties
    c, e = M.mxfp4_quantize_rows(x.cuda())
    wc, we = OMX.quantize(f64(x))
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(e.cpu().numpy(), we)
    v = M.mxfp4_dequantize(c, e)
    assert v.dtype == BF and np.array_equal(f64(v), OMX.dequantize(wc, we))


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("rows,K", [(1, 128), (33, 768)])
def test_gated_rows(rows, K, act):
    x = (torch.randn(rows, 2 * K, generator=torch.Generator().manual_seed(K)) * 2).to(BF)
    c, e = M.mxfp4_quantize_rows(x.cuda(), act=act)
    gate, up = x[:, :K].double(), x[:, K:].double()
    f = torch.nn.functional.silu if act == "swiglu" else torch.nn.functional.gelu
    h = (f(gate) * up).numpy()
    amax = np.abs(h).reshape(rows, -1, 32).max(2)
    # the exponent, but where the largest is at a power of two to within the activation's error
    lo, hi = (np.floor(np.log2(amax * s)) + 125 for s in (1 - 1e-5, 1 + 1e-5))
    e = e.cpu().numpy()
    assert np.all((e >= lo) & (e <= hi))
    scale = np.repeat(np.ldexp(1.0, e.astype(int) - 127), 32, 1)
    m = np.abs(h) / scale
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    # half a step, what lies between 6 and 8, and the activation's own error (sigmoid 2^-20 relative, the normal
    # distribution function 1e-6 of the gate)
    tol = (step / 2 + np.maximum(m - 6, 0)) * scale * (1 + 1e-5) + 1e-6 * (x[:, :K].double() * up).abs().numpy()
    got = values(c, torch.from_numpy(e))
    assert np.all(np.abs(got - h) <= tol)


def test_zero_tiny_huge_and_nonfinite_blocks():
    x = torch.randn(6, 256).to(BF)
    x[0, :32] = 0
    x[1, 32:64] = 1e-39  # subnormal in bf16
    x[2, 70] = float("nan")
    x[3, 100] = -float("inf")
    x[4, 128:160] = 3e38
    x[5, 0:32] = 2.0 ** -126
    c, e = M.mxfp4_quantize_rows(x.cuda())
    wc, we = OMX.quantize(f64(x))
    assert np.array_equal(e.cpu().numpy(), we) and we[2, 2] == 255 and we[3, 3] == 255
    keep = np.repeat(we != 255, 16, 1)
    assert np.array_equal(c.cpu().numpy()[keep], wc[keep])
    v = f64(M.mxfp4_dequantize(c, e))
    bad = np.repeat(we == 255, 32, 1)
    assert np.isnan(v[bad]).all() and np.array_equal(v[~bad], OMX.dequantize(wc, we)[~bad])


def test_every_code_and_exponent_back():
    """All 16 codes under all 255 exponents: exact in bf16, subnormal values too; beyond bf16's range infinite."""
    codes = torch.arange(256 * 64, dtype=torch.int32).to(torch.uint8).reshape(256, 64)
    codes = (codes * 37 + torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None])
    exps = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].expand(256, 4).contiguous()
    got = f64(M.mxfp4_dequantize(codes.cuda(), exps.cuda()))
    with np.errstate(over="ignore"):
        want = OMX.dequantize(codes.numpy(), exps.numpy())
    assert np.isnan(got[255]).all()
    fine = np.abs(want) < 2.0 ** 128
    fine[255] = False
    assert np.array_equal(got[fine], want[fine])
    assert np.all(np.isinf(got[~fine & (np.arange(256) < 255)[:, None]]))


def test_no_rows():
    c, e = M.mxfp4_quantize_rows(torch.zeros(0, 256, dtype=BF, device="cuda"))
    assert c.shape == (0, 128) and e.shape == (0, 8) and M.mxfp4_dequantize(c, e).shape == (0, 256)


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 256, 384)])
def test_weights_and_their_transpose(E, N, K):
    w = (torch.randn(E, N, K, generator=torch.Generator().manual_seed(N)) * 0.02).to(BF)
    c, e, ct, et = M.mxfp4_quantize_weight(w.cuda(), transposed=True)
    for got, want in ((c, OMX.quantize(f64(w))[0]), (e, OMX.quantize(f64(w))[1]),
                      (ct, OMX.quantize(f64(w.transpose(1, 2)))[0]), (et, OMX.quantize(f64(w.transpose(1, 2)))[1])):
        assert np.array_equal(got.cpu().numpy(), want)
    c2, e2 = M.mxfp4_quantize_weight(w.cuda())
    assert torch.equal(c2, c) and torch.equal(e2, e)


def operands(rows, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a = M.mxfp4_quantize_rows(spread(g, rows, K).cuda())
    w = M.mxfp4_quantize_rows((torch.randn(E * N, K, generator=g) * K ** -0.5 * torch.exp(torch.randn(E * N, 1, generator=g))).to(BF).cuda())
    return *a, w[0].view(E, N, K // 2), w[1].view(E, N, K // 32)


def check(idx, E, N, K, gather, seed=0):
    T, k = idx.shape
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    a, ea, w, ew = operands(T if gather else cap, E, N, K, seed)
    out = torch.full((cap, N), -77.0, dtype=BF, device="cuda")
    got = M.mxfp4_product(pool, a, ea, w, ew, topk=k if gather else 0, out=out)
    assert got.data_ptr() == out.data_ptr()
    got, av, wv = f64(got), values(a, ea), values(w, ew)
    assert (got[pool["row_to_route"].cpu().numpy() < 0] == -77.0).all()
    for e, rows, routes in extents(pool):
        # within eight neighbours of one block the products are multiples of a quarter up to 36 and add exactly; the
        # groups and instructions are joined in at least 24 bits
        ref, tol = OP.product(av[routes // k if gather else rows], wv[e])
        tol = half_step(ref, tol)
        assert np.all(np.abs(got[rows] - ref) <= tol), (e, rows.size, np.max(np.abs(got[rows] - ref) / tol))


SHAPES = [
    (1, 8, 2, 64, 128, 0.0, None), (1, 1, 1, 32, 128, 0.0, None), (5, 3, 1, 96, 384, 0.0, None),
    (40, 16, 2, 256, 640, 0.2, None), (33, 64, 6, 160, 256, 0.2, None), (300, 4, 2, 544, 1152, 0.2, None),
    (700, 3, 2, 288, 1024, 0.0, [1]), (257, 2, 1, 512, 2048, 0.0, None), (90, 512, 3, 64, 128, 0.2, None),
    (1100, 2, 2, 1056, 384, 0.0, None), (6, 5, 2, 32, 256, 1.0, None),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,N,K,drop,only", SHAPES)
def test_product(T, E, k, N, K, drop, only, gather):
    check(routing(T, E, k, T + N, drop, only), E, N, K, gather, seed=K)


@pytest.mark.parametrize("name,T,E,k,N,K,gather", [
    ("k_mxfp4_few", 9, 3, 1, 64, 1152, True), ("k_mxfp4_few", 100, 4, 1, 256, 128, False),
    ("k_mxfp4_tile64", 600, 3, 2, 544, 384, True), ("k_mxfp4_tile64", 900, 5, 1, 288, 512, False),
    ("k_mxfp4_tile256", 8000, 3, 1, 4128, 512, True), ("k_mxfp4_tile256", 8000, 2, 1, 4096, 640, True),
    ("k_mxfp4_tile256", 8000, 3, 1, 3872, 1024, False), ("k_mxfp4_tile256", 8000, 2, 1, 4096, 128, False)])
def test_every_kernel(name, T, E, k, N, K, gather):
    with Kernels() as ran:
        check(routing(T, E, k, T, 0.1), E, N, K, gather, seed=N)
    assert name in ran.names, ran.names


def test_nan_exponents_in_a_large_tile():
    """One token's and one weight row's last block, where pairs of stages and single ones are loaded."""
    for K in (512, 640):
        idx = torch.zeros(8192, 1, dtype=torch.int32)
        idx[::2] = 1
        pool = build(idx, 2)
        a, ea, w, ew = operands(8192, 2, 4096, K, K)
        ea[777, K // 32 - 1] = 255
        ew[0, 4001, K // 32 - 1] = 255
        with Kernels() as ran:
            out = M.mxfp4_product(pool, a, ea, w, ew, topk=1)
        assert "k_mxfp4_tile256" in ran.names
        bad = torch.isnan(out).cpu()
        for e, rows, routes in extents(pool):
            want = torch.zeros(rows.size, 4096, dtype=torch.bool)
            want[torch.from_numpy(routes == 777)] = True
            if e == 0:
                want[:, 4001] = True
            assert torch.equal(bad[rows], want), (K, e)


def test_nan_exponents_stay_in_their_rows_and_columns():
    """A NaN block of one token, of one weight row, and in the row behind a short last stage."""
    idx = torch.tensor([[0, 1], [1, 2], [0, 2]], dtype=torch.int32)
    pool = build(idx, 3)
    for K in (128, 384, 512):
        a, ea, w, ew = operands(3, 3, 64, K, K)
        ea[1, K // 64] = 255
        ew[2, 7, 0] = 255
        out = f64(M.mxfp4_product(pool, a, ea, w, ew, topk=2))
        for e, rows, routes in extents(pool):
            bad = np.zeros((rows.size, 64), bool)
            bad[routes // 2 == 1] = True
            if e == 2:
                bad[:, 7] = True
            assert np.array_equal(np.isnan(out[rows]), bad), (K, e)


def test_far_apart_exponents():
    """Blocks of very large and very small scale in one row; results below bf16's normal range."""
    idx = torch.zeros(1, 1, dtype=torch.int32)
    pool = build(idx, 1)
    a, ea, w, ew = operands(1, 1, 32, 512, 3)
    ea[0, :] = torch.tensor([127, 20, 230, 127] * 4, dtype=torch.uint8)
    ew[0, :, :] = torch.tensor([127, 234, 24, 90] * 4, dtype=torch.uint8)
    out = f64(M.mxfp4_product(pool, a, ea, w, ew, topk=1))
    ref, tol = OP.product(values(a, ea), values(w, ew)[0])
    assert np.all(np.abs(out[0] - ref[0]) <= half_step(ref, tol)[0])


def test_streams_and_graph():
    idx = routing(60, 4, 2, 3)
    pool = build(idx, 4)
    g = torch.Generator().manual_seed(4)
    x = spread(g, 60, 256).cuda()
    w, ew = M.mxfp4_quantize_weight((torch.randn(4, 128, 256, generator=g) / 16).to(BF).cuda())

    def run(stream=None, **out):
        a, ea = M.mxfp4_quantize_rows(x, stream=stream)
        return M.mxfp4_product(pool, a, ea, w, ew, topk=2, stream=stream, **out)
    want = run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(s)
    s.synchronize()
    assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out=out)
    for i in range(3):
        x.copy_(spread(g, 60, 256))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(run().view(torch.int16), out.view(torch.int16)), i


def test_weights_of_the_layers_base():
    """The layer's own 4-bit weights as the product's: same codes, same exponents, and the down product of a layer."""
    idx = routing(20, 4, 2, 1)
    pool = build(idx, 4)
    case = {n: torch.randn(4, 256, 256).mul(0.1).to(BF) for n in ("W13", "W2")}
    mx, deq = Hn.mxfp4_base({n: t.view(torch.int16).numpy().view(np.uint16) for n, t in case.items()})
    c, e = M.mxfp4_quantize_weight(case["W2"].cuda())
    assert np.array_equal(c.cpu().numpy(), mx["W2"]) and np.array_equal(e.cpu().numpy(), mx["W2_scale"])
    v = f64(M.mxfp4_dequantize(c, e))
    assert np.array_equal(v, OMX.dequantize(mx["W2"], mx["W2_scale"]))

"""Every remainder of both widths, with rows of every remainder, through every
kernel of the expert products and of the weight's gradient; 4-bit products with
exponents at the alignment that is asked of them, and of a layer's own base."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from oracle import mxfp4 as OMX
from oracle import products as OP
from tests import harness as Hn
from tests import test_gpu_mxfp4_ops as MX
from tests.test_gpu_product import Kernels, build, check_grad, check_product, extents, f64, half_step, routing

pytestmark = pytest.mark.gpu
BF, U8 = torch.bfloat16, torch.uint8

# remainders of N modulo 256 and of K modulo 64
REST = [(8, 56), (24, 48), (72, 40), (120, 32), (136, 24), (200, 16), (248, 8)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


@pytest.mark.parametrize("name,T,E,k,N,K,transposed", [
    ("k_product_few", 9, 3, 1, 0, 1024, False), ("k_product_tile64", 600, 3, 2, 512, 192, False),
    ("k_product_tile256", 5900, 3, 1, 2048, 512, False), ("k_product_t_tile64", 600, 3, 2, 512, 192, True),
    ("k_product_t_tile256", 5900, 3, 1, 2048, 512, True)])
@pytest.mark.parametrize("i", range(len(REST)))
def test_widths(name, T, E, k, N, K, transposed, i):
    n, m = REST[i]
    T += 37 * i if T > 9 else i
    with Kernels() as ran:
        check_product(routing(T, E, k, T, 0.1), E, N + n, K + m, i % 2 == 0, transposed, seed=i)
    assert name in ran.names, ran.names


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("i", range(len(REST)))
def test_widths_of_the_gradient(gather, i):
    n, m = REST[i]
    check_grad(routing(150 + 9 * i, 3, 2, i, 0.1), 3, 256 + n, 256 + m + 64 * (i % 4), gather, (BF, torch.float32)[i % 2], i % 3 == 0, seed=i)


@pytest.mark.parametrize("name,T,E,N,K", [
    ("k_mxfp4_few", 9, 3, 0, 1152), ("k_mxfp4_tile64", 600, 3, 512, 384), ("k_mxfp4_tile256", 8000, 3, 4096, 512),
    ("k_mxfp4_tile256", 8000, 2, 4096, 640)])
@pytest.mark.parametrize("n", [32, 96, 160, 224])
def test_widths_in_4_bits(name, T, E, N, K, n):
    with Kernels() as ran:
        MX.check(routing(T + n, E, 1, n, 0.1), E, N + n, K, n % 64 == 32, seed=n)
    assert name in ran.names, ran.names


def off_by_four(t):
    """The same bytes, 4 past a multiple of 16."""
    b = torch.empty(t.numel() + 16, dtype=U8, device="cuda")
    o = b[4:4 + t.numel()].view(t.shape)
    assert o.data_ptr() % 16 == 4
    return o.copy_(t)


@pytest.mark.parametrize("name,T,E,N,K", [
    ("k_mxfp4_few", 9, 3, 64, 1152), ("k_mxfp4_tile64", 600, 3, 544, 384), ("k_mxfp4_tile256", 8000, 3, 4128, 512),
    ("k_mxfp4_tile256", 8000, 2, 4096, 640)])
@pytest.mark.parametrize("gather", [False, True])
def test_exponents_of_four_bytes_alignment(name, T, E, N, K, gather):
    pool = build(routing(T, E, 1, T), E)
    a, ea, w, ew = MX.operands(T if gather else pool["row_to_route"].numel(), E, N, K, 5)
    want = M.mxfp4_product(pool, a, ea, w, ew, topk=int(gather))
    with Kernels() as ran:
        got = M.mxfp4_product(pool, a, off_by_four(ea), w, off_by_four(ew), topk=int(gather))
    assert name in ran.names, ran.names
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_rows_to_and_from_exponents_of_four_bytes_alignment():
    x = MX.spread(torch.Generator().manual_seed(6), 70, 384).cuda()
    c, e = M.mxfp4_quantize_rows(x)
    to = off_by_four(torch.zeros_like(e))
    M.mxfp4_quantize_rows(x, exponents=to)
    assert torch.equal(to, e)
    assert torch.equal(M.mxfp4_dequantize(c, to), M.mxfp4_dequantize(c, e))


@pytest.mark.parametrize("which", ["W13", "W2"])
def test_products_of_the_layers_own_base(which):
    """Gate / up and down of an MXFP4 layer: its codes and scales, as the layer holds them, as a product's weight."""
    E, H, I, k = 4, 256, 512, 2
    g = torch.Generator().manual_seed(7)
    base = {"W13": torch.randn(E, 2 * I, H, generator=g).mul(0.1).to(BF), "W2": torch.randn(E, H, I, generator=g).mul(0.1).to(BF)}
    mx, _ = Hn.mxfp4_base({n: t.view(torch.int16).numpy().view(np.uint16) for n, t in base.items()})
    w, ew = (torch.from_numpy(np.ascontiguousarray(mx[n])).cuda() for n in (which, which + "_scale"))
    idx = routing(50, E, k, 8)
    pool = build(idx, E)
    gather = which == "W13"
    x = MX.spread(g, 50 if gather else pool["row_to_route"].numel(), base[which].shape[2])
    a, ea = M.mxfp4_quantize_rows(x.cuda())
    out = f64(M.mxfp4_product(pool, a, ea, w, ew, topk=k if gather else 0))
    av, wv = MX.values(a, ea), OMX.dequantize(mx[which], mx[which + "_scale"])
    for e, rows, routes in extents(pool):
        ref, tol = OP.product(av[routes // k if gather else rows], wv[e])
        assert len(rows) and np.all(np.abs(out[rows] - ref) <= half_step(ref, tol)), e


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("T,N,K", [(20, 65536, 72), (20, 72, 65536), (500, 65536, 72), (500, 72, 65536)])
def test_widest(T, N, K, transposed):
    """Single waves and tiles at the largest widths."""
    check_product(routing(T, 2, 1, T, 0.1), 2, N, K, T > 100, transposed, seed=T)


@pytest.mark.parametrize("N,K", [(65536, 72), (72, 65536)])
def test_widest_gradient(N, K):
    check_grad(routing(100, 2, 1, 3, 0.1), 2, N, K, True, torch.float32, False)


@pytest.mark.parametrize("T,N,K", [(20, 65536, 128), (20, 32, 65536), (500, 65536, 128), (500, 96, 65536)])
def test_widest_in_4_bits(T, N, K):
    MX.check(routing(T, 2, 1, T, 0.1), 2, N, K, T > 100, seed=T)

"""Calls of the expert products, 4-bit products and MoeMuon at the edges of what
they allow: no routes at all, one expert twice in a token, the smallest widths,
512 experts, activations shorter than the pool, pools of several adapters, what
stands in rows of no route; and MoeMuon's refusals of device tensors."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import mxfp4 as OMX
from oracle import products as OP
from tests import harness as Hn
from tests.test_gpu_product import build, check_product, extents, f64, half_step, rand, routing

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def check_grad(pool, d, a, topk, got, before=None):
    d, a = f64(d), f64(a)
    for e, rows, routes in extents(pool):
        ref, tol = OP.weight_grad(d[rows], a[routes // topk if topk else rows])
        if before is not None:
            ref, tol = ref + f64(before[e]), tol + 2.0 ** -24 * (np.abs(ref + f64(before[e])) + tol)
        assert np.all(np.abs(f64(got[e]) - ref) <= tol), e


def test_no_routes():
    pool = build(torch.full((30, 2), -1, dtype=torch.int32), 4)
    g = torch.Generator().manual_seed(1)
    cap = pool["row_to_route"].numel()
    a, w, d = rand(g, 30, 128), rand(g, 4, 64, 128), rand(g, cap, 64)
    for transposed in (False, True):
        out = torch.full((cap, 128 if transposed else 64), 3.0, dtype=BF, device="cuda")
        M.expert_product(pool, d if transposed else a, w, topk=0 if transposed else 2, transposed=transposed, out=out)
        assert (out == 3).all()
    dw = torch.full((4, 64, 128), 5.0, device="cuda")
    M.expert_weight_grad(pool, d, a, topk=2, out=dw, accumulate=True)
    assert (dw == 5).all()
    M.expert_weight_grad(pool, d, a, topk=2, out=dw)
    assert (dw == 0).all()
    q, x = M.mxfp4_quantize_rows(a)
    wq, wx = M.mxfp4_quantize_weight(rand(g, 4, 128, 128))
    out = torch.full((cap, 128), 3.0, dtype=BF, device="cuda")
    M.mxfp4_product(pool, q, x, wq, wx, topk=2, out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("transposed", [False, True])
def test_one_expert_twice_in_a_token(transposed):
    check_product(torch.tensor([[1, 1], [0, 1], [2, 2], [1, 1]], dtype=torch.int32), 3, 48, 80, True, transposed)


@pytest.mark.parametrize("N,K", [(8, 8), (8, 72), (72, 8)])
def test_smallest_widths(N, K):
    idx = routing(40, 5, 2, N + K)
    for transposed in (False, True):
        check_product(idx, 5, N, K, True, transposed)
    pool = build(idx, 5)
    g = torch.Generator().manual_seed(2)
    d, a = rand(g, pool["row_to_route"].numel(), N), rand(g, 40, K)
    check_grad(pool, d, a, 2, M.expert_weight_grad(pool, d, a, topk=2, dtype=F32))


def test_512_experts():
    idx = routing(700, 512, 3, 5, 0.1)
    for transposed in (False, True):
        check_product(idx, 512, 40, 136, True, transposed)
    pool = build(idx, 512)
    g = torch.Generator().manual_seed(3)
    d, a = rand(g, pool["row_to_route"].numel(), 40), rand(g, 700, 136)
    check_grad(pool, d, a, 3, M.expert_weight_grad(pool, d, a, topk=3, dtype=F32))


def test_rows_of_no_route_hold_anything():
    """NaN in the pool's padding and unused rows of every operand that has them."""
    idx = routing(90, 5, 2, 7, 0.3)
    pool = build(idx, 5)
    g = torch.Generator().manual_seed(4)
    cap = pool["row_to_route"].numel()
    pad = pool["row_to_route"] < 0
    d, a, w = rand(g, cap, 136), rand(g, cap, 72), rand(g, 5, 136, 72)
    d[pad], a[pad] = NAN, NAN
    assert int(pad.sum()) > 0
    out = torch.zeros(cap, 136, dtype=BF, device="cuda")
    assert not torch.isnan(M.expert_product(pool, a, w, out=out)).any()
    assert not torch.isnan(M.expert_product(pool, d, w, transposed=True)).any()
    check_grad(pool, d, a, 0, M.expert_weight_grad(pool, d, a, dtype=F32))
    x = rand(g, 90, 72)
    before = torch.randn(5, 136, 72, generator=g).cuda()
    dw = before.clone()
    M.expert_weight_grad(pool, d, x, topk=2, out=dw, accumulate=True)
    check_grad(pool, d, x, 2, dw, before)
    q, e = M.mxfp4_quantize_rows(rand(g, cap, 128))
    e[pad] = 255
    wq, we = M.mxfp4_quantize_weight(rand(g, 5, 128, 128))
    assert not torch.isnan(M.mxfp4_product(pool, q, e, wq, we)).any()


@pytest.mark.parametrize("rows", [1, 17, 40])
def test_activations_shorter_than_the_pool(rows):
    """Pool rows past a's are zeros."""
    idx = routing(60, 3, 1, 8)
    pool = build(idx, 3)
    cap = pool["row_to_route"].numel()
    g = torch.Generator().manual_seed(5)
    a, w, d = rand(g, cap, 72), rand(g, 3, 40, 72), rand(g, cap, 40)
    zeroed = a.clone()
    zeroed[rows:] = 0
    got, want = M.expert_product(pool, a[:rows], w), M.expert_product(pool, zeroed, w)
    assert torch.equal(got, want)
    got, want = (M.expert_weight_grad(pool, d, x, dtype=F32) for x in (a[:rows], zeroed))
    assert torch.equal(got, want)


def test_pool_of_several_adapters():
    """A pool grouped by (expert, adapter): weights one per group."""
    T, E, k, roots = 64, 4, 2, [0, 20, 20, 64]
    desc = B.make_desc(T, 256, 256, E, k, 8)
    layer = B.MoeLoraLayer(desc, roots=roots)
    layer.build_pool(routing(T, E, k, 9).cuda())
    pool = layer.pool
    G = pool["counts"].numel()
    g = torch.Generator().manual_seed(6)
    a, w = rand(g, T, 72), rand(g, G, 40, 72)
    out = f64(M.expert_product(pool, a, w, topk=k))
    d = rand(g, pool["row_to_route"].numel(), 40)
    assert G == E * 3 and int(pool["counts"].sum()) == T * k
    for e, rows, routes in extents(pool):
        ref, tol = OP.product(f64(a)[routes // k], f64(w[e]))
        assert np.all(np.abs(out[rows] - ref) <= half_step(ref, tol)), e
    check_grad(pool, d, a, k, M.expert_weight_grad(pool, d, a, topk=k, dtype=F32))


def test_a_stream_by_its_handle():
    idx = routing(40, 3, 2, 10)
    pool = build(idx, 3)
    g = torch.Generator().manual_seed(7)
    a, w = rand(g, 40, 128), rand(g, 3, 128, 128)
    want = M.expert_product(pool, a, w, topk=2)
    q, e = M.mxfp4_quantize_rows(a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = M.expert_product(pool, a, w, topk=2, stream=s.cuda_stream)
    q2, e2 = M.mxfp4_quantize_rows(a, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(q, q2) and torch.equal(e, e2)
    v = f64(M.mxfp4_dequantize(q, e))
    assert np.array_equal(v, OMX.dequantize(q.cpu().numpy(), e.cpu().numpy()))


def test_muon_refusals():
    def z(*s, dtype=F32):
        return torch.zeros(*s, dtype=dtype, device="cuda")
    both = z(8, 40)
    for params, grads, kw in (
            ([z(8, 40)], [z(8, 41)], {}), ([z(8, 40)], [z(8, 40, dtype=torch.float16)], {}),
            ([z(8, 40, dtype=torch.float16)], [z(8, 40)], {}), ([z(40, 8).t()], [z(8, 40)], {}),
            ([z(8, 40), z(8, 40, dtype=BF)], [z(8, 40), z(8, 40)], {}), ([both, both], [z(8, 40), z(8, 40)], {}),
            ([both], [both], {}), ([z(8, 40)], [z(8, 40)], dict(masters=[z(8, 40)])),
            ([z(8, 40, dtype=BF)], [z(8, 40)], dict(masters=[z(8, 40, dtype=BF)])),
            ([z(8, 40)], [z(8, 40)], dict(states={"momentum": [z(8, 39)]})),
            ([z(8, 40)], [z(8, 40)], dict(states={"m": [z(8, 40)]})), ([z(8, 40)], [torch.zeros(8, 40)], {})):
        with pytest.raises(ValueError):
            M.MoeMuon(params, grads, **kw)
    for shape in ((257, 300), (2, 300, 257)):
        with pytest.raises(B.MoeLoraError):
            M.MoeMuon([z(*shape)], [z(*shape)])
    for kw in (dict(lr=-1.0), dict(lr=NAN), dict(momentum=1.0), dict(eps=0.0), dict(rounds=0), dict(rounds=17),
               dict(weight_decay=-0.1), dict(rms=float("inf"))):
        p = z(8, 40)
        with pytest.raises(B.MoeLoraError):
            M.MoeMuon([p], [z(8, 40)], **kw).step()
        assert not p.any()
    opt = M.MoeMuon([z(8, 40)], [z(8, 40)])
    for control in (z(3), z(2, dtype=BF), torch.zeros(2)):
        with pytest.raises(ValueError):
            opt.step(control=control)
    for lr, gs in ((-1.0, 1.0), (0.1, NAN), (1e300, 1.0)):
        with pytest.raises(ValueError):
            opt.write_control(z(2), lr, gs)
    opt._ws = (opt._ws[0], opt._ws[1] - 16)  # a workspace shorter than asked for
    with pytest.raises(B.MoeLoraError):
        opt.step()


def test_muon_rate_zero_moves_the_momentum_alone():
    g = torch.Generator().manual_seed(11)
    p, gr = rand(g, 3, 20, 60), rand(g, 3, 20, 60)
    before = p.clone()
    opt = M.MoeMuon([p], [gr], lr=0.0, weight_decay=0.5)
    opt.step()
    assert torch.equal(p, before) and torch.equal(opt.states["momentum"][0], gr.float())

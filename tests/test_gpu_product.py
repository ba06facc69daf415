"""Expert products in bf16 and the weight's gradient against float64: gathered
and pool rows, both weight layouts, experts with none, one and many rows, every
remainder of both widths, rows of no route left alone, gradients added to what
was there, other streams, replayed graphs, and a layer's forward and backward
made of them."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import products as OP
from tests import harness as Hn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def f64(t):
    return t.double().cpu().numpy()


def build(idx, E):
    T, k = idx.shape
    desc = B.make_desc(T, 256, 256, E, k, 8)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
            "route_to_row": torch.empty(T * k, **i32), "row_to_route": torch.empty(B.moe_lora_pool_capacity(desc), **i32)}
    M.build_pool(desc, idx.cuda(), pool["counts"], pool["offsets"], pool["route_to_row"], pool["row_to_route"])
    return pool


def routing(T, E, k, seed, drop=0.0, only=None):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)])
    if only is not None:
        idx = torch.tensor(only)[idx % len(only)]
    if drop:
        idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx.to(torch.int32)


def rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def extents(pool):
    """(expert, its rows, the routes of them)."""
    off, cnt, r2r = (pool[n].cpu().numpy() for n in ("offsets", "counts", "row_to_route"))
    return [(e, np.arange(off[e], off[e] + c), r2r[off[e]:off[e] + c]) for e, c in enumerate(cnt)]


def half_step(ref, tol):
    return tol + 2.0 ** -8 * (np.abs(ref) + tol)  # the rounding to bf16


def check_product(idx, E, N, K, gather, transposed, seed=0):
    T, k = idx.shape
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    g = torch.Generator().manual_seed(seed)
    a = rand(g, T if gather else cap, K)
    w = rand(g, E, *((K, N) if transposed else (N, K)), std=K ** -0.5)
    out = torch.full((cap, N), -77.0, dtype=BF, device="cuda")
    got = M.expert_product(pool, a, w, topk=k if gather else 0, transposed=transposed, out=out)
    assert got.data_ptr() == out.data_ptr()
    got, a, w = f64(got), f64(a), f64(w)
    assert (got[pool["row_to_route"].cpu().numpy() < 0] == -77.0).all()  # padding and unused rows
    for e, rows, routes in extents(pool):
        ref, tol = OP.product(a[routes // k if gather else rows], w[e].T if transposed else w[e])
        tol = half_step(ref, tol)
        assert np.all(np.abs(got[rows] - ref) <= tol), (e, rows.size, np.max(np.abs(got[rows] - ref) / tol))


def check_grad(idx, E, N, K, gather, dtype, add, seed=0):
    T, k = idx.shape
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    g = torch.Generator().manual_seed(seed)
    a, grad = rand(g, T if gather else cap, K), rand(g, cap, N)
    grad[pool["row_to_route"] < 0] = float("nan")  # rows of no route are not used
    if not gather:
        a[pool["row_to_route"] < 0] = float("nan")
    out = torch.full((E, N, K), 3.0 if add else float("nan"), dtype=dtype, device="cuda")
    got = M.expert_weight_grad(pool, grad, a, topk=k if gather else 0, out=out, accumulate=add)
    assert got.data_ptr() == out.data_ptr()
    got, a, grad = f64(got), f64(a), f64(grad)
    for e, rows, routes in extents(pool):
        ref, tol = OP.weight_grad(grad[rows], a[routes // k if gather else rows])
        if add and rows.size:
            ref, tol = ref + 3.0, tol + 2.0 ** -23 * (np.abs(ref) + 3.0)
        elif add:
            ref = ref + 3.0
        if rows.size == 0:
            assert np.array_equal(got[e], ref)
            continue
        tol = half_step(ref, tol) if dtype == BF else tol
        assert np.all(np.abs(got[e] - ref) <= tol), (e, rows.size, np.max(np.abs(got[e] - ref) / tol))


# one token; a few; many experts without rows; one expert with all rows; tiles of every kernel
SHAPES = [
    (1, 8, 2, 64, 128, 0.0, None), (1, 1, 1, 8, 8, 0.0, None), (5, 3, 1, 24, 40, 0.0, None),
    (40, 16, 2, 256, 72, 0.2, None), (33, 64, 6, 136, 264, 0.2, None), (300, 4, 2, 520, 200, 0.2, None),
    (700, 3, 2, 264, 1000, 0.0, [1]), (257, 2, 1, 512, 512, 0.0, None), (90, 512, 3, 48, 64, 0.2, None),
    (520, 2, 2, 1032, 136, 0.0, None), (6, 5, 2, 40, 32, 1.0, None),
]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,N,K,drop,only", SHAPES)
def test_product(T, E, k, N, K, drop, only, gather, transposed):
    check_product(routing(T, E, k, T + N, drop, only), E, N, K, gather, transposed, seed=K)


@pytest.mark.parametrize("dtype,add", [(BF, False), (torch.float32, False), (BF, True), (torch.float32, True)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("T,E,k,N,K,drop,only", SHAPES)
def test_weight_gradient(T, E, k, N, K, drop, only, gather, dtype, add):
    check_grad(routing(T, E, k, T + N, drop, only), E, N, K, gather, dtype, add, seed=K)


class Kernels:
    """The kernels that calls take, from the library's own trace."""

    def __enter__(self):
        B.moe_lora_trace_reset()
        B.moe_lora_trace_enable(True)
        return self

    def __exit__(self, *a):
        B.moe_lora_trace_enable(False)
        self.names = set(B.moe_lora_trace_collect())
        B.moe_lora_trace_reset()


@pytest.mark.parametrize("name,T,E,k,N,K,gather,transposed", [
    ("k_product_few", 9, 3, 1, 40, 1048, True, False), ("k_product_few", 100, 4, 1, 256, 72, False, False),
    ("k_product_tile64", 600, 3, 2, 520, 200, True, False), ("k_product_tile64", 900, 5, 1, 264, 64, False, False),
    ("k_product_tile256", 6000, 3, 1, 2056, 520, True, False), ("k_product_tile256", 5000, 2, 1, 2304, 1024, False, False),
    ("k_product_t_tile64", 600, 3, 2, 520, 200, True, True), ("k_product_t_tile64", 40, 5, 1, 264, 72, False, True),
    ("k_product_t_tile256", 6000, 3, 1, 2056, 520, True, True), ("k_product_t_tile256", 5000, 2, 1, 2304, 1024, False, True)])
def test_every_kernel(name, T, E, k, N, K, gather, transposed):
    with Kernels() as ran:
        check_product(routing(T, E, k, T, 0.1), E, N, K, gather, transposed, seed=N)
    assert name in ran.names, ran.names


def test_infinities_stay_in_their_rows():
    """A NaN or an infinity in one token, one expert's weight, and past the widths' ends in memory."""
    idx = torch.tensor([[0, 1], [1, 2], [0, 2]], dtype=torch.int32)
    pool = build(idx, 3)
    g = torch.Generator().manual_seed(5)
    for transposed in (False, True):
        N, K = 40, 72
        a, w = rand(g, 3, K), rand(g, 3, *((K, N) if transposed else (N, K)))
        a[1, 3] = float("inf")
        if transposed:
            w[2, 5, 7] = float("nan")
        else:
            w[2, 7, 5] = float("nan")
        out = f64(M.expert_product(pool, a, w, topk=2, transposed=transposed))
        for e, rows, routes in extents(pool):
            t = routes // 2
            bad = np.zeros((rows.size, N), bool)
            bad[t == 1] = True
            if e == 2:
                bad[:, 7] = True
            assert np.array_equal(~np.isfinite(out[rows]), bad), (transposed, e)


def test_a_row_does_not_depend_on_the_others():
    idx = routing(300, 4, 2, 7)
    pool = build(idx, 4)
    g = torch.Generator().manual_seed(8)
    a, w = rand(g, 300, 512), rand(g, 4, 256, 512)
    first = M.expert_product(pool, a, w, topk=2).clone()
    again = M.expert_product(pool, a, w, topk=2)
    assert torch.equal(first.view(torch.int16), again.view(torch.int16))
    b = a.clone()
    b[5] = 99.0
    other = M.expert_product(pool, b, w, topk=2)
    keep = (pool["row_to_route"] // 2 != 5) & (pool["row_to_route"] >= 0)
    assert torch.equal(first[keep].view(torch.int16), other[keep].view(torch.int16))


def test_routes_beyond_the_activations_read_zeros():
    idx = torch.tensor([[0], [1], [0], [1]], dtype=torch.int32)
    pool = build(idx, 2)
    g = torch.Generator().manual_seed(1)
    a, w = rand(g, 2, 64), rand(g, 2, 32, 64)  # tokens 2 and 3 are not there
    out = f64(M.expert_product(pool, a, w, topk=1))
    dw = f64(M.expert_weight_grad(pool, torch.ones(pool["row_to_route"].numel(), 32, dtype=BF, device="cuda"), a, topk=1))
    for e, rows, routes in extents(pool):
        assert not out[rows[routes >= 2]].any() and out[rows[routes < 2]].any()
        assert np.allclose(dw[e], np.tile(f64(a)[e], (32, 1)), rtol=2.0 ** -8)


def test_streams_and_graph():
    idx = routing(60, 4, 2, 3)
    pool = build(idx, 4)
    g = torch.Generator().manual_seed(4)
    a, w, d = rand(g, 60, 256), rand(g, 4, 128, 256), rand(g, pool["row_to_route"].numel(), 128)
    want = M.expert_product(pool, a, w, topk=2), M.expert_weight_grad(pool, d, a, topk=2), M.expert_product(pool, d, w, transposed=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = (M.expert_product(pool, a, w, topk=2, stream=s), M.expert_weight_grad(pool, d, a, topk=2, stream=s),
           M.expert_product(pool, d, w, transposed=True, stream=s))
    s.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.expert_product(pool, a, w, topk=2, out=outs[0])
        M.expert_weight_grad(pool, d, a, topk=2, out=outs[1])
        M.expert_product(pool, d, w, transposed=True, out=outs[2])
    for i in range(3):
        a.copy_(rand(g, 60, 256))
        M.build_pool(B.make_desc(60, 256, 256, 4, 2, 8), routing(60, 4, 2, 30 + i).cuda(), *[pool[n] for n in (
            "counts", "offsets", "route_to_row", "row_to_route")])
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = M.expert_product(pool, a, w, topk=2), M.expert_weight_grad(pool, d, a, topk=2), M.expert_product(pool, d, w, transposed=True)
        for x, y in zip(want, outs):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16)), i


def test_two_layers_of_products_and_their_gradients():
    """Gate / up and down as products, against autograd in float64 on the CPU; a gradient added over two micro-batches."""
    T, E, k, H, I = 50, 6, 2, 136, 72
    idx = routing(T, E, k, 9, drop=0.1)
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    g = torch.Generator().manual_seed(11)
    x, w1, w2 = rand(g, T, H), rand(g, E, I, H, std=H ** -0.5), rand(g, E, H, I, std=I ** -0.5)
    dy = rand(g, cap, H)
    h = M.expert_product(pool, x, w1, topk=k)
    M.expert_product(pool, h, w2)
    dh = M.expert_product(pool, dy, w2, transposed=True)
    dw2 = M.expert_weight_grad(pool, dy, h, dtype=torch.float32)
    dw1 = M.expert_weight_grad(pool, dh, x, topk=k, dtype=torch.float32)
    M.expert_weight_grad(pool, dh, x, topk=k, out=dw1, accumulate=True)
    dx = M.expert_product(pool, dh, w1, transposed=True)
    tx, t1, t2 = (t.double().cpu().requires_grad_() for t in (x, w1, w2))
    loss = 0
    for e, rows, routes in extents(pool):
        loss = loss + ((tx[routes // k] @ t1[e].T) @ t2[e].T * dy.double().cpu()[rows]).sum()
    loss.backward()
    # what the roundings of h and dh to bf16 (2^-8 of each value, and the sums' own bound below that) carry on, by the
    # magnitudes of what they meet; 1.1: the second order, and the fp32 sums
    X, W1, W2, DY = f64(x), f64(w1), f64(w2), f64(dy)
    sum_dx, tol_dx = np.zeros((T, H)), np.zeros((T, H))
    for e, rows, routes in extents(pool):
        t = routes // k
        hv, dhv = X[t] @ W1[e].T, DY[rows] @ W2[e]
        eh = 2.0 ** -8 * np.abs(hv) + OP.product(X[t], W1[e])[1]
        ed = 2.0 ** -8 * np.abs(dhv) + OP.product(DY[rows], W2[e].T)[1]
        assert np.all(np.abs(f64(dw1)[e] - 2 * t1.grad[e].numpy()) <= 2.2 * (ed.T @ np.abs(X[t])) + 1e-12)
        assert np.all(np.abs(f64(dw2)[e] - t2.grad[e].numpy()) <= 1.1 * (np.abs(DY[rows]).T @ eh) + 1e-12)
        exact = dhv @ W1[e]
        np.add.at(sum_dx, t, f64(dx)[rows])
        np.add.at(tol_dx, t, 1.1 * (ed @ np.abs(W1[e]) + 2.0 ** -8 * np.abs(exact)) + 1e-12)
    assert np.all(np.abs(sum_dx - tx.grad.numpy()) <= tol_dx)

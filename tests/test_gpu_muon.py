"""The optimiser step with an orthogonalised update against float64: every
type, wide, tall and square matrices of odd sizes, one row, stacks and several
tensors in a call, matrices of zeros and of one direction, spectra over six
decades, non-finite gradients, streams and replayed graphs."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from oracle import muon as OMU
from tests import harness as Hn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=0.05, momentum=0.9, nesterov=True, weight_decay=0.1, rms=0.2, eps=1e-7)
SLOPE = OMU.slope(5)


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def f64(t):
    return t.double().cpu().numpy()


def update_tolerance(U, X, eps):
    """How far the update may be, in the root of its sum of squares: U is rounded to fp32 twice (2^-24 of each value
    each time), which the rounds enlarge by their slope at most; Q has 2^-24 of its own values, and Q U is summed in
    fp32 over the short side."""
    n = np.sqrt((U * U).sum()) + eps
    if U.shape[0] > U.shape[1]:
        U, X = U.T, X.T
    u, s, v = np.linalg.svd(U / n, full_matrices=False)
    q = (u * (np.where(s > 0, np.einsum("ij,ij->i", u.T @ X, v) / np.where(s > 0, s, 1), 0))) @ u.T
    return 2.0 ** -23 * SLOPE + (U.shape[0] + 1) * 2.0 ** -23 * np.linalg.norm(np.abs(q) @ np.abs(U / n))


def make(g, shape, ptype, gtype, masters, momentum=0.01):
    p = torch.randn(*shape, generator=g) * 0.05
    return {"master": p.cuda() if masters else None, "param": p.to(ptype).cuda(),
            "grad": (torch.randn(*shape, generator=g) * 0.01).to(gtype).cuda(),
            "momentum": (torch.randn(*shape, generator=g) * momentum).cuda()}


def optimiser(ts, **kw):
    kw = {**HYPER, **kw}
    return M.MoeMuon([t["param"] for t in ts], [t["grad"] for t in ts],
                     masters=[t["master"] for t in ts] if ts[0]["master"] is not None else None,
                     states={"momentum": [t["momentum"] for t in ts]}, **kw)


def expect(t, grad_scale=1.0, **kw):
    """What a step gives for each matrix of a tensor: p, momentum, update, U."""
    h = {**HYPER, **kw}
    p = f64(t["param"] if t["master"] is None else t["master"])
    p, g, m = (x.reshape(-1, *x.shape[-2:]) for x in (p, f64(t["grad"]), f64(t["momentum"])))
    out = []
    f = lambda v: float(np.float32(v))  # noqa: E731  (the step's constants are fp32)
    for i in range(p.shape[0]):
        kw2 = dict(lr=f(h["lr"]), mu=f(h["momentum"]), nesterov=h["nesterov"], weight_decay=f(h["weight_decay"]),
                   rms=f(h["rms"]), eps=h["eps"], grad_scale=f(grad_scale), rounds=h.get("rounds", 5))
        q, mm, x = OMU.step(p[i], g[i], m[i], **kw2)
        u = f(grad_scale) * g[i] + f(h["momentum"]) * mm if h["nesterov"] else mm
        out.append((q, mm, x, u, p[i]))
    return out


def check(t, want, **kw):
    h = {**HYPER, **kw}
    p = f64(t["param"] if t["master"] is None else t["master"])
    m = f64(t["momentum"])
    p, m = (x.reshape(-1, *x.shape[-2:]) for x in (p, m))
    rounds_to = t["param"].dtype if t["master"] is None else F32
    for i, (q, mm, x, u, p0) in enumerate(want):
        assert np.all(np.abs(m[i] - mm) <= 2.0 ** -23 * (np.abs(mm) + 0.2)), i
        tol = h["lr"] * h["rms"] * np.sqrt(max(p0.shape)) * update_tolerance(u, x, h["eps"])
        # the change's own roundings, and p's
        each = 4 * 2.0 ** -24 * (np.abs(q - p0) + h["lr"] * h["weight_decay"] * np.abs(p0)) + 2.0 ** -24 * np.abs(q)
        each = each + (2.0 ** -8 * (np.abs(q) + tol) if rounds_to == BF else 0)
        assert np.linalg.norm(np.maximum(np.abs(p[i] - q) - each, 0)) <= tol, i
    if t["master"] is not None:
        assert torch.equal(t["param"], t["master"].to(BF))


SHAPES = [(8, 512), (512, 8), (3, 5, 1000), (2, 300, 7), (4, 128, 256), (3, 256, 128), (1, 64, 64), (2, 1, 9), (2, 9, 1),
          (1, 1), (2, 130, 515), (1, 200, 210), (1, 700, 255), (256, 256), (16, 33, 40), (1, 5000, 20), (20, 4097)]


@pytest.mark.parametrize("ptype,gtype,masters", [(BF, BF, True), (F32, F32, False), (BF, F32, False), (F32, BF, False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_step(shape, ptype, gtype, masters):
    t = make(torch.Generator().manual_seed(sum(shape)), shape, ptype, gtype, masters)
    want = expect(t, 0.5)
    optimiser([t]).step(grad_scale=0.5)
    check(t, want)


@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(weight_decay=0.0), dict(momentum=0.0), dict(rounds=1),
                                dict(rounds=2), dict(eps=0.5)])
def test_options(kw):
    t = make(torch.Generator().manual_seed(1), (2, 20, 300), F32, F32, False)
    want = expect(t, **kw)
    optimiser([t], **kw).step()
    check(t, want, **kw)


def test_many_tensors_in_one_call():
    """Short and long sides of all kernels, more tensors than one launch's table, an empty one, three steps."""
    g = torch.Generator().manual_seed(2)
    shapes = [(8, 64), (3, 64, 8), (0, 4, 4), (130, 140), (2, 260, 200)] + [(2, 5, 11 + i) for i in range(45)]
    ts = [make(g, s, BF, BF, True) for s in shapes]
    opt = optimiser(ts)
    for _ in range(3):
        want = [expect(t) for t in ts]
        opt.step()
        for t, w in zip(ts, want):
            check(t, w)


def test_first_step_from_zeros():
    t = make(torch.Generator().manual_seed(3), (2, 30, 50), F32, F32, False)
    t["momentum"].zero_()
    want = expect(t)
    opt = M.MoeMuon([t["param"]], [t["grad"]], **HYPER)
    opt.step()
    t["momentum"] = opt.states["momentum"][0]
    check(t, want)


def test_matrices_of_zeros_and_one_direction():
    t = make(torch.Generator().manual_seed(4), (4, 24, 100), F32, F32, False)
    for n in ("grad", "momentum"):
        t[n][1] = 0
        t[n][2] = t[n][2, :, :1] * t[n][2, :1]  # rank one
        t[n][3] = 0
        t[n][3, 7, 9] = 1.0
    p0 = t["param"].clone()
    want = expect(t)
    optimiser([t]).step()
    check(t, want)
    decay = float(np.float32(np.float32(0.05) * np.float32(0.1)))
    assert torch.allclose(t["param"][1].double(), p0[1].double() * (1 - decay), rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("shape", [(16, 600), (128, 256), (250, 300)])
def test_spectra_over_six_decades(shape):
    """Singular values from 1 to 1e-6: the smallest are raised by the rounds, and their errors with them."""
    r = np.random.default_rng(5)
    m, n = shape
    u, v = np.linalg.qr(r.standard_normal((m, m)))[0], np.linalg.qr(r.standard_normal((n, m)))[0]
    g = torch.from_numpy(u * np.logspace(0, -6, m) @ v.T).float()
    t = {"param": torch.zeros(m, n).cuda(), "master": None, "grad": g.cuda(), "momentum": torch.zeros(m, n).cuda()}
    want = expect(t)
    optimiser([t]).step()
    check(t, want)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e25])
def test_scale_of_the_gradient(scale):
    """Squares far outside fp32's range; eps beside the smallest."""
    t = make(torch.Generator().manual_seed(6), (12, 90), F32, F32, False)
    t["grad"] *= scale * 100
    t["momentum"] *= scale
    want = expect(t, eps=1e-38)
    optimiser([t], eps=1e-38).step()
    q, mm, x, u, p0 = want[0]
    tol = 0.05 * 0.2 * np.sqrt(90) * update_tolerance(u, x, 1e-38)
    assert np.linalg.norm(f64(t["param"]) - q) <= tol + 2.0 ** -22 * np.linalg.norm(q)
    assert np.all(np.abs(f64(t["momentum"]) - mm) <= 2.0 ** -22 * (np.abs(mm) + scale))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_gradients_stay_in_their_matrix(bad):
    t = make(torch.Generator().manual_seed(7), (3, 20, 70), BF, BF, True)
    want = expect(t)
    t["grad"][1, 3, 50] = bad
    optimiser([t]).step()
    assert torch.isnan(t["master"][1]).all() and torch.isnan(t["param"][1]).all()
    for i in (0, 2):
        one = {n: x[i] for n, x in t.items()}
        check(one, [want[i]])


def test_steps_repeat_bit_for_bit_on_another_stream():
    g = torch.Generator().manual_seed(8)
    ts = [make(g, s, BF, BF, True) for s in ((3, 200, 16), (60, 900))]
    copies = [{n: x.clone() for n, x in t.items()} for t in ts]
    optimiser(ts).step()
    s = torch.cuda.Stream()
    other = optimiser(copies)
    torch.cuda.synchronize()
    other.step(stream=s)
    s.synchronize()
    for t, c in zip(ts, copies):
        for n in t:
            assert torch.equal(t[n], c[n])


def test_replayed_graph_with_other_rates():
    g = torch.Generator().manual_seed(9)
    a = [make(g, s, BF, BF, True) for s in ((3, 200, 16), (60, 900))]
    b = [{n: x.clone() for n, x in t.items()} for t in a]
    oa, ob = optimiser(a), optimiser(b)
    control = torch.zeros(2, device="cuda")
    oa.write_control(control, lr=0.0)
    oa.step(control=control)  # moves the momentum only
    ob.step(lr=0.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        oa.step(control=control)
    for i, (lr, gs) in enumerate(((0.01, 1.0), (0.5, 0.25), (0.002, 3.0))):
        for x, y in zip(a, b):
            new = (torch.randn(x["grad"].shape, generator=g) * 0.01).to(BF).cuda()
            x["grad"].copy_(new)
            y["grad"].copy_(new)
        oa.write_control(control, lr=lr, grad_scale=gs)
        graph.replay()
        torch.cuda.synchronize()
        ob.step(lr=lr, grad_scale=gs)
        for x, y in zip(a, b):
            for n in x:
                assert torch.equal(x[n], y[n]), (i, n)


def test_memory_is_kept():
    """A tensor given other memory: the optimiser goes on with what it was made for."""
    t = make(torch.Generator().manual_seed(10), (8, 40), F32, F32, False)
    opt = optimiser([t])
    old = t["param"].detach().clone()
    held = torch.empty(0).cuda().set_(t["param"].untyped_storage(), 0, (8, 40))
    t["param"].data = torch.zeros(8, 40, device="cuda")
    opt.step()
    assert not torch.equal(held, old) and not t["param"].any()

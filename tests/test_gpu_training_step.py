"""The operators as they are used together: a training step (router, layer,
router gradient, optimiser) against the oracles in one chain, eager and as a
replayed graph; and a frozen 8-bit expert pass (router, pool, rows, products)
stage by stage."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from mixture_experts_grouped_amd import inputs as I
from oracle import float8 as O8
from oracle import moe_lora as OM
from oracle import router as OR
from tests import harness as Hn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPE = I.Shape(T=150, H=256, I=256, E=8, topk=2, rank=8)
FACTORS = ("A1", "A3", "B1", "B3", "A2", "B2")
LR, WD = 1e-3, 0.01


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


class Step:
    """One adapter's training step from a router weight and the layer's case."""

    def __init__(self, bits):
        self.case = I.layer_inputs(SHAPE, (83,))
        self.run = Hn.GpuRun(SHAPE, self.case)
        g = torch.Generator().manual_seed(4)
        self.logits = (self.run.x.float().cpu() @ torch.randn(SHAPE.E, SHAPE.H, generator=g).t() * SHAPE.H ** -0.5).cuda()
        self.valid = (torch.rand(SHAPE.T, generator=g) > 0.1).to(torch.uint8).cuda()
        self.grad_loss = torch.full((1,), 3.0, device="cuda")
        self.router = M.MoeRouter(SHAPE.T, SHAPE.E, SHAPE.topk)
        L = self.run.layer
        params = [self.run.params[n] for n in FACTORS]
        self.masters = [p.float() for p in params]
        self.opt = M.MoeAdamW(params, [L.grads["d" + n] for n in FACTORS], masters=self.masters, state_bits=bits, lr=LR,
                              weight_decay=WD)

    def __call__(self, control=None):
        L, r = self.run.layer, self.router
        idx, w, counts, active, loss = r.forward(self.logits, self.valid)
        _, gw, _ = L.step(idx, self.run.x, w, self.run.params, self.run.go)
        r.backward(self.logits, idx, counts, active, gw, self.grad_loss, self.valid)
        self.opt.step(control=control)

    def results(self):
        r = self.router
        return [t.clone() for t in (r.topk_idx, r.topk_w, r.counts, r.loss, r.grad_logits, self.run.layer.out,
                                    self.run.layer.grad_x, *self.masters, *self.opt.params, *self.opt.states["m"],
                                    *self.opt.states["v"])]


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_against_the_oracles(bits):
    s = Step(bits)
    p64 = {n: Hn.f64(s.case[n]) for n in OM.PARAM_NAMES}
    x, go = Hn.f64(s.case["x"]), Hn.f64(s.case["grad_out"])
    s()
    res = s.run.fetch()
    l = s.logits.cpu().double().numpy()
    f = OR.forward(l, SHAPE.topk, True, valid=s.valid.cpu().numpy())
    assert np.array_equal(s.router.topk_idx.cpu().numpy(), f["topk_idx"])
    assert np.array_equal(s.run.layer.pool["counts"].cpu().numpy(), f["counts"][0])  # the pool's are the router's
    w = s.router.topk_w.cpu().double().numpy()
    out = OM.forward(x, f["topk_idx"], w, p64, SHAPE.scale)
    grads = OM.backward(go, x, f["topk_idx"], w, p64, SHAPE.scale)
    Hn.compare_all(res, out, grads, tag=f"step{bits}:")
    dl, scale = OR.backward(l, f, SHAPE.topk, True, res["grad_w"].astype(np.float64), np.array([3.0]))
    got = s.router.grad_logits.cpu().double().numpy()
    assert np.all(np.abs(got - dl) <= 2.0 ** -16 * scale + 2.0 ** -126)
    for n, m in zip(FACTORS, s.masters):
        g = Hn.f64(res["d" + n])
        want, _, _ = O8.adamw(p64[n], g, 0.0 * g, 0.0 * g, lr=LR, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=WD, step=1)
        # the update is at most lr (1 + a little); fp32 in about twenty roundings of it, two of the value
        tol = 24 * 2.0 ** -24 * LR + 4 * 2.0 ** -24 * np.abs(p64[n])
        assert np.all(np.abs(m.cpu().double().numpy().reshape(want.shape) - want) <= tol), n


def test_training_steps_captured_and_replayed():
    eager, other = Step(8), Step(8)
    control = torch.zeros(5, dtype=torch.int32, device="cuda")
    warm = Step(8)
    warm()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other(control=control)
    for step in range(1, 4):
        eager()
        other.opt.write_control(control, LR, step)
        graph.replay()
        warm()
        torch.cuda.synchronize()
        for a, b in zip(eager.results(), other.results()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), step
    del graph


def test_frozen_pass_in_8_bits():
    T, H, Id, E, k = 90, 384, 256, 6, 3
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, H, generator=g).to(BF)
    w13 = (torch.randn(E, 2 * Id, H, generator=g) * H ** -0.5).to(BF).cuda()
    w2 = (torch.randn(E, H, Id, generator=g) * Id ** -0.5).to(BF).cuda()
    q13, s13 = M.fp8_quantize_weight(w13)
    q2, s2 = M.fp8_quantize_weight(w2)
    router = M.MoeRouter(T, E, k)
    idx, w, *_ = router.forward(torch.randn(T, E, generator=g).cuda())
    desc = B.make_desc(T, 256, 256, E, k, 8)
    layer = B.MoeLoraLayer(desc)  # its pool
    layer.build_pool(idx)
    pool = layer.pool
    a, sa = M.fp8_quantize_rows(x.cuda())
    gu = M.fp8_product(pool, a, sa, q13, s13, topk=k)
    h, sh = M.fp8_quantize_rows(gu, act="swiglu")
    y = M.fp8_product(pool, h, sh, q2, s2)
    rows = pool["route_to_row"].view(T, k).long()
    out = (y[rows].float() * w[:, :, None]).sum(1).cpu().double().numpy()

    def c(t):
        return t.view(torch.uint8).cpu().numpy()

    def d(t):
        return t.double().cpu().numpy()
    ref = np.zeros((T, H))
    bound = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e, r = int(idx[t, j]), int(rows[t, j])
            up, tol = O8.product(c(a)[t:t + 1], d(sa)[t:t + 1], c(q13[e]), d(s13[e]))
            assert np.all(np.abs(d(gu)[r] - up[0]) <= tol + 2.0 ** -8 * (np.abs(up) + tol))
            v, tol = O8.product(c(h)[r:r + 1], d(sh)[r:r + 1], c(q2[e]), d(s2[e]))
            wt = float(w[t, j])
            ref[t] += wt * v[0]
            bound[t] += wt * (tol[0] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(v[0]))
    assert np.all(np.abs(out - ref) <= bound * (1 + 1e-5))

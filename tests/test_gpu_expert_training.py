"""The expert products, their gradients, the 4-bit rows and the orthogonalising
optimiser as they are used together: a layer's training step with MoeMuon on
its factors; experts trained whole over two micro-batches (products, data and
weight gradients, the optimiser), eager and as a replayed graph; a frozen
4-bit expert pass stage by stage."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from mixture_experts_grouped_amd import inputs as I
from oracle import moe_lora as OM
from oracle import mxfp4 as OMX
from oracle import products as OP
from tests import harness as Hn
from tests.test_gpu_muon import check, expect
from tests.test_gpu_product import extents, f64, half_step, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FACTORS = ("A1", "A3", "B1", "B3", "A2", "B2")
HYPER = dict(lr=0.05, momentum=0.9, nesterov=True, weight_decay=0.1, rms=0.2, eps=1e-7)  # those of `expect`


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


class LayerStep:
    """Router, layer, router gradient, MoeMuon on the six factors."""

    SHAPE = I.Shape(T=150, H=256, I=256, E=8, topk=2, rank=8)

    def __init__(self):
        s = self.SHAPE
        self.case = I.layer_inputs(s, (83,))
        self.run = Hn.GpuRun(s, self.case)
        g = torch.Generator().manual_seed(4)
        self.logits = rand(g, s.T, s.E).float()
        self.router = M.MoeRouter(s.T, s.E, s.topk)
        L = self.run.layer
        self.ts = [{"param": self.run.params[n], "grad": L.grads["d" + n], "master": self.run.params[n].float(),
                    "momentum": (torch.randn(self.run.params[n].shape, generator=g) * 1e-3).cuda()} for n in FACTORS]
        self.opt = M.MoeMuon([t["param"] for t in self.ts], [t["grad"] for t in self.ts],
                             masters=[t["master"] for t in self.ts],
                             states={"momentum": [t["momentum"] for t in self.ts]}, **HYPER)

    def grads(self):
        r = self.router
        idx, w, counts, active, _ = r.forward(self.logits)
        _, gw, _ = self.run.layer.step(idx, self.run.x, w, self.run.params, self.run.go)
        r.backward(self.logits, idx, counts, active, gw)

    def __call__(self, control=None):
        self.grads()
        self.opt.step(control=control)

    def results(self):
        return [t.clone() for t in (self.run.layer.out, self.run.layer.grad_x, self.router.grad_logits,
                                    *[t[n] for t in self.ts for n in t])]


def test_layer_step_against_the_oracles():
    s = LayerStep()
    p64 = {n: Hn.f64(s.case[n]) for n in OM.PARAM_NAMES}
    before = [{n: t[n].clone() for n in ("param", "master", "momentum")} for t in s.ts]
    s()
    res = s.run.fetch()
    x, go = Hn.f64(s.case["x"]), Hn.f64(s.case["grad_out"])
    idx, w = s.router.topk_idx.cpu().numpy(), f64(s.router.topk_w)
    Hn.compare_all(res, OM.forward(x, idx, w, p64, s.SHAPE.scale),
                   OM.backward(go, x, idx, w, p64, s.SHAPE.scale), tag="muon step:")
    for t, b in zip(s.ts, before):
        check(t, expect({**b, "grad": t["grad"]}))


def test_layer_steps_captured_and_replayed():
    eager, other, warm = LayerStep(), LayerStep(), LayerStep()
    warm()
    control = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other(control=control)
    for lr in (0.05, 0.01, 0.2):
        eager.opt.lr = lr
        eager()
        other.opt.write_control(control, lr=lr)
        graph.replay()
        warm()  # work of the same kernels between the replays
        torch.cuda.synchronize()
        for a, b in zip(eager.results(), other.results()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), lr


class ExpertStep:
    """Experts x -> x w1^T -> (x w1^T) w2^T trained whole: products, the data gradient, both weights' gradients in fp32
    added over two micro-batches, MoeMuon on the weights."""

    T, E, k, H, I = 70, 6, 2, 136, 72

    def __init__(self):
        T, E, k, H, I_ = self.T, self.E, self.k, self.H, self.I
        g = torch.Generator().manual_seed(6)
        self.desc = B.make_desc(T, 256, 256, E, k, 8)
        cap = B.moe_lora_pool_capacity(self.desc)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pool = {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
                     "route_to_row": torch.empty(T * k, **i32), "row_to_route": torch.empty(cap, **i32)}
        self.router = M.MoeRouter(T, E, k)
        self.batches = [(rand(g, T, H), rand(g, T, E).float(), rand(g, cap, H, std=0.1)) for _ in range(2)]
        self.ts = []
        for shape in ((E, I_, H), (E, H, I_)):
            m = torch.randn(*shape, generator=g) * shape[2] ** -0.5
            self.ts.append({"master": m.cuda(), "param": m.to(BF).cuda(), "grad": torch.empty(*shape, device="cuda"),
                            "momentum": (torch.randn(*shape, generator=g) * 0.1).cuda()})
        self.h, self.dh = (torch.zeros(cap, I_, dtype=BF, device="cuda") for _ in range(2))
        self.y, self.dx = (torch.zeros(cap, H, dtype=BF, device="cuda") for _ in range(2))
        self.opt = M.MoeMuon([t["param"] for t in self.ts], [t["grad"] for t in self.ts],
                             masters=[t["master"] for t in self.ts],
                             states={"momentum": [t["momentum"] for t in self.ts]}, **HYPER)
        self.kept = []

    def __call__(self, control=None, keep=False):
        (w1, g1), (w2, g2) = ((t["param"], t["grad"]) for t in self.ts)
        for i, (x, logits, dy) in enumerate(self.batches):
            idx, *_ = self.router.forward(logits)
            p = self.pool
            M.build_pool(self.desc, idx, p["counts"], p["offsets"], p["route_to_row"], p["row_to_route"])
            M.expert_product(p, x, w1, topk=self.k, out=self.h)
            M.expert_product(p, self.h, w2, out=self.y)
            M.expert_product(p, dy, w2, transposed=True, out=self.dh)
            M.expert_product(p, self.dh, w1, transposed=True, out=self.dx)
            M.expert_weight_grad(p, dy, self.h, out=g2, accumulate=i > 0)
            M.expert_weight_grad(p, self.dh, x, topk=self.k, out=g1, accumulate=i > 0)
            if keep:
                self.kept.append((extents(p), f64(self.h), f64(self.y), f64(self.dh), f64(self.dx)))
        self.opt.step(control=control)

    def results(self):
        return [t.clone() for t in (self.h, self.y, self.dh, self.dx, *[t[n] for t in self.ts for n in t])]


def test_expert_step_stage_by_stage():
    s = ExpertStep()
    w1, w2 = (f64(t["param"]) for t in s.ts)
    before = [{n: t[n].clone() for n in ("param", "master", "momentum")} for t in s.ts]
    s(keep=True)
    sums = [np.zeros_like(w1), np.zeros_like(w2)]
    tols = [np.zeros_like(w1), np.zeros_like(w2)]
    for (x, _, dy), (ext, h, y, dh, dx) in zip(s.batches, s.kept):
        x, dy = f64(x), f64(dy)
        for e, rows, routes in ext:
            xe = x[routes // s.k]
            for got, a, w in ((h, xe, w1[e]), (y, h[rows], w2[e]), (dh, dy[rows], w2[e].T), (dx, dh[rows], w1[e].T)):
                ref, tol = OP.product(a, w)
                assert np.all(np.abs(got[rows] - ref) <= half_step(ref, tol)), e
            for j, (d, a) in enumerate(((dh[rows], xe), (dy[rows], h[rows]))):
                ref, tol = OP.weight_grad(d, a)
                sums[j][e] += ref
                tols[j][e] += tol
    for t, ref, tol in zip(s.ts, sums, tols):  # two sums added in fp32: one more rounding of the total
        assert np.all(np.abs(f64(t["grad"]) - ref) <= tol + 2.0 ** -24 * (np.abs(ref) + tol))
    for t, b in zip(s.ts, before):
        check(t, expect({**b, "grad": t["grad"]}))


def test_expert_steps_captured_and_replayed():
    eager, other, warm = ExpertStep(), ExpertStep(), ExpertStep()
    warm()
    control = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other(control=control)
    g = torch.Generator().manual_seed(8)
    for lr in (0.05, 0.3, 0.01):
        for a, b in zip(eager.batches, other.batches):
            for x, y in zip(a, b):
                x.copy_(rand(g, *x.shape))
                y.copy_(x)
        eager.opt.lr = lr
        eager()
        other.opt.write_control(control, lr=lr)
        graph.replay()
        warm()
        torch.cuda.synchronize()
        pad = eager.pool["row_to_route"] < 0  # rows of no route keep what an earlier pool left: the same in both
        assert torch.equal(pad, other.pool["row_to_route"] < 0)
        for a, b in zip(eager.results(), other.results()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), lr


def test_two_expert_steps_on_two_streams():
    """Each with its own memory, at the same time: what each gives alone."""
    alone, a, b = ExpertStep(), ExpertStep(), ExpertStep()
    for _ in range(3):
        alone()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for step, stream in ((a, sa), (b, sb)):
            with torch.cuda.stream(stream):
                step()
    torch.cuda.synchronize()
    for x, y, z in zip(alone.results(), a.results(), b.results()):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_frozen_pass_in_4_bits():
    T, H, Id, E, k = 90, 384, 256, 6, 3
    g = torch.Generator().manual_seed(2)
    x = rand(g, T, H)
    w13, w2 = rand(g, E, 2 * Id, H, std=H ** -0.5), rand(g, E, H, Id, std=Id ** -0.5)
    q13, e13 = M.mxfp4_quantize_weight(w13)
    q2, e2 = M.mxfp4_quantize_weight(w2)
    router = M.MoeRouter(T, E, k)
    idx, *_ = router.forward(rand(g, T, E).float())
    layer = B.MoeLoraLayer(B.make_desc(T, 256, 256, E, k, 8))  # its pool
    layer.build_pool(idx)
    pool = layer.pool
    a, ea = M.mxfp4_quantize_rows(x)
    gu = M.mxfp4_product(pool, a, ea, q13, e13, topk=k)
    h, eh = M.mxfp4_quantize_rows(gu, act="swiglu")
    y = M.mxfp4_product(pool, h, eh, q2, e2)

    def v(c, e):
        return OMX.dequantize(c.cpu().numpy(), e.cpu().numpy())
    xv, w13v, w2v, hv = v(a, ea), v(q13, e13), v(q2, e2), v(h, eh)
    want = OMX.quantize(f64(x))
    assert np.array_equal(a.cpu().numpy(), want[0]) and np.array_equal(ea.cpu().numpy(), want[1])
    for e, rows, routes in extents(pool):
        for got, p, w in ((gu, xv[routes // k], w13v[e]), (y, hv[rows], w2v[e])):
            ref, tol = OP.product(p, w)
            assert np.all(np.abs(f64(got)[rows] - ref) <= half_step(ref, tol)), e
        # the gated value in 64 bits, within half a step of 4 bits of its block: at most a sixth of the block's largest
        # (from 4 to 6 the codes lie 2 apart; larger values are cut by a fourth at most), and fp32's error of the gate
        gate, up = np.split(f64(gu)[rows], 2, axis=1)
        ref = gate / (1 + np.exp(-gate)) * up
        top = np.abs(ref).reshape(len(rows), -1, 32).max(2).repeat(32, 1)
        assert np.all(np.abs(hv[rows] - ref) <= 0.25 * top * (1 + 1e-5)), e

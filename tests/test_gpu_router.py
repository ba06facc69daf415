"""The router's forward and backward against the float64 oracle: ties, closed
experts, padding tokens, empty roots, NaN and infinite logits, every expert
count class, one token to several chunks."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from oracle import router as OR
from tests import harness as Hn

pytestmark = pytest.mark.gpu

# A weight or a mean probability is e^(l - max) over a sum of such terms.  With
# |l - max| <= 30: the exponent l - max and its product with log2 e are each
# rounded (2 * 30 * 2^-24, relative to the result), the exponential is off by
# 2^-23, the sum over at most 32 values a lane and 16 lanes by 36 * 2^-24, the
# reciprocal and the product by 3 * 2^-24, the mean over tokens by another few:
# below 128 * 2^-24.
REL = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def make(T, E, dtype, seed, cut=0.0, mask=0.0, grid=None):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2
    if grid:  # few distinct values: ties
        l = torch.round(l * grid) / grid
    if cut:
        l[torch.rand(T, E, generator=g) < cut] = -np.inf
    l = l.to(dtype)
    valid = (torch.rand(T, generator=g) >= mask).to(torch.uint8) if mask else None
    return l, valid, torch.randn(T, 16, generator=g), torch.randn(8, generator=g)


def check(l, valid, k, renorm, roots, gw, gl, dev="cuda"):
    T, E = l.shape
    na = 1 if roots is None else len(roots) - 1
    r = M.MoeRouter(T, E, k, dtype=l.dtype, renorm=renorm, roots=roots, device=dev)
    for b in (r.topk_idx, r.topk_w, r.counts, r.active, r.loss, r.device_error, r.workspace, r.grad_logits):
        b.view(torch.uint8).fill_(0xFF)
    ld = l.to(dev)
    vd = None if valid is None else valid.to(dev)
    idx, w, counts, active, loss = r.forward(ld, vd)
    o = OR.forward(l.double().numpy(), k, renorm, roots, None if valid is None else valid.numpy())
    assert np.array_equal(idx.cpu().numpy(), o["topk_idx"])
    assert np.array_equal(counts.cpu().numpy(), o["counts"])
    assert np.array_equal(active.cpu().numpy(), o["active"])
    assert int(r.device_error) == o["bad"]
    assert np.all(np.abs(w.cpu().double().numpy() - o["topk_w"]) <= REL * o["topk_w"])
    assert np.all(np.abs(loss.cpu().double().numpy() - o["loss"]) <= REL * o["loss"])
    gw = gw[:, :k].contiguous()
    gl = gl[:na].contiguous()
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        ref, scale = OR.backward(l.double().numpy(), o, k, renorm, gw.double().numpy() if use_w else None,
                                 gl.double().numpy() if use_l else None, roots)
        got = r.backward(ld, idx, counts, active, gw.to(dev) if use_w else None, gl.to(dev) if use_l else None, vd)
        got = got.cpu().double().numpy()
        out = 2.0 ** -8 if l.dtype == torch.bfloat16 else 0.0  # the output's own rounding
        # every term is a product of quantities with relative error REL, summed in fp32;
        # the last term: fp32's and bf16's smallest normal value
        assert np.all(np.abs(got - ref) <= 2 * REL * scale + out * (np.abs(ref) + 2 * REL * scale) + 2.0 ** -126)
    return r


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 5, 5), (65, 16, 2), (130, 63, 6), (64, 65, 8), (70, 128, 1),
                                   (33, 250, 16), (200, 257, 4), (17, 512, 16)])
def test_router_shapes(T, E, k, dtype, renorm):
    l, _, gw, gl = make(T, E, dtype, T + E)
    check(l, None, k, renorm, None, gw, gl)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_roots_padding_and_closed_experts(dtype):
    l, valid, gw, gl = make(300, 40, dtype, 9, cut=0.3, mask=0.3)
    check(l, valid, 6, True, [0, 100, 100, 101, 300], gw, gl)
    check(l, valid, 6, False, [0, 0, 170, 300], gw, gl)


def test_router_ties_and_signed_zero():
    l, _, gw, gl = make(90, 70, torch.float32, 4, grid=2)
    l[5] = 0.0
    l[5, ::2] = -0.0  # equal to +0: experts 0, 1, 2, ...
    r = check(l, None, 6, True, None, gw, gl)
    assert r.topk_idx[5].tolist() == [0, 1, 2, 3, 4, 5]


def test_router_rows_that_leave_nothing():
    l, valid, gw, gl = make(40, 9, torch.float32, 6, mask=0.2)
    low = torch.finfo(torch.float32).min
    l[0] = -np.inf                 # nothing open
    l[1] = -np.inf
    l[1, 7] = 3.0                  # one expert for four routes
    l[2] = low                     # the type's lowest value everywhere: uniform
    l[3] = low
    l[3, 2] = 0.0                  # the lowest value beside an ordinary one: chosen, weight 0
    l[4, 3] = np.nan
    l[5, 0] = np.inf
    l[6] = np.nan
    l[7, :] = torch.tensor([88.0] * 8 + [-88.0])
    valid[:8] = 1
    valid[8] = 0
    l[8, 1] = np.nan               # a NaN in a padding token is nobody's error
    r = check(l, valid, 4, True, None, gw, gl)
    assert int(r.device_error) == 3 and r.dropped_tokens() == 3
    assert not r.grad_logits[[0, 4, 5, 6, 8]].any()
    check(l, valid, 4, False, None, gw, gl)
    with pytest.raises(FloatingPointError):
        M.MoeRouter(40, 9, 4, checked=True).forward(l.cuda())
    all_out = torch.zeros(40, dtype=torch.uint8)
    r = check(l, all_out, 4, True, [0, 7, 40], gw, gl)
    assert not r.counts.any() and not r.loss.any()


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_where_there_is_no_route(renorm):
    """The weights' gradient at ids of -1 is whatever its buffer holds."""
    l, valid, gw, gl = make(60, 12, torch.float32, 14, cut=0.7, mask=0.2)
    r = check(l, valid, 6, renorm, None, gw, gl)
    none = r.topk_idx.cpu() < 0
    assert none.any() and not none.all()
    clean = gw[:, :6].contiguous()
    ld, vd, gld = l.cuda(), valid.cuda(), gl[:1].cuda()
    args = ld, r.topk_idx, r.counts, r.active
    want = r.backward(*args, clean.masked_fill(none, 0).cuda(), gld, vd).clone()
    for x in (np.nan, np.inf, -np.inf):
        assert torch.equal(r.backward(*args, clean.masked_fill(none, x).cuda(), gld, vd), want)


def test_router_gradient_of_more_tokens_than_workgroups():
    """Past 2^24 tokens a workgroup takes several rounds.  One expert: p = w = 1,
    so the gradient is exactly 0; NaN tokens too."""
    T = (1 << 24) + 5
    r = M.MoeRouter(T, 1, 1)
    l = torch.zeros(T, 1, device="cuda")
    l[::1000003] = float("nan")
    idx, w, counts, active, loss = r.forward(l)
    bad = len(range(0, T, 1000003))
    assert int(counts) == int(active) == T - bad and r.dropped_tokens() == bad
    r.grad_logits.fill_(float("nan"))
    r.backward(l, idx, counts, active, torch.ones(T, 1, device="cuda"), torch.ones(1, device="cuda"))
    assert not r.grad_logits.any()


def test_router_gradient_in_place_and_repeatable():
    l, valid, gw, gl = make(500, 64, torch.float32, 3, mask=0.1)
    r = check(l, valid, 6, True, None, gw, gl)
    ld, vd, gwd, gld = l.cuda(), valid.cuda(), gw[:, :6].contiguous().cuda(), gl[:1].cuda()
    idx, w, counts, active, loss = [t.clone() for t in r.forward(ld, vd)]
    g0 = r.backward(ld, idx, counts, active, gwd, gld, vd).clone()
    for _ in range(3):
        again = r.forward(ld, vd)
        assert all(torch.equal(a, b) for a, b in zip(again, (idx, w, counts, active, loss)))
        r.grad_logits = ld.clone()  # the logits' own buffer
        assert torch.equal(r.backward(r.grad_logits, idx, counts, active, gwd, gld, vd), g0)


def test_router_by_differences():
    """The gradient against central differences of the fp32 forward: step h,
    truncation h^2 and rounding 2^-24 / h of values near 1."""
    T, E, k = 3, 8, 2
    l, _, gw, gl = make(T, E, torch.float32, 12)
    r = M.MoeRouter(T, E, k, renorm=True)
    ld, gwd, gld = l.cuda(), gw[:, :k].contiguous().cuda(), gl[:1].cuda()
    idx, w, counts, active, loss = [t.clone() for t in r.forward(ld)]
    grad = r.backward(ld, idx, counts, active, gwd, gld).cpu()

    def value(x):
        _, w, _, _, loss = r.forward(x.cuda())
        return float((w.double() * gwd.double()).sum() + (loss.double() * gld.double()).sum())
    h = 2.0 ** -7
    size = float(gwd.abs().sum() + gld.abs().sum())
    for t in range(T):
        for e in range(E):
            d = torch.zeros(T, E)
            d[t, e] = h
            r2 = r.forward((l + d).cuda())[0].clone(), r.forward((l - d).cuda())[0].clone()
            if not (torch.equal(r2[0], idx) and torch.equal(r2[1], idx)):
                continue  # the step crosses a change of choice
            assert abs((value(l + d) - value(l - d)) / (2 * h) - float(grad[t, e])) <= size * (h * h + REL / h)


def test_router_on_another_stream_and_in_a_graph():
    l, valid, gw, gl = make(700, 64, torch.bfloat16, 8, mask=0.1)
    ld, vd, gwd, gld = l.cuda(), valid.cuda(), gw[:, :6].contiguous().cuda(), gl[:1].cuda()
    r = M.MoeRouter(700, 64, 6, dtype=torch.bfloat16)
    want = [t.clone() for t in r.forward(ld, vd)]
    want.append(r.backward(ld, want[0], want[2], want[3], gwd, gld, vd).clone())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = r.forward(ld, vd, stream=s)
    r.backward(ld, got[0], got[2], got[3], gwd, gld, vd, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip((*got, r.grad_logits), want))
    noise = M.MoeRouter(700, 64, 6, dtype=torch.bfloat16)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = r.forward(ld, vd)
        r.backward(ld, got[0], got[2], got[3], gwd, gld, vd)
    for _ in range(3):
        for b in (*got, r.grad_logits):
            b.view(torch.uint8).fill_(0xFF)
        noise.forward(torch.flip(ld, [0]))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, r.grad_logits), want))
    del g


def test_router_writes_its_own_buffers_only():
    """The results are the buffers made with the router, also where an attribute
    has been given another tensor since; their memory is not another's."""
    T, E, k = 4096, 64, 6
    l, _, _, _ = make(T, E, torch.float32, 31)
    r, ref = M.MoeRouter(T, E, k), M.MoeRouter(T, E, k)
    want = [t.clone() for t in ref.forward(l.cuda())]
    names = ("topk_idx", "topk_w", "counts", "active", "loss", "device_error", "workspace")
    for n in names:
        setattr(r, n, torch.zeros_like(getattr(r, n)))
    shapes = [(getattr(r, n).shape, getattr(r, n).dtype) for n in names]
    others = [torch.full(s, 7, dtype=dt, device="cuda") for s, dt in shapes]
    got = r.forward(l.cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 7).all() for t in others)
    for n in names[:5]:
        assert not getattr(r, n).any()
    idx, _, counts, active, _ = got
    for other in (torch.zeros(T - 1, E), torch.zeros(T, E, dtype=torch.bfloat16), torch.zeros(E, T).t()):
        r.grad_logits = other.cuda()
        with pytest.raises(ValueError, match="grad_logits"):
            r.backward(l.cuda(), idx, counts, active)


@pytest.mark.parametrize("T,roots", [(1 << 27, None), ((1 << 22) + 3, None), (1 << 26, [0, 5, 5, (1 << 25) + 77, 1 << 26])])
def test_router_loss_of_very_many_tokens(T, roots):
    """Tokens that are all alike: p = (1/7, 4/7, 2/7), every route on expert 1,
    so the loss is 3 * 4/7 whatever their number.  No sum may grow so long in
    fp32 that its roundings, which are alike too, add up past REL."""
    l = torch.tensor([0.0, 2.0, 1.0]) * float(np.log(2.0))
    r = M.MoeRouter(T, 3, 1, roots=roots)
    idx, w, counts, active, loss = r.forward(l.cuda().expand(T, 3).contiguous())
    sizes = np.diff(roots or [0, T])
    assert active.tolist() == sizes.tolist() and counts[:, 1].tolist() == sizes.tolist()
    assert not counts[:, 0].any() and not counts[:, 2].any() and (idx == 1).all() and r.dropped_tokens() == 0
    want = np.where(sizes > 0, 12 / 7, 0.0)
    assert np.all(np.abs(loss.cpu().double().numpy() - want) <= REL * want), loss

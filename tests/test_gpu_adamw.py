"""The AdamW step against float64: parameter, gradient and state types, odd
lengths and many tensors, the 8-bit states' codes and scales, non-finite
gradients, device-side control values in a replayed graph."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from oracle import float8 as O8
from tests import harness as Hn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HYPER = dict(betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)
# fp32 moments: two products and a sum of terms of the same order, three
# roundings, the betas' own rounding to fp32: within 4 * 2^-24 of the terms'
# magnitudes.  The update: sqrt, two quotients, a few products: 16 * 2^-24 of it.
MOM, UPD = 4 * 2.0 ** -24, 16 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def tensors(sizes, ptype, gtype, seed):
    g = torch.Generator().manual_seed(seed)
    ps = [torch.randn(n, generator=g).to(ptype).cuda() for n in sizes]
    gs = [(torch.randn(n, generator=g) * torch.exp(torch.randn(n, generator=g))).to(gtype).cuda() for n in sizes]
    return ps, gs


def f64(t):
    return t.detach().double().cpu().numpy()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def values8(opt, i, name):
    fmt = "e4m3" if name == "m" else "e5m2"
    s = f64(opt.states[name + "_scale"][i])
    c = codes(opt.states[name][i]).reshape(-1)
    return O8.decode(c, fmt) * np.repeat(s, 128)[:c.size]


SIZES = [1, 7, 8, 127, 128, 129, 2048, 2049, 5000, 40960]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ptype,gtype,master", [(BF, BF, True), (BF, BF, False), (BF, F32, True), (BF, F32, False),
                                                (F32, F32, False), (F32, BF, False)])
def test_steps(ptype, gtype, master, bits):
    ps, gs = tensors(SIZES, ptype, gtype, 1)
    masters = [p.float() for p in ps] if master else None
    opt = M.MoeAdamW(ps, gs, masters=masters, state_bits=bits, lr=1e-2, **HYPER)
    for step in range(1, 4):
        before = [f64(t) for t in (masters or ps)]
        if bits == 32:
            m0, v0 = [f64(t) for t in opt.states["m"]], [f64(t) for t in opt.states["v"]]
        else:
            m0, v0 = ([values8(opt, i, n) for i in range(len(ps))] for n in "mv")
        opt.step(grad_scale=0.5)
        for i, n in enumerate(SIZES):
            g = f64(gs[i])
            p, m, v = O8.adamw(before[i], g, m0[i], v0[i], lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1,
                               step=step, grad_scale=0.5)
            # the update feels the moments' errors (m may cancel) and v's by its root
            mterm = 0.9 * np.abs(m0[i]) + 0.1 * np.abs(0.5 * g)
            upd = 1e-2 * mterm / (1 - 0.9 ** step) / (np.sqrt(v / (1 - 0.99 ** step)) + 1e-6)
            tol = (UPD + 2 * MOM) * upd + 4 * 2.0 ** -24 * np.abs(before[i])
            got = f64((masters or ps)[i])
            if not master and ptype == BF:
                tol = tol + 2.0 ** -8 * (np.abs(p) + tol)
            assert np.all(np.abs(got - p) <= tol + 2.0 ** -126)
            if master:
                assert torch.equal(ps[i], masters[i].to(BF))
            if bits == 32:
                assert np.all(np.abs(f64(opt.states["m"][i]) - m) <= MOM * mterm + 2.0 ** -149)
                assert np.all(np.abs(f64(opt.states["v"][i]) - v) <= MOM * v + 2.0 ** -149)
                continue
            rnd = O8.noise(n, step)
            for name, x, xt, r, fmt, man in (("m", m, mterm, rnd & 0xFFFF, "e4m3", 3), ("v", v, v, rnd >> np.uint64(16), "e5m2", 2)):
                want, scale = O8.moments8(x, r.astype(np.float64), fmt)
                gs_ = f64(opt.states[name + "_scale"][i])
                # the run's largest |moment|: its fp32 error, and the quotient's
                big = np.array([xt[128 * q:128 * q + 128].max() for q in range(len(scale))]) / O8.FORMATS[fmt][1]
                assert np.all(np.abs(gs_ - scale) <= 2 * MOM * big + 2.0 ** -23 * scale)
                have = codes(opt.states[name][i]).reshape(-1)
                same = have == want
                # where fp32 crosses a cut the code is the neighbour: rare, and one step away
                assert np.mean(~same) <= 1e-3 or (~same).sum() <= 1
                per = np.repeat(scale, 128)[:n]
                a, b = O8.decode(have, fmt) * per, O8.decode(want, fmt) * per
                low = 2.0 ** (-9 if fmt == "e4m3" else -16) * per
                assert np.all(np.abs(a - b) <= np.maximum(np.abs(a), np.abs(b)) * 2.0 ** -man * (1 + 1e-5) + low)
                if name == "v":
                    assert np.all((have == 0) == (v == 0))


def test_rounding_follows_the_seed_and_repeats():
    def run(seed):
        ps, gs = tensors([4096], BF, BF, 2)
        opt = M.MoeAdamW(ps, gs, state_bits=8)
        opt.step(seed=seed)
        return codes(opt.states["m"][0]), codes(opt.states["v"][0]), f64(ps[0])
    a, b, c = run(5), run(5), run(6)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    assert not np.array_equal(a[0], c[0]) and not np.array_equal(a[1], c[1]) and np.array_equal(a[2], c[2])


def test_small_decay_is_not_lost_in_8_bits():
    """v under a vanished gradient: 300 steps of 0.99 leave 0.049 of it.  Each
    code is right on the mean; a run's largest value is held exactly.  The
    mean of 4,064 codes, each rounded 300 times (a spread of a quarter of the
    value at most, summed over an average of 100 remembered roundings each
    hitting with the decay's share 0.01 / 0.25 of a code), is within 5 %."""
    n = 4096
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 1.0, device="cuda")
    g[1::2] = 0.5
    opt = M.MoeAdamW([p], [g], state_bits=8, betas=(0.9, 0.99))
    opt.step()
    v1 = values8(opt, 0, "v")
    g.zero_()
    for _ in range(300):
        opt.step(lr=0.0)
    v2 = values8(opt, 0, "v")
    assert abs(v2[::2].mean() / (v1[::2].mean() * 0.99 ** 300) - 1) < 0.05
    assert abs(v2[1::2].mean() / (0.0025 * 0.99 ** 300) - 1) < 0.05


def test_many_tensors_and_views_leave_neighbours_alone():
    flat = torch.full((130 * 256,), 7.0, device="cuda")
    grads = torch.ones(130, 200, device="cuda")
    ps = [flat[256 * i:256 * i + 197] for i in range(130)] + [flat[:0]]
    gs = [grads[i, :].clone()[:197] for i in range(130)] + [grads[0, :0]]
    opt = M.MoeAdamW(ps, gs, lr=0.5, eps=1e-8)
    opt.step()
    view = flat.view(130, 256)
    assert (view[:, 197:] == 7.0).all()
    assert torch.allclose(view[:, :197], torch.full_like(view[:, :197], 6.5), rtol=1e-6)


def test_nonfinite_gradients_stay_in_their_run():
    ps, gs = tensors([1024], F32, F32, 4)
    gs[0][130], gs[0][700] = float("nan"), float("inf")
    keep = ps[0].clone()
    opt = M.MoeAdamW(ps, gs, state_bits=8)
    opt.step()
    m, v = values8(opt, 0, "m"), values8(opt, 0, "v")
    bad = np.zeros(1024, bool)
    bad[128:256] = bad[640:768] = True
    assert not np.isfinite(m[bad]).any() and not np.isfinite(v[bad]).any()
    assert np.isfinite(m[~bad]).all() and np.isfinite(v[~bad]).all()
    assert torch.isfinite(ps[0]).sum() >= 1022 and not torch.equal(keep, ps[0])


def test_tiny_and_zero_moments():
    g = torch.zeros(256, device="cuda")
    g[128:] = 1e-25
    p = torch.ones(256, device="cuda")
    opt = M.MoeAdamW([p], [g], state_bits=8)
    for _ in range(3):
        opt.step()
    assert torch.equal(p, torch.ones_like(p)) and np.isfinite(values8(opt, 0, "m")).all()
    assert not values8(opt, 0, "v").any()  # 1e-50: below the smallest scale


def test_control_in_a_replayed_graph():
    def fresh():
        ps, gs = tensors([3000, 129], BF, BF, 6)
        return ps, gs, M.MoeAdamW(ps, gs, masters=[p.float() for p in ps], state_bits=8, **HYPER)
    ps, gs, opt = fresh()
    qs, hs, other = fresh()
    control = torch.zeros(5, dtype=torch.int32, device="cuda")
    warm = M.MoeAdamW([torch.zeros(8, device="cuda")], [torch.zeros(8, device="cuda")])
    warm.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step(control=control)
    for step in range(1, 5):
        lr = 1e-2 / step
        opt.step(lr=lr, step=step, seed=step * 7, grad_scale=0.25)
        other.write_control(control, lr, step, grad_scale=0.25, seed=step * 7)
        warm.step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ps + opt.masters + opt.states["m"] + opt.states["v_scale"],
                        qs + other.masters + other.states["m"] + other.states["v_scale"]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del graph


def test_goes_on_from_given_states_on_another_stream():
    ps, gs = tensors([500, 300], F32, BF, 9)
    qs = [p.clone() for p in ps]
    a = M.MoeAdamW(ps, gs, state_bits=8)
    a.step()
    a.step()
    b = M.MoeAdamW(qs, gs, state_bits=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.step(stream=s)
    c = M.MoeAdamW(qs, gs, state_bits=8, states=b.states)
    c.step(step=2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(ps, qs))


def test_refused_steps_and_shared_memory():
    ps, gs = tensors([100, 300], F32, F32, 21)
    opt = M.MoeAdamW(ps, gs)
    opt.step()
    with pytest.raises(M.MoeLoraError):
        opt.step(lr=-1.0)
    assert opt.steps == 1  # a refused step is not counted
    M.MoeAdamW(ps, [gs[1][:100], gs[1]])  # gradients are only read
    p = torch.zeros(512, device="cuda")
    for params, grads in (([ps[0], ps[0]], [gs[0], gs[0]]), ([p[:300], p[256:]], [gs[1], gs[0].repeat(3)[:256]]),
                          ([p[:256], ps[0]], [p[256:], p[200:300]])):
        with pytest.raises(ValueError):
            M.MoeAdamW(params, grads)


def test_control_values_are_checked():
    ps, gs = tensors([8], F32, F32, 22)
    opt, c = M.MoeAdamW(ps, gs), torch.zeros(5, dtype=torch.int32, device="cuda")
    for kw in (dict(lr=1e-3, step=0), dict(lr=-1.0, step=1), dict(lr=np.nan, step=1), dict(lr=1.0, step=1, grad_scale=np.inf)):
        with pytest.raises(ValueError):
            opt.write_control(c, **kw)
    assert not c.any()


def test_more_elements_than_32_bits_count():
    n, tail = 2 ** 31 + 517, 5000
    g = torch.Generator().manual_seed(5)
    p, gr = torch.randn(tail, generator=g).to(BF).cuda(), torch.randn(tail, generator=g).to(BF).cuda()
    big, grad = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))
    big[-tail:], grad[-tail:] = p, gr
    opt, ref = M.MoeAdamW([big], [grad], lr=1e-2), M.MoeAdamW([p], [gr], lr=1e-2)
    opt.step()
    ref.step()
    assert torch.equal(big[-tail:], p) and torch.equal(opt.states["v"][0][-tail:], ref.states["v"][0])
    assert not big[:2 ** 20].any()


def low_run(ratio):
    """Gradients of 512 runs: the first element of each 1, the others `ratio`."""
    g = torch.full((128 * 512,), ratio, device="cuda")
    g[::128] = 1.0
    return g, np.arange(128 * 512) % 128 != 0


@pytest.mark.parametrize("name,ratio", [("m", 1e-5), ("m", 3e-6), ("m", 1e-6), ("v", 3e-5), ("v", 2e-5)])
def test_moments_far_below_their_runs_largest_are_right_on_the_mean(name, ratio):
    """Below the formats' normal range (m 3.5e-5, v 1.1e-9 of the largest) the
    codes are whole steps of 2^-9 or 2^-16, taken up or down at random: one
    rounding's variance is at most a quarter of a squared step, and the mean of
    65,024 of them stays within five of its deviations (and fp32's own
    roundings of the moment and of its quotient)."""
    g, rest = low_run(ratio)
    opt = M.MoeAdamW([torch.zeros_like(g)], [g], state_bits=8, betas=(0.9, 0.99))
    opt.step()
    want = 0.1 * ratio if name == "m" else 0.01 * ratio ** 2
    step = (2.0 ** -9 if name == "m" else 2.0 ** -16) * float(opt.states[name + "_scale"][0][0])
    got = values8(opt, 0, name)[rest]
    assert 0.1 < want / step < 8 and got.min() <= want <= got.max() and got.max() - got.min() <= step * (1 + 1e-6)
    assert abs(got.mean() - want) <= 5 * 0.5 * step / np.sqrt(rest.sum()) + 8 * 2.0 ** -24 * want


def test_first_moments_far_below_their_runs_largest_decay():
    """A gradient that ends: eleven steps of 0.9 later the mean is 0.9^11 of
    what it was, within five deviations of the roundings' sum (each at most a
    quarter of a squared step, the older ones decayed: in all at most 1/4 / (1
    - 0.81) squared steps of the last scale, the scales only grow)."""
    g, rest = low_run(2e-5)
    opt = M.MoeAdamW([torch.zeros_like(g)], [g], state_bits=8, betas=(0.9, 0.99))
    opt.step()
    g[torch.from_numpy(rest).cuda()] = 0.0
    for _ in range(11):
        opt.step()
    step = 2.0 ** -9 * float(opt.states["m_scale"][0][0])
    got, want = values8(opt, 0, "m")[rest].mean(), 2e-6 * 0.9 ** 11
    assert abs(got - want) <= 5 * np.sqrt(0.25 / 0.19) * step / np.sqrt(rest.sum())


def test_the_smallest_second_moments_keep_the_lowest_code():
    g, rest = low_run(1e-6)
    opt = M.MoeAdamW([torch.zeros_like(g)], [g], state_bits=8)
    for _ in range(5):
        opt.step()
        assert (codes(opt.states["v"][0])[rest] == 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_small_weight_decay_of_one_step(bits):
    """lr weight_decay = 1e-7 of values in [1, 2): 0.84 to 1.7 of their last
    place.  The change is exact to a few fp32 roundings of itself, so the
    result is the rounding of the exact one (half a place, 2^-24)."""
    p = (1 + torch.rand(1 << 16, generator=torch.Generator().manual_seed(3))).cuda()
    before = f64(p)
    M.MoeAdamW([p], [torch.zeros_like(p)], state_bits=bits, lr=1e-5, weight_decay=0.01).step()
    want = before * (1 - 1e-7)
    assert np.all(np.abs(f64(p) - want) <= 2.0 ** -24 + 4 * 2.0 ** -24 * 1e-7 * before)


def test_small_weight_decay_over_many_steps():
    """lr weight_decay = 2e-8, a sixth to a third of half a place, beside
    updates of many places: each step's rounding is up or down at random, so
    the mean of 65,536 elements over 200 steps is off by five deviations of
    their sum, 5 * 2^-23 / sqrt(12) * sqrt(200 / 65536) = 0.08 * 2^-23, and by
    the updates' own relative error, at most 24 * 2^-24 of 200 * lr in magnitude
    (each is lr m / sqrt(v), at most a few lr).  A decay that is left out is 33 places off."""
    n, lr, wd = 1 << 16, 2e-6, 0.01
    g = torch.Generator(device="cuda").manual_seed(7)
    p, grad = 1 + torch.rand(n, generator=g, device="cuda"), torch.zeros(n, device="cuda")
    q, m, v = p.double(), torch.zeros(n, device="cuda").double(), torch.zeros(n, device="cuda").double()
    opt = M.MoeAdamW([p], [grad], lr=lr, betas=(0.9, 0.99), weight_decay=wd)
    for step in range(1, 201):
        grad.normal_(generator=g)
        opt.step()
        m = 0.9 * m + 0.1 * grad.double()
        v = 0.99 * v + 0.01 * grad.double().square()
        q = q - lr * wd * q - lr * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
    off = float((p.double() - q).mean())
    assert abs(off) <= 0.08 * 2.0 ** -23 + 24 * 2.0 ** -24 * 200 * 4 * lr


def test_memory_replaced_after_construction_stays_the_optimisers():
    """`p.data = ...` leaves the optimiser with the memory it was made for: it
    is not handed to another tensor while the optimiser writes it."""
    n = 1 << 20
    p, grad, master = torch.zeros(n, dtype=BF, device="cuda"), torch.ones(n, dtype=BF, device="cuda"), torch.zeros(n, device="cuda")
    opt = M.MoeAdamW([p], [grad], masters=[master], state_bits=8, lr=0.5)
    held = {t.data_ptr() for t in (p, grad, master)}
    for t in (p, grad, master):
        t.data = torch.zeros_like(t)
    others = [torch.full((n,), 7.0, dtype=dt, device="cuda") for dt in (BF, BF, F32)]
    assert not held & {t.data_ptr() for t in others}
    opt.step()
    assert all((t == 7.0).all() for t in others) and not any(t.any() for t in (p, grad, master))


def test_control_values_beyond_fp32_and_wrong_buffers():
    ps, gs = tensors([8], F32, F32, 22)
    opt, c = M.MoeAdamW(ps, gs), torch.zeros(5, dtype=torch.int32, device="cuda")
    for kw in (dict(lr=1e39, step=1), dict(lr=1.0, step=1, grad_scale=-1e39), dict(lr=1.0, step=-1)):
        with pytest.raises(ValueError, match="write_control"):
            opt.write_control(c, **kw)
    for other in (c.float(), c.long(), torch.zeros(6, dtype=torch.int32, device="cuda"), c[None].clone()):
        with pytest.raises(ValueError, match="control"):
            opt.write_control(other, 1e-3, 1)
        assert not other.any()
    opt.write_control(c, 0.25, 3, grad_scale=0.5, seed=1 << 31)
    f = c[:4].view(torch.float32).tolist()
    assert f[0] == 0.25 and f[3] == 0.5 and abs(f[1] - 0.271) < 1e-6 and int(c[4]) == -(1 << 31)

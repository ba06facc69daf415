"""The float64 oracles of the router, the 8-bit formats and the optimiser step
pinned to other routes to the same numbers: torch autograd, finite
differences, hand-worked values and torch's own 8-bit types."""
import numpy as np
import pytest
import torch

from oracle import float8 as O8
from oracle import router as OR


def test_router_by_hand():
    """Two tokens, three experts: logits ln of 1, 2, 1 and 4, 2, 2."""
    l = np.log(np.array([[1.0, 2.0, 1.0], [4.0, 2.0, 2.0]]))
    o = OR.forward(l, 2, False)
    assert o["topk_idx"].tolist() == [[1, 0], [0, 1]]  # the tie goes to the lower expert
    assert np.allclose(o["topk_w"], [[0.5, 0.25], [0.5, 0.25]])
    assert o["counts"].tolist() == [[2, 2, 0]] and o["active"].tolist() == [2]
    # E / (k n^2) = 3/8, masses .75, .75, .5
    assert np.isclose(o["loss"][0], 3 / 8 * (2 * 0.75 + 2 * 0.75))
    r = OR.forward(l, 2, True)
    assert np.allclose(r["topk_w"], [[2 / 3, 1 / 3], [2 / 3, 1 / 3]])


def test_router_drops():
    inf, nan = np.inf, np.nan
    l = np.array([[0.0, -inf, -inf], [-inf, -inf, -inf], [0.0, nan, 1.0], [inf, 0.0, 0.0], [1.0, 1.0, 1.0]])
    o = OR.forward(l, 2, True, valid=np.array([1, 1, 1, 1, 0]))
    assert o["topk_idx"].tolist() == [[0, -1], [-1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert o["topk_w"].tolist()[0] == [1.0, 0.0] and o["bad"] == 2 and o["active"].tolist() == [1]


def test_balanced_routing_has_loss_one():
    l = np.full((8, 4), -1.0)
    for t in range(8):
        l[t, [t % 4, (t + 1) % 4]] = 1.0
    assert np.isclose(OR.forward(l, 2, True)["loss"][0], 1.0)


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_by_autograd_and_differences(renorm):
    g = np.random.default_rng(5)
    T, E, k, roots = 11, 7, 3, [0, 4, 4, 11]
    l = g.standard_normal((T, E))
    l[2, :5] = -np.inf
    gw, gl = g.standard_normal((T, k)), g.standard_normal(3)
    f = OR.forward(l, k, renorm, roots)
    grad, scale = OR.backward(l, f, k, renorm, gw, gl, roots)
    t = torch.tensor(l, requires_grad=True)
    p = torch.softmax(t, 1)
    idx = torch.tensor(f["topk_idx"]).long()
    w = p.gather(1, idx.clamp(min=0)) * (idx >= 0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    loss = (w * torch.tensor(gw)).sum()
    for a in range(3):
        n = max(1, int(f["active"][a]))
        loss = loss + gl[a] * E / (k * n * n) * (torch.tensor(f["counts"][a]) * p[roots[a]:roots[a + 1]].sum(0)).sum()
    loss.backward()
    assert np.allclose(np.nan_to_num(t.grad.numpy()), grad, rtol=1e-12, atol=1e-14)
    assert (np.abs(grad) <= scale * (1 + 1e-12)).all()

    def value(x):
        h = OR.forward(x, k, renorm, roots)
        return float((h["topk_w"] * gw).sum() + (h["loss"] * gl).sum())
    for t_, e in [(0, 0), (3, 6), (7, 2), (10, 5)]:
        d = np.zeros_like(l)
        d[t_, e] = 1e-6
        assert abs((value(l + d) - value(l - d)) / 2e-6 - grad[t_, e]) < 1e-7


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_formats_equal_torchs(fmt, dtype):
    codes = np.arange(256, dtype=np.uint8)
    ours = O8.decode(codes, fmt)
    theirs = torch.from_numpy(codes).view(dtype).float().numpy()
    fine = np.isfinite(theirs)
    assert np.array_equal(ours[fine], theirs[fine])
    top = O8.FORMATS[fmt][1]
    y = np.concatenate([np.random.default_rng(1).uniform(-top, top, 4000), ours[fine],
                        (np.sort(ours[fine])[1:] + np.sort(ours[fine])[:-1]) / 2])  # values, ties
    y = y.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(y.astype(np.float32)).to(dtype).view(torch.uint8).numpy()
    got = O8.nearest(y, fmt)
    assert np.array_equal(O8.decode(got, fmt), O8.decode(want, fmt))


def test_moments_round_without_bias():
    """A code's mean over the noise is the value (normal range)."""
    x = np.full(1 << 16, 0.3)
    x[0] = 1.0  # the run's largest
    for fmt in ("e4m3", "e5m2"):
        runs = x.reshape(-1, 128).copy()
        runs[:, 0] = 1.0
        c, s = O8.moments8(runs.reshape(-1), np.arange(1 << 16), fmt)
        v = (O8.decode(c, fmt) * np.repeat(s, 128)).reshape(-1, 128)[:, 1:]
        assert abs(v.mean() - 0.3) < 1e-3 and len(np.unique(v)) == 2
        assert np.allclose(O8.decode(c, fmt).reshape(-1, 128)[:, 0], O8.FORMATS[fmt][1])


def test_moments_below_the_normal_range_round_without_bias():
    """Over all 2^16 noise values the mean is the value to 2^-16 of a step."""
    for fmt, low in (("e4m3", 2.0 ** -9), ("e5m2", 2.0 ** -16)):
        top = O8.FORMATS[fmt][1]
        for steps in (1.0, 1.3, 2.29, 3.6, 7.9):
            x = np.full((1 << 16, 128), steps * low / top)
            x[:, 0] = 1.0
            c, s = O8.moments8(x.reshape(-1), np.repeat(np.arange(1 << 16), 128), fmt)
            v = (O8.decode(c, fmt).reshape(-1, 128) / low)[:, 1]
            assert abs(v.mean() - steps) <= 2.0 ** -16 and set(v) <= {np.floor(steps), np.ceil(steps)}
    x = np.zeros(128)
    x[:3] = 448.0, 0.229 * 2.0 ** -9, -0.229 * 2.0 ** -9
    up = np.array([O8.decode(O8.moments8(x, np.full(128, r), "e4m3")[0], "e4m3")[1:3] for r in range(0, 1 << 16, 7)])
    assert abs(up[:, 0].mean() / 2.0 ** -9 - 0.229) < 1e-3 and np.array_equal(up[:, 1], -up[:, 0])


def test_positive_second_moment_keeps_a_code():
    x = np.concatenate([[1.0], np.full(127, 1e-12), [0.0]])
    c, s = O8.moments8(x, np.zeros(129), "e5m2")
    assert (c[1:128] >= 1).all() and c[128] == 0 and s[1] == 0


def test_adamw_equals_torchs():
    g = np.random.default_rng(3)
    p, m, v = g.standard_normal(50), np.zeros(50), np.zeros(50)
    t = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    for step in range(1, 5):
        gr = g.standard_normal(50)
        t.grad = torch.tensor(gr * 0.5)
        opt.step()
        p, m, v = O8.adamw(p, gr, m, v, lr=1e-2, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.1, step=step,
                           grad_scale=0.5)
        assert np.allclose(t.detach().numpy(), p, rtol=1e-12)


def test_block_scaled_product_by_hand():
    """One block: codes of 1 with scales 2 and 3 over 128 terms."""
    one = O8.nearest(np.ones((1, 128)), "e4m3")
    out, tol = O8.product(one, np.array([[2.0]]), np.repeat(one, 128, 0), np.array([[3.0]]))
    assert out.shape == (1, 128) and (out == 128 * 6).all()
    # 16 groups of 8 with products of 1, 128 terms of 6
    assert np.allclose(tol, 16 * 8 * 2.0 ** -13 * 6 + (16 * 2.0 ** -23 + 4 * 2.0 ** -24) * 768, rtol=1e-12)
    x = np.random.default_rng(2).standard_normal((3, 256))
    c, s = O8.quantize_rows(x)
    back = O8.decode(c, "e4m3") * np.repeat(s, 128, 1)
    # half a step of e4m3 in the normal range, half of the smallest step below it
    assert (np.abs(back - x) <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + np.repeat(s, 128, 1) * 2.0 ** -10).all()

"""8-bit rows, weights and expert products against float64: gathered and pool
rows, experts with none, one and many rows, every N and K remainder, rows of
no route left alone, non-finite inputs, other streams and replayed graphs."""
import numpy as np
import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from oracle import float8 as O8
from tests import harness as Hn

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def f64(t):
    return t.double().cpu().numpy()


def same_codes(got, want, share):
    """Equal codes but for a share of ties that fp32 turns the other way, each
    then a neighbour."""
    off = got != want
    assert np.mean(off) <= share or off.sum() <= 1
    step = np.abs((got[off] & 127).astype(int) - (want[off] & 127).astype(int))
    assert (step <= 1).all()


@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (17, 640), (130, 2048)])
def test_rows(rows, K):
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, K, generator=g) * torch.exp(2 * torch.randn(1, K, generator=g))).to(BF)
    c, s = M.fp8_quantize_rows(x.cuda())
    wc, ws = O8.quantize_rows(f64(x))
    # scale: one division, half a step; codes: bf16 quotients hit ties of the
    # format, which the rounded reciprocal of the maximum can turn
    assert np.all(np.abs(f64(s) - ws) <= 2.0 ** -24 * ws)
    same_codes(codes(c), wc, 0.02)


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
@pytest.mark.parametrize("rows,K", [(1, 128), (33, 768)])
def test_gated_rows(rows, K, act):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(rows, 2 * K, generator=g) * 2).to(BF)
    c, s = M.fp8_quantize_rows(x.cuda(), act=act)
    gate, up = x[:, :K].double(), x[:, K:].double()
    f = torch.nn.functional.silu if act == "swiglu" else torch.nn.functional.gelu
    h = (f(gate) * up).numpy()
    back = O8.decode(codes(c), "e4m3") * np.repeat(f64(s), 128, 1)
    # e4m3's half step, half its smallest step at the bottom, the activation's
    # own error (sigmoid: 2^-20 relative; the normal distribution function: 1e-6
    # of the gate)
    tol = 2.0 ** -4 * np.abs(h) * (1 + 1e-5) + np.repeat(f64(s), 128, 1) * 2.0 ** -10 + 1e-6 * (x[:, :K].double() * up).abs().numpy()
    assert np.all(np.abs(back - h) <= tol)
    amax = np.abs(h).reshape(rows, -1, 128).max(2) / 448
    assert np.all(np.abs(f64(s) - amax) <= 2.0 ** -18 * amax + 1e-8)


def test_rows_of_zero_tiny_and_nonfinite_blocks():
    x = torch.randn(4, 512).to(BF)
    x[0, :128] = 0
    x[1, 128:256] = 1e-35
    x[2, 300] = float("nan")
    x[3, 400] = -float("inf")
    c, s = M.fp8_quantize_rows(x.cuda())
    v = O8.decode(codes(c), "e4m3") * np.repeat(f64(s), 128, 1)
    assert not codes(c)[0, :128].any() and float(s[0, 0]) == 0
    assert not (codes(c)[1, 128:256] & 127).any() and float(s[1, 1]) == 0
    assert not np.isfinite(f64(s)[2, 2]) and not np.isfinite(f64(s)[3, 3])
    keep = np.ones((4, 512), bool)
    keep[2, 256:384] = keep[3, 384:] = False
    assert np.isfinite(v[keep]).all()


def test_no_rows():
    c, s = M.fp8_quantize_rows(torch.zeros(0, 256, dtype=BF, device="cuda"))
    assert c.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (3, 256, 384)])
def test_weights_and_their_transpose(E, N, K):
    w = (torch.randn(E, N, K, generator=torch.Generator().manual_seed(N)) * 0.02).to(BF)
    c, s, ct, st = M.fp8_quantize_weight(w.cuda(), transposed=True)
    for e in range(E):
        wc, ws = O8.quantize_weight(f64(w[e]))
        assert np.all(np.abs(f64(s[e]) - ws) <= 2.0 ** -24 * ws)
        same_codes(codes(c[e]), wc, 0.02)
    assert np.array_equal(codes(ct), codes(c).transpose(0, 2, 1))
    assert torch.equal(st, s.transpose(1, 2).contiguous())
    c2, s2 = M.fp8_quantize_weight(w.cuda())
    assert torch.equal(c2.view(torch.uint8), c.view(torch.uint8)) and torch.equal(s2, s)


def build(idx, E):
    T, k = idx.shape
    layer = B.make_desc(T, 256, 256, E, k, 8)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
            "route_to_row": torch.empty(T * k, **i32), "row_to_route": torch.empty(B.moe_lora_pool_capacity(layer), **i32)}
    M.build_pool(layer, idx.cuda(), pool["counts"], pool["offsets"], pool["route_to_row"], pool["row_to_route"])
    return pool


def operands(rows, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    a, sa = M.fp8_quantize_rows(torch.randn(rows, K, generator=g).to(BF).cuda())
    w, sw = M.fp8_quantize_weight((torch.randn(E, N, K, generator=g) * K ** -0.5).to(BF).cuda())
    return a, sa, w, sw


def check(idx, E, N, K, gather, seed=0):
    T, k = idx.shape
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    a, sa, w, sw = operands(T if gather else cap, E, N, K, seed)
    out = torch.full((cap, N), -77.0, dtype=BF, device="cuda")
    got = M.fp8_product(pool, a, sa, w, sw, topk=k if gather else 0, out=out)
    assert got.data_ptr() == out.data_ptr()
    r2r = pool["row_to_route"].cpu().numpy()
    off, cnt = pool["offsets"].cpu().numpy(), pool["counts"].cpu().numpy()
    got = f64(got)
    assert (got[r2r < 0] == -77.0).all()  # padding and unused rows
    for e in range(E):
        rows = np.arange(off[e], off[e] + cnt[e])
        if rows.size == 0:
            continue
        src = r2r[rows] // k if gather else rows
        ref, tol = O8.product(codes(a)[src], f64(sa)[src], codes(w[e]), f64(sw[e]))
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)  # the output's half step
        assert np.all(np.abs(got[rows] - ref) <= tol), (e, np.max(np.abs(got[rows] - ref) / tol))
    return pool


def routing(T, E, k, seed, drop=0.0, only=None):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)])
    if only is not None:
        idx = torch.tensor(only)[idx % len(only)]
    if drop:
        idx[torch.rand(T, k, generator=g) < drop] = -1
    return idx.to(torch.int32)


class Kernel:
    """Which product kernel a call takes, from the library's own trace."""

    def __enter__(self):
        B.moe_lora_trace_reset()
        B.moe_lora_trace_enable(True)
        return self

    def __exit__(self, *exc):
        B.moe_lora_trace_enable(False)
        self.names = {n[6:] for n in B.moe_lora_trace_collect() if n.startswith(("k_fp8_few", "k_fp8_tile"))}
        B.moe_lora_trace_reset()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,E,k,N,K,kernel", [
    (1, 1, 1, 128, 128, "few"),          # one row, one tile, one block
    (1, 64, 6, 256, 512, "few"),         # a decoded token
    (5, 8, 2, 384, 128, "few"),
    (40, 3, 2, 128, 1024, "few"),
    (33, 100, 2, 1024, 384, "tile64"),
    (200, 4, 2, 1408, 128, "tile64"),    # fewer K blocks than stages
    (300, 3, 2, 2176, 256, "tile64"),
    (700, 2, 1, 1152, 640, "tile64"),    # odd numbers of K blocks
    (200, 4, 2, 1408, 896, "tile64"),
    (4200, 1, 1, 4224, 128, "tile256"),  # N not a multiple of a tile's columns, one K block
    (4000, 3, 1, 4224, 256, "tile256"),
    (3000, 20, 2, 3968, 384, "tile256"),
    (4096, 1, 1, 4096, 640, "tile256"),
])
def test_product(T, E, k, N, K, kernel, gather):
    with Kernel() as ran:
        check(routing(T, E, k, T + N), E, N, K, gather, seed=T)
    assert ran.names == {kernel}


@pytest.mark.parametrize("gather", [True, False])
def test_product_of_uneven_experts(gather):
    """Experts without rows, with one row and with hundreds, dropped routes."""
    E = 100
    idx = routing(300, E, 3, 2, drop=0.3, only=[0, 0, 0, 0, 7, 63, 64, 64, 98])
    idx[0, 0] = 99
    check(idx, E, 384, 256, gather)


def test_product_of_tails():
    """256-row tiles, the last of an expert with 0, 1, 64, 65, 128, 129 and 255 rows,
    experts below one tile, and one without rows."""
    counts = [768, 513, 576, 1089, 640, 641, 511, 1, 130, 100, 0, 1500]
    idx = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).to(torch.int32)
    idx = idx[torch.randperm(idx.numel(), generator=torch.Generator().manual_seed(1))][:, None].contiguous()
    with Kernel() as ran:
        check(idx, len(counts), 4096, 256, True)
    assert ran.names == {"tile256"}


def test_product_of_no_routes():
    pool = check(torch.full((7, 2), -1, dtype=torch.int32), 5, 128, 128, True)
    assert int(pool["counts"].sum()) == 0


def test_small_products_beside_large_ones():
    """256 * 256 and its negative cancel; what is left of a third product: all
    of it down to 2^-13 of them in the same 8 columns, to 2^-23 elsewhere."""
    idx = torch.zeros(4, 1, dtype=torch.int32)
    pool = build(idx, 1)
    one = torch.ones(4, 1, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    for k, small in ((2, 2.0 ** 3), (7, 1.5 * 2.0 ** 4), (8, 2.0 ** -7), (127, 2.0 ** -7), (64, 1.5 * 2.0 ** -6)):
        a, w = torch.zeros(4, 128), torch.zeros(1, 128, 128)
        a[:, 0], a[:, 1], w[0, :, 0], w[0, :, 1], w[0, :, k] = 256, -256, 256, 256, 1
        a[0, k], a[1, k] = small, -small
        out = M.fp8_product(pool, a.to(F8).cuda(), one[0], w.to(F8).cuda(), one[1], topk=1)
        assert (out[0] == small).all() and (out[1] == -small).all() and not out[2:4].any(), (k, small)


def test_data_gradient_is_the_product_with_the_transpose():
    E, N, K = 3, 256, 384
    idx = routing(50, E, 2, 8)
    pool = build(idx, E)
    cap = pool["row_to_route"].numel()
    w = (torch.randn(E, N, K, generator=torch.Generator().manual_seed(1)) * 0.05).to(BF).cuda()
    c, s, ct, st = M.fp8_quantize_weight(w, transposed=True)
    dy, sdy = M.fp8_quantize_rows(torch.randn(cap, N, generator=torch.Generator().manual_seed(2)).to(BF).cuda())
    dx = f64(M.fp8_product(pool, dy, sdy, ct, st))
    off, cnt = pool["offsets"].tolist(), pool["counts"].tolist()
    for e in range(E):
        rows = slice(off[e], off[e] + cnt[e])
        wt = codes(c[e]).T.copy()
        ref, tol = O8.product(codes(dy)[rows], f64(sdy)[rows], wt, f64(s[e]).T)
        assert np.all(np.abs(dx[rows] - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))


def test_nonfinite_rows_stay_in_their_rows():
    E, N, K = 2, 256, 256
    idx = routing(20, E, 1, 3)
    pool = build(idx, E)
    x = torch.randn(20, K).to(BF)
    x[4, 200] = float("nan")
    x[9, 3] = float("inf")
    a, sa = M.fp8_quantize_rows(x.cuda())
    _, _, w, sw = operands(4, E, N, K, 5)
    out = M.fp8_product(pool, a, sa, w, sw, topk=1)
    tok = (pool["row_to_route"].cpu()).numpy()
    fine = np.isfinite(f64(out)).all(1)
    assert not np.isfinite(f64(out))[np.isin(tok, [4, 9])].any()
    assert fine[~np.isin(tok, [4, 9])].all()


def test_one_row_alone_equals_the_row_in_a_batch():
    """A row's sums depend neither on the other rows nor on the kernel."""
    E, N, K = 1, 4096, 896
    a, sa, w, sw = operands(4300, E, N, K, 11)
    idx = torch.zeros(4300, 1, dtype=torch.int32)
    outs, ran = {}, set()
    for n in (1, 100, 700, 4200, 4300):
        with Kernel() as kern:
            outs[n] = M.fp8_product(build(idx[:n], E), a[:n].contiguous(), sa[:n].contiguous(), w, sw, topk=1)[:n]
        ran |= kern.names
    assert ran == {"few", "tile64", "tile256"}
    for n in (1, 100, 700, 4200):
        assert torch.equal(outs[n], outs[4300][:n])
    for t in (255, 256, 4299):
        one = M.fp8_product(build(idx[:1], E), a[t:t + 1].contiguous(), sa[t:t + 1].contiguous(), w, sw, topk=1)
        assert torch.equal(one[0], outs[4300][t])


@pytest.mark.parametrize("T,N", [(40, 256), (600, 2176), (4200, 4096)])
def test_rows_past_the_activations_and_the_pool(T, N):
    """Routes of tokens past a's rows read zeros; a pool whose arrays claim more
    rows than its capacity writes none past it."""
    E, K = 2, 256
    idx = routing(T, E, 1, 5)
    pool = build(idx, E)
    a, sa, w, sw = operands(T, E, N, K, 3)
    full = M.fp8_product(pool, a, sa, w, sw, topk=1)
    few = T - 7
    part = M.fp8_product(pool, a[:few].contiguous(), sa[:few].contiguous(), w, sw, topk=1)
    tok = pool["row_to_route"].long()
    assert torch.equal(part[(tok >= 0) & (tok < few)], full[(tok >= 0) & (tok < few)])
    assert not part[tok >= few].any()
    cap = pool["row_to_route"].numel()
    broken = dict(pool, counts=pool["counts"] + torch.tensor([0, 1000], dtype=torch.int32, device="cuda"))
    room = torch.full((cap + 2000, N), -7.0, dtype=BF, device="cuda")
    M.fp8_product(broken, a, sa, w, sw, topk=1, out=room[:cap])
    assert (room[cap:] == -7.0).all()
    live = tok >= 0
    assert torch.equal(room[:cap][live], full[live])
    # every expert claims every row: more tiles than a pool can have
    M.fp8_product(dict(pool, counts=torch.full_like(pool["counts"], 2 ** 31 - 1), offsets=torch.zeros_like(pool["offsets"])),
                  a, sa, w, sw, topk=1, out=room[:cap])
    assert (room[cap:] == -7.0).all()


def test_streams_and_graphs():
    E, N, K = 6, 256, 256
    idx = routing(30, E, 2, 4)
    pool = build(idx, E)
    x = torch.randn(30, K).to(BF).cuda()
    _, _, w, sw = operands(4, E, N, K, 6)
    a, sa = M.fp8_quantize_rows(x)
    want = M.fp8_product(pool, a, sa, w, sw, topk=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a2, sa2 = M.fp8_quantize_rows(x, stream=s)
    with torch.cuda.stream(s):
        out = torch.zeros_like(want)
    M.fp8_product(pool, a2, sa2, w, sw, topk=2, out=out, stream=s)
    made = M.fp8_product(pool, a2, sa2, w, sw, topk=2, stream=s)  # zeroed on the call's stream
    raw = M.fp8_product(pool, a2, sa2, w, sw, topk=2, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and torch.equal(made, want) and torch.equal(raw, want)
    got = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.fp8_quantize_rows(x, codes=a2, scales=sa2)
        M.fp8_product(pool, a2, sa2, w, sw, topk=2, out=got)
    for _ in range(3):
        got.zero_()
        a2.view(torch.uint8).zero_()
        M.fp8_product(pool, a, sa, w, sw, topk=2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    del g


@pytest.mark.parametrize("T,E,k,N,K,kernel", [
    (1, 1, 1, 128, 65536, "few"), (400, 1, 1, 512, 65536, "tile64"), (6000, 1, 1, 2048, 65536, "tile256"),
    (1, 1, 1, 65536, 128, "tile64"), (900, 1, 1, 65536, 128, "tile256"), (3, 512, 16, 128, 128, "few"),
    (900, 512, 16, 256, 256, "tile64")])
def test_largest_sizes(T, E, k, N, K, kernel):
    """The ends of the ranges; the last block of columns and some rows checked."""
    idx = routing(T, E, k, T)
    pool = build(idx, E)
    a, sa, w, sw = operands(T, E, N, K, T)
    with Kernel() as ran:
        out = M.fp8_product(pool, a, sa, w, sw, topk=k)
    assert ran.names == {kernel}
    r2r = pool["row_to_route"].cpu().numpy()
    off, cnt = pool["offsets"].cpu().numpy(), pool["counts"].cpu().numpy()
    for e in sorted({0, 1, E // 2, E - 1} & set(range(E))):
        rows = np.arange(off[e], off[e] + cnt[e])[:: max(1, cnt[e] // 8)]
        if rows.size == 0:
            continue
        src = torch.from_numpy(r2r[rows] // k).long().cuda()
        ref, tol = O8.product(codes(a.view(torch.uint8)[src]), f64(sa[src]), codes(w[e, N - 128:]), f64(sw[e, -1:]))
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        got = f64(out[torch.from_numpy(rows).cuda()][:, N - 128:])
        assert np.all(np.abs(got - ref) <= tol), (e, np.max(np.abs(got - ref) / tol))


def test_rows_past_32_bits():
    rows, K = 2 ** 31 // 4096 + 40, 4096
    x = torch.zeros(rows, K, dtype=BF, device="cuda")
    x[-40:] = torch.randn(40, K, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    c, s = M.fp8_quantize_rows(x)
    wc, ws = M.fp8_quantize_rows(x[-40:].contiguous())
    assert torch.equal(c[-40:].view(torch.uint8), wc.view(torch.uint8)) and torch.equal(s[-40:], ws)
    assert not s[:1000].any()


@pytest.mark.parametrize("T,kernel", [(1, "few"), (100, "tile64"), (9000, "tile256")])
def test_weights_past_32_bits(T, kernel):
    """All routes on the last of so many experts that its weights lie past 2^31."""
    E, N, K = 33, 8192, 8192
    g = torch.Generator().manual_seed(T)
    last = (torch.randn(1, N, K, generator=g) * K ** -0.5).to(BF).cuda()
    big = torch.zeros(E, N, K, dtype=BF, device="cuda")
    big[-1] = last[0]
    w, sw = M.fp8_quantize_weight(big)
    del big
    w1, sw1 = M.fp8_quantize_weight(last)
    assert torch.equal(w[-1].view(torch.uint8), w1[0].view(torch.uint8)) and torch.equal(sw[-1], sw1[0])
    a, sa = M.fp8_quantize_rows(torch.randn(T, K, generator=g).to(BF).cuda())
    one = build(torch.zeros(T, 1, dtype=torch.int32), 1)
    want = M.fp8_product(one, a, sa, w1, sw1, topk=1)
    pool = build(torch.full((T, 1), E - 1, dtype=torch.int32), E)
    with Kernel() as ran:
        got = M.fp8_product(pool, a, sa, w, sw, topk=1)
    assert ran.names == {kernel}
    live, live1 = pool["row_to_route"] >= 0, one["row_to_route"] >= 0
    assert int(live.sum()) == T and torch.equal(got[live], want[live1])


def test_outputs_past_32_bits():
    T, N, K = 2 ** 31 // 32768 + 300, 32768, 128
    a, sa, w, sw = operands(T, 1, N, K, 2)
    pool = build(torch.zeros(T, 1, dtype=torch.int32), 1)
    for topk in (1, 0):
        with Kernel() as ran:
            out = M.fp8_product(pool, a, sa, w, sw, topk=topk)
        tail = build(torch.zeros(300, 1, dtype=torch.int32), 1)
        rows = pool["row_to_route"][T - 300:T].long()  # one expert: pool row r is a route of it
        src = rows if topk else torch.arange(T - 300, T, device="cuda")
        want = M.fp8_product(tail, a.view(torch.uint8)[src].view(F8), sa[src], w, sw, topk=0)
        assert ran.names == {"tile256"} and torch.equal(out[T - 300:T], want[:300])
        del out


@pytest.mark.parametrize("T,N", [(12, 256), (300, 1024), (4200, 4096)])
def test_replays_for_other_routes(T, N):
    """Pool and product captured once, replayed for routes that fall otherwise:
    spread, all on one expert, mostly dropped, none."""
    E, k, K = 8, 2, 256
    layer = B.make_desc(T, 256, 256, E, k, 8)
    idx = routing(T, E, k, 1).cuda()
    pool = build(idx, E)
    a, sa, w, sw = operands(T, E, N, K, 4)
    out = torch.zeros(pool["row_to_route"].numel(), N, dtype=BF, device="cuda")
    names = ("counts", "offsets", "route_to_row", "row_to_route")
    M.fp8_product(pool, a, sa, w, sw, topk=k, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.build_pool(layer, idx, *(pool[n] for n in names))
        M.fp8_product(pool, a, sa, w, sw, topk=k, out=out)
    one = torch.full((T, k), -1, dtype=torch.int32)
    one[:, 1] = E - 1
    for other in (routing(T, E, k, 2), one, routing(T, E, k, 3, drop=0.95), torch.full_like(one, -1), routing(T, E, k, 2)):
        want = M.fp8_product(build(other, E), a, sa, w, sw, topk=k)
        idx.copy_(other)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del g


@pytest.mark.parametrize("T,E,N,K,kernel", [(1536, 24, 8192, 512, "tile64"), (4096, 4, 8192, 384, "tile256")])
def test_nonfinite_blocks_stay_in_their_tiles(T, E, N, K, kernel):
    """A NaN or an infinity in the last 128 columns of a token or of an
    expert's weight, with more tiles than workgroups that run at once (each
    walks several): every other result is the clean run's, bit for bit."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, E, (T, 1), generator=g).to(torch.int32)
    pool = build(idx, E)
    x, w = torch.randn(T, K, generator=g).to(BF), (torch.randn(E, N, K, generator=g) * K ** -0.5).to(BF)
    q = M.fp8_quantize_weight(w.cuda())
    rows = M.fp8_quantize_rows(x.cuda())
    with Kernel() as ran:
        clean = M.fp8_product(pool, *rows, *q, topk=1)
    assert ran.names == {kernel}
    tok = pool["row_to_route"].long()
    live = tok >= 0
    bad = [int(torch.nonzero(idx[:, 0] == e)[0]) for e in (0, E // 2, E - 1)]
    for t, value in zip(bad, (float("nan"), float("inf"), -float("inf"))):
        x[t, K - 1] = value
    got = M.fp8_product(pool, *M.fp8_quantize_rows(x.cuda()), *q, topk=1)
    hit = live & torch.isin(tok, torch.tensor(bad, device="cuda"))
    assert int(hit.sum()) == len(bad) and not torch.isfinite(got[hit]).any()
    assert torch.equal(got[live & ~hit], clean[live & ~hit])
    for value in (float("nan"), float("inf")):
        e, n = E // 2, N - 256 + 5  # the block of rows N - 256 .. N - 129
        sick = w.clone()
        sick[e, n, K - 1] = value
        got = M.fp8_product(pool, *rows, *M.fp8_quantize_weight(sick.cuda()), topk=1)
        its = live.clone()
        its[live] = (idx[:, 0].cuda()[tok[live]] == e)
        assert not torch.isfinite(got[its, N - 256:N - 128]).any()
        got[its, N - 256:N - 128] = clean[its, N - 256:N - 128]
        assert torch.equal(got[live], clean[live])


@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_gated_rows_of_small_activations(act):
    """Blocks whose gates lie all in the activation's lower tail: their scale is
    that of small values alone.  x = gate Phi(gate) up or gate sigmoid(gate) up in
    fp32: the tail's exponent, gate^2 / 2 or -gate, is off by two roundings of
    itself (2^-23), the functions and products by 32 * 2^-24 in all."""
    rows, K = 10, 256
    g = torch.Generator().manual_seed(6)
    x = torch.cat([-(torch.arange(2.0, 2.0 + rows)[:, None] + torch.rand(rows, K, generator=g)),
                   1 + torch.rand(rows, K, generator=g)], 1).to(BF)
    c, s = M.fp8_quantize_rows(x.cuda(), act=act)
    gate, up = x[:, :K].double(), x[:, K:].double()
    tail = 0.5 * torch.erfc(-gate * 0.5 ** 0.5) if act == "geglu" else torch.sigmoid(gate)
    h = (gate * tail * up).numpy()
    size = (gate.square() if act == "geglu" else gate.abs()).numpy()
    rel = 2.0 ** -23 * size + 32 * 2.0 ** -24
    amax = np.abs(h).reshape(rows, -1, 128).max(2) / 448
    assert amax.min() > 2.0 ** -98
    assert np.all(np.abs(f64(s) - amax) <= rel.reshape(rows, -1, 128).max(2) * amax)
    back, spread = O8.decode(codes(c), "e4m3") * np.repeat(f64(s), 128, 1), np.repeat(f64(s), 128, 1)
    assert np.all(np.abs(back - h) <= 2.0 ** -4 * np.abs(h) * (1 + rel) + rel * np.abs(h) + spread * 2.0 ** -10)

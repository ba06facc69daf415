"""Measured cases of the expert products in bf16 and their gradients, of the
4-bit block-scaled rows and expert products, and of the optimiser step that
orthogonalises its update: their inputs, their plain form in torch operations,
the framework's calls, and their values in 64 bits.

The sizes are the layer's: the production share (16,384 tokens, 64 experts,
top-6, H 4096, I 2048, rank 128), the token sweep (1 to 2,048 tokens, a fifth
of the routes dropped), the small oracle shape (H 512, I 256, 16 experts,
rank 8), and odd sizes between them.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLK = 32  # elements per shared exponent
ABC = (3.4445, -4.7750, 2.0315)  # the quintic of the orthogonalisation
ROUNDS = 5

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token through gate and up: reading six experts' weights
        {"name": "product one token", "op": "product", "T": 1, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "transposed": False, "mask": 0.0},
        # a sweep point's down product: ragged experts, a fifth of the routes dropped
        {"name": "product sweep", "op": "product", "T": 689, "E": 64, "k": 6, "N": 4096, "K": 2048,
         "gather": False, "transposed": False, "mask": 0.2},
        # gate and up at the production share
        {"name": "product production", "op": "product", "T": 16384, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "transposed": False, "mask": 0.0},
        # the down projection's data gradient at the production share, from the weight as the forward has it
        {"name": "data gradient production", "op": "product", "T": 16384, "E": 64, "k": 6, "N": 2048, "K": 4096,
         "gather": False, "transposed": True, "mask": 0.0},
        # the gradient of the gate and up weights at the production share
        {"name": "weight gradient production", "op": "wgrad", "T": 16384, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "type": "bf16", "add": False, "mask": 0.0},
        # a small layer of odd widths, added to an fp32 gradient over micro-batches; experts with few rows or none
        {"name": "weight gradient odd", "op": "wgrad", "T": 347, "E": 40, "k": 2, "N": 520, "K": 1000,
         "gather": False, "type": "fp32", "add": True, "mask": 0.2},
        # the layer input of the production share through 4-bit rows
        {"name": "mxfp4 rows production", "op": "rows", "rows": 16384, "K": 4096, "gated": False},
        # the gated activation of a sweep point's routes through 4-bit rows
        {"name": "mxfp4 gated rows", "op": "rows", "rows": 2064, "K": 2048, "gated": True},
        # one decoded token on 4-bit weights
        {"name": "mxfp4 product one token", "op": "mx", "T": 1, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "mask": 0.0},
        # gate and up at the production share in 4 bits
        {"name": "mxfp4 product production", "op": "mx", "T": 16384, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "mask": 0.0},
        # the six factors of the small oracle shape: launch latency
        {"name": "muon small", "op": "muon", "H": 512, "I": 256, "E": 16, "rank": 8, "adapters": 1,
         "param": "bf16", "grad": "bf16", "master": True, "nesterov": True},
        # the six factors at the production share
        {"name": "muon production", "op": "muon", "H": 4096, "I": 2048, "E": 64, "rank": 128, "adapters": 1,
         "param": "bf16", "grad": "bf16", "master": True, "nesterov": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "wgrad", "rows", "mx", "muon"])
    if op == "rows":
        return {"op": op, "rows": _log(rng, 1, 16384), "K": 128 * rng.randint(1, 32), "gated": rng.random() < 0.5}
    if op == "muon":
        param = rng.choice(["bf16", "fp32"])
        return {"op": op, "H": 256 * rng.randint(1, 16), "I": 256 * rng.randint(1, 8), "E": _log(rng, 1, 32),
                "rank": _log(rng, 1, 160), "adapters": rng.randint(1, 2), "param": param,
                "grad": rng.choice(["bf16", "fp32"]), "master": param == "bf16" and rng.random() < 0.5,
                "nesterov": rng.random() < 0.7}
    c = {"op": op, "T": _log(rng, 1, 4096), "E": _log(rng, 1, 64), "k": rng.randint(1, 6),
         "gather": rng.random() < 0.5, "mask": rng.choice([0.0, 0.2])}
    if op == "mx":
        return {**c, "N": 32 * rng.randint(1, 128), "K": 128 * rng.randint(1, 32)}
    c.update(N=8 * _log(rng, 1, 512), K=8 * _log(rng, 1, 512))
    if op == "product":
        return {**c, "transposed": rng.random() < 0.5}
    return {**c, "type": rng.choice(["bf16", "fp32"]), "add": rng.random() < 0.5}


def _shapes(c):
    """The factors of one adapter."""
    H, I, E, r = c["H"], c["I"], c["E"], c["rank"]
    return [(r, H), (r, H), (E, I, r), (E, I, r), (E, r, I), (H, r)]


def work(c):
    op = c["op"]
    if op == "rows":
        n = c["rows"] * c["K"]
        return {"bytes": n * (6 if c["gated"] else 4), "flops": n * (10 if c["gated"] else 3)}
    if op == "muon":
        one = (2 if c["grad"] == "bf16" else 4) + 8 + (2 + 8 if c["master"] else 4 if c["param"] == "bf16" else 8)
        n, flops = 0, 0
        for s in _shapes(c):
            size, r = math.prod(s), min(s[-2:])
            n += size
            # its Gram matrix, one product with a matrix of its side, and that matrix: in each round the square, in
            # all but the first one product, in all but the last two for the next round
            flops += 4 * size * r + (size // (s[-1] * s[-2])) * 2 * r ** 3 * (ROUNDS + ROUNDS - 1 + 2 * (ROUNDS - 1))
        return {"bytes": n * one * c["adapters"], "flops": flops * c["adapters"]}
    routes = c["T"] * c["k"] * (1 - c["mask"])
    experts = c["E"] * (1 - (1 - 1 / c["E"]) ** routes)  # experts that a random routing reaches
    flops = int(2 * routes * c["N"] * c["K"])
    a = (c["T"] if c["gather"] else routes) * c["K"]
    if op == "product":
        return {"bytes": int(2 * (experts * c["N"] * c["K"] + a + routes * c["N"])), "flops": flops}
    if op == "mx":
        four = 0.5 + 1 / BLK
        return {"bytes": int(four * (experts * c["N"] * c["K"] + a) + routes * c["N"] * 2), "flops": flops}
    size = 2 if c["type"] == "bf16" else 4
    out = (2 * experts if c["add"] else c["E"]) * c["N"] * c["K"] * size
    return {"bytes": int(2 * (a + routes * c["N"]) + out), "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _e2m1(x):
    """x [..., K] in blocks of 32: each block's exponent and its values in units of two to it, rounded to
    0, 0.5, 1, 1.5, 2, 3, 4, 6."""
    b = x.reshape(*x.shape[:-1], -1, BLK)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    y = torch.ldexp(b, -e)
    m = y.abs().clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return e, torch.copysign(torch.round(m / step) * step, y)


def _mxfp4(x):
    """Codes [..., K/2] and exponents [..., K/32], as the layer's 4-bit weights are held."""
    e, v = _e2m1(x.float())
    m = v.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m <= 4, m + 2, 7)).to(torch.uint8)
    code = (code + 8 * (v < 0).to(torch.uint8)).reshape(x.shape)
    return code[..., 0::2] + 16 * code[..., 1::2], (e[..., 0] + 127).to(torch.uint8)


def _value(codes, exponents):
    """What they stand for, in fp32."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    v = v.reshape(*codes.shape[:-1], -1, BLK)
    return torch.ldexp(v, exponents.int()[..., None] - 127).reshape(*codes.shape[:-1], -1)


def _pool(c, g):
    """A routing of T tokens and the pool that the framework lays out for it: each expert's routes in ascending
    order, padded to 16 rows."""
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.rand(T, max(E, k), generator=g, device=DEV)
    idx = torch.topk(score, k, dim=1).indices % E
    if c["mask"]:
        idx = torch.where(torch.rand(T, k, generator=g, device=DEV) < c["mask"], -1, idx)
    f = idx.reshape(-1)
    n = T * k
    counts = torch.bincount(f[f >= 0], minlength=E)
    padded = (counts + 15) // 16 * 16
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), padded.cumsum(0)])
    capacity = n + min(E, n) * 15
    key = torch.where(f >= 0, f, E)
    order = torch.sort(key, stable=True).indices[: int(counts.sum())]
    first = counts.cumsum(0) - counts
    row = offsets[f[order]] + torch.arange(order.numel(), device=DEV) - first[f[order]]
    row_to_route = torch.full((capacity,), -1, dtype=torch.int64, device=DEV)
    row_to_route[row] = order
    route_to_row = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    route_to_row[order] = row
    pool = {"counts": counts, "offsets": offsets, "route_to_row": route_to_row, "row_to_route": row_to_route}
    return {"pool": {n: t.to(torch.int32) for n, t in pool.items()}, "capacity": capacity,
            "extents": list(zip(offsets.tolist(), counts.tolist()))}


def _prepare_product(c, g):
    st = _pool(c, g)
    E, N, K = c["E"], c["N"], c["K"]
    st["a"] = _normal(g, c["T"] if c["gather"] else st["capacity"], K, dtype=torch.bfloat16)
    st["w"] = torch.empty(E, *((K, N) if c["transposed"] else (N, K)), dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        st["w"][e] = _normal(g, *st["w"].shape[1:], std=K ** -0.5)
    st["out"] = torch.zeros(st["capacity"], N, dtype=torch.bfloat16, device=DEV)
    return st


def _prepare_wgrad(c, g):
    st = _pool(c, g)
    # rows of no route hold whatever is there
    st["grad"] = _normal(g, st["capacity"], c["N"], std=1e-2, dtype=torch.bfloat16)
    st["a"] = _normal(g, c["T"] if c["gather"] else st["capacity"], c["K"], dtype=torch.bfloat16)
    shape = (c["E"], c["N"], c["K"])
    st["out"] = torch.zeros(shape, dtype=TYPES[c["type"]], device=DEV)
    if c["add"]:
        st["out"] += _normal(g, *shape, std=0.1)
    return st


def _prepare_rows(c, g):
    # activations with a few columns far above the rest
    x = _normal(g, c["rows"], c["K"] * (2 if c["gated"] else 1))
    x = x * torch.exp(_normal(g, 1, x.shape[1]))
    return {"x": x.to(torch.bfloat16)}


def _prepare_mx(c, g):
    st = _pool(c, g)
    E, N, K = c["E"], c["N"], c["K"]
    st["a"], st["ea"] = _mxfp4(_normal(g, c["T"] if c["gather"] else st["capacity"], K))
    st["w"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    st["ew"] = torch.empty(E, N, K // BLK, dtype=torch.uint8, device=DEV)
    for e in range(E):
        st["w"][e], st["ew"][e] = _mxfp4(_normal(g, N, K, std=K ** -0.5))
    st["out"] = torch.zeros(st["capacity"], N, dtype=torch.bfloat16, device=DEV)
    return st


def _prepare_muon(c, g):
    st = {"param": [], "grad": [], "momentum": [], "hyper": {
        "lr": 0.02, "momentum": 0.95, "nesterov": c["nesterov"], "weight_decay": 0.01, "rms": 0.2, "grad_scale": 0.5,
        "eps": 1e-7}}
    if c["master"]:
        st["master"] = []
    for shape in _shapes(c) * c["adapters"]:
        p = _normal(g, *shape, std=0.02)
        # gradients whose directions differ in size
        size = torch.exp(0.5 * _normal(g, *shape[:-1], 1))
        st["param"].append(p.to(TYPES[c["param"]]))
        if c["master"]:
            st["master"].append(p)
        st["grad"].append((_normal(g, *shape, std=1e-3) * size).to(TYPES[c["grad"]]))
        st["momentum"].append(_normal(g, *shape, std=2e-3) * size)
    return st


_PREPARE = {"product": _prepare_product, "wgrad": _prepare_wgrad, "rows": _prepare_rows, "mx": _prepare_mx,
            "muon": _prepare_muon}


def _handle(st):
    """What a program that trains with the framework keeps: the optimiser over its tensors."""
    import mixture_experts_grouped_amd as M

    h = st["hyper"]
    return M.MoeMuon(st["param"], st["grad"], masters=st.get("master"), momentum=h["momentum"], nesterov=h["nesterov"],
                     weight_decay=h["weight_decay"], rms=h["rms"], eps=h["eps"], rounds=ROUNDS, coefficients=ABC,
                     states={"momentum": st["momentum"]})


def prepare(case, seed):
    st = _PREPARE[case["op"]](case, _gen(seed))
    st["case"] = case
    if own and case["op"] == "muon":
        st["handle"] = _handle(st)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _rows_of(c, st, at, n):
    """The activation rows of pool rows at .. at + n - 1."""
    a = st["a"]
    return a[st["pool"]["row_to_route"][at:at + n].long() // c["k"]] if c["gather"] else a[at:at + n]


def _product_plain(c, st):
    for e, (at, n) in enumerate(st["extents"]):
        if n:
            w = st["w"][e].float()
            st["out"][at:at + n] = (_rows_of(c, st, at, n).float() @ (w if c["transposed"] else w.t())).to(torch.bfloat16)
    return st["out"]


def _wgrad_plain(c, st):
    out = st["out"]
    for e, (at, n) in enumerate(st["extents"]):
        if n:
            d = st["grad"][at:at + n].float().t() @ _rows_of(c, st, at, n).float()
            out[e] = (out[e].float() + d if c["add"] else d).to(out.dtype)
        elif not c["add"]:
            out[e] = 0
    return out


def _rows_plain(c, st):
    x = st["x"].float()
    if c["gated"]:
        gate, up = x[:, :c["K"]], x[:, c["K"]:]
        x = gate / (1 + torch.exp(-gate)) * up
    e, v = _e2m1(x)
    return torch.ldexp(v, e).reshape(x.shape).to(torch.bfloat16)


def _mx_plain(c, st):
    a = {**st, "a": _value(st["a"], st["ea"])}
    for e, (at, n) in enumerate(st["extents"]):
        if n:
            w = _value(st["w"][e], st["ew"][e])
            st["out"][at:at + n] = (_rows_of(c, a, at, n) @ w.t()).to(torch.bfloat16)
    return st["out"]


def _orthogonal_plain(u, eps):
    """u [..., m, n], m <= n, over its norm and through the rounds of the quintic."""
    a, b, c = ABC
    x = u / (u.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(ROUNDS):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def _muon_plain(c, st):
    h = st["hyper"]
    for i, p in enumerate(st["param"]):
        master = st["master"][i] if c["master"] else p
        g = st["grad"][i].float() * h["grad_scale"]
        m = st["momentum"][i]
        m.copy_(m * h["momentum"] + g)
        u = g + m * h["momentum"] if h["nesterov"] else m
        tall = u.shape[-2] > u.shape[-1]
        o = _orthogonal_plain(u.mT.contiguous() if tall else u, h["eps"])
        o = (o.mT if tall else o) * (h["rms"] * math.sqrt(max(u.shape[-2:])))
        new = master.float() - h["lr"] * (o + h["weight_decay"] * master.float())
        master.copy_(new)
        if c["master"]:
            p.copy_(new)
    return {n: st[n] for n in ("param", "momentum", "master") if n in st}


_PLAIN = {"product": _product_plain, "wgrad": _wgrad_plain, "rows": _rows_plain, "mx": _mx_plain, "muon": _muon_plain}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------


def _own(c, st):
    import mixture_experts_grouped_amd as M

    op = c["op"]
    topk = c["k"] if c.get("gather") else 0
    if op == "product":
        return M.expert_product(st["pool"], st["a"], st["w"], topk=topk, transposed=c["transposed"], out=st["out"])
    if op == "wgrad":
        return M.expert_weight_grad(st["pool"], st["grad"], st["a"], topk=topk, out=st["out"], accumulate=c["add"])
    if op == "rows":
        return M.mxfp4_dequantize(*M.mxfp4_quantize_rows(st["x"], act="swiglu" if c["gated"] else None))
    if op == "mx":
        return M.mxfp4_product(st["pool"], st["a"], st["ea"], st["w"], st["ew"], topk=topk, out=st["out"])
    h = st["hyper"]
    st["handle"].step(lr=h["lr"], grad_scale=h["grad_scale"])
    return {n: st[n] for n in ("param", "momentum", "master") if n in st}


def run(state):
    c = state["case"]
    return _own(c, state) if own else _PLAIN[c["op"]](c, state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _pairs(c, st):
    """Expert, its pool rows and the activation row of each."""
    rows = st["pool"]["row_to_route"].long()
    for e, (at, n) in enumerate(st["extents"]):
        if n:
            at = torch.arange(at, at + n, device=DEV)
            yield e, at, torch.div(rows[at], c["k"], rounding_mode="floor") if c["gather"] else at


def _product_exact(c, st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for e, at, src in _pairs(c, st):
        w = st["w"][e].double()
        out[at] = torch.mm(w.t().contiguous() if c["transposed"] else w, st["a"][src].double().t().contiguous()).t()
    return out


def _wgrad_exact(c, st):
    out = st["out"].double() if c["add"] else torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for e, at, src in _pairs(c, st):
        out[e] += torch.mm(st["a"][src].double().t().contiguous(), st["grad"][at].double()).t()
    return out


def _nearest(y):
    """The nearest of the eight magnitudes, a tie to the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    half = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5], dtype=torch.float64, device=DEV)
    lo = torch.bucketize(y, half)  # borders below y
    tie = (lo < 7) & (y == half[lo.clamp(max=6)])
    return grid[torch.where(tie & (lo % 2 == 1), lo + 1, lo)]


def _rows_exact(c, st):
    x = st["x"].double()
    if c["gated"]:
        x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
    b = x.view(c["rows"], -1, BLK)
    scale = torch.exp2(torch.floor(torch.log2(b.abs().amax(2, keepdim=True).clamp(min=1e-40))) - 2)
    return (torch.sign(b) * _nearest(b.abs() / scale) * scale).view(x.shape)


def _mx_exact(c, st):
    def values(codes, exponents):
        n = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
        m = n % 8
        v = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5).double() * torch.exp2((m // 2 - 1).double()))
        return torch.where(n > 7, -v, v) * torch.exp2(exponents.double() - 127).repeat_interleave(BLK, -1)

    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    a = values(st["a"], st["ea"])
    for e, at, src in _pairs(c, st):
        out[at] = torch.mm(values(st["w"][e], st["ew"][e]), a[src].t().contiguous()).t()
    return out


def _muon_exact(c, st):
    h = st["hyper"]
    out = {"param": [], "momentum": [], **({"master": []} if c["master"] else {})}
    for i, p in enumerate(st["param"]):
        p = (st["master"][i] if c["master"] else p).double()
        g = h["grad_scale"] * st["grad"][i].double()
        m = h["momentum"] * st["momentum"][i].double() + g
        u = h["momentum"] * m + g if h["nesterov"] else m
        wide = u.shape[-2] <= u.shape[-1]
        y = (u.mT if wide else u).contiguous()  # columns: the short side
        y = y / (torch.linalg.matrix_norm(y)[..., None, None] + h["eps"])
        one = torch.eye(y.shape[-1], dtype=torch.float64, device=DEV)
        for _ in range(ROUNDS):
            s = torch.matmul(y.mT.contiguous(), y)
            y = torch.matmul(y, ABC[0] * one + torch.matmul(s, ABC[1] * one + ABC[2] * s))
        o = y.mT if wide else y
        new = p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * h["rms"] * max(u.shape[-2:]) ** 0.5 * o
        out["momentum"].append(m)
        out["param"].append(new)
        if c["master"]:
            out["master"].append(new)
    return out


_EXACT = {"product": _product_exact, "wgrad": _wgrad_exact, "rows": _rows_exact, "mx": _mx_exact, "muon": _muon_exact}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))

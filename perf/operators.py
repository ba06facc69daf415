"""Measured cases of the router, the optimiser step and the 8-bit block-scaled
expert products: their inputs, their plain form in torch operations, the
framework's calls, and their values in 64 bits.

The sizes are the layer's: the production share (16,384 tokens, 64 experts,
top-6, H 4096, I 2048, rank 128), the token sweep (1 to 2,048 tokens, a fifth
of the routes dropped), the small oracle shape (H 512, I 256, 16 experts,
rank 8), and odd sizes between them.
"""
import math

import torch

own = False

DEV = "cuda"
F8, F8V = torch.float8_e4m3fn, torch.float8_e5m2
BLK = 128  # elements per scale: fp8 blocks, 8-bit optimiser states
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token: the router's latency before the expert layer
        {"name": "route one token", "op": "route", "T": 1, "E": 64, "k": 6, "type": "fp32", "renorm": True,
         "roots": 1, "mask": 0.0, "cut": 0.0},
        # the training step's router at the production share
        {"name": "route production", "op": "route", "T": 16384, "E": 64, "k": 6, "type": "fp32", "renorm": True,
         "roots": 1, "mask": 0.0, "cut": 0.0},
        # its gradient, from the layer's router-weight gradients and the balance loss
        {"name": "route grad production", "op": "route_grad", "T": 16384, "E": 64, "k": 6, "type": "fp32",
         "renorm": True, "roots": 1, "mask": 0.0, "cut": 0.0},
        # many experts, four adapters' roots in one padded bf16 batch, some experts closed to some tokens
        {"name": "route grad ragged", "op": "route_grad", "T": 2057, "E": 250, "k": 8, "type": "bf16",
         "renorm": False, "roots": 4, "mask": 0.2, "cut": 0.1},
        # the six factors of the small oracle shape, one adapter: launch latency
        {"name": "adamw small", "op": "adamw", "H": 512, "I": 256, "E": 16, "rank": 8, "adapters": 1,
         "param": "bf16", "grad": "bf16", "master": True, "bits": 32},
        # the six factors at the production share, states in 8 bits beside fp32 masters
        {"name": "adamw production 8 bit", "op": "adamw", "H": 4096, "I": 2048, "E": 64, "rank": 128, "adapters": 1,
         "param": "bf16", "grad": "bf16", "master": True, "bits": 8},
        # several adapters of an odd rank, plain 32-bit training
        {"name": "adamw odd adapters", "op": "adamw", "H": 1024, "I": 512, "E": 9, "rank": 5, "adapters": 16,
         "param": "fp32", "grad": "fp32", "master": False, "bits": 32},
        # the layer input of the production share into 8-bit rows
        {"name": "fp8 rows production", "op": "rows", "rows": 16384, "K": 4096, "gated": False},
        # the gated activation of a sweep point's routes into 8-bit rows
        {"name": "fp8 gated rows", "op": "rows", "rows": 2064, "K": 2048, "gated": True},
        # one token through gate and up: reading six experts' weights
        {"name": "fp8 product one token", "op": "product", "T": 1, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "mask": 0.0},
        # a sweep point's down product: ragged experts, a fifth of the routes dropped
        {"name": "fp8 product sweep", "op": "product", "T": 689, "E": 64, "k": 6, "N": 4096, "K": 2048,
         "gather": False, "mask": 0.2},
        # gate and up at the production share
        {"name": "fp8 product production", "op": "product", "T": 16384, "E": 64, "k": 6, "N": 4096, "K": 4096,
         "gather": True, "mask": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "adamw", "rows", "product"])
    if op in ("route", "route_grad"):
        E = _log(rng, 2, 512)
        return {"op": op, "T": min(_log(rng, 1, 16384), (1 << 20) // E), "E": E, "k": rng.randint(1, min(16, E)),
                "type": rng.choice(["fp32", "bf16"]), "renorm": rng.random() < 0.5, "roots": rng.choice([1, 1, 2, 5]),
                "mask": rng.choice([0.0, 0.2]), "cut": rng.choice([0.0, 0.1, 0.6])}
    if op == "adamw":
        param = rng.choice(["bf16", "fp32"])
        return {"op": op, "H": 256 * rng.randint(1, 16), "I": 256 * rng.randint(1, 8), "E": _log(rng, 1, 32),
                "rank": _log(rng, 1, 128), "adapters": rng.randint(1, 2), "param": param,
                "grad": rng.choice(["bf16", "fp32"]), "master": param == "bf16" and rng.random() < 0.5,
                "bits": rng.choice([8, 32])}
    if op == "rows":
        return {"op": op, "rows": _log(rng, 1, 16384), "K": 128 * rng.randint(1, 32), "gated": rng.random() < 0.5}
    return {"op": op, "T": _log(rng, 1, 4096), "E": _log(rng, 1, 64), "k": rng.randint(1, 6),
            "N": 128 * rng.randint(1, 32), "K": 128 * rng.randint(1, 32), "gather": rng.random() < 0.5,
            "mask": rng.choice([0.0, 0.2])}


def _sizes(c):
    """The factors' element counts of one adapter."""
    H, I, E, r = c["H"], c["I"], c["E"], c["rank"]
    return [r * H, r * H, E * I * r, E * I * r, E * r * I, H * r]


def work(c):
    op = c["op"]
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        logits = T * E * (4 if c["type"] == "fp32" else 2)
        if op == "route":
            return {"bytes": logits + T * (1 + 8 * k) + c["roots"] * (4 * E + 8), "flops": 5 * T * E}
        return {"bytes": 2 * logits + T * (1 + 8 * k) + c["roots"] * (4 * E + 8), "flops": 10 * T * E}
    if op == "adamw":
        n = sum(_sizes(c)) * c["adapters"]
        p = 2 if c["param"] == "bf16" else 4
        one = (2 if c["grad"] == "bf16" else 4) + (8 + p if c["master"] else 2 * p)
        one += 16 if c["bits"] == 32 else 4 + 16 / BLK
        return {"bytes": n * one, "flops": 16 * n}
    if op == "rows":
        n = c["rows"] * c["K"]
        return {"bytes": n * (5 if c["gated"] else 3) + 4 * n // BLK, "flops": n * (10 if c["gated"] else 3)}
    routes = c["T"] * c["k"] * (1 - c["mask"])
    experts = c["E"] * (1 - (1 - 1 / c["E"]) ** routes)  # experts that a random routing reaches
    a = (c["T"] if c["gather"] else routes) * c["K"]
    return {"bytes": int(experts * c["N"] * c["K"] + a + routes * c["N"] * 2),
            "flops": int(2 * routes * c["N"] * c["K"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _cuts(T, roots):
    """Root boundaries: unequal token ranges, one of them empty where there are several."""
    if roots == 1:
        return [0, T]
    inner = sorted(((i * i + 1) * T) // (roots * roots + 1) for i in range(1, roots))
    inner[-1] = inner[-2] if len(inner) > 1 else inner[-1]
    return [0] + inner + [T]


def _pad(n):
    return -(-n // 64) * 64


def _block_scale(x, axis_blocks, top):
    """(codes, scales) of x by blocks: x viewed so that the dims in axis_blocks make up one block."""
    amax = x.abs().amax(dim=axis_blocks, keepdim=True)
    return x * torch.where(amax > 0, top / amax, 0.0), amax / top


def _rows8(x):
    y, s = _block_scale(x.float().view(x.shape[0], -1, BLK), (2,), 448.0)
    return y.view(x.shape).to(F8), s.squeeze(2)


def _weights8(w):
    E, N, K = w.shape
    y, s = _block_scale(w.float().view(E, N // BLK, BLK, K // BLK, BLK), (2, 4), 448.0)
    return y.view(E, N, K).to(F8), s.view(E, N // BLK, K // BLK).contiguous()


def _prepare_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    # a router that prefers some experts, as one does before it is balanced
    logits = _normal(g, T, E) + 0.5 * _normal(g, 1, E)
    if c["cut"]:
        logits[torch.rand(T, E, generator=g, device=DEV) < c["cut"]] = -math.inf
    st = {"logits": logits.to(TYPES[c["type"]]).contiguous(), "roots": _cuts(T, c["roots"]),
          "valid": (torch.rand(T, generator=g, device=DEV) >= c["mask"]).to(torch.uint8) if c["mask"] else None}
    st["root_of"] = torch.repeat_interleave(
        torch.arange(c["roots"], device=DEV),
        torch.tensor([b - a for a, b in zip(st["roots"], st["roots"][1:])], device=DEV))
    if c["op"] == "route_grad":
        idx, w, counts, active, loss = _route_plain(c, st)
        st.update(idx=idx, counts=counts, active=active, grad_w=_normal(g, T, k),
                  grad_loss=_normal(g, c["roots"], std=0.1 * math.sqrt(T)))
    return st


def _prepare_adamw(c, g):
    sizes = _sizes(c) * c["adapters"]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + (-(-n // BLK) * BLK))  # flat buffers, every tensor at an aligned start
    total = starts[-1]
    at = [(s, n) for s, n in zip(starts, sizes)]
    used = torch.zeros(total, dtype=torch.bool, device=DEV)
    for s, n in at:
        used[s:s + n] = True
    p = _normal(g, total, std=0.1) * used
    grad = _normal(g, total, std=1e-3) * torch.exp(_normal(g, total)) * used
    m = _normal(g, total, std=3e-4) * used
    v = (_normal(g, total, std=1e-3).square() + 1e-8) * used
    flat = {"param": p.to(TYPES[c["param"]]), "grad": grad.to(TYPES[c["grad"]])}
    if c["master"]:
        flat["master"] = p
    if c["bits"] == 32:
        flat["m"], flat["v"] = m, v
    else:
        y, s = _block_scale(m.view(-1, BLK), (1,), 448.0)
        flat["m"], flat["m_scale"] = y.to(F8).view(-1), s.view(-1).contiguous()
        y, s = _block_scale(v.view(-1, BLK), (1,), 57344.0)
        y = torch.where(v.view(-1, BLK) > 0, y.clamp(min=2.0 ** -16), 0.0)
        flat["v"], flat["v_scale"] = y.to(F8V).view(-1), s.view(-1).contiguous()
    # where each element stands in its own tensor: what seeds its rounding
    index = torch.arange(total, device=DEV)
    index = index - torch.repeat_interleave(torch.tensor(starts[:-1], device=DEV),
                                            torch.tensor([b - a for a, b in zip(starts, starts[1:])], device=DEV))
    return {"flat": flat, "at": at, "index": index, "hyper": {
        "lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "step": 7, "grad_scale": 0.5,
        "seed": 12345}}


def _prepare_rows(c, g):
    # activations with a few columns far above the rest
    x = _normal(g, c["rows"], c["K"] * (2 if c["gated"] else 1))
    x = x * torch.exp(_normal(g, 1, x.shape[1]))
    return {"x": x.to(torch.bfloat16)}


def _prepare_product(c, g):
    T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
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
    a, sa = _rows8(_normal(g, T if c["gather"] else capacity, K, dtype=torch.bfloat16))
    w, sw = torch.empty(E, N, K, dtype=F8, device=DEV), torch.empty(E, N // BLK, K // BLK, device=DEV)
    for e in range(E):
        we, se = _weights8(_normal(g, 1, N, K, std=K ** -0.5, dtype=torch.bfloat16))
        w[e], sw[e] = we[0], se[0]
    return {"pool": {n: t.to(torch.int32) for n, t in pool.items()}, "a": a, "sa": sa, "w": w, "sw": sw,
            "out": torch.zeros(capacity, N, dtype=torch.bfloat16, device=DEV),
            "extents": list(zip(offsets.tolist(), counts.tolist()))}


_PREPARE = {"route": _prepare_route, "route_grad": _prepare_route, "adamw": _prepare_adamw, "rows": _prepare_rows,
            "product": _prepare_product}


def _handle(c, st):
    """What a program that trains with the framework keeps for one shape: the router's buffers, the optimiser over
    its tensors."""
    import mixture_experts_grouped_amd as M

    if c["op"] in ("route", "route_grad"):
        return M.MoeRouter(c["T"], c["E"], c["k"], dtype=TYPES[c["type"]], renorm=c["renorm"], roots=st["roots"],
                           device=DEV)
    f, h = st["flat"], st["hyper"]
    cut = {n: [t[s // BLK:-(-(s + k) // BLK)] if n.endswith("scale") else t[s:s + k] for s, k in st["at"]]
           for n, t in f.items()}
    return M.MoeAdamW(cut["param"], cut["grad"], masters=cut.get("master"), state_bits=c["bits"],
                      betas=(h["beta1"], h["beta2"]), eps=h["eps"], weight_decay=h["weight_decay"],
                      states={n: cut[n] for n in ("m", "v", "m_scale", "v_scale") if n in cut})


def prepare(case, seed):
    st = _PREPARE[case["op"]](case, _gen(seed))
    st["case"] = case
    if own and case["op"] in ("route", "route_grad", "adamw"):
        st["handle"] = _handle(case, st)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _active(st):
    """Tokens that route: not masked, and with an expert open to them."""
    l = st["logits"].float()
    open_ = (l > -math.inf).any(1)
    return open_ if st["valid"] is None else open_ & (st["valid"] != 0)


def _softmax(l, on):
    m = torch.where(on, l.amax(1), 0.0)
    e = torch.exp(l - m[:, None]) * on[:, None]
    return e / torch.where(on, e.sum(1), 1.0)[:, None]


def _by_root(x, st, roots):
    """Sums over each root's tokens."""
    out = torch.zeros(roots, *x.shape[1:], dtype=x.dtype, device=x.device)
    return out.index_add_(0, st["root_of"], x) if roots > 1 else x.sum(0, keepdim=True)


def _route_plain(c, st):
    E, k, roots = c["E"], c["k"], c["roots"]
    l = st["logits"].float()
    on = _active(st)
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    taken = on[:, None] & (val > -math.inf)
    p = _softmax(l, on)
    w = torch.where(taken, p.gather(1, idx), 0.0)
    if c["renorm"]:
        e = torch.exp(val - torch.where(on, val[:, 0], 0.0)[:, None]) * taken
        w = e / torch.where(on, e.sum(1), 1.0)[:, None]
    hits = torch.zeros(l.shape, device=DEV).scatter_add_(1, idx, taken.float())
    counts = _by_root(hits, st, roots)
    n = _by_root(on.float()[:, None], st, roots)[:, 0]
    mass = _by_root(p.double(), st, roots)
    loss = (counts.double() * mass).sum(1) * E / (k * torch.clamp(n, min=1.0).double().square())
    return torch.where(taken, idx, -1).to(torch.int32), w, counts.to(torch.int32), n.to(torch.int32), loss.float()


def _route_grad_plain(c, st):
    E, k = c["E"], c["k"]
    l = st["logits"].float()
    on = _active(st)
    p = _softmax(l, on)
    taken = st["idx"] >= 0
    idx = st["idx"].clamp(min=0).long()
    gw = torch.where(taken, st["grad_w"], 0.0)
    n = torch.clamp(st["active"].float(), min=1.0)
    coef = (st["grad_loss"] * E / (k * n.square()))[:, None] * st["counts"].float()  # [roots, E]
    up = coef[st["root_of"]]
    if c["renorm"]:
        ps = torch.where(taken, p.gather(1, idx), 0.0)
        w = ps / torch.where(on, ps.sum(1), 1.0)[:, None]
        sel = w * (gw - (w * gw).sum(1, keepdim=True))
        out = p * (up - (p * up).sum(1, keepdim=True))
        return out.scatter_add_(1, idx, sel).to(st["logits"].dtype)
    up = up.scatter_add(1, idx, gw)
    return (p * (up - (p * up).sum(1, keepdim=True))).to(st["logits"].dtype)


def _noise(index, seed):
    """32 random bits of each element: its index and the step's seed through a mixing function."""
    m32 = 0xFFFFFFFF
    x = (index * 0x9E3779B9 + seed) & m32
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & m32
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & m32
    return x ^ (x >> 16)


def _state8(x, noise16, bits, top, dtype):
    """x in blocks of 128 as 8-bit codes and scales, rounded at random: noise is added below the last kept bit."""
    y, s = _block_scale(x.view(-1, BLK), (1,), top)
    y = y.view(-1).clamp(-top, top)
    if dtype == F8V:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -16), 0.0)
    y = ((y.view(torch.int32) + (noise16 << (bits - 16))) & -(1 << bits)).view(torch.float32)
    return y.to(dtype), s.view(-1)


def _adamw_plain(c, st):
    f, h = st["flat"], st["hyper"]
    g = f["grad"].float() * h["grad_scale"]
    p = (f["master"] if c["master"] else f["param"]).float()
    if c["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m = (f["m"].float().view(-1, BLK) * f["m_scale"][:, None]).view(-1)
        v = (f["v"].float().view(-1, BLK) * f["v_scale"][:, None]).view(-1)
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + g * g * (1 - h["beta2"])
    c1, c2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    p = p * (1 - h["lr"] * h["weight_decay"]) - (m * (h["lr"] / c1)) / (torch.sqrt(v * (1 / c2)) + h["eps"])
    f["param"].copy_(p)
    if c["master"]:
        f["master"].copy_(p)
    if c["bits"] == 32:
        f["m"].copy_(m)
        f["v"].copy_(v)
    else:
        r = _noise(st["index"], h["seed"])
        for name, x, noise, bits, top, t in (("m", m, r & 0xFFFF, 20, 448.0, F8), ("v", v, r >> 16, 21, 57344.0, F8V)):
            code, scale = _state8(x, noise.to(torch.int32), bits, top, t)
            f[name].copy_(code)
            f[name + "_scale"].copy_(scale)
    return {n: t for n, t in f.items() if n != "grad"}


def _rows_plain(c, st):
    x = st["x"].float()
    if c["gated"]:
        gate, up = x[:, :c["K"]], x[:, c["K"]:]
        x = gate / (1 + torch.exp(-gate)) * up
    return _rows8(x)


def _product_plain(c, st):
    k, N, K = c["k"], c["N"], c["K"]
    a = (st["a"].float().view(-1, K // BLK, BLK) * st["sa"][:, :, None]).view(-1, K)
    rows = st["pool"]["row_to_route"]
    for e, (at, n) in enumerate(st["extents"]):
        if n:
            w = (st["w"][e].float().view(N // BLK, BLK, K // BLK, BLK) * st["sw"][e][:, None, :, None]).view(N, K)
            ae = a[rows[at:at + n].long() // k] if c["gather"] else a[at:at + n]
            st["out"][at:at + n] = (ae @ w.t()).to(torch.bfloat16)
    return st["out"]


_PLAIN = {"route": _route_plain, "route_grad": _route_grad_plain, "adamw": _adamw_plain, "rows": _rows_plain,
          "product": _product_plain}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------


def _own(c, st):
    import mixture_experts_grouped_amd as M

    op = c["op"]
    if op == "route":
        return st["handle"].forward(st["logits"], valid=st["valid"])
    if op == "route_grad":
        return st["handle"].backward(st["logits"], st["idx"], st["counts"], st["active"], st["grad_w"],
                                     st["grad_loss"], valid=st["valid"])
    if op == "adamw":
        h = st["hyper"]
        st["handle"].step(lr=h["lr"], step=h["step"], grad_scale=h["grad_scale"], seed=h["seed"])
        return {n: t for n, t in st["flat"].items() if n != "grad"}
    if op == "rows":
        return M.fp8_quantize_rows(st["x"], act="swiglu" if c["gated"] else None)
    return M.fp8_product(st["pool"], st["a"], st["sa"], st["w"], st["sw"], topk=c["k"] if c["gather"] else 0,
                         out=st["out"])


def run(state):
    c = state["case"]
    return _own(c, state) if own else _PLAIN[c["op"]](c, state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _tokens64(st):
    l = st["logits"].double()
    on = torch.isfinite(l).any(1)
    if st["valid"] is not None:
        on &= st["valid"].bool()
    return l, on


def _route_exact(c, st):
    l, on = _tokens64(st)
    E, k = c["E"], c["k"]
    # an expert's rank among a token's logits: those above it, and its equals before it
    idx = torch.empty(c["T"], k, dtype=torch.int64, device=DEV)
    rest = l.clone()
    for j in range(k):
        top = rest.amax(1, keepdim=True)
        idx[:, j] = torch.where(rest == top, torch.arange(E, device=DEV), E).amin(1)
        idx[:, j][torch.isinf(top[:, 0])] = -1
        rest.scatter_(1, idx[:, j:j + 1].clamp(min=0), -math.inf)
    idx[~on] = -1
    lse = torch.where(on, torch.logsumexp(l, 1), 0.0)
    p = torch.where(on[:, None], torch.exp(l - lse[:, None]), 0.0)
    w = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        w = w / torch.where(on, w.sum(1), 1.0)[:, None]
    counts, active, loss = [], [], []
    for a, b in zip(st["roots"], st["roots"][1:]):
        got = idx[a:b].reshape(-1)
        cnt = torch.bincount(got[got >= 0], minlength=E)
        n = max(1, int(on[a:b].sum()))
        counts.append(cnt)
        active.append(on[a:b].sum())
        loss.append((cnt.double() / (k * n) * (p[a:b].sum(0) / n)).sum() * E)
    return (idx.to(torch.int32), w, torch.stack(counts).to(torch.int32), torch.stack(active).to(torch.int32),
            torch.stack(loss))


def _route_grad_exact(c, st):
    l, on = _tokens64(st)
    E, k = c["E"], c["k"]
    lse = torch.where(on, torch.logsumexp(l, 1), 0.0)
    p = torch.where(on[:, None], torch.exp(l - lse[:, None]), 0.0)
    up = torch.zeros_like(p)  # the gradient with respect to p
    idx = st["idx"].long()
    gw = st["grad_w"].double()
    total = torch.where(on, torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), 0.0).sum(1), 1.0)
    for j in range(k):
        i = idx[:, j:j + 1]
        g = torch.where(i >= 0, gw[:, j:j + 1], 0.0)
        if c["renorm"]:  # w = p / total: the quotient's two terms
            every = torch.where(idx >= 0, gw * p.gather(1, idx.clamp(min=0)), 0.0).sum(1, keepdim=True)
            g = torch.where(i >= 0, g / total[:, None] - every / total[:, None] ** 2, 0.0)
        up.scatter_add_(1, i.clamp(min=0), g)
    for q, (a, b) in enumerate(zip(st["roots"], st["roots"][1:])):
        n = max(1, int(on[a:b].sum()))
        up[a:b] += st["grad_loss"][q].double() * E / (k * n * n) * st["counts"][q].double()
    return p * up - p * (p * up).sum(1, keepdim=True)


def _state_exact(x, u, mant, lowest, top, dtype):
    """Codes and scales of x: |x| / scale moved up by u of its last place, cut there, then to the format."""
    blocks = x.view(-1, BLK)
    scale = (blocks.abs().amax(1) / top).float().double()
    y = torch.where(scale[:, None] > 0, blocks / scale[:, None], 0.0).view(-1).abs().clamp(max=top)
    if dtype == F8V:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -16), 0.0)
    last = torch.exp2(torch.floor(torch.log2(y.clamp(min=1e-30))) - mant)
    q = torch.floor(y / last + u) * last
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(q.clamp(min=1e-30))), min=lowest) - mant)
    return torch.copysign(torch.round(q / step) * step, x), scale


def _adamw_exact(c, st):
    f, h = st["flat"], st["hyper"]
    d = {n: t.double() for n, t in f.items()}
    g = d["grad"] * h["grad_scale"]
    m, v = d["m"], d["v"]
    if c["bits"] == 8:
        m = m * d["m_scale"].repeat_interleave(BLK)
        v = v * d["v_scale"].repeat_interleave(BLK)
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = d["master"] if c["master"] else d["param"]
    p = p - h["lr"] * (mh / (vh.sqrt() + h["eps"]) + h["weight_decay"] * p)
    out = {"param": p, "m": m, "v": v}
    if c["master"]:
        out["master"] = p
    if c["bits"] == 8:
        r = _noise(st["index"], h["seed"])
        out["m"], out["m_scale"] = _state_exact(m, (r & 0xFFFF).double() / 65536, 3, -6, 448.0, F8)
        out["v"], out["v_scale"] = _state_exact(v, (r >> 16).double() / 65536, 2, -14, 57344.0, F8V)
    return out


def _rows_exact(c, st):
    x = st["x"].double()
    if c["gated"]:
        x = x[:, :c["K"]] * torch.sigmoid(x[:, :c["K"]]) * x[:, c["K"]:]
    b = x.view(c["rows"], -1, BLK)
    scale = (b.abs().amax(2) / 448.0).float().double()
    y = torch.where(scale[:, :, None] > 0, b / scale[:, :, None], 0.0).reshape(x.shape)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp(min=1e-30))), min=-6.0) - 3)
    return torch.round(y / step) * step, scale


def _product_exact(c, st):
    K = c["K"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    a, w = st["a"].double(), st["w"]
    a = a * st["sa"].double().repeat_interleave(BLK, 1)
    rows = st["pool"]["row_to_route"].long()
    for e, (at, n) in enumerate(st["extents"]):
        if n == 0:
            continue
        use = rows[at:at + n] // c["k"] if c["gather"] else torch.arange(at, at + n, device=DEV)
        we = w[e].double() * st["sw"][e].double().repeat_interleave(BLK, 0).repeat_interleave(BLK, 1)
        out[at:at + n] = torch.mm(we, a[use].t().contiguous()).t()
    return out


_EXACT = {"route": _route_exact, "route_grad": _route_grad_exact, "adamw": _adamw_exact, "rows": _rows_exact,
          "product": _product_exact}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))

"""Refusals of the router, optimiser and 8-bit product calls on the host: bad
arguments come back as status codes before any launch (the pointers here are
never dereferenced)."""
import ctypes

import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from tests import harness as Hn

INV, UNS, WS = B.MOE_ERR_INVALID, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
MB = 1 << 20  # fake device addresses: multiples of it


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("field,value,status", [
    ("T", 0, INV), ("E", 0, INV), ("topk", 0, INV), ("topk", 9, INV), ("renorm", 2, INV), ("E", 513, UNS),
    ("logits_type", 2, UNS), ("T", 1 << 28, UNS)])
def test_router_desc(field, value, status):
    d = B.make_router_desc(64, 8, 2)
    setattr(d, field, value)
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_router_workspace_size(d)
    assert e.value.status == status


def test_router_longest_batch():
    assert B.moe_router_workspace_size(B.make_router_desc(1 << 30, 1, 1)) > 0
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_router_workspace_size(B.make_router_desc((1 << 30) + 1, 1, 1))
    assert e.value.status == UNS


def test_router_topk_beyond_sixteen():
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_router_workspace_size(B.make_router_desc(4, 64, 17))
    assert e.value.status == UNS


@pytest.mark.parametrize("roots,status", [([0], INV), ([1, 64], INV), ([0, 63], INV), ([0, 40, 30, 64], INV),
                                          (list(range(66)), UNS)])
def test_router_roots(roots, status):
    with pytest.raises(B.MoeLoraError) as e:
        B.moe_router_workspace_size(B.make_router_desc(64, 8, 2), roots)
    assert e.value.status == status


def test_router_calls():
    lib, d = B.library(), B.make_router_desc(64, 8, 2)
    n = B.moe_router_workspace_size(d)
    good = [MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, 8 * MB, 9 * MB]  # logits valid idx w counts active loss err ws

    def fwd(args, size=n, desc=d):
        return lib.moe_router_forward(None if desc is None else ref(desc), None, *args, size, None)
    assert fwd(good, desc=None) == INV
    assert fwd(good, size=n - 1) == WS
    for i in (0, 2, 3, 4, 5, 6, 8):  # valid and device_error may be NULL
        assert fwd(good[:i] + [None] + good[i + 1:]) == INV
    for i, off in ((0, 4), (2, 2), (3, 1), (8, 8)):
        assert fwd(good[:i] + [good[i] + off] + good[i + 1:]) == INV
    assert fwd(good[:3] + [good[2] + 256] + good[4:]) == INV  # topk_w inside topk_idx
    assert fwd(good[:8] + [good[0] + 1024]) == INV            # workspace inside the logits
    bwd = [MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB, 6 * MB, 7 * MB, 8 * MB]  # logits valid idx counts active gw gloss out

    def back(args):
        return lib.moe_router_backward(ref(d), None, *args, None)
    for i in (0, 2, 3, 4, 7):
        assert back(bwd[:i] + [None] + bwd[i + 1:]) == INV
    assert back(bwd[:7] + [bwd[0] + 16]) == INV  # shifted over the logits
    assert back(bwd[:7] + [bwd[5]]) == INV       # over grad_topk_w


def adam_desc(**kw):
    d = B.MoeAdamwDesc(B.MOE_TYPE_BF16, B.MOE_TYPE_BF16, 32, 0, 1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def adam_tensor(n=100, **kw):
    t = B.MoeAdamwTensor(MB, None, 2 * MB, 3 * MB, 4 * MB, None, None, n)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def adam(d, *ts, count=None):
    arr = (B.MoeAdamwTensor * max(1, len(ts)))(*ts)
    return B.library().moe_adamw_step(None if d is None else ref(d), arr, len(ts) if count is None else count, None)


nan, inf = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(param_type=2), UNS), (dict(grad_type=-1), UNS), (dict(state_bits=16), UNS), (dict(beta1=1.0), INV),
    (dict(beta2=nan), INV), (dict(beta1=-0.1), INV), (dict(eps=0.0), INV), (dict(eps=1e-60), INV), (dict(eps=inf), INV),
    (dict(weight_decay=-1.0), INV), (dict(lr=nan), INV), (dict(lr=-1e-3), INV), (dict(step=0), INV),
    (dict(grad_scale=inf), INV), (dict(control=MB + 2), INV)])
def test_adamw_desc(kw, status):
    assert adam(adam_desc(**kw), adam_tensor()) == status


@pytest.mark.parametrize("kw,desc", [
    (dict(param=None), {}), (dict(param=MB + 2), {}), (dict(grad=None), {}), (dict(m=None), {}), (dict(v=4 * MB + 8), {}),
    (dict(m=4 * MB), {}), (dict(grad=MB), {}), (dict(m_scale=5 * MB), {}), (dict(n=-1), {}),
    (dict(), dict(state_bits=8)), (dict(m_scale=5 * MB, v_scale=6 * MB + 1), dict(state_bits=8)),
    (dict(master=5 * MB), dict(param_type=B.MOE_TYPE_F32)), (dict(master=5 * MB + 4), {})])
def test_adamw_tensors(kw, desc):
    assert adam(adam_desc(**desc), adam_tensor(**kw)) == INV


def test_adamw_lists():
    assert adam(None, adam_tensor()) == INV
    assert adam(adam_desc(), count=-1) == INV
    assert B.library().moe_adamw_step(ref(adam_desc()), None, 1, None) == INV
    assert adam(adam_desc(), count=0) == B.MOE_OK
    assert adam(adam_desc(), adam_tensor(n=0, param=None, grad=None)) == B.MOE_OK  # an empty tensor is not looked at
    assert adam(adam_desc(), adam_tensor(master=8 * MB), adam_tensor()) == INV       # masters for all or none
    assert adam(adam_desc(), adam_tensor(), adam_tensor(grad=None)) == INV           # the second is checked too
    assert adam(adam_desc(), adam_tensor(n=(1 << 34) + 1)) == UNS
    assert adam(adam_desc(), adam_tensor(n=(1 << 62) + 1)) == UNS


def test_fp8_rows():
    f = B.library().moe_fp8_quantize_rows
    assert f(MB, -1, 128, -1, 2 * MB, 3 * MB, None) == INV
    assert f(MB, 4, 0, -1, 2 * MB, 3 * MB, None) == INV
    assert f(MB, 4, 192, -1, 2 * MB, 3 * MB, None) == UNS
    assert f(MB, 4, 65664, -1, 2 * MB, 3 * MB, None) == UNS
    assert f(MB, 1 << 28, 128, -1, 2 * MB, 3 * MB, None) == UNS  # more threads than a launch holds
    assert f(MB, 1 << 31, 128, -1, 2 * MB, 3 * MB, None) == UNS
    assert f(MB, 4, 128, 2, 2 * MB, 3 * MB, None) == UNS
    assert f(MB + 2, 4, 128, -1, 2 * MB, 3 * MB, None) == INV
    assert f(MB, 4, 128, -1, None, 3 * MB, None) == INV
    assert f(MB, 4, 128, -1, 2 * MB, 3 * MB + 2, None) == INV
    assert f(MB, 4096, 256, -1, 2 * MB, 3 * MB, None) == INV      # 2 MB of src over the codes
    assert f(MB, 2048, 256, B.MOE_ACT_SWIGLU, 2 * MB, 8 * MB, None) == INV  # gated: src is twice as wide
    assert f(None, 0, 128, -1, None, None, None) == B.MOE_OK


def test_fp8_weight():
    f = B.library().moe_fp8_quantize_weight
    for E, N, K, st in ((0, 128, 128, INV), (1, 0, 128, INV), (513, 128, 128, UNS), (1, 130, 128, UNS), (1, 128, 64, UNS),
                        (1, 65536, 65536, UNS), (1, 65664, 128, UNS)):
        assert f(MB, E, N, K, 2 * MB, 3 * MB, None, None, None) == st, (E, N, K)
    assert f(MB + 8, 1, 128, 128, 2 * MB, 3 * MB, None, None, None) == INV
    assert f(MB, 1, 128, 128, 2 * MB, 3 * MB, 4 * MB, None, None) == INV   # both transposed outputs or none
    assert f(MB, 1, 128, 128, 2 * MB, 3 * MB, 2 * MB + 1024, 5 * MB, None) == INV
    assert f(MB, 1, 128, 128, MB + 1024, 3 * MB, None, None, None) == INV


def test_fp8_product():
    def call(pool_kw={}, a=20 * MB, sa=30 * MB, w=40 * MB, sw=50 * MB, out=60 * MB, desc_none=False, pool_none=False, **kw):
        d = B.MoeFp8Desc(8, 256, 256, 2, 64)
        p = B.MoePool(MB, 2 * MB, None, 3 * MB, 256, 16)
        for k, v in kw.items():
            setattr(d, k, v)
        for k, v in pool_kw.items():
            setattr(p, k, v)
        return B.library().moe_fp8_product(None if desc_none else ref(d), None if pool_none else ref(p), a, sa, w, sw, out,
                                           None)
    assert call(desc_none=True) == INV and call(pool_none=True) == INV
    assert call(E=0) == INV and call(E=513) == UNS and call(N=200) == UNS and call(K=64) == UNS
    assert call(topk=-1) == INV and call(a_rows=0) == INV and call(a_rows=1 << 24) == UNS
    assert call(pool_kw=dict(capacity=0)) == INV and call(pool_kw=dict(capacity=1 << 31)) == UNS
    for k in ("counts", "offsets", "row_to_route"):
        assert call(pool_kw={k: None}) == INV
    assert call(a=None) == INV and call(sa=30 * MB + 2) == INV and call(w=40 * MB + 4) == INV and call(out=None) == INV
    assert call(out=20 * MB) == INV and call(out=40 * MB + 4096) == INV and call(out=3 * MB) == INV


def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        M.fp8_quantize_rows(torch.zeros(4, 128, dtype=bf))
    with pytest.raises(ValueError):
        M.fp8_quantize_rows(torch.zeros(4, 128, dtype=bf), act="relu")
    with pytest.raises(ValueError):
        M.fp8_quantize_weight(torch.zeros(128, 128, dtype=bf))
    with pytest.raises(ValueError):
        M.MoeAdamW([torch.zeros(8)], [torch.zeros(8)])
    with pytest.raises(ValueError):
        M.MoeAdamW([], [])
    with pytest.raises(ValueError):
        M.MoeAdamW([torch.zeros(8)], [torch.zeros(8)], state_bits=16)
    with pytest.raises(ValueError):
        M.MoeRouter(4, 8, 2, dtype=torch.float16, device="cpu")
    r = M.MoeRouter(4, 8, 2, device="cpu")
    with pytest.raises(ValueError):
        r.forward(torch.zeros(4, 8))


def test_fp8_rows_fill_a_launch():
    """A launch holds fewer than 2^32 threads in whole workgroups of 256, eight
    columns a thread: rows * K is at most 2^35 - 2048."""
    f = B.library().moe_fp8_quantize_rows
    src, codes, scales = 1 << 40, 1 << 42, 1 << 43  # far apart: nothing overlaps
    for rows, K in (((1 << 28) - 1, 128), ((1 << 28) - 15, 128), ((1 << 26) - 1, 512), (1 << 26, 512)):
        for act in (-1, B.MOE_ACT_SWIGLU, B.MOE_ACT_GEGLU):
            assert f(src, rows, K, act, codes, scales, None) == UNS, (rows, K)


@pytest.mark.parametrize("kw", [dict(lr=1e39), dict(weight_decay=1e39), dict(grad_scale=-1e39), dict(eps=1e39)])
def test_adamw_values_beyond_fp32(kw):
    """The step computes in fp32: a value that is infinite there is refused."""
    assert adam(adam_desc(**kw), adam_tensor()) == INV


@pytest.mark.parametrize("control", [torch.zeros(5), torch.zeros(5, dtype=torch.int64), torch.zeros(6, dtype=torch.int32),
                                     torch.zeros(1, 5, dtype=torch.int32), torch.zeros(10, dtype=torch.int32)[::2],
                                     torch.zeros(5, dtype=torch.int32)])
def test_control_buffers_are_checked(control):
    """A control buffer is int32 [5], contiguous, on the optimiser's device."""
    opt = object.__new__(M.MoeAdamW)
    opt.betas, opt._dev = (0.9, 0.99), 0
    before = control.clone()
    with pytest.raises(ValueError, match="control"):
        opt.write_control(control, 1e-3, 1)
    assert torch.equal(control, before)


@pytest.mark.parametrize("stream", [None, 1234])
def test_dropped_tokens_waits_for_the_routers_device(stream, monkeypatch):
    """Without a stream object to wait for it is the router's device that is
    waited for, not the current one."""
    r, waited = M.MoeRouter(4, 8, 2, device="cpu"), []
    r.device_error.fill_(2)
    r._dev = 3
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: waited.append(device))
    assert r.dropped_tokens(stream) == 2 and waited == [3]

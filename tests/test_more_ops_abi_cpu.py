"""Refusals of the expert products, the 4-bit calls and the orthogonalising
optimiser step on the host: bad arguments come back as status codes before any
launch (the pointers here are never dereferenced)."""
import ctypes

import pytest
import torch

import mixture_experts_grouped_amd as M
from mixture_experts_grouped_amd import binding as B
from tests import harness as Hn

INV, UNS, WS, OK = B.MOE_ERR_INVALID, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK
MB = 1 << 20  # fake device addresses: multiples of it
nan, inf = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def ref(x):
    return None if x is None else ctypes.byref(x)


def pool(**kw):
    p = B.MoePool(MB, 2 * MB, None, 3 * MB, 256, 16)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def expert_desc(**kw):
    d = B.MoeExpertDesc(4, 64, 128, 2, 100, 0, B.MOE_TYPE_BF16, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def product(d, p, a=4 * MB, w=5 * MB, out=6 * MB):
    return B.library().moe_expert_product(ref(d), ref(p), a, w, out, None)


def grad(d, p, g=4 * MB, a=5 * MB, dw=6 * MB):
    return B.library().moe_expert_weight_grad(ref(d), ref(p), g, a, dw, None)


DESCS = [(dict(E=0), INV), (dict(N=0), INV), (dict(K=-8), INV), (dict(E=513), UNS), (dict(N=60), UNS), (dict(K=100), UNS),
         (dict(N=65544), UNS), (dict(K=65544), UNS), (dict(N=32768, K=32768), UNS), (dict(topk=-1), INV),
         (dict(a_rows=0), INV), (dict(a_rows=1 << 31), UNS), (dict(a_rows=1 << 23), UNS)]
POOLS = [(dict(capacity=0), INV), (dict(block_m=0), INV), (dict(capacity=1 << 31), UNS), (dict(counts=None), INV),
         (dict(offsets=2 * MB + 2), INV), (dict(row_to_route=None), INV)]


@pytest.mark.parametrize("call", [product, grad])
@pytest.mark.parametrize("kw,status", DESCS)
def test_expert_desc(call, kw, status):
    assert call(expert_desc(**kw), pool()) == status


@pytest.mark.parametrize("call", [product, grad])
@pytest.mark.parametrize("kw,status", POOLS)
def test_expert_pool(call, kw, status):
    assert call(expert_desc(), pool(**kw)) == status


def test_expert_more_tiles_than_an_index():
    assert product(expert_desc(N=65528), pool(capacity=(1 << 31) - 1)) == UNS


@pytest.mark.parametrize("call", [product, grad])
def test_expert_pointers(call):
    assert call(None, pool()) == INV and call(expert_desc(), None) == INV
    names = ("a", "w", "out") if call is product else ("g", "a", "dw")
    for n in names:
        assert call(expert_desc(), pool(), **{n: None}) == INV
        assert call(expert_desc(), pool(), **{n: 7 * MB + 8}) == INV
    for other in (4 * MB, 5 * MB, MB, 2 * MB, 3 * MB):  # the output over an input
        assert call(expert_desc(), pool(), **{names[2]: other}) == INV
    if call is product:
        assert call(expert_desc(transposed=2), pool()) == INV
    else:
        assert call(expert_desc(out_type=2), pool()) == UNS
        assert call(expert_desc(accumulate=3), pool()) == INV


def mx_desc(**kw):
    d = B.MoeMxfp4Desc(4, 64, 128, 2, 100)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def mx(d, p, a=4 * MB, ea=5 * MB, w=6 * MB, ew=7 * MB, out=8 * MB):
    return B.library().moe_mxfp4_product(ref(d), ref(p), a, ea, w, ew, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(E=513), UNS), (dict(N=48), UNS), (dict(K=96), UNS),
    (dict(N=65568), UNS), (dict(K=65664), UNS), (dict(N=32768, K=65536), UNS), (dict(topk=-1), INV), (dict(a_rows=0), INV),
    (dict(a_rows=1 << 31), UNS), (dict(a_rows=1 << 25), UNS)])
def test_mxfp4_desc(kw, status):
    assert mx(mx_desc(**kw), pool()) == status


@pytest.mark.parametrize("kw,status", POOLS)
def test_mxfp4_pool(kw, status):
    assert mx(mx_desc(), pool(**kw)) == status


def test_mxfp4_pointers():
    assert mx(None, pool()) == INV and mx(mx_desc(), None) == INV
    for n, off in (("a", 8), ("ea", 2), ("w", 8), ("ew", 2), ("out", 8)):
        assert mx(mx_desc(), pool(), **{n: None}) == INV
        assert mx(mx_desc(), pool(), **{n: 9 * MB + off}) == INV
    for other in (4, 5, 6, 7, 1, 2, 3):
        assert mx(mx_desc(), pool(), out=other * MB) == INV


def test_mxfp4_rows():
    def rows(src=MB, n=4, K=256, act=B.MOE_FP8_PLAIN, c=2 * MB, e=3 * MB):
        return B.library().moe_mxfp4_quantize_rows(src, n, K, act, c, e, None)

    def back(c=MB, e=2 * MB, n=4, K=256, out=3 * MB):
        return B.library().moe_mxfp4_dequantize(c, e, n, K, out, None)
    assert rows(n=0, src=None, c=None, e=None) == OK and back(n=0, c=None, e=None, out=None) == OK
    assert rows(n=-1) == INV and rows(K=0) == INV and rows(K=96) == UNS and rows(K=65664) == UNS and rows(act=2) == UNS
    assert rows(n=1 << 31, K=128) == UNS and rows(n=1 << 20, K=65536) == UNS
    assert back(n=-1) == INV and back(K=0) == INV and back(K=64) == UNS and back(n=1 << 20, K=65536) == UNS
    for kw in (dict(src=None), dict(src=MB + 8), dict(c=None), dict(e=3 * MB + 2), dict(c=MB), dict(e=MB), dict(e=2 * MB)):
        assert rows(**kw) == INV
    for kw in (dict(c=None), dict(c=MB + 8), dict(e=2 * MB + 1), dict(out=None), dict(out=MB), dict(out=2 * MB)):
        assert back(**kw) == INV


def test_mxfp4_weight():
    def weight(E=2, N=128, K=256, ptr=(MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB)):
        return B.library().moe_mxfp4_quantize_weight(ptr[0], E, N, K, *ptr[1:], None)
    assert weight(E=0) == INV and weight(E=513) == UNS and weight(N=64) == UNS and weight(K=64) == UNS
    assert weight(N=65536, K=32768) == UNS
    good = (MB, 2 * MB, 3 * MB, 4 * MB, 5 * MB)
    for i in range(5):  # the transposed pair comes together
        assert weight(ptr=good[:i] + (None,) + good[i + 1:]) == INV
        assert weight(ptr=good[:i] + (good[i] + 2,) + good[i + 1:]) == INV
        for j in range(i):
            assert weight(ptr=good[:i] + (good[j],) + good[i + 1:]) == INV


def muon_desc(**kw):
    d = B.MoeMuonDesc(B.MOE_TYPE_BF16, B.MOE_TYPE_BF16, 1, 5, 0.02, 0.95, 0.01, 0.2, 1e-7, 1.0, 3.4445, -4.775, 2.0315, None)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def muon_tensor(batch=2, m=8, n=100, **kw):
    t = B.MoeMuonTensor(MB, None, 2 * MB, 3 * MB, batch, m, n)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def muon_size(d, *ts, count=None):
    arr = (B.MoeMuonTensor * max(1, len(ts)))(*ts)
    v = ctypes.c_size_t()
    return B.library().moe_muon_workspace_size(ref(d), arr, len(ts) if count is None else count, ctypes.byref(v))


@pytest.mark.parametrize("kw,status", [
    (dict(param_type=2), UNS), (dict(grad_type=-1), UNS), (dict(nesterov=2), INV), (dict(rounds=0), INV), (dict(rounds=17), UNS),
    (dict(lr=-1.0), INV), (dict(lr=nan), INV), (dict(momentum=1.0), INV), (dict(momentum=-0.1), INV),
    (dict(momentum=0.99999999999), INV), (dict(weight_decay=-1.0), INV), (dict(rms=inf), INV), (dict(rms=-0.2), INV),
    (dict(eps=0.0), INV), (dict(eps=1e-60), INV), (dict(grad_scale=inf), INV), (dict(grad_scale=1e300), INV), (dict(a=nan), INV),
    (dict(b=inf), INV), (dict(c=nan), INV)])
def test_muon_desc(kw, status):
    assert muon_size(muon_desc(**kw), muon_tensor()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INV), (dict(m=0), INV), (dict(n=-5), INV), (dict(m=257, n=257), UNS), (dict(m=256, n=1 << 23), UNS),
    (dict(batch=(1 << 18) + 1), UNS), (dict(batch=1 << 18, m=256, n=1 << 14), UNS)])
def test_muon_sizes(kw, status):
    assert muon_size(muon_desc(), muon_tensor(**kw)) == status
    assert muon_size(None, muon_tensor()) == INV and muon_size(muon_desc(), count=-1) == INV


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_python_calls_refuse_tensors_of_the_host():
    p = {n: cpu(4, dtype=torch.int32) for n in ("counts", "offsets", "row_to_route")}
    with pytest.raises(ValueError):
        M.expert_product(p, cpu(4, 8), cpu(4, 8, 8))
    with pytest.raises(ValueError):
        M.expert_weight_grad(p, cpu(4, 8), cpu(4, 8))
    with pytest.raises(ValueError):
        M.mxfp4_quantize_rows(cpu(4, 128))
    with pytest.raises(ValueError):
        M.mxfp4_dequantize(cpu(4, 64, dtype=torch.uint8), cpu(4, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        M.mxfp4_product(p, cpu(4, 64, dtype=torch.uint8), cpu(4, 4), cpu(4, 8, 64, dtype=torch.uint8), cpu(4, 8, 4))
    with pytest.raises(ValueError):
        M.MoeMuon([cpu(4, 8)], [cpu(4, 8)])


def test_python_calls_refuse_shapes():
    for call in (lambda: M.expert_product({}, cpu(4, 8, 8), cpu(4, 8, 8)), lambda: M.expert_weight_grad({}, cpu(4), cpu(4, 8)),
                 lambda: M.mxfp4_quantize_rows(cpu(4, 128, 1)), lambda: M.mxfp4_quantize_rows(cpu(4, 128), act="relu"),
                 lambda: M.mxfp4_quantize_rows(cpu(4, 129), act="swiglu"), lambda: M.mxfp4_quantize_weight(cpu(4, 8)),
                 lambda: M.mxfp4_dequantize(cpu(4, 60, dtype=torch.uint8), cpu(4, 4)),
                 lambda: M.mxfp4_product({}, cpu(4, 64), cpu(4, 4), cpu(4, 8), cpu(4, 8)),
                 lambda: M.MoeMuon([], []), lambda: M.MoeMuon([cpu(4, 8)], []), lambda: M.MoeMuon([cpu(8)], [cpu(8)])):
        with pytest.raises(ValueError):
            call()


def fp8(p, a=4 * MB):
    d = B.MoeFp8Desc(4, 128, 128, 2, 100)
    return B.library().moe_fp8_product(ref(d), ref(p), a, 5 * MB, 6 * MB, 7 * MB, 8 * MB, None)


@pytest.mark.parametrize("call", [lambda p, a: product(expert_desc(), p, a=a), lambda p, a: grad(expert_desc(), p, a=a),
                                  lambda p, a: mx(mx_desc(), p, a=a), fp8])
def test_most_rows_of_a_pool(call):
    """An expert's rows and a tile's less one: 32 bits.  (At the limit the call gets to the pointer that is missing.)"""
    for capacity in ((1 << 31) - 1, (1 << 31) - 255):
        assert call(pool(capacity=capacity), None) == UNS
    assert call(pool(capacity=(1 << 31) - 256), None) == INV


def test_a_products_tiles_are_no_limit_of_the_gradient():
    p = pool(capacity=(1 << 31) - 256)
    assert product(expert_desc(N=65528), p, a=None) == UNS
    assert grad(expert_desc(N=65528), p, g=None) == INV  # gets to the pointer that is missing


def test_mxfp4_most_values():
    """2^35 - 2048 values; one row or matrix more is refused (at the limit a call gets to the pointer that is missing)."""
    lib = B.library()

    def rows(n, K):
        return lib.moe_mxfp4_quantize_rows(None, n, K, B.MOE_FP8_PLAIN, 2 * MB, 3 * MB, None)

    def back(n, K):
        return lib.moe_mxfp4_dequantize(None, 2 * MB, n, K, 3 * MB, None)

    def weight(E, N, K):
        return lib.moe_mxfp4_quantize_weight(None, E, N, K, 2 * MB, 3 * MB, None, None, None)
    for f in (rows, back):
        assert f(1 << 24, 2048) == UNS and f((1 << 24) - 1, 2048) == INV
        assert f(1 << 28, 128) == UNS and f((1 << 28) - 16, 128) == INV and f((1 << 28) - 15, 128) == UNS
    assert weight(64, 32768, 16384) == UNS and weight(63, 32768, 16384) == INV and weight(64, 32640, 16384) == INV


def test_python_calls_refuse_sizes_that_32_bits_do_not_hold():
    """They would run as what the lower 32 bits say."""
    def wide(*shape, dtype=torch.bfloat16):
        return torch.empty(1, dtype=dtype).expand(*shape)
    far, u8 = (1 << 32) + 128, torch.uint8
    p = {n: cpu(4, dtype=torch.int32) for n in ("counts", "offsets", "row_to_route")}
    e4 = torch.float8_e4m3fn
    for call in (lambda: M.expert_product(p, wide(1, far), wide(1, 8, far)), lambda: M.expert_product(p, wide(1, 8), wide(1, far, 8)),
                 lambda: M.expert_product(p, cpu(4, 8), cpu(4, 8, 8), topk=1 << 32),
                 lambda: M.expert_product(p, cpu(4, 8), cpu(4, 8, 8), block_m=(1 << 32) + 16),
                 lambda: M.expert_weight_grad(p, wide(4, far), cpu(4, 8)), lambda: M.expert_weight_grad(p, cpu(4, 8), wide(4, far)),
                 lambda: M.mxfp4_quantize_rows(wide(1, far)), lambda: M.mxfp4_quantize_rows(wide(1, 2 * far), act="swiglu"),
                 lambda: M.mxfp4_quantize_weight(wide(1, far, 128)), lambda: M.mxfp4_quantize_weight(wide(1, 128, far)),
                 lambda: M.mxfp4_dequantize(torch.empty(1, 1 << 30, dtype=u8), cpu(1, 1 << 20, dtype=u8)),
                 lambda: M.mxfp4_product(p, wide(1, far, dtype=u8), wide(1, 4, dtype=u8), wide(1, 32, far, dtype=u8), wide(1, dtype=u8)),
                 lambda: M.MoeMuon([wide(1, far)], [wide(1, far)]), lambda: M.MoeMuon([wide(far, 1)], [wide(far, 1)]),
                 lambda: M.fp8_quantize_rows(wide(1, far)), lambda: M.fp8_quantize_weight(wide(1, 128, far)),
                 lambda: M.fp8_product(p, wide(1, far, dtype=e4), cpu(1, 1), wide(1, 128, far, dtype=e4), cpu(1, 1)),
                 lambda: B.moe_lora_split_e2m3x2(wide(1, far))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()

"""Optimisers whose steps run on another stream than the one they were made on:
the memory they made for themselves is filled before the first step, and is
not handed out again while a step of a dropped one still runs."""
import pytest
import torch

import mixture_experts_grouped_amd as M
from tests import harness as Hn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
MAKE = {"muon": lambda p, g: M.MoeMuon([p], [g], lr=0.05), "adamw": lambda p, g: M.MoeAdamW([p], [g], lr=0.05),
        "adamw8": lambda p, g: M.MoeAdamW([p], [g], lr=0.05, state_bits=8)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    Hn.ensure_built()


def busy(n):
    """n large products on the current stream, a millisecond each."""
    a = torch.ones(8192, 8192, dtype=BF, device="cuda")
    b = torch.empty_like(a)
    for _ in range(n):
        torch.mm(a, a, out=b)
    return a, b


def own(opt):
    """What an optimiser made for itself."""
    return [t for ts in opt.states.values() for t in ts] + ([opt.workspace] if hasattr(opt, "workspace") else [])


def tensors(seed, shape):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*shape, generator=g) * 0.1).cuda() for _ in range(2)]


@pytest.mark.parametrize("kind", MAKE)
def test_first_step_on_another_stream(kind):
    shape = (40, 1000, 200)
    p, g = tensors(1, shape)
    q = p.clone()
    MAKE[kind](q, g).step()
    s = torch.cuda.Stream()
    torch.cuda.empty_cache()
    # the memory that the states will have holds NaN, and their fill waits behind other work
    poison = [torch.full_like(p, float("nan")) for _ in range(3)]
    keep = busy(1)
    torch.cuda.synchronize()
    del poison
    keep = busy(60), keep
    opt = MAKE[kind](p, g)
    opt.step(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(p, q)


@pytest.mark.parametrize("how", ["argument", "current"])
@pytest.mark.parametrize("kind", MAKE)
def test_dropped_while_a_step_runs(kind, how):
    p, g = tensors(2, (8, 400, 200))
    s = torch.cuda.Stream()
    opt = MAKE[kind](p, g)
    with torch.cuda.stream(s):
        keep = busy(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        keep = busy(100), keep
        if how == "current":
            opt.step()
    if how == "argument":
        opt.step(stream=s)
    done = torch.cuda.Event()
    done.record(s)
    at = {t.data_ptr(): t.numel() * t.element_size() for t in own(opt) if t.numel()}
    del opt
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in at.values()]
    assert done.query() or not any(t.data_ptr() in at for t in again)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", MAKE)
def test_steps_on_several_streams_in_turn(kind):
    """Handles and stream objects, and back to the stream it was made on."""
    p, g = tensors(3, (4, 60, 100))
    q = p.clone()
    one, other = MAKE[kind](p, g), MAKE[kind](q, g)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for stream in (a, None, b.cuda_stream, a, b, None):
        one.step(stream=stream)
        other.step()
        torch.cuda.synchronize()
    assert torch.equal(p, q)


@pytest.mark.parametrize("kind", MAKE)
def test_made_in_a_capture(kind):
    """The fill of the states is captured with the first step: every replay is a first step."""
    p, g = tensors(4, (4, 60, 100))
    start, q = p.clone(), p.clone()
    MAKE[kind](q, g).step()
    MAKE[kind](torch.zeros_like(p), g).step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt = MAKE[kind](p, g)
        opt.step()
    for _ in range(3):
        p.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, q)
    del opt


@pytest.mark.parametrize("kind", MAKE)
def test_nothing_to_update_on_another_stream(kind):
    p, g = torch.zeros(0, 4, 6, device="cuda"), torch.zeros(0, 4, 6, device="cuda")
    opt, s = MAKE[kind](p, g), torch.cuda.Stream()
    opt.step(stream=s)
    opt.step()
    torch.cuda.synchronize()

"""The base operators on streams other than the one their memory came from:
tensors that the library made are not handed out again before the work that
uses them has run, nor written while their last owner's work still runs.

Each check looks at addresses: memory that is still in use must not be what
the allocator hands out next.
"""
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_attn import Batch
from test_gpu_i8 import acts, quant64, weight

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SLEEP = 20_000_000


def handed_out(side, n, at, count=6):
    """Whether memory of n bytes at `at` is handed out to the current stream
    while `side` still works; what is handed out is written over."""
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(count)]
    assert not side.query()
    for j in junk:
        j.fill_(85)
    return any(j.data_ptr() <= at < j.data_ptr() + n for j in junk)


@pytest.fixture
def side():
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    yield st
    torch.cuda.synchronize()


def test_a_plan_mapped_under_another_current_stream_and_dropped(side):
    b = Batch(50, [(300, [(1, 90), (1, 70), (40, 100)])], 4, 2, 64, 32)
    t = b.table()
    plan = b.plan()
    torch.cuda.synchronize()
    n, at = plan.buf.numel(), plan.buf.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
        plan.remap(*t)
    del plan
    assert not handed_out(side, n, at)


def test_a_plan_whose_status_was_asked_under_another_current_stream(side):
    b = Batch(51, [(300, [(1, 90), (1, 70)])], 4, 2, 64, 32)
    plan = b.plan()
    torch.cuda.synchronize()
    n, at = plan.buf.numel(), plan.buf.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
        out = plan.status_async()
    del plan
    assert not handed_out(side, n, at)
    torch.cuda.synchronize()
    assert int(out[0]) == tclora.OK


def test_queries_of_an_append_under_another_current_stream(side):
    cache = tclora.KVCache(*(torch.zeros(40, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    T = 512
    q, k = (torch.randn(T, h * 64, device=DEV).to(torch.bfloat16) for h in (8, 2))
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    slot = torch.arange(T, device=DEV)
    call = tclora.AppendCall(cache, k, k, pos, slot, q=q)
    torch.cuda.synchronize()
    n, at = call.q_out.numel() * 2, call.q_out.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
        call()
    del call
    assert not handed_out(side, n, at)


@pytest.mark.parametrize("how", ["product", "call", "made and called"])
def test_a_packed_weight_used_under_another_current_stream(how, side):
    """The weight's copy was made on the default stream, also where the call
    was made on the other one."""
    W, ws = weight(52, 1024, 512)
    x = acts(52, 64, 512, torch.bfloat16)
    n8, s = (t.to(DEV) for t in quant64(x))
    want = tclora.i8_linear(tclora.I8Weight(W, ws), x)
    y = torch.zeros_like(want)
    w = tclora.I8Weight(W, ws)
    call = tclora.I8Call(w, x, y) if how == "call" else None
    torch.cuda.synchronize()
    n, at = w.W_p.numel(), w.W_p.data_ptr()
    with torch.cuda.stream(side):
        if how == "made and called":
            call = tclora.I8Call(w, x, y)
        torch.cuda._sleep(SLEEP)
        if call is not None:
            call()
        else:
            tclora.i8_product(w, n8, s, y=y)
    del w, call
    assert not handed_out(side, n, at)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_attention_made_on_one_stream_over_a_plan_of_another(side):
    b = Batch(53, [(300, [(1, 90), (1, 70), (40, 100)])], 4, 2, 64, 32)
    want = tclora.attention(b.plan(), b.qd)
    plan = b.plan()
    torch.cuda.synchronize()
    n, at = plan.buf.numel(), plan.buf.data_ptr()
    with torch.cuda.stream(side):
        call = tclora.AttnCall(plan, b.qd)
        torch.cuda._sleep(SLEEP)
        call()
    o = call.o
    del call, plan
    assert not handed_out(side, n, at)
    torch.cuda.synchronize()
    assert torch.equal(o, want)

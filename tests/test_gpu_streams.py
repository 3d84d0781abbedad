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
SLEEP = 100_000_000


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
    torch.cuda.empty_cache()  # (blocks of other tests are not handed out instead)
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


class Freed:
    """Memory of n bytes, freed on the current stream with a copy of it still
    to be made there; whatever owns it next has to leave it until then."""

    def __init__(self, n):
        old = torch.full((n,), 3, dtype=torch.uint8, device=DEV)
        self.at = old.data_ptr()
        torch.cuda._sleep(SLEEP)
        self.copy = old.clone()

    def left_alone(self):
        torch.cuda.synchronize()
        return bool((self.copy == 3).all())


@pytest.mark.parametrize("how", ["given", "raw", "current"])
def test_calls_made_over_memory_that_is_still_read(how, side):
    """Calls whose own tensors lie in such memory, their first run on another
    stream that nothing else orders behind it."""
    def go(call):
        if how == "current":
            with torch.cuda.stream(side):
                call()
        else:
            call(side.cuda_stream if how == "raw" else side)

    W, ws = weight(60, 256, 4096)
    w = tclora.I8Weight(W, ws)
    x = acts(60, 512, 4096, torch.bfloat16)
    want = tclora.i8_linear(w, x)
    y = torch.zeros_like(want)
    n = tclora.I8Call(w, x, y).ws.numel()
    torch.cuda.synchronize()
    f = Freed(n)
    call = tclora.I8Call(w, x, y)
    assert call.ws.data_ptr() == f.at
    go(call)
    assert f.left_alone() and torch.equal(y, want)

    cache = tclora.KVCache(*(torch.zeros(40, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    q, k = (torch.randn(512, h * 64, device=DEV).to(torch.bfloat16) for h in (64, 2))
    pos = torch.arange(512, dtype=torch.int32, device=DEV)
    rope = tclora.Rope(torch.ones(32, device=DEV))
    want = tclora.kv_append(cache, k, k, pos, pos.long(), rope, q=q)
    slot = pos.long()
    torch.cuda.synchronize()
    f = Freed(q.numel() * 2)
    call = tclora.AppendCall(cache, k, k, pos, slot, rope, q=q)
    assert call.q_out.data_ptr() == f.at
    go(call)
    assert f.left_alone() and torch.equal(call.q_out, want)

    b = Batch(61, [(300, [(1, 90), (1, 70), (40, 100)])], 64, 8, 64, 32)
    plan = b.plan()
    want = tclora.attention(plan, b.qd)
    o = torch.zeros_like(want)
    torch.cuda.synchronize()
    f = Freed(plan.workspace_bytes)
    call = tclora.AttnCall(plan, b.qd, o=o)
    assert call.ws.data_ptr() == f.at
    go(call)
    assert f.left_alone() and torch.equal(o, want)
    f = Freed(want.numel() * 2)
    call = tclora.AttnCall(plan, b.qd, ws=call.ws)
    assert call.o.data_ptr() == f.at
    go(call)
    assert f.left_alone() and torch.equal(call.o, want)


def test_a_call_made_and_forked_inside_a_capture(side):
    """Made in the capture, run on a stream forked from it before: the replay
    runs it behind what the capture had put into the same memory."""
    W, ws = weight(62, 256, 4096)
    w = tclora.I8Weight(W, ws)
    x = acts(62, 512, 4096, torch.bfloat16)
    want = tclora.i8_linear(w, x)
    y = torch.zeros_like(want)
    n = tclora.I8Call(w, x, y).ws.numel()
    src = torch.full((n,), 3, dtype=torch.uint8, device=DEV)
    kept = torch.zeros_like(src)
    fork = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        fork.wait_stream(side)
        old = src.clone()
        kept.copy_(old)
        at = old.data_ptr()
        del old
        call = tclora.I8Call(w, x, y)
        same = call.ws.data_ptr() == at
        call(fork)
        side.wait_stream(fork)
    assert same
    for _ in range(4):
        y.zero_(), kept.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and bool((kept == 3).all())


def test_calls_made_before_a_capture(side):
    """Captured on streams other than their own, forked ones among them."""
    W, ws = weight(63, 264, 1040)
    w = tclora.I8Weight(W, ws)
    x = acts(63, 40, 1040, torch.bfloat16)
    want = tclora.i8_linear(w, x)
    ys = [torch.zeros_like(want) for _ in range(2)]
    calls = [tclora.I8Call(w, x, y) for y in ys]
    fork = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        fork.wait_stream(side)
        calls[0]()
        calls[1](fork)
        side.wait_stream(fork)
    for _ in range(3):
        for y in ys:
            y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in ys)
    calls[1](fork)  # eager, on the stream of the capture
    torch.cuda.synchronize()
    assert torch.equal(ys[1], want)


def test_given_workspaces():
    """A workspace that is given and large enough is the one that is used; one
    whose elements do not lie one behind another is refused."""
    W, ws = weight(64, 264, 1040)
    w = tclora.I8Weight(W, ws)
    x = acts(64, 40, 1040, torch.bfloat16)
    y = torch.zeros(40, 264, device=DEV)
    b = Batch(65, [(300, [(1, 90), (40, 100)])], 4, 2, 64, 32)
    plan = b.plan()
    for make, n in ((lambda ws: tclora.I8Call(w, x, y, ws=ws), 1 << 17),
                    (lambda ws: tclora.AttnCall(plan, b.qd, ws=ws), plan.workspace_bytes)):
        own = torch.empty(n, dtype=torch.uint8, device=DEV)
        assert make(own).ws is own and make(own[:256]).ws is not own
        for bad in (own[:1].expand(n), torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
            with pytest.raises(ValueError):
                make(bad)

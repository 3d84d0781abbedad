"""How the mapping cuts a windowed batch, and the windows that it refuses."""
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_attn import DEV, Batch
from test_gpu_attn_window import Windowed

pytestmark = pytest.mark.gpu


LONG = {  # (long enough that items are cut by the batch's size)
    "one prefix": [(8192, [(1, 300)] * 64)],
    "several": [(5000, [(1, 40 + i) for i in range(40)]), (3000, [(3, 100)] * 20), (700, [(90, 400), (1, 9)])],
}


@pytest.mark.parametrize("window,sinks", [((1 << 31) - 1, 0), (9000, 4), (1, 1 << 30), (300, 9000)])
@pytest.mark.parametrize("name", LONG)
def test_a_window_that_hides_nothing_is_cut_as_none(name, window, sinks):
    """The same items, and bit for bit the attention without a window."""
    b = Windowed(7, LONG[name], 32, 8, 64, 32, window, sinks)
    plans = [Batch.plan(b), b.plan()]
    status = [p.status_async().tolist() for p in plans]
    assert status[0][0] == tclora.OK and status[0] == status[1]
    lse = [torch.zeros(b.T, 32, device=DEV) for _ in range(2)]
    o = [tclora.attention(p, b.qd, lse=x) for p, x in zip(plans, lse)]
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


@pytest.mark.parametrize("kw", [dict(window=5 - (1 << 32)), dict(window=-(1 << 40)),
                                dict(window=4, sinks=3 - (1 << 32))])
def test_negative_windows_of_any_size_are_refused(kw):
    b = Windowed(14, [(20, [(1, 3)])], 4, 2, 64, 16, 3, 1)
    with pytest.raises(tclora.TclError) as e:
        tclora.AttnPlan(b.cache, 4, *b.table(), n_tokens=b.T, **kw)
    assert e.value.code == tclora.EINVAL

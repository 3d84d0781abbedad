"""How the mapping cuts a windowed batch, and the windows that it refuses."""
import pytest

from tenant_composite_lora_amd import tclora
from test_gpu_attn_window import Windowed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(window=5 - (1 << 32)), dict(window=-(1 << 40)),
                                dict(window=4, sinks=3 - (1 << 32))])
def test_negative_windows_of_any_size_are_refused(kw):
    b = Windowed(14, [(20, [(1, 3)])], 4, 2, 64, 16, 3, 1)
    with pytest.raises(tclora.TclError) as e:
        tclora.AttnPlan(b.cache, 4, *b.table(), n_tokens=b.T, **kw)
    assert e.value.code == tclora.EINVAL

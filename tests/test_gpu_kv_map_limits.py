"""tcl_kv_map at the largest position."""
import pytest

from tenant_composite_lora_amd import tclora
from test_gpu_kv_map import cache_of, up

pytestmark = pytest.mark.gpu
LAST = (1 << 31) - 1


@pytest.mark.parametrize("n_tokens", [6, 5000])  # (by the first launch, by the second)
def test_positions_up_to_the_last(n_tokens):
    """Request 0 brings no token behind keys that pass the last position,
    request 1 three tokens up to it and request 2 one at 9."""
    def call(prefix):
        return tclora.kv_map(cache_of(9, 16), up([0, 3, 1]), up([0, 1, 2, 3]), up([LAST, prefix, 4]),
                             up([7, 14, 5]), up([[0, 0], [1, 0], [2, 0]]), up([7, 8, 6]), up([0]), n_tokens)

    c = call(LAST - 16)
    assert c.status() == (tclora.OK, 4, 1, 2)
    assert c.pos.tolist()[:6] == [LAST - 2, LAST - 1, LAST, 9, 0, 0]
    assert c.slot.tolist()[:6] == [30, 31, 7 * 16, 37, -1, -1]
    assert c.seq_tok_ptr.tolist() == [0, 0, 3, 4] and c.own_len.tolist() == [7, 17, 6]
    assert (c.pos[4:] == 0).all() and (c.slot[4:] == -1).all()
    # one further
    c = call(LAST - 15)
    assert c.status()[0] == tclora.EINVAL and (c.slot == -1).all() and c.own_len.tolist() == [7, 14, 5]

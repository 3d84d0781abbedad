"""The weights of tcl_attn_apply: what their rounding leaves of the output's
accuracy, and rows whose scores leave no usable weight.

Tolerance of a request of fewer than 64 query rows a key head.  As in
test_gpu_attn, but its weights enter the second product as two bf16 parts: the
first is the weight cut to 8 bits (2^-7 of it left over at most), the second
what is left, rounded (2^-8 of that), so 2^-15, and 2^-20 that the second part
is raised by: less than 2^-14 of A = sum w |V| in place of 2^-8.
"""
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_attn import DEV, HALF, Batch

pytestmark = pytest.mark.gpu


def tight(b):
    """(o, bound) in 64 bits with weights of two parts."""
    wo, _, tol = b.want()
    V, b.Vh = b.Vh, b.Vh.abs()
    A, _, _ = b.want()
    b.Vh = V
    return wo, tol - (HALF - 2.0 ** -14) * A


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (8, 1, 128), (6, 2, 256)])
@pytest.mark.parametrize("name,groups", [
    ("two share", [(600, [(1, 30), (1, 90)])]),
    ("five share", [(600, [(1, 30)] * 5), (333, [(1, 1)] * 5)]),
    ("forty share", [(900, [(1, 1 + 5 * i) for i in range(40)])]),
    ("some tokens each", [(500, [(3, 40), (7, 70), (1, 9)]), (0, [(7, 300), (5, 64)])]),
])
def test_a_short_requests_accuracy_does_not_depend_on_its_batch(name, groups, Hq, Hkv, D):
    b = Batch(len(name) + D, groups, Hq, Hkv, D, 16)
    wo, tol = tight(b)
    got = tclora.attention(b.plan(), b.qd).double().cpu().view(wo.shape)
    assert float(((got - wo).abs() - tol).max()) <= 1e-30

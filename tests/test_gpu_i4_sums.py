"""Sums of tcl_i4_linear where the two sums of a group nearly cancel, each kernel
by the mean square of its errors.

All activations have one sign, so that a group's sum of x (16 + n), p, and its sum
of x times 16 + z, f q, are many times their difference c.  Bound of the mean
square, for sums that are fp32 and joined a group at a time: p and q take one
rounding a column at most, so L each, and two more join them; a rounding moves a
number v by no more than 2^-24 |v|, evenly spread, in the mean square by a third
of its square.  The running sums of the groups take three roundings a group
(scaling, the wave's or workgroup's sums, the result).  The groups are drawn
alike, so a partial sum of them has in the mean square no more than the whole
sum's square and the sum of the squares, whichever kernel takes them in whichever
order.  A kernel that joins `late` groups at a time holds up to `late` p s beside
its running sum, which is rounded twice a group meanwhile:

    2^-48 / 3 (sum_g s^2 ((L + 2) (p^2 + f^2 q^2) + 2 late^2 p^2) + 3 G (y^2 + sum_g s^2 c^2))

(late 0: none).  Sums joined only at the end would hold the whole of sum_g s p.
"""
import pytest
import torch

from tenant_composite_lora_amd import tclora
from test_gpu_i4 import DEV, close, product64, weight

pytestmark = pytest.mark.gpu


def moments(w, n, x, late):
    """(y, bound of the mean square) in 64 bits."""
    _, scale, zero = w
    G = scale.shape[1]
    L = n.shape[1] // G
    y = torch.zeros(len(x), len(n), dtype=torch.float64, device=DEV)
    groups, c2 = y.clone(), y.clone()
    n = n.to(DEV)
    for g in range(G):
        at = slice(g * L, (g + 1) * L)
        xg, s = x[:, at].double(), scale[:, g].double()
        f = 24.0 if zero is None else 16 + zero[:, g].double()
        p, fq = xg @ (16 + n[:, at].double()).T, xg.sum(1, keepdim=True) * f
        groups += s.square() * ((L + 2) * (p.square() + fq.square()) + 2 * late ** 2 * p.square())
        c = (p - fq) * s
        y += c
        c2 += c.square()
    return y, 2.0 ** -48 / 3 * (groups + 3 * G * (y.square() + c2))


def balanced(w, n):
    """Zero points on both sides of the integers' mean (7.5)."""
    if w[2] is not None:
        w[2].copy_(7 + torch.rand(w[2].shape, device=DEV).round().to(torch.uint8))


def run(T, d_in, d_out, group, zeros, late):
    torch.manual_seed(T + d_in)
    w, n = weight(T + d_in, d_out, d_in, group, zeros, full=True)
    balanced(w, n)
    x = (torch.randn(T, d_in, device=DEV).abs() + 4).to(torch.bfloat16)
    got = tclora.i4_linear(tclora.I4Weight(*w), x, y_dtype=torch.float32)
    y, bound = moments(w, n, x, late)
    err = (got.double() - y).square().mean()
    assert float(err) <= float(bound.mean()), (float(err) / float(bound.mean())) ** 0.5
    return w, n, x, got


# (one size a kernel and its variants: few rows; rows turned in LDS, 32, 64 and 128
# channels, split over workgroups; laid-out rows in blocks; tiles of 64, 128 tokens)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T,d_in,d_out,group,late", [
    (3, 4096, 264, 32, 0), (16, 4096, 14336, 64, 0), (64, 4096, 264, 32, 0), (64, 2048, 4104, 64, 0),
    (64, 2048, 14336, 128, 0), (40, 8192, 2056, 32, 0),
    (64, 4096, 14336, 32, 0), (100, 2048, 14336, 64, 0), (250, 1056, 8200, 32, 0),
    (1024, 2048, 4096, 32, 4), (1000, 2048, 4096, 64, 4), (1024, 2048, 4096, 128, 4),
    (2048, 2048, 4096, 32, 4), (2030, 2048, 4096, 64, 4), (2048, 2048, 4096, 128, 4)])
def test_one_signed_activations(T, d_in, d_out, group, late, zeros):
    w, n, x, got = run(T, d_in, d_out, group, zeros, late)
    close(got, *product64(w, n, x))


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("T", [16, 64, 1024])
def test_one_signed_activations_of_long_rows(T, group):
    """Sums that were joined only at the end would be off by many times the bound,
    and more the longer the row (1024 tokens: laid-out rows in blocks)."""
    run(T, 65536, 520, group, True, 0)


@pytest.mark.parametrize("T,d_in,d_out,group", [
    (3, 4096, 264, 32), (64, 4096, 264, 128), (64, 4096, 14336, 128), (64, 4096, 14336, 32), (40, 8192, 2056, 32),
    (1024, 1024, 4096, 64), (2048, 1024, 4096, 128)])
def test_one_strong_activation_at_its_zero_points(T, d_in, d_out, group):
    """It adds nothing to the result, yet sums are as exact as |x| (16 + n) lets
    them be, not as |x| |n - z|: the bound is that of all products."""
    (W, s, _), n = weight(T, d_out, d_in, group, full=True)
    n[:, 7] = 8
    W[:, 3] = (W[:, 3] & 15) | 8 << 4
    torch.manual_seed(T)
    x = torch.randn(T, d_in, device=DEV)
    x[:, 7] = 3000
    x = x.to(torch.bfloat16)
    got = tclora.i4_linear(tclora.I4Weight(W, s), x, y_dtype=torch.float32)
    close(got, *product64((W, s, None), n, x))

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


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (4, 1, 128, 32), (3, 1, 256, 8)])
def test_rows_whose_scores_are_all_minus_infinity(Hq, Hkv, D, page):
    """Their softmax is NaN (as of any row of -infinity); rows beside them
    that see another key, or none, are as ever.  Rows of one item, of few and
    of many rows, and rows joined from several."""
    groups = [
        (0, [(1, 9), (1, 40), (70, 70), (70, 60), (3, 0)]),   # no prefix: written at once
        (130, [(1, 20), (1, 30), (5, 40), (90, 100)]),        # joined with the prefix's
        (900, [(1, 5), (2, 30), (1, 0)]),
    ]
    b = Batch(70 + D, groups, Hq, Hkv, D, page)
    b.q.view(b.T, Hq, D)[..., 0] = 1.0
    low = -float("inf")
    hide = {0: (0, 9), 2: (0, 70), 3: (0, 30), 5: (0, 20), 7: (0, 38), 9: (0, 5)}
    for pages, n in [(b.prefix_pages[1], 130), (b.prefix_pages[2], 900)] + [
            (b.own_pages[s], hi) for s, (_, hi) in hide.items()]:
        for j in range(n):
            b.Kh[int(pages[j // page]), j % page, :, 0] = low
    b.up(b.Kh, b.Vh)
    lse = torch.zeros(b.T, Hq, device=DEV)
    o = tclora.attention(b.plan(), b.qd, lse=lse).double().cpu().view(b.T, Hq, D)
    wo, wl, _ = b.want()
    assert torch.equal(torch.isnan(o), torch.isnan(wo))
    nan = torch.isnan(wo).all(-1)
    assert 0.2 < float(nan.double().mean()) < 0.8
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(wl)) and bool((lse.cpu()[nan] == low).all())
    none = torch.zeros(b.T, dtype=torch.bool)
    for s, (q, n) in enumerate(b.seqs):
        p = groups[0 if s < 5 else 1 if s < 9 else 2][0]
        none[int(b.seq_tok[s]):int(b.seq_tok[s]) + max(0, q - p - n)] = True
    assert int(none.sum()) == 13 and not o[none].any() and bool((lse.cpu()[none] == low).all())
    # finite rows: as ever, with sum |q k| * scale of the finite scores at most
    # D * D^-0.5 * max |q| * max |K|
    ok = ~nan & ~none[:, None]
    V, b.Vh = b.Vh, b.Vh.abs()
    A, _, _ = b.want()
    b.Vh = V
    K0 = torch.where(torch.isinf(b.Kh.float()), 0.0, b.Kh.float().abs()).amax()
    E = (D + 2) * 2.0 ** -24 * D ** 0.5 * float(K0) * float(b.q.float().abs().max())
    tol = (2 * E + 2.0 ** -19 + HALF) * A + HALF * wo.abs()
    assert float(((o - wo).abs() - tol)[ok].max()) <= 1e-30


@pytest.mark.parametrize("scale", [0.0, 1e-45, -1e-40, 1e-38])
def test_scales_near_zero_and_large_scores(scale):
    """A scale of zero weighs every key alike, however large its score: the
    smallest one in use must not make a difference of it.  (Scores up to
    1e38 here.)"""
    b = Batch(80, [(150, [(1, 40), (1, 70), (20, 30), (90, 100)])], 4, 2, 64, 16)
    b.q.mul_(2.0 ** 60)
    b.Kh.mul_(2.0 ** 60)
    b.up(b.Kh, b.Vh)
    o = tclora.attention(b.plan(), b.qd, scale=scale).double().cpu().view(b.T, 4, 64)
    wo, _, _ = b.want(scale)
    V, b.Vh = b.Vh, b.Vh.abs()
    A, _, _ = b.want(scale)
    b.Vh = V
    # a score times the scale is off by what the scale loses in fp32, in the
    # call and times log2(e) (half of the smallest number each; all of it for
    # zero), and by 66 roundings of the sum, 64 * 2^120 * 32 at most in magnitude
    top = 2.0 ** 131
    E = top * (2.0 ** -149 + 66 * 2.0 ** -24 * abs(scale)) + 2.0 ** -20
    tol = (2 * E + 2.0 ** -19 + HALF) * A + HALF * wo.abs()
    assert float(((o - wo).abs() - tol).max()) <= 1e-30


@pytest.mark.parametrize("factor", [16.0, 64.0])
def test_every_row_of_extreme_scores(factor):
    """Scores of hundreds and thousands.  Their fp32 sums are off by up to E,
    no longer small beside one, so a weight by exp(2 E) and the output by
    (exp(2 E) - 1) A; for 2 E below 0.35 that is less than 1.2 * 2 E A."""
    b = Batch(8, [(150, [(1, 40), (1, 70), (20, 30), (90, 100)])], 4, 2, 64, 16)
    q, K = b.q * factor, b.Kh * factor
    b.q, b.Kh = q.abs(), K.abs()
    e = float(b.want()[1].max())  # (at least the largest sum of |q k|)
    assert 2 * (b.D + 2) * 2.0 ** -24 * e < 0.35
    b.q, b.Kh = q, K
    b.up(b.Kh, b.Vh)
    o = tclora.attention(b.plan(), b.qd).double().cpu().view(b.T, b.Hq, b.D)
    wo, _, tol = b.want()
    assert float(((o - wo).abs() - 1.2 * tol).max()) <= 1e-30

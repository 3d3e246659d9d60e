"""The sums of the 16-bit expert products on the GPU: what long contractions may lose, and sums that must be exact.

The tensor core's fp32 sums may cut off every term where the running sum's last bit ends, a loss below 2^-23 of that
sum for each.  The kernels sum at most 1024 terms that way; partial sums are added rounded to nearest.
"""
import pytest
import torch

from test_gpu_y_products import _cuda, gen, normal, offsets_of, spans, TYPES  # noqa: F401
from weight_only_bit_route_b200 import moe

pytestmark = pytest.mark.gpu


# few tiles (clusters share the contraction, an eighth each), single CTAs, CTA pairs
@pytest.mark.parametrize("rows,K,N", [(64, 131072, 1024), (4800, 16384, 128), (4800, 16384, 512)])
@pytest.mark.parametrize("grad", [False, True])
def test_long_sums_are_not_cut_off(rows, K, N, grad):
    """Positive terms, so that every cut-off counts the same way, in fp16.  With 1024 terms at a time the running sum
    grows from 0, and the loss is below 2^-23 * (1 + ... + 1024) / 1024 = 2^-13.998 of the result whatever K.  (A step
    of 16 terms aligns each of them with the running sum, so it is the terms that count, not the steps: 64 cut-offs of
    half a last bit would be 1.4e-6, and 6.2e-6 are seen.)  One sum over 16 times the terms may lose 16 times that, and
    loses 16 * 6.2e-6 = 9.9e-5, above the bound.  The rounding to fp16 is off by 2^-11 at most, as often up as down: the
    mean over M results is within 5 standard deviations, 5 * 2^-11 / sqrt(3 M), of zero (the fp32 sums' own rounding,
    2^-24 each, as little one-sided, is far below).  The reference is in 64 bits."""
    g = gen(30)
    x = (torch.rand(rows, K, generator=g, device="cuda") * 0.5 + 0.5).half()
    w = ((torch.rand(N, K, generator=g, device="cuda") * 0.5 + 0.5) * (1024.0 / K)).half()
    off, ws = offsets_of([rows]), moe.control_block()
    if grad:
        y = moe.grouped_mm_dgrad(x, w.t().contiguous().unsqueeze(0), off, ws)
    else:
        y = moe.grouped_mm(x, w.unsqueeze(0), off, ws)
    assert moe.read_status(ws) == 0
    wd = w.double()
    err = torch.cat([y[a:a + 512].double() / (x[a:a + 512].double() @ wd.T) - 1 for a in range(0, rows, 512)])
    cut, half = 2.0 ** -13.998, 2.0 ** -11
    assert err.mean().abs() <= cut + 5 * half / (3 * err.numel()) ** 0.5, err.mean().item()
    # one result: half a step, the chunks' cut-offs, and the fp32 additions of the partial sums
    assert err.abs().max() <= (half + cut + (K / 1024 + 8) * 2.0 ** -24) * (1 + half), err.abs().max().item()

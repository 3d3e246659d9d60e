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


def whole(g, *shape, density, dtype):
    """Entries -1, 0 and 1."""
    sign = torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1
    return (sign * (torch.rand(*shape, generator=g, device="cuda") < density)).to(dtype)


def same_sums(got, ref, dtype):
    """Sums of whole numbers are exact in fp32, and in the output type up to 2^8 (bf16) or 2^11 (fp16): a term left out
    or counted twice is off by one."""
    assert ref.abs().max() <= (256 if dtype is torch.bfloat16 else 2048) and ref.any()
    assert torch.equal(got.double(), ref)


# One expert of 60 rows: clusters of 8, 4 and 2 share the contraction, then none does; few and many rows on CTA pairs;
# experts without and with few rows on single CTAs.  Contractions that end inside a stage, a chunk and a share of it.
LAYOUTS = {"eight": ([60], 1024), "four": ([60], 3200), "two": ([60], 6400), "one": ([60], 12800),
           "experts": ([0, 1, 17, 64, 65, 0, 130, 3] * 4, 520), "pair": ([4800], 1032), "pairs": ([700, 0, 1300, 33, 800], 1288)}


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K", [4096, 4104, 5000, 8192])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_every_term_counts_once(layout, K, dtype):
    (counts, M), dt = LAYOUTS[layout], TYPES[dtype]
    E, rows, g = len(counts), sum(counts), gen(37)
    density = 1 / 4 if dt is torch.bfloat16 else 1.0              # sums stay below 2^8: sqrt(8192 / 8) = 32, times 8
    x, w = whole(g, rows, K, density=0.5, dtype=dt), whole(g, E, M, K, density=density, dtype=dt)
    off, ws = offsets_of(counts), moe.control_block()
    y = moe.grouped_mm(x, w, off, ws)
    dx = moe.grouped_mm_dgrad(x, w.transpose(1, 2).contiguous(), off, ws)
    assert moe.read_status(ws) == 0
    ref = torch.cat([x[a:b].double() @ w[e].double().T for e, a, b in spans(counts)])
    same_sums(y, ref, dt)
    same_sums(dx, ref, dt)


# clusters of four share the rows; CTA pairs; single CTAs
@pytest.mark.parametrize("counts,K,N", [([8200], 264, 1000), ([3000, 0, 5177], 136, 264), ([4500, 0, 4111, 700], 1032, 1032),
                                        ([100] * 40, 520, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_row_counts_once(counts, K, N, dtype):
    dt, rows, g = TYPES[dtype], sum(counts), gen(38)
    x, dy = whole(g, rows, K, density=0.25, dtype=dt), whole(g, rows, N, density=0.5, dtype=dt)
    off, ws = offsets_of(counts), moe.control_block()
    ref = torch.stack([dy[a:b].double().T @ x[a:b].double() for e, a, b in spans(counts)])
    base = whole(g, *ref.shape, density=1.0, dtype=torch.float32)
    same_sums(moe.grouped_mm_wgrad(dy, x, off, ws), ref, dt)
    same_sums(moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32), ref, dt)
    same_sums(moe.grouped_mm_wgrad(dy, x, off, ws, out=base.clone(), accumulate=True), ref + base.double(), dt)
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("K", [4096, 4224, 8192])
@pytest.mark.parametrize("counts,M", [([60], 1024), ([60], 3200), ([60], 6400), ([60], 12800), ([4800], 1024),
                                      ([0, 1, 17, 64, 65, 0, 130, 3] * 4, 512)])
def test_every_term_counts_once_in_8_bits(counts, M, K):
    """Rows of -1, 0 and 1 have the codes -127, 0 and 127 and the scale 1/127: the sum times the scale is the whole
    number within 2^-22 of itself, and that number in bf16."""
    E, rows, g = len(counts), sum(counts), gen(39)
    h = whole(g, rows, K, density=0.5, dtype=torch.bfloat16)
    h[:, 0] = 1                                                   # (a row has a largest magnitude of 1)
    q = whole(g, E, M, K, density=0.25, dtype=torch.int8)
    down = moe.Bank(moe.FMT_INT8, q, torch.ones(E, M, device="cuda"))
    off, rs = offsets_of(counts), torch.arange(rows, dtype=torch.int32, device="cuda")
    ws = moe.workspace(rows, M, E, K, 1)
    y = moe.grouped_down(h, off, rs, None, down, ws)
    assert moe.read_status(ws) == 0
    same_sums(y, torch.cat([h[a:b].double() @ q[e].double().T for e, a, b in spans(counts)]), torch.bfloat16)

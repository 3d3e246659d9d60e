"""Offsets of the expert products that leave the rows or decrease, on the GPU: reported, and each counted as the largest
up to it, clipped to the rows, so that no two experts share a row."""
import pytest
import torch

from test_gpu_y_products import ERR_INDEX, _cuda, gen, int8_bank, normal  # noqa: F401
from weight_only_bit_route_b200 import moe

pytestmark = pytest.mark.gpu


def _offsets(kind, E, rows):
    even = [rows * e // E for e in range(E + 1)]
    if kind == "see-saw":                            # every second expert asks for all the rows
        return [0 if e % 2 == 0 else rows for e in range(E + 1)]
    if kind == "falls":                              # an expert's rows begin inside those of one before it
        even[E // 2] = even[E // 4] // 2
        return even
    if kind == "outside":
        return [-7] + even[1:E] + [rows + 1000]
    return [0, 2 ** 31 - 1] + [-2 ** 31] * (E - 2) + [rows // 2]


def _clipped(offsets, rows):
    out, top = [], 0
    for o in offsets:
        top = max(top, min(o, rows))
        out.append(top)
    return out


# few tiles (clusters share them), single CTAs, CTA pairs, in the products and in the weight gradient
@pytest.mark.parametrize("E,rows,K,N", [(4, 61, 2048, 136), (4, 2100, 264, 136), (200, 900, 128, 264), (1024, 700, 64, 72),
                                        (4, 4800, 1024, 1032), (48, 9000, 264, 520)])
@pytest.mark.parametrize("kind", ["see-saw", "falls", "outside", "extremes"])
def test_bad_offsets_count_as_the_clipped_ones(kind, E, rows, K, N):
    g = gen(33)
    x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, E, N, K, std=0.1)
    bad = _offsets(kind, E, rows)
    got, want = [], []
    for offsets, outs, status in ((_clipped(bad, rows), want, 0), (bad, got, ERR_INDEX)):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        y = torch.full((rows, N), 7.0, dtype=x.dtype, device="cuda")
        dx = torch.full((rows, K), 7.0, dtype=x.dtype, device="cuda")
        for call in (lambda ws: moe.grouped_mm(x, w, off, ws, out=y), lambda ws: moe.grouped_mm_dgrad(dy, w, off, ws, out=dx),
                     lambda ws: moe.grouped_mm_wgrad(dy, x, off, ws),
                     lambda ws: moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32)):
            ws = moe.control_block()
            outs.append(call(ws))
            assert moe.read_status(ws) == status
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("E,rows", [(4, 24), (4, 1000), (64, 5000)])
def test_bad_offsets_of_the_8_bit_experts(E, rows):
    """Rows behind the last offset hold no codes: here the last offset is the rows' end."""
    H, F = 512, 256
    g = gen(34)
    x = normal(g, rows, H)
    gate, up = int8_bank(g, E, F, H), int8_bank(g, E, F, H)
    rs = torch.arange(rows, dtype=torch.int32, device="cuda")
    bad = _offsets("falls", E, rows)
    ws = moe.workspace(rows, H, E, F, 1)
    h = [moe.grouped_swiglu(x, torch.tensor(o, dtype=torch.int32, device="cuda"), rs, 1, gate, up, rows, ws)
         for o in (_clipped(bad, rows), bad)]
    assert moe.read_status(ws) == ERR_INDEX
    assert torch.equal(*h)

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


@pytest.mark.parametrize("E,T,k,H,F", [(3, 20, 2, 512, 256), (16, 1100, 8, 2048, 128)])     # (the second copies the codes)
def test_rows_of_no_expert_in_8_bits(E, T, k, H, F):
    """Rows in front of the first expert and behind the last: their slots are not looked at, their values are nobody's
    error, and the outputs' rows keep what they held."""
    g = gen(35)
    rows, first, last = T * k, 5, T * k - 9
    x = normal(g, T, H)
    gate, up, down = int8_bank(g, E, F, H), int8_bank(g, E, F, H), int8_bank(g, E, H, F)
    off = torch.tensor([first + (last - first) * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    rs = torch.arange(rows, dtype=torch.int32, device="cuda")
    rs[:first], rs[last:] = -5, 2 ** 31 - 1
    ws = moe.workspace(T, H, E, F, min(k, E))
    h = torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_swiglu(x, off, rs, k, gate, up, rows, ws, out=h)
    assert moe.read_status(ws) == 0
    assert (h[:first] == 7.0).all() and (h[last:] == 7.0).all()
    h[:first], h[last:] = float("nan"), float("inf")
    y = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_down(h, off, rs, torch.rand(rows, generator=g, device="cuda"), down, ws, out=y)
    assert moe.read_status(ws) == 0
    assert (y[:first] == 7.0).all() and (y[last:] == 7.0).all() and torch.isfinite(y).all()


def test_rows_behind_a_falling_last_offset_in_8_bits():
    """The last offset below the others: rows from it on have no codes, and none is multiplied."""
    E, T, H, F = 3, 40, 512, 256
    g = gen(36)
    x, gate, up = normal(g, T, H), int8_bank(g, E, F, H), int8_bank(g, E, F, H)
    rs = torch.arange(T, dtype=torch.int32, device="cuda")
    ws = moe.workspace(T, H, E, F, 1)
    h = []
    for offsets in ([0, 10, 12, 12], [0, 10, 30, 12]):
        h.append(torch.full((T, F), 7.0, dtype=torch.bfloat16, device="cuda"))
        moe.grouped_swiglu(x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), rs, 1, gate, up, T, ws, out=h[-1])
    assert moe.read_status(ws) == ERR_INDEX
    assert torch.equal(*h) and (h[1][12:] == 7.0).all()

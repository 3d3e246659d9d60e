"""The expert products in 16 bits (forward and both gradients) and in 8-bit integers on the GPU, against the
formulas in 64 bits.

Tolerances.  16-bit products: each of the K fp32 additions is off by at most 2^-23 of the sum of the terms'
magnitudes (the tensor core may truncate), then one rounding to the output type (half a step, finfo.eps / 2).
8-bit products: the integer sum is exact; its conversion, the scales' product and the two multiplications are
four roundings of 2^-24, the row and channel scales one each; silu's relative sensitivity to g is at most
1 + |g|, expf and the division add less than 2^-21; then one rounding to bf16.
"""
import threading

import numpy as np
import pytest
import torch

from weight_only_bit_route_b200 import moe

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ERR_TIMEOUT, ERR_INDEX, ERR_NONFINITE = -4, -6, -7


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.init()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32, device="cuda")


def spans(counts, first=0):
    o = np.concatenate([[0], np.cumsum(counts)]) + first
    return [(e, int(o[e]), int(o[e + 1])) for e in range(len(counts))]


def product_bound(mag, K, ref, dtype):
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * half * 2
    return mag * (K * 2.0 ** -23) * (1 + half) + ref.abs() * half + tiny


COUNTS = {
    "many": [1100, 0],
    "long": [2049],
    "ragged": [0, 1, 16, 17, 0, 63, 64, 65, 255, 0],
    "one_each": [1] * 9,
    "big": [600, 0, 257, 5],
    "single": [37],
    "none": [0, 0, 0],
}
WIDTHS = [(8, 8), (64, 128), (72, 136), (1000, 264), (256, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("load", list(COUNTS))
def test_products_match_the_formula(load, K, N, dtype):
    """All three directions.  Rows in front of the first expert and behind the last hold NaN: they must reach
    nothing, and the outputs' rows there must keep what they held."""
    counts, dt = COUNTS[load], TYPES[dtype]
    E, first, rows = len(counts), 3, sum(counts) + 3 + 21
    g = gen(1)
    x, dy = normal(g, rows, K, dtype=dt), normal(g, rows, N, dtype=dt, std=0.5)
    w = normal(g, E, N, K, dtype=dt, std=0.1)
    off = offsets_of(counts, first)
    end = first + sum(counts)
    for t in (x, dy):
        t[:first], t[end:] = float("nan"), float("nan")
    ws = moe.control_block()
    y = torch.full((rows, N), 7.0, dtype=dt, device="cuda")
    dx = torch.full((rows, K), 7.0, dtype=dt, device="cuda")
    moe.grouped_mm(x, w, off, ws, out=y)
    moe.grouped_mm_dgrad(dy, w, off, ws, out=dx)
    dw = moe.grouped_mm_wgrad(dy, x, off, ws)
    dwf = moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32)
    base = normal(g, E, N, K, dtype=torch.float32)
    acc = moe.grouped_mm_wgrad(dy, x, off, ws, out=base.clone(), accumulate=True)
    assert moe.read_status(ws) == 0
    for out in (y, dx):
        assert (out[:first] == 7.0).all() and (out[end:] == 7.0).all()
    for e, a, b in spans(counts, first):
        xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
        for name, got, ref, mag, terms in (
                ("y", y[a:b], xe @ we.T, xe.abs() @ we.abs().T, K),
                ("dx", dx[a:b], de @ we, de.abs() @ we.abs(), N),
                ("dw", dw[e], de.T @ xe, de.abs().T @ xe.abs(), b - a),
                ("dw fp32", dwf[e], de.T @ xe, de.abs().T @ xe.abs(), b - a)):
            err = (got.double() - ref).abs()
            assert (err <= product_bound(mag, terms, ref, got.dtype)).all(), (name, e, err.max().item())
        ref = base[e].double() + de.T @ xe
        bound = product_bound(de.abs().T @ xe.abs(), b - a, ref, torch.float32)
        assert ((acc[e].double() - ref).abs() <= bound).all(), ("accumulated", e)


@pytest.mark.parametrize("K,N", [(4096, 136), (2056, 392), (1024, 1000), (320, 64)])
@pytest.mark.parametrize("counts", [[3], [61], [1, 0, 16, 17], [64], [40, 64, 3]], ids=str)
def test_few_tiles_share_a_long_contraction(counts, K, N):
    """Few tiles: clusters split the contraction (of K forward, of N in the gradient), and the parts are joined."""
    E, rows = len(counts), sum(counts) + 5
    g = gen(20)
    x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, E, N, K, std=0.1)
    wt = w.transpose(1, 2).contiguous()
    off, ws = offsets_of(counts), moe.control_block()
    y, dx = moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(x, wt, off, ws)
    assert moe.read_status(ws) == 0
    for e, a, b in spans(counts):
        xe, we = x[a:b].double(), w[e].double()
        ref, mag = xe @ we.T, xe.abs() @ we.abs().T
        for got in (y, dx):                      # dx by the transposed weights is the same product
            assert ((got[a:b].double() - ref).abs() <= product_bound(mag, K, ref, torch.bfloat16)).all(), e
    for _ in range(2):
        assert torch.equal(moe.grouped_mm(x, w, off, ws)[:sum(counts)], y[:sum(counts)])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(2056, 2040), (2048, 2048)])
@pytest.mark.parametrize("counts", [[700, 0, 129, 300, 1], [2000, 3, 0, 1000, 500]], ids=str)
def test_products_of_many_rows(counts, K, N, dtype):
    """Sizes that run on CTA pairs, in both directions, with rows in front and behind that nothing may read."""
    dt, E, first, rows = TYPES[dtype], len(counts), 5, sum(counts) + 60
    g = gen(27)
    x, dy, w = normal(g, rows, K, dtype=dt), normal(g, rows, N, dtype=dt), normal(g, E, N, K, dtype=dt, std=0.1)
    end = first + sum(counts)
    for t in (x, dy):
        t[:first], t[end:] = float("nan"), float("inf")
    off, ws = offsets_of(counts, first), moe.control_block()
    y = torch.full((rows, N), 7.0, dtype=dt, device="cuda")
    dx = torch.full((rows, K), 7.0, dtype=dt, device="cuda")
    moe.grouped_mm(x, w, off, ws, out=y)
    moe.grouped_mm_dgrad(dy, w, off, ws, out=dx)
    assert moe.read_status(ws) == 0
    for out in (y, dx):
        assert (out[:first] == 7.0).all() and (out[end:] == 7.0).all()
    for e, a, b in spans(counts, first):
        we = w[e].double()
        for got, p, q, terms in ((y[a:b], x[a:b].double(), we.T, K), (dx[a:b], dy[a:b].double(), we, N)):
            ref = p @ q
            assert ((got.double() - ref).abs() <= product_bound(p.abs() @ q.abs(), terms, ref, dt)).all(), e


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(520, 1528), (512, 1536)])
@pytest.mark.parametrize("counts", [[700, 0, 129, 300], [15, 513, 0, 1024], [2, 3, 4, 640]], ids=str)
def test_weight_gradients_of_many_rows(counts, K, N, dtype):
    """Sizes that run on CTA pairs: several partial sums of 512 rows, ragged ends, experts without rows."""
    dt, E, rows = TYPES[dtype], len(counts), sum(counts) + 40
    g = gen(26)
    x, dy = normal(g, rows, K, dtype=dt), normal(g, rows, N, dtype=dt, std=0.5)
    x[sum(counts):], dy[sum(counts):] = float("inf"), float("nan")
    off, ws = offsets_of(counts), moe.control_block()
    base = normal(g, E, N, K, dtype=torch.float32)
    dw, dwf = moe.grouped_mm_wgrad(dy, x, off, ws), moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32)
    acc = moe.grouped_mm_wgrad(dy, x, off, ws, out=base.clone(), accumulate=True)
    assert moe.read_status(ws) == 0
    for e, a, b in spans(counts):
        xe, de = x[a:b].double(), dy[a:b].double()
        ref, mag = de.T @ xe, de.abs().T @ xe.abs()
        for got, want in ((dw[e], ref), (dwf[e], ref), (acc[e], ref + base[e].double())):
            assert ((got.double() - want).abs() <= product_bound(mag, b - a, want, got.dtype)).all(), (e, got.dtype)


@pytest.mark.parametrize("E,n_experts,rows_of", [(44, 16, 1), (44, 16, 3), (44, 40, 1), (3, 3, 65), (5, 5, 66), (44, 9, 40)])
def test_clusters_take_several_tiles(E, n_experts, rows_of):
    """Long contractions over more tiles than clusters: a cluster joins tile after tile, most of whose epilogue warps
    have nothing to send or to sum when an expert holds few rows."""
    K, N = 2048, 1536
    counts = [rows_of] * n_experts + [0] * (E - n_experts)
    g = gen(28)
    rows = sum(counts)
    x, w = normal(g, rows, K), normal(g, E, N, K, std=0.1)
    x8, gate, up, down = normal(g, rows, K), int8_bank(g, E, N, K), int8_bank(g, E, N, K), int8_bank(g, E, K, N)
    off, rs = offsets_of(counts), torch.arange(rows, dtype=torch.int32, device="cuda")
    ws = moe.workspace(rows, K, E, N, 1)
    wt = w.transpose(1, 2).contiguous()
    runs = [[moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(x, wt, off, ws),
             moe.grouped_swiglu(x8, off, rs, 1, gate, up, rows, ws), moe.grouped_down(x8[:, :N].contiguous(), off, rs, None, down, ws)]
            for _ in range(5)]
    assert moe.read_status(ws) == 0
    for r in runs[1:]:
        for a, b in zip(r, runs[0]):
            assert torch.equal(a, b)
    y, dx, h, d = runs[0]
    q, s = codes_of(x8)
    qd, sd = codes_of(x8[:, :N].contiguous())
    for e, a, b in spans(counts)[:n_experts]:
        xe, we = x[a:b].double(), w[e].double()
        ref, mag = xe @ we.T, xe.abs() @ we.abs().T
        for got in (y, dx):
            assert ((got[a:b].double() - ref).abs() <= product_bound(mag, K, ref, torch.bfloat16)).all(), e
        gg, uu = product8(q[a:b], s[a:b], gate, e), product8(q[a:b], s[a:b], up, e)
        ref = gg * torch.sigmoid(gg) * uu
        assert ((h[a:b].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + (1 + gg.abs()) * 2.0 ** -20) + 1e-30).all(), e
        ref = product8(qd[a:b], sd[a:b], down, e)
        assert ((d[a:b].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all(), e


def test_no_rows_at_all():
    """Empty row tensors: nothing to multiply, a zero gradient, an accumulated one left as it was."""
    off, ws, K, N = offsets_of([0, 0]), moe.control_block(), 72, 136
    x, dy = torch.empty(0, K, dtype=torch.bfloat16, device="cuda"), torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    w = normal(gen(25), 2, N, K)
    assert moe.grouped_mm(x, w, off, ws).shape == (0, N) and moe.grouped_mm_dgrad(dy, w, off, ws).shape == (0, K)
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full((2, N, K), 3.0, dtype=dt, device="cuda")
        assert (moe.grouped_mm_wgrad(dy, x, off, ws, out=out) == 0).all()
    out = torch.full((2, N, K), 3.0, device="cuda")
    assert (moe.grouped_mm_wgrad(dy, x, off, ws, out=out, accumulate=True) == 3.0).all()
    assert moe.read_status(ws) == 0


def test_an_expert_keeps_its_infinities():
    """Inf and NaN in one expert's rows or weights reach only that expert's results."""
    counts = [5, 19, 30]
    K, N, rows = 72, 136, sum(counts)
    g = gen(2)
    x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, 3, N, K)
    off, ws = offsets_of(counts), moe.control_block()
    clean = [moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws), moe.grouped_mm_wgrad(dy, x, off, ws)]
    x[5:24], dy[5:24], w[1] = float("inf"), float("nan"), float("-inf")
    got = [moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws), moe.grouped_mm_wgrad(dy, x, off, ws)]
    for a, b in zip(got[:2], clean[:2]):
        assert torch.equal(a[:5], b[:5]) and torch.equal(a[24:], b[24:])
        assert not torch.isfinite(a[5:24]).any()
    assert torch.equal(got[2][0], clean[2][0]) and torch.equal(got[2][2], clean[2][2])


def test_most_experts():
    """1024 experts, few and many rows: the whole table, and its order by size."""
    E, K, N = 1024, 72, 136
    g = gen(21)
    for rows_per in (1, 70):
        counts = torch.randint(0, 2 * rows_per + 1, (E,), generator=g, device="cuda").tolist()
        counts[3] = 40 * rows_per
        rows = sum(counts)
        x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, E, N, K, std=0.1)
        off, ws = offsets_of(counts), moe.control_block()
        y, dx = moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws)
        dw = moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32)
        assert moe.read_status(ws) == 0
        for e, a, b in spans(counts):
            xe, de, we = x[a:b].double(), dy[a:b].double(), w[e].double()
            for got, p, q, terms in ((y[a:b], xe, we.T, K), (dx[a:b], de, we, N), (dw[e], de.T, xe, b - a)):
                ref = p @ q
                assert ((got.double() - ref).abs() <= product_bound(p.abs() @ q.abs(), terms, ref, got.dtype)).all(), e


def test_offsets_past_32_bits():
    """Outputs of more than 2^31 elements: the last rows (and the last expert's gradient) are where they belong."""
    K, N, rows, E = 64, 4096, 560_000, 3
    g = gen(22)
    x, w = normal(g, rows, K), normal(g, E, N, K, std=0.1)
    off, ws = offsets_of([200_000, 0, 360_000]), moe.control_block()
    y = moe.grouped_mm(x, w, off, ws)
    assert y.numel() > 2 ** 31
    for a, e in ((0, 0), (199_990, 0), (200_000, 2), (530_000, 2), (rows - 10, 2)):
        xe, we = x[a:a + 10].double(), w[e].double()
        ref = xe @ we.T
        assert ((y[a:a + 10].double() - ref).abs() <= product_bound(xe.abs() @ we.abs().T, K, ref, y.dtype)).all(), a
    dx = moe.grouped_mm_dgrad(y, w, off, ws)                   # an input of more than 2^31 elements
    for a, e in ((0, 0), (rows - 10, 2)):
        ye, we = y[a:a + 10].double(), w[e].double()
        ref = ye @ we
        assert ((dx[a:a + 10].double() - ref).abs() <= product_bound(ye.abs() @ we.abs(), N, ref, dx.dtype)).all(), a
    assert moe.read_status(ws) == 0


def test_products_repeat_bit_for_bit():
    counts = [300, 0, 77, 1, 512]
    g = gen(3)
    rows, K, N = sum(counts), 520, 392
    x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, 5, N, K)
    off, ws = offsets_of(counts), moe.control_block()

    def all_three():
        return (moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws),
                moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32))

    first = all_three()
    for _ in range(3):
        for a, b in zip(all_three(), first):
            assert torch.equal(a, b)


def test_bad_offsets_are_clipped_and_reported():
    """Offsets that leave the rows or decrease: nothing outside the tensors is touched and the status says so."""
    rows, K, N = 40, 64, 64
    g = gen(4)
    x, dy, w = normal(g, rows, K), normal(g, rows, N), normal(g, 3, N, K)
    for bad in ([0, 10, 5, 40], [-3, 10, 20, 40], [0, 10, 20, 4000], [0, 2 ** 31 - 1, 7, 12]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda ws: moe.grouped_mm(x, w, off, ws), lambda ws: moe.grouped_mm_dgrad(dy, w, off, ws),
                     lambda ws: moe.grouped_mm_wgrad(dy, x, off, ws)):
            ws = moe.control_block()
            call(ws)
            assert moe.read_status(ws) == ERR_INDEX, bad
            assert moe.read_status(ws) == 0


def test_gradients_against_differences():
    """f = sum(c * (x W^T)) in fp32 outputs' precision: a directional difference of f (exact in the step, f is
    linear in x and in W) equals the gradients' inner products."""
    counts = [33, 0, 70]
    rows, K, N = sum(counts), 136, 72
    g = gen(5)
    x, w, c = normal(g, rows, K), normal(g, 3, N, K, std=0.1), normal(g, rows, N)
    vx, vw = normal(g, rows, K), normal(g, 3, N, K, std=0.1)
    off, ws = offsets_of(counts), moe.control_block()
    dx = moe.grouped_mm_dgrad(c, w, off, ws)
    dw = moe.grouped_mm_wgrad(c, x, off, ws, out_dtype=torch.float32)

    def f(xx, ww):
        return sum((c[a:b].double() * (xx[a:b] @ ww[e].T)).sum() for e, a, b in spans(counts))

    xd, wd = x.double(), w.double()
    by_x = (f(xd + vx.double(), wd) - f(xd - vx.double(), wd)) / 2
    by_w = (f(xd, wd + vw.double()) - f(xd, wd - vw.double())) / 2
    # bf16 dx: each element off by 2^-8 of itself (and the sums' 2^-23 N, far below)
    tol_x = (dx.double().abs() * vx.double().abs()).sum() * 2.0 ** -7.9
    assert (by_x - (dx.double() * vx.double()).sum()).abs() <= tol_x
    mag = sum(((c[a:b].double().abs().T @ xd[a:b].abs()) * vw[e].double().abs()).sum() for e, a, b in spans(counts))
    assert (by_w - (dw.double() * vw.double()).sum()).abs() <= mag * 71 * 2.0 ** -23


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------
def codes_of(x):
    """The definition in 64 bits: whole numbers and scales (a row that holds an infinity or a NaN: zeros, NaN)."""
    v = x.double()
    bad = ~torch.isfinite(v).all(1)
    v = torch.where(bad.unsqueeze(1), torch.zeros_like(v), v)
    top = v.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(v * 127.0 / torch.where(top > 0, top, torch.ones_like(top))), 0.0 * v)
    return q, torch.where(bad, float("nan"), (top / 127.0).squeeze(1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (7, 128), (5, 1008), (33, 4096), (3, 20000), (2051, 1536), (2048, 2048)])
def test_quantize_int8_is_exact(rows, cols, dtype):
    dt = TYPES[dtype]
    g = gen(6)
    x = normal(g, rows, cols, dtype=dt)
    x[0] = 0
    for r, f in ((1, 1e-6), (2, 3e4), (3, torch.finfo(dt).smallest_normal), (4, torch.finfo(dt).max / 8)):
        if r < rows:
            x[r] = (x[r].float().clamp(-8, 8) * f).to(dt)
    codes, scales = moe.quantize_int8(x)
    q, s = codes_of(x)
    assert torch.equal(codes.double(), q)
    assert torch.equal(scales.isnan(), s.isnan())
    s, scales = s.nan_to_num(), scales.nan_to_num()
    assert ((scales.double() - s).abs() <= s * 2.0 ** -24 + 2.0 ** -150).all()


def test_quantize_int8_ties_and_every_ratio():
    """Largest magnitude 127 and multiples of a half: ties to even.  Then every bf16 in a row against each of
    some largest magnitudes: the codes of the real quotient."""
    row = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 63.5, 64.5] * 4, dtype=torch.bfloat16, device="cuda")
    codes, scales = moe.quantize_int8(row.unsqueeze(0))
    assert codes[0, :8].tolist() == [127, 0, 2, 2, 0, -2, 64, 64] and scales.item() == 1.0
    bits = torch.arange(0, 0x7F80, device="cuda", dtype=torch.int32)
    values = bits.to(torch.int16).view(torch.bfloat16)
    rows = []
    for top in (1.0, 1.9921875, 3.0e38, 2.0 ** -100, 2.0 ** -126, 2.0 ** -133, 2.0 ** 101, 2.0 ** -90, 254.0):
        t = torch.tensor(top, dtype=torch.bfloat16, device="cuda")
        row = torch.where(values <= t, values, torch.zeros_like(values))
        rows.append(torch.cat([row, t.reshape(1), torch.zeros(15, dtype=torch.bfloat16, device="cuda")]))
    x = torch.stack(rows)
    x = x[:, :x.shape[1] // 16 * 16].contiguous()
    for r in range(x.shape[0]):
        x[r, 0] = x[r].max()
    codes, _ = moe.quantize_int8(x)
    q, _ = codes_of(x)
    assert torch.equal(codes.double(), q)


def test_quantize_int8_nonfinite_rows():
    x = normal(gen(7), 4, 256)
    x[1, 200], x[2, 3] = float("inf"), float("nan")
    codes, scales = moe.quantize_int8(x)
    assert scales.isnan().tolist() == [False, True, True, False]
    assert (codes[1:3] == 0).all() and (codes[0] != 0).any()


def routing(counts, k, g):
    """Slots of the rows: any permutation of T * k slots, bucketed as given."""
    return torch.randperm(sum(counts), generator=g, device="cuda").to(torch.int32)


def int8_bank(g, E, n_out, n_in):
    q = torch.randint(-128, 128, (E, n_out, n_in), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(E, n_out, generator=g, device="cuda") * 2e-3 / n_in ** 0.5
    return moe.Bank(moe.FMT_INT8, q, s)


def product8(q, s, bank, e):
    return (q @ bank.packed[e].double().T) * s.unsqueeze(1) * bank.scales[e].double()


COUNTS8 = {
    "ragged": ([0, 1, 16, 17, 0, 63, 64, 65, 6, 0], 8),
    "decode": ([1, 0, 2, 1, 0, 0, 4, 1, 1, 6], 8),
    "big": ([600, 0, 257, 7], 8),
    "single": ([37], 1),
    "pair": ([61, 3], 2),
    "many": ([700, 0, 129, 300, 7], 8),
}


@pytest.mark.parametrize("load", list(COUNTS8))
@pytest.mark.parametrize("H,F", [(256, 128), (1024, 384), (640, 256), (4096, 1152), (2048, 2048)])
def test_int8_steps_match_the_formula(load, H, F):
    counts, k = COUNTS8[load]
    E, rows = len(counts), sum(counts)
    T = rows // k
    assert T * k == rows
    g = gen(8)
    x = normal(g, T, H, std=1.0)
    x[0] = 0
    gate, up, down = int8_bank(g, E, F, H), int8_bank(g, E, F, H), int8_bank(g, E, H, F)
    rs, off = routing(counts, k, g), offsets_of(counts)
    tw = torch.rand(rows, generator=g, device="cuda")
    ws = moe.workspace(T, H, E, F, min(k, E))
    h = moe.grouped_swiglu(x, off, rs, k, gate, up, rows, ws)
    y = moe.grouped_down(h, off, rs, tw, down, ws)
    y1 = moe.grouped_down(h, off, rs, None, down, ws)
    assert moe.read_status(ws) == 0
    qx, sx = codes_of(x)
    qh, sh = codes_of(h)
    for e, a, b in spans(counts):
        tok = (rs[a:b] // k).long()
        gg, uu = product8(qx[tok], sx[tok], gate, e), product8(qx[tok], sx[tok], up, e)
        ref = gg * torch.sigmoid(gg) * uu
        bound = ref.abs() * (2.0 ** -8 + (1 + gg.abs()) * 2.0 ** -20) + 1e-30
        assert ((h[a:b].double() - ref).abs() <= bound).all(), e
        ref = product8(qh[a:b], sh[a:b], down, e)
        assert ((y1[a:b].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all(), e
        ref = ref * tw[rs[a:b].long()].double().unsqueeze(1)
        assert ((y[a:b].double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-30).all(), e


def test_int8_largest_sums():
    """All codes at +-127 / -128 over a long contraction: the integer sums pass 2^24 and stay exact before the
    one rounding to fp32."""
    E, T, H, F = 2, 16, 16384, 128
    g = gen(9)
    sign = torch.randint(0, 2, (T, 1), generator=g, device="cuda") * 2 - 1
    h = (sign * torch.ones(T, H, device="cuda")).to(torch.bfloat16)
    q = torch.full((E, F, H), -128, dtype=torch.int8, device="cuda")
    q[1] = 127
    down = moe.Bank(moe.FMT_INT8, q, torch.ones(E, F, device="cuda"))
    off = offsets_of([9, 7])
    rs = torch.arange(T, dtype=torch.int32, device="cuda")
    ws = moe.workspace(T, 128, E, H, 1)
    y = moe.grouped_down(h, off, rs, None, down, ws)
    v = torch.tensor([-128.0] * 9 + [127.0] * 7, device="cuda").double().unsqueeze(1) * sign.double() * H
    assert ((y.double() - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -20)).all()


def test_int8_slots_out_of_range_and_repeated():
    """row_slot as a caller may make it: the same token for several rows is fine; a slot outside the batch gives a
    zero row and is reported."""
    counts, k, H, F = [12, 20], 8, 256, 128
    g = gen(23)
    x = normal(g, 4, H)
    gate, up, down = int8_bank(g, 2, F, H), int8_bank(g, 2, F, H), int8_bank(g, 2, H, F)
    off, ws = offsets_of(counts), moe.workspace(4, H, 2, F, 2)
    same = torch.full((32,), 17, dtype=torch.int32, device="cuda")                 # token 2, every row
    h = moe.grouped_swiglu(x, off, same, k, gate, up, 32, ws)
    assert moe.read_status(ws) == 0
    assert torch.equal(h[:12], h[:1].expand(12, F)) and torch.equal(h[12:], h[12:13].expand(20, F))
    rs = routing(counts, k, g)
    ref = moe.grouped_swiglu(x, off, rs, k, gate, up, 32, ws)
    for bad in (-1, 32, 2 ** 31 - 1, -2 ** 31):
        r = rs.clone()
        r[5] = bad
        h = moe.grouped_swiglu(x, off, r, k, gate, up, 32, ws)
        assert moe.read_status(ws) == ERR_INDEX
        keep = torch.arange(32, device="cuda") != 5
        assert (h[5] == 0).all() and torch.equal(h[keep], ref[keep])
        tw = torch.ones(32, device="cuda")
        y = moe.grouped_down(ref, off, r, tw, down, ws)
        assert moe.read_status(ws) == ERR_INDEX and (y[5] == 0).all()


def test_int8_many_tokens_take_the_copy():
    """A batch large enough that tokens are quantised once and their codes copied gives the bits of the small one."""
    T, k, E, H, F = 1100, 8, 8, 2048, 128
    g = gen(24)
    x = normal(g, T, H)
    gate, up = int8_bank(g, E, F, H), int8_bank(g, E, F, H)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1).to(torch.int32).contiguous()
    ws = moe.workspace(T, H, E, F, k)
    off, rs, sr = moe.permute(ids, E, ws)
    h = moe.grouped_swiglu(x, off, rs, k, gate, up, T * k, ws)
    assert moe.read_status(ws) == 0
    qx, sx = codes_of(x)
    o = off.tolist()
    for e in range(E):
        tok = (rs[o[e]:o[e + 1]] // k).long()
        gg, uu = product8(qx[tok], sx[tok], gate, e), product8(qx[tok], sx[tok], up, e)
        ref = gg * torch.sigmoid(gg) * uu
        bound = ref.abs() * (2.0 ** -8 + (1 + gg.abs()) * 2.0 ** -20) + 1e-30
        assert ((h[o[e]:o[e + 1]].double() - ref).abs() <= bound).all(), e
    x[7, 3] = float("inf")                         # seen by the token pass, carried by the copy
    h2 = moe.grouped_swiglu(x, off, rs, k, gate, up, T * k, ws)
    assert moe.read_status(ws) == ERR_NONFINITE
    bad = (rs // k) == 7
    assert h2[bad].isnan().all() and torch.equal(h2[~bad], h[~bad])


def test_int8_nonfinite_row_is_reported():
    counts, k, H, F = [8, 0, 24], 8, 256, 128
    g = gen(10)
    x = normal(g, 4, H)
    gate, up = int8_bank(g, 3, F, H), int8_bank(g, 3, F, H)
    rs, off, ws = routing(counts, k, g), offsets_of(counts), moe.workspace(4, H, 3, F, 3)
    clean = moe.grouped_swiglu(x, off, rs, k, gate, up, 32, ws)
    assert moe.read_status(ws) == 0
    x[2, 9] = float("nan")
    h = moe.grouped_swiglu(x, off, rs, k, gate, up, 32, ws)
    assert moe.read_status(ws) == ERR_NONFINITE
    bad = (rs // k) == 2
    assert h[bad].isnan().all() and torch.equal(h[~bad], clean[~bad])


def layer8(g, E, H, F, k, shared, act_f16=False):
    wr = torch.randn(E, H, generator=g, device="cuda") / H ** 0.5
    sh = None
    if shared:
        sh = [moe.Bank(moe.FMT_BF16, normal(g, 1, o, i, std=0.02)) for o, i in ((F, H), (F, H), (H, F))]
    return moe.MoELayer(int8_bank(g, E, F, H), int8_bank(g, E, F, H), int8_bank(g, E, H, F), wr, top_k=k, shared=sh,
                        act_f16=act_f16)


@pytest.mark.parametrize("T,shared,f16", [(1, False, False), (5, True, False), (64, False, True), (200, True, False),
                                          (130, True, True)])
def test_int8_layer_runs_the_steps(T, shared, f16):
    """moe_layer_forward (and, to 64 tokens, moe_layer_decode and its recording) on int8 banks: the router, the
    steps and the combine as one call.  Every step's formula is tested above; here the layer must give the bits
    of the steps called one by one."""
    E, H, F, k = 16, 512, 256, 8
    g = gen(11)
    L = layer8(g, E, H, F, k, shared, f16)
    x = normal(g, T, H, dtype=torch.float16 if f16 else torch.bfloat16)
    ws = moe.workspace(T, H, E, F, k)
    y = moe.layer_forward(x, L, ws)
    assert moe.read_status(ws) == 0
    if T <= 64:
        assert torch.equal(moe.layer_decode(x, L, ws), y)
    rec = moe.LayerGraph(x, L, moe.workspace(T, H, E, F, k))
    for _ in range(2):
        rec.launch()
    assert torch.equal(rec.y, y) and moe.read_status(rec.ws) == 0
    rec.close()
    if f16:
        return                                   # the steps take bf16 tokens
    ids, tw = moe.route_topk(x, L.router_w, None, k, ws)
    off, rs, sr = moe.permute(ids, E, ws)
    h = moe.grouped_swiglu(x, off, rs, k, L.gate, L.up, T * k, ws)
    yp = moe.grouped_down(h, off, rs, tw.reshape(-1), L.down, ws)
    ys = None
    if shared:
        o1 = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        r1 = (torch.arange(T, device="cuda") * k).to(torch.int32)
        hs = moe.grouped_swiglu(x, o1, r1, k, L.shared[0], L.shared[1], T, ws)
        ys = moe.grouped_down(hs, o1, r1, None, L.shared[2], ws)
    assert torch.equal(moe.unpermute_combine(yp, sr, T, k, ys), y)


# ---------------------------------------------------------------------------
# a run of them together; streams, graphs, threads, failures
# ---------------------------------------------------------------------------
def test_training_step_of_the_experts():
    """Gather, three products, SwiGLU between them, and their gradients: against the same network in 64 bits.
    Every product rounds to bf16 once; h and its gradients are computed from the rounded products, so the
    64-bit network takes the same rounded values at each product's input."""
    T, E, H, F, k = 40, 6, 128, 72, 2
    g = gen(12)
    x = normal(g, T, H)
    wg, wu, wd = (normal(g, E, o, i, std=0.1) for o, i in ((F, H), (F, H), (H, F)))
    wr = torch.randn(E, H, generator=g, device="cuda")
    ws = moe.workspace(T, 128, E, 128, k)
    ids, tw = moe.route_topk(x, wr, None, k, ws)
    off, rs, sr = moe.permute(ids, E, ws)
    xp = x[(rs // k).long()]
    gate, up = moe.grouped_mm(xp, wg, off, ws), moe.grouped_mm(xp, wu, off, ws)
    gf, uf = gate.float(), up.float()
    sig = torch.sigmoid(gf)
    h = (gf * sig * uf).to(torch.bfloat16)
    y = moe.grouped_mm(h, wd, off, ws)
    dy = normal(g, T * k, H)
    dh = moe.grouped_mm_dgrad(dy, wd, off, ws)
    dwd = moe.grouped_mm_wgrad(dy, h, off, ws, out_dtype=torch.float32)
    du = (dh.float() * gf * sig).to(torch.bfloat16)
    dg = (dh.float() * uf * sig * (1 + gf * (1 - sig))).to(torch.bfloat16)
    dwg = moe.grouped_mm_wgrad(dg, xp, off, ws, out_dtype=torch.float32)
    dwu = moe.grouped_mm_wgrad(du, xp, off, ws, out_dtype=torch.float32)
    dxg, dxu = moe.grouped_mm_dgrad(dg, wg, off, ws), moe.grouped_mm_dgrad(du, wu, off, ws)
    assert moe.read_status(ws) == 0
    o = off.tolist()
    for e in range(E):
        a, b = o[e], o[e + 1]
        X, Hh, DY, DG, DU = (t[a:b].double() for t in (xp, h, dy, dg, du))
        for got, p, q, terms in ((gate[a:b], X, wg[e].double().T, H), (up[a:b], X, wu[e].double().T, H),
                                 (y[a:b], Hh, wd[e].double().T, F), (dh[a:b], DY, wd[e].double(), H),
                                 (dwd[e], DY.T, Hh, b - a), (dwg[e], DG.T, X, b - a), (dwu[e], DU.T, X, b - a),
                                 (dxg[a:b], DG, wg[e].double(), F), (dxu[a:b], DU, wu[e].double(), F)):
            ref = p @ q
            assert ((got.double() - ref).abs() <= product_bound(p.abs() @ q.abs(), terms, ref, got.dtype)).all()


def _calls(seed=13):
    counts, k, H, F = [40, 0, 1, 23], 8, 256, 128
    g = gen(seed)
    rows = sum(counts)
    x, dy = normal(g, rows, 264), normal(g, rows, 136)
    w = normal(g, 4, 136, 264)
    off, rs = offsets_of(counts), routing(counts, k, g)
    x8 = normal(g, rows // k, H)
    gate, up, down = int8_bank(g, 4, F, H), int8_bank(g, 4, F, H), int8_bank(g, 4, H, F)

    def run(ws):
        h = moe.grouped_swiglu(x8, off, rs, k, gate, up, rows, ws)
        return [moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws), moe.grouped_mm_wgrad(dy, x, off, ws),
                h, moe.grouped_down(h, off, rs, None, down, ws)]

    return run, lambda: moe.workspace(rows // k, H, 4, F, 4)


def _large_calls(seed=16):
    """The same calls at sizes that run on CTA pairs, and with few tiles on clusters that share a contraction."""
    counts, few, k, H, F = [700, 0, 300, 24], [3, 60], 8, 2560, 2560
    g = gen(seed)
    rows = sum(counts)
    x, dy, w = normal(g, rows, 2600), normal(g, rows, 2568), normal(g, 4, 2568, 2600)
    xs, ws_ = normal(g, 63, 2048), normal(g, 2, 136, 2048)
    xl, dyl, offl = normal(g, 601, 2048), normal(g, 601, 1536), offsets_of([601])
    off, offs, rs = offsets_of(counts), offsets_of(few), routing(counts, k, g)
    x8 = normal(g, rows // k, H)
    gate, up, down = int8_bank(g, 4, F, H), int8_bank(g, 4, F, H), int8_bank(g, 4, H, F)

    def run(ws):
        h = moe.grouped_swiglu(x8, off, rs, k, gate, up, rows, ws)
        return [moe.grouped_mm(x, w, off, ws), moe.grouped_mm_dgrad(dy, w, off, ws), moe.grouped_mm_wgrad(dy, x, off, ws),
                moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float32), moe.grouped_mm(xs, ws_, offs, ws), h,
                moe.grouped_mm_wgrad(dyl, xl, offl, ws), moe.grouped_mm_wgrad(dyl[:, :136].contiguous(), xl, offl, ws),
                moe.grouped_down(h, off, rs, None, down, ws)]

    return run, lambda: moe.workspace(rows // k, H, 4, F, 4)


@pytest.mark.parametrize("calls", [_calls, _large_calls], ids=["small", "large"])
def test_captured_and_replayed(calls):
    """Two graphs captured over one workspace, replayed in turn."""
    run, new_ws = calls()
    ws = new_ws()
    ref = run(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(run(ws))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert moe.read_status(ws) == 0
    for gr in graphs:
        gr.reset()


@pytest.mark.parametrize("calls", [_calls, _large_calls], ids=["small", "large"])
def test_two_streams_and_threads(calls):
    """Calls on two streams from two host threads with separate workspaces: the bits of one thread."""
    made = [calls(s) for s in (14, 15)]
    refs = [run(new()) for run, new in made]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            run, new = made[i]
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                ws = new()
                for _ in range(10):
                    got[i] = run(ws)
            st.synchronize()
        except Exception as e:                    # noqa: BLE001
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not errors, errors
    for out, ref in zip(got, refs):
        for a, b in zip(out, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("calls", [_calls, _large_calls], ids=["small", "large"])
def test_wait_limit_runs_out_then_recovers(calls):
    run, new_ws = calls()
    ws = new_ws()
    ref = run(ws)
    assert moe.read_status(ws) == 0
    moe.set_wait_limit(ws, 1_000_000)
    moe.set_wait_hold(ws, 1)
    run(ws)
    torch.cuda.synchronize()                      # the kernels returned
    assert moe.read_status(ws) == ERR_TIMEOUT
    moe.set_wait_hold(ws, 0)
    moe.set_wait_limit(ws, 0)
    for a, b in zip(run(ws), ref):
        assert torch.equal(a, b)
    assert moe.read_status(ws) == 0


def test_binding_checks_shapes_and_types():
    x, w = normal(gen(1), 8, 64), normal(gen(1), 2, 32, 64)
    off, ws = offsets_of([4, 4]), moe.control_block()
    dy = normal(gen(1), 8, 32)
    bad = [lambda: moe.grouped_mm(x.t(), w, off, ws), lambda: moe.grouped_mm(x[:, ::2], w, off, ws),
           lambda: moe.grouped_mm(x, w[:1], off, ws), lambda: moe.grouped_mm(x, w, off.long(), ws),
           lambda: moe.grouped_mm(x, w.half(), off, ws), lambda: moe.grouped_mm(x, w, off.cpu(), ws),
           lambda: moe.grouped_mm(x, w, off, ws, out=dy.float()), lambda: moe.grouped_mm_dgrad(x, w, off, ws),
           lambda: moe.grouped_mm_wgrad(dy[:4], x, off, ws), lambda: moe.grouped_mm_wgrad(dy, x, off, ws, accumulate=True),
           lambda: moe.grouped_mm_wgrad(dy, x, off, ws, out_dtype=torch.float16),
           lambda: moe.grouped_mm(x, w, off[:2], ws), lambda: moe.grouped_mm(x, w, off, ws.float()),
           lambda: moe.Bank(moe.FMT_INT8, w, dy), lambda: moe.Bank(moe.FMT_INT8, w.to(torch.int8), None),
           lambda: moe.Bank(moe.FMT_INT8, w.to(torch.int8), torch.ones(2, 31, device="cuda")),
           lambda: moe.Bank(moe.FMT_INT8, w.to(torch.int8), torch.ones(2, 32, dtype=torch.bfloat16, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.code == -1, i
    with pytest.raises(moe.MoEError) as err:
        moe.grouped_mm_wgrad(dy, x, off, ws, out=torch.zeros(2, 32, 64, dtype=torch.bfloat16, device="cuda"),
                             accumulate=True)
    assert err.value.code == -2

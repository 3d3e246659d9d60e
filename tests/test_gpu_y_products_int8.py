"""Both ways of quantising the tokens of the 8-bit experts on the GPU: each row from its token, and (from 2^24 codes)
the tokens once, whose codes are then copied to the rows."""
import pytest
import torch

from test_gpu_y_products import ERR_INDEX, ERR_NONFINITE, _cuda, gen, int8_bank, normal  # noqa: F401
from weight_only_bit_route_b200 import moe

pytestmark = pytest.mark.gpu

E, H, F, K = 16, 2048, 128, 8
SMALL, LARGE = 1000, 1100                        # 8000 * 2048 codes < 2^24 <= 8800 * 2048


def _setup(seed):
    g = gen(seed)
    x = normal(g, LARGE, H)
    x[3] = 0
    ids = torch.rand(LARGE, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32).contiguous()
    return x, ids, int8_bank(g, E, F, H), int8_bank(g, E, F, H), moe.workspace(LARGE, H, E, F, K)


def _by_slot(x, ids, gate, up, ws, T, want_permute=0):
    """h by slot ([T * K, F]; slots that no expert takes: zeros) and the status of the call."""
    off, rs, sr = moe.permute(ids[:T].contiguous(), E, ws)
    assert moe.read_status(ws) == want_permute
    h = moe.grouped_swiglu(x[:T].contiguous(), off, rs, K, gate, up, T * K, ws)
    status = moe.read_status(ws)
    out = torch.zeros_like(h)
    live = sr.reshape(-1) >= 0
    out[live] = h[sr.reshape(-1)[live].long()]
    return out, status


def test_the_copy_gives_the_bits_of_the_rows():
    """The codes, scales and products of a slot do not depend on how its token was quantised."""
    x, ids, gate, up, ws = _setup(31)
    small, s0 = _by_slot(x, ids, gate, up, ws, SMALL)
    large, s1 = _by_slot(x, ids, gate, up, ws, LARGE)
    assert (s0, s1) == (0, 0) and small.abs().max() > 0
    assert torch.equal(small, large[:SMALL * K])


@pytest.mark.parametrize("T", [SMALL, LARGE])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_no_row_refers_to_is_not_reported(T, bad):
    """Token 7 is routed nowhere: what it holds is nobody's error, at any batch size.  Token 8 is: its rows are."""
    x, ids, gate, up, ws = _setup(32)
    ids[7] = -1
    clean, status = _by_slot(x, ids, gate, up, ws, T, want_permute=ERR_INDEX)
    assert status == 0
    x[7, 11] = bad
    got, status = _by_slot(x, ids, gate, up, ws, T, want_permute=ERR_INDEX)
    assert status == 0 and torch.equal(got, clean)
    x[8, 5] = bad
    got, status = _by_slot(x, ids, gate, up, ws, T, want_permute=ERR_INDEX)
    assert status == ERR_NONFINITE
    rows = torch.zeros(T * K, dtype=torch.bool, device="cuda")
    rows[8 * K:9 * K] = True
    assert got[rows].isnan().all() and torch.equal(got[~rows], clean[~rows])

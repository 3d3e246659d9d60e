"""The binding's refusals of tensors that are not on a GPU, before any pointer reaches the library (no GPU needed)."""
import pytest
import torch

from weight_only_bit_route_b200 import moe


def test_grouped_calls_refuse_host_tensors():
    T, k, H, F, E = 4, 2, 256, 128, 3
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    gate = moe.Bank(moe.FMT_INT8, torch.zeros(E, F, H, dtype=torch.int8), torch.ones(E, F))
    down = moe.Bank(moe.FMT_INT8, torch.zeros(E, H, F, dtype=torch.int8), torch.ones(E, H))
    off, rs = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(T * k, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    h = torch.zeros(T * k, F, dtype=torch.bfloat16)
    for call in (lambda: moe.grouped_swiglu(x, off, rs, k, gate, gate, T * k, ws),
                 lambda: moe.grouped_down(h, off, rs, None, down, ws)):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.code == -1

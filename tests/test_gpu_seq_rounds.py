"""The fp32 backward of packed-sequence attention by a few rounds of blocks an SM, where how many lie on one, and how the
row terms' kernel goes before them, is chosen by the number of units.  Sizes follow the device."""
import pytest
import torch

from test_gpu_seq_large import check, sms

pytestmark = pytest.mark.gpu


# units an SM on each side of what the choices go by
@pytest.mark.parametrize("D,H,Hk,causal,per_sm", [
    (64, 4, 4, True, 1.4), (64, 4, 4, True, 1.9), (64, 8, 8, True, 2.4), (64, 8, 8, False, 1.9), (64, 8, 8, False, 2.4), (64, 8, 8, False, 2.9),
    (64, 8, 4, False, 2.4), (32, 8, 8, False, 1.9), (32, 8, 8, False, 2.7), (32, 8, 8, False, 3.3), (32, 8, 8, False, 3.7), (32, 8, 8, False, 4.3),
    (32, 8, 4, False, 3.5), (32, 8, 4, False, 4.2), (32, 8, 4, False, 4.8), (32, 8, 2, False, 4.8), (32, 8, 8, True, 2.5), (32, 8, 4, True, 3.9),
    (32, 8, 4, True, 4.5), (128, 4, 4, False, 2.2)])
def test_units_an_sm(D, H, Hk, causal, per_sm):
    tiles = int(per_sm * sms() / (2 * (H + Hk)))
    rows = 64 * tiles - 7
    _, _, first = check([rows - 70, 70], H, Hk, D, "f32", causal)
    _, _, again = check([rows - 70, 70], H, Hk, D, "f32", causal)
    assert all(torch.equal(a, b) for a, b in zip(first, again))

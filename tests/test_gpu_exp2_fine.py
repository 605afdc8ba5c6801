"""The exponential on the FMA pipe that the prompt weights use, over the whole
range of its argument.

Bound: the polynomial is off by at most 1.6e-7 of 2^f for f in [-1/2, 1/2]; the
last of its fp32 steps by half a unit of a result in [0.7, 1.42], 2^-24 relative,
and the ones before it, each multiplied by |f| <= 1/2 once more, by less than 2^-25
together: 2.5e-7."""
import pytest
import torch

import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu


def test_against_64_bits():
    swa.build()
    x = torch.cat([torch.linspace(-126.0, 100.0, 4_000_001, device="cuda"),
                   torch.rand(4_000_000, device="cuda") - 0.5, torch.arange(-126.0, 101.0, device="cuda"),
                   torch.arange(-126.0, 101.0, device="cuda") + 0.49999997,
                   torch.arange(-125.0, 101.0, device="cuda") - 0.49999997])
    y = swa.swa_selftest_exp2_fine(x).double()
    want = torch.exp2(x.double())
    assert ((y - want).abs() / want).max().item() <= 2.5e-7


def test_below_the_clamp_and_odd_counts():
    lo = torch.tensor([-126.0, -126.5, -1e30, float("-inf"), float("nan")], device="cuda")
    assert (swa.swa_selftest_exp2_fine(lo) == 2.0 ** -126).all()
    for n in (1, 2, 3, 511, 513):
        x = torch.linspace(-3, 3, n, device="cuda")
        y = swa.swa_selftest_exp2_fine(x)
        assert ((y - torch.exp2(x)).abs() <= 5e-7 * torch.exp2(x)).all()

"""A 16-bit rolling buffer that is not yet full, converted as include/swa.h says:
its own positions alone, whatever the rest of it holds."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    swa.build()
    swa.lib()
    yield
    assert swa.swa_get_device_status() == swa.SWA_OK


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("junk", [3e38, float("nan"), float("inf")])
def test_partly_filled_sequences(block, junk):
    """Lengths inside a block, at its border, of one position, and full; the slots
    behind them hold what a fresh allocation may."""
    rng = np.random.default_rng(block)
    W, H, D, lens = 100, 2, 64, [1, 15, 16, 37, 64, 99, 100, 250]
    B = len(lens)
    k16 = torch.full((B, W, H, D), junk, dtype=torch.bfloat16, device="cuda")
    v16 = k16.clone()
    for b, n in enumerate(lens):
        k = torch.tensor(rng.standard_normal((1, min(n, W), H, D)), dtype=torch.bfloat16, device="cuda")
        first = torch.tensor([max(0, n - W)], dtype=torch.int32, device="cuda")
        swa.swa_cache_append(k, 2 * k, k16[b:b + 1], v16[b:b + 1], first)
    k8 = torch.full((B, W, H, D), 0x7F, dtype=torch.uint8, device="cuda").view(F8)
    v8, ks = k8.clone(), torch.full((B, -(-W // block), H), float("nan"), device="cuda")
    vs = ks.clone()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        m = min(n, W)
        swa.swa_cache_append_q8(k16[b:b + 1, :m], v16[b:b + 1, :m], k8[b:b + 1], v8[b:b + 1], ks[b:b + 1], vs[b:b + 1],
                                zero, block=block)
    for b, n in enumerate(lens):
        m = min(n, W)
        for x16, x8, s in ((k16, k8, ks), (v16, v8, vs)):
            want = ref.f64(x16[b, :m])
            step = np.repeat(ref.f64(s[b]), block, 0)[:m, :, None]
            got = ref.f64(x8[b, :m]) * step
            # half a step of e4m3: 2^-4 relative, 2^-10 of the scale for its subnormals
            assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step)).all(), n
            assert (step <= 2.0 ** -5).all() and (x8[b, m:].view(torch.uint8) == 0x7F).all()

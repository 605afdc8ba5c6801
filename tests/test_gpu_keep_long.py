"""The cut of prompts around and above the length whose order numbers fit in
shared memory (40960), against the plain form: positions, rows and weights bit
for bit."""
import numpy as np
import pytest
import torch

import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    swa.build()
    swa.lib()
    yield
    assert swa.swa_get_device_status() == swa.SWA_OK


def kept(w, n, M, S, R):
    """The positions of a prompt of n that stay, in order (ties: the lowest)."""
    if n <= M:
        return np.arange(n)
    order = np.where(np.isnan(w), np.inf, w)[S:n - R]
    middle = S + np.argsort(-order, kind="stable")[:M - S - R]
    return np.concatenate([np.arange(S), np.sort(middle), np.arange(n - R, n)])


@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
@pytest.mark.parametrize("N,M,S,R", [(40959, 3000, 4, 100), (40960, 5000, 0, 1), (40961, 40000, 16, 333),
                                     (70001, 2048, 4, 256), (70000, 20, 4, 16)])
def test_long_prompts(N, M, S, R, kind):
    rng = np.random.default_rng(N + M)
    B, H, D = 3, 2, 64
    lens = [N, N - 777, M - 1]
    w = rng.random((B, H, N)) ** 4 * 8
    if kind == "ties":
        w = np.floor(w * 3) / 3
    w = w.astype(np.float32)
    if kind == "special":
        w[:, :, ::5] = np.nan
        w[:, :, 1::5] = np.inf
        w[:, :, 2::5] = -0.0
        w[:, :, 3::5] = 0.0
        w[:, 1] = -w[:, 1]
    g = torch.Generator(device="cuda").manual_seed(N)
    k, v = (torch.randn(B, N, H, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    kc, vc = torch.full((B, M, H, D), 7.0, dtype=BF16, device="cuda"), torch.full((B, M, H, D), 9.0, dtype=BF16, device="cuda")
    at = torch.full((B, H, M), 12345, dtype=torch.int32, device="cuda")
    wo, wt = torch.full((B, H, M), 3.0, device="cuda"), torch.tensor(w, device="cuda")
    swa.swa_cache_keep(k, v, wt, torch.tensor(lens, dtype=torch.int32, device="cuda"), kc, vc, at, wo, S, R)
    for b, n in enumerate(lens):
        for h in range(H):
            want = kept(w[b, h], n, M, S, R)
            m = len(want)
            np.testing.assert_array_equal(at[b, h].cpu().numpy(), np.concatenate([want, np.full(M - m, -1)]))
            idx = torch.tensor(want, device="cuda")
            assert torch.equal(wo[b, h, :m].view(torch.int32), wt[b, h, idx].view(torch.int32))
            assert torch.equal(kc[b, :m, h], k[b, idx, h]) and torch.equal(vc[b, :m, h], v[b, idx, h])
            assert not wo[b, h, m:].any() and (kc[b, m:, h] == 7).all() and (vc[b, m:, h] == 9).all()

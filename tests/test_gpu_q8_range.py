"""Values over the whole range an 8-bit buffer holds (scales from 2^-117 to
2^119), through every way the splits of a decode are joined, against the plain
64-bit form (tests/cache_ref.py).

Bound, element by element: the rounding of the output to bf16, 2^-8 |ref|; of
each weight to f16, 2^-11, in a quotient by the sum of the rounded weights, so
twice it times the largest |v| of that column; and the scores, off by d = 2^-18
scale sum |q k|, which moves the output by at most 2 d times it."""
import math

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


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.tensor(x, dtype=torch.float64).to(torch.bfloat16).cuda()


def decode_and_check(k, v, q, pos, block):
    B, W, H, D = k.shape
    Hq, scale = q.shape[1], 1 / math.sqrt(D)
    k8 = torch.zeros(B, W, H, D, device="cuda").to(F8)
    v8, ks = k8.clone(), torch.zeros(B, -(-W // block), H, device="cuda")
    vs = ks.clone()
    swa.swa_cache_append_q8(bf16(k), bf16(v), k8, v8, ks, vs, i32([0] * B), block=block)
    out = swa.swa_decode_q8(bf16(q), k8, v8, ks, vs, i32(pos), scale, block=block)
    for b, p in enumerate(pos):
        n = min(p + 1, W)
        kk = ref.widen(ref.f64(k8[b]), ref.f64(ks[b]), block)[:n]
        vv = ref.widen(ref.f64(v8[b]), ref.f64(vs[b]), block)[:n]
        want, _, big = ref.attend(ref.f64(bf16(q[b])), kk, vv, np.ones(n, bool), scale)
        d = 2.0 ** -18 * big * scale
        top = np.repeat(np.abs(vv).max(0), Hq // H, 0)
        got = ref.f64(out[b])
        assert np.isfinite(got).all(), f"sequence {b}: {np.isinf(got).sum()} infinite, {np.isnan(got).sum()} NaN"
        bad = np.abs(got - want) / (2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -11 + 2 * d) * top + 1e-42)
        assert bad.max() <= 1, f"sequence {b}: {bad.max():.3f} of the bound"


# one split; four, merged in a cluster; several, through the workspace; a group in two pieces
SHAPES = [(2, 2, 2, 100), (2, 4, 2, 1024), (1, 4, 1, 4500), (1, 12, 1, 1500)]


@pytest.mark.parametrize("power", [-115, -60, 0, 50, 68, 70, 100, 115, 126])
@pytest.mark.parametrize("B,Hq,H,W", SHAPES)
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_one_magnitude(D, B, Hq, H, W, power):
    """All of one sign, so that the sums are as large as the values allow."""
    rng = np.random.default_rng(200 + power + W)
    v = (1 + 0.7 * rng.random((B, W, H, D))) * 2.0 ** power
    k, q = rng.standard_normal((B, W, H, D)), rng.standard_normal((B, Hq, D))
    decode_and_check(k, v, q, [W - 1 - 13 * b for b in range(B)], 64)


@pytest.mark.parametrize("at", [0, 37, 700, 1499])
@pytest.mark.parametrize("B,Hq,H,W", SHAPES)
def test_one_large_value_among_ordinary_ones(B, Hq, H, W, at):
    """One key's value is near the top of the range in one column: that column
    shows it, the other columns keep the precision of their own values."""
    rng = np.random.default_rng(at + W)
    v = rng.standard_normal((B, W, H, 64))
    v[:, min(at, W - 1), :, 5] = 1.6 * 2.0 ** 127
    k, q = rng.standard_normal((B, W, H, 64)), rng.standard_normal((B, Hq, 64))
    decode_and_check(k, v, q, [3 * W] * B, 16)


def test_an_even_weight_on_the_largest_values():
    """4096 keys of the same weight and of the largest value."""
    v = np.full((1, 4096, 1, 64), 448 * 2.0 ** 119)
    decode_and_check(np.zeros_like(v), v, np.ones((1, 1, 64)), [4095], 128)

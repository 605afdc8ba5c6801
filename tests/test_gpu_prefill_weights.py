"""The softmax weights a prompt's keys receive from its last T queries, against
a plain 64-bit form (tests/cache_ref.py), and the whole way of a prompt through
the fixed-size cache.

Bound, per weight, relative to the sum: scores are sums of D exact products in
D/16 steps, each off by at most 2^-22 of sum |q k|, and rounded three times
(d = 2^-18 scale sum |q k|, entering once through the score and once through
lse); lse is rounded at its own magnitude, at most scale log2(e) sum |q k| +
log2 N, by 2^-24; the exponential, the logarithm and the joining of the parts
add 2^-20; the sum over a tile's columns runs in chains of 32 and then over the
tiles, each addition off by 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
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


def rows(rng, *shape, outliers=False):
    x = rng.standard_normal(shape)
    if outliers:
        x[..., ::17, :, :] *= 8
    return torch.tensor(x, dtype=BF16, device="cuda")


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def check(q, k, lens, W, scale, got):
    B, T, Hq, D = q.shape
    N, H = k.shape[1], k.shape[2]
    tiles = T * (Hq // H) / 64 + 2
    got = ref.f64(got)
    assert np.isfinite(got).all()
    for b in range(B):
        n = lens[b] if 0 <= lens[b] <= N else 0
        kk = np.where((np.arange(N) < n)[:, None, None], ref.f64(k[b]), 0.0)
        want = ref.prompt_weights(ref.f64(q[b]), kk, n, W, scale)
        big = float(np.abs(ref.f64(q[b])).max(1).sum(-1).max() * np.abs(kk).max(initial=0.0))
        d = 2.0 ** -18 * scale * big
        tol = (2 * d + (scale * math.log2(math.e) * big + math.log2(N) + 1) * 2.0 ** -24 + 2.0 ** -20
               + (36 + tiles) * 2.0 ** -24) * want + 1e-30
        bad = np.abs(got[b] - want) / tol
        assert bad.max() <= 1, f"sequence {b}: {bad.max():.3f} of the bound"
        assert not got[b][:, n:].any()


def run(rng, B, N, T, Hq, H, D, W, lens, outliers=False):
    q, k = rows(rng, B, T, Hq, D), rows(rng, B, N, H, D, outliers=outliers)
    for b, n in enumerate(lens):
        if 0 <= n < N:
            k[b, n:] = float("nan")          # beyond the prompt: never to be used
    scale = 1 / math.sqrt(D)
    got = swa.swa_prefill_weights(q, k, i32(lens), W, scale)
    check(q, k, lens, W, scale, got)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 12, 33, 128])
def test_groups(D, G):
    rng = np.random.default_rng(G * D)
    run(rng, 2, 150, 20 if G < 32 else 3, 2 * G, 2, D, 150, [150, 77])


@pytest.mark.parametrize("N,T", [(1, 1), (2, 2), (127, 127), (128, 1), (129, 129), (200, 31), (300, 300), (513, 64)])
@pytest.mark.parametrize("W", [1, 7, 128, 1000])
def test_lengths_and_windows(N, T, W):
    """Prompts around the tiles, from the last query alone to all of them, and
    lengths shorter than T, of one position and of none."""
    rng = np.random.default_rng(N * T + W)
    run(rng, 4, N, T, 4, 2, 64, W, [N, max(1, N // 2), 1, 0])


def test_many_tiles_to_a_unit():
    """One head with many key tiles and many query tiles: units split, results
    joined; the ring and the tensor-memory buffers turn over many times."""
    rng = np.random.default_rng(1)
    run(rng, 1, 2500, 40, 2, 1, 128, 2500, [2500], outliers=True)
    run(rng, 1, 1300, 1300, 1, 1, 64, 1300, [1300], outliers=True)


def test_more_units_than_blocks():
    rng = np.random.default_rng(2)
    run(rng, 12, 400, 30, 8, 8, 64, 100, [400 - 31 * b for b in range(12)])


def test_sharp_softmax():
    """Scores of several hundred: one key takes the weight of each query."""
    rng = np.random.default_rng(3)
    q, k = rows(rng, 1, 60, 4, 64) * 8, rows(rng, 1, 200, 2, 64) * 8
    scale = 0.125
    got = swa.swa_prefill_weights(q, k, i32([200]), 200, scale)
    check(q, k, [200], 200, scale, got)


def test_every_query_gives_one_unit_of_weight():
    rng = np.random.default_rng(4)
    q, k = rows(rng, 2, 700, 6, 128), rows(rng, 2, 700, 2, 128)
    w = swa.swa_prefill_weights(q, k, i32([700, 500]), 300, 0.09)
    total = w.double().sum(-1)
    assert (total - torch.tensor([[2100.0], [1500.0]], device="cuda")).abs().max() < 2100 * 2.0 ** -16


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_shows_where_it_is_seen(value):
    """A key (or query) that is not finite makes the weights of the queries that
    see it, and so of the keys they see, not finite; other sequences and heads
    keep theirs."""
    rng = np.random.default_rng(9)
    for where in range(40, 56):                        # every column pair of the exponentials
        q, k = rows(rng, 2, 200, 2, 64), rows(rng, 2, 200, 2, 64)
        q[..., 5] = q[..., 5].abs() + 0.1              # an infinite key scores +infinity
        clean = swa.swa_prefill_weights(q, k, i32([200, 200]), 200, 0.1)
        k[0, where, 0, 5] = value
        w = swa.swa_prefill_weights(q, k, i32([200, 200]), 200, 0.1)
        assert not torch.isfinite(w[0, 0]).any()       # query 199 sees all of them
        assert torch.equal(w[1], clean[1]) and torch.equal(w[0, 1], clean[0, 1])
    q, k = rows(rng, 1, 200, 1, 64), rows(rng, 1, 200, 1, 64)
    q[0, 150, 0, 3] = value
    w = swa.swa_prefill_weights(q, k, i32([200]), 200, 0.1)
    assert not torch.isfinite(w[0, 0, :151]).any() and torch.isfinite(w[0, 0, 151:]).all()


def test_a_length_outside_the_prompt_gives_zeros_and_is_recorded():
    rng = np.random.default_rng(5)
    run(rng, 3, 140, 9, 4, 2, 64, 140, [141, -1, 140])
    assert swa.swa_get_device_status() == swa.SWA_ERR_INVALID_ARG


def test_repeated_and_on_another_stream_the_same_bits():
    rng = np.random.default_rng(6)
    q, k, lens = rows(rng, 2, 100, 8, 128), rows(rng, 2, 900, 2, 128), i32([900, 850])
    want = swa.swa_prefill_weights(q, k, lens, 900, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [swa.swa_prefill_weights(q, k, lens, 900, 0.1, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_a_prompt_through_the_fixed_size_cache():
    """Prefill, weights, the cut to M slots, then tokens: each step against the
    plain form on the state the GPU had."""
    rng = np.random.default_rng(8)
    B, N, Hq, H, D, M, S, R, T = 2, 300, 6, 2, 64, 64, 4, 16, 32
    lens, scale = [300, 251], 0.125
    q, k, v = rows(rng, B, N, Hq, D), rows(rng, B, N, H, D), rows(rng, B, N, H, D)
    swa.swa_prefill(q, k, v, N, scale)
    last = torch.stack([q[b, n - T:n] for b, n in enumerate(lens)]).contiguous()
    w = swa.swa_prefill_weights(last, k, i32(lens), N, scale)
    check(last, k, lens, N, scale, w)
    kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
    vc, at = torch.zeros_like(kc), torch.zeros(B, H, M, dtype=torch.int32, device="cuda")
    wc = torch.zeros(B, H, M, device="cuda")
    swa.swa_cache_keep(k, v, w, i32(lens), kc, vc, at, wc, S, R)
    for b, n in enumerate(lens):
        for h in range(H):
            kept = ref.keep(w[b, h].cpu().numpy(), n, M, S, R)
            assert at[b, h].tolist() == kept
            assert torch.equal(kc[b, :, h], k[b, kept, h]) and torch.equal(vc[b, :, h], v[b, kept, h])
    for step in range(20):
        pos = [n + step for n in lens]
        k1, v1, q1 = rows(rng, B, H, D), rows(rng, B, H, D), rows(rng, B, Hq, D)
        want = [[ref.evict(at[b, h].tolist(), wc[b, h].cpu().numpy(), pos[b], S, R) for h in range(H)] for b in range(B)]
        assert swa.swa_cache_evict_append(k1, v1, kc, vc, at, wc, i32(pos), S, R).tolist() == want
        out, _ = swa.swa_decode_weights(q1, kc, vc, at, wc, i32(pos), scale)
        for b in range(B):
            o, _, big = ref.attend(ref.f64(q1[b]), ref.f64(kc[b]), ref.f64(vc[b]), np.ones((H, M), bool), scale)
            d = big * scale * 2.0 ** -18
            assert (np.abs(ref.f64(out[b]) - o)
                    <= 2.0 ** -8 * np.abs(o) + (2.0 ** -7 + 2 * d) * np.abs(ref.f64(vc[b])).max()).all()

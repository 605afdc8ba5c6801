"""Queries that are not finite, in every column of the products in which the
queries are the columns, whichever exponential that column takes: the keys the
query sees get weights that are not finite, the others keep theirs."""
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


def rows(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=BF16, device="cuda")


# (N, T, G, first query that is spoilt): all queries in two tiles, which stay
# while keys are streamed; and more, streamed past the keys
FORMS = [(400, 64, 1, 0), (400, 16, 4, 0), (600, 600, 1, 384), (500, 500, 2, 384)]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("N,T,G,first", FORMS)
def test_a_query_that_is_not_finite_shows_in_every_key_it_sees(N, T, G, first, value):
    rng = np.random.default_rng(N + G)
    B = 64                                             # sequence b: row b of a run of 64 (query, head) rows
    one_q, one_k = rows(rng, 1, T, G, 64), rows(rng, 1, N, 1, 64)
    q, k = one_q.repeat(B, 1, 1, 1), one_k.repeat(B, 1, 1, 1).contiguous()
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    clean = swa.swa_prefill_weights(q, k, lens, N, 0.1)
    assert torch.isfinite(clean).all()
    at = [first + b // G for b in range(B)]            # query spoilt, its head b % G
    for b in range(B):
        q[b, at[b], b % G, 3] = value
    got = swa.swa_prefill_weights(q, k, lens, N, 0.1)
    for b in range(B):
        seen = N - T + at[b] + 1
        hidden = int(torch.isfinite(got[b, 0, :seen]).sum())
        assert hidden == 0, f"row {b}: {hidden} of {seen} weights are finite"
        assert torch.equal(got[b, 0, seen:], clean[b, 0, seen:]), f"row {b}: keys behind the query changed"


def test_in_a_window():
    """Keys outside the query's window keep their weights."""
    rng = np.random.default_rng(7)
    N, W, at = 700, 300, 600
    q, k = rows(rng, 1, N, 1, 128), rows(rng, 1, N, 1, 128)
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    clean = swa.swa_prefill_weights(q, k, lens, W, 0.1)
    q[0, at, 0, 100] = float("nan")
    got = swa.swa_prefill_weights(q, k, lens, W, 0.1)
    assert not torch.isfinite(got[0, 0, at - W + 1:at + 1]).any()
    assert torch.equal(got[0, 0, :at - W + 1], clean[0, 0, :at - W + 1])
    assert torch.equal(got[0, 0, at + 1:], clean[0, 0, at + 1:])


@pytest.mark.parametrize("T", [3, 400])
def test_a_query_whose_scores_are_all_minus_infinity(T):
    """It has no softmax: the weights of the keys it sees are not finite."""
    rng = np.random.default_rng(T)
    N = 400
    q, k = rows(rng, 1, T, 1, 64), rows(rng, 1, N, 1, 64)
    k[..., 9] = k[..., 9].abs() + 0.1
    q[0, T - 2, 0] = 0
    q[0, T - 2, 0, 9] = -float("inf")
    got = swa.swa_prefill_weights(q, k, torch.tensor([N], dtype=torch.int32, device="cuda"), N, 0.1)
    assert not torch.isfinite(got[0, 0, :N - 1]).any() and torch.isfinite(got[0, 0, N - 1])

"""A fixed-size cache whose sequence is taken back (tokens proposed and then
rejected): slots of positions behind the sequence's are not attended to, receive
nothing and are taken before anything is evicted.

Bounds as in tests/test_gpu_evict.py."""
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


def rows(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=BF16, device="cuda")


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def check_decode(q, kc, vc, at, w0, w, out, pos, scale):
    B, Hq, D = q.shape
    M, H = kc.shape[1], kc.shape[2]
    for b in range(B):
        held = at[b].cpu().numpy()
        seen = (held >= 0) & (held <= pos[b])
        kk = np.where(seen.T[..., None], ref.f64(kc[b]), 0.0)
        vv = np.where(seen.T[..., None], ref.f64(vc[b]), 0.0)
        want, p, big = ref.attend(ref.f64(q[b]), kk, vv, seen, scale)
        d = 2.0 ** -18 * big * scale
        got = ref.f64(out[b])
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -7 + 2 * d) * np.abs(vv).max()).all(), b
        add = ref.f64(w0[b]) + p.reshape(H, Hq // H, M).sum(1)
        assert (np.abs(ref.f64(w[b]) - add) <= (2 * d + 2.0 ** -20 + (Hq // H + 1) * 2.0 ** -24) * add).all(), b
        assert torch.equal(w[b][torch.tensor(~seen)], w0[b][torch.tensor(~seen)])


# merged in a cluster; through the workspace; a group in two pieces
@pytest.mark.parametrize("B,Hq,H,D,M", [(2, 6, 2, 64, 40), (1, 4, 1, 128, 6000), (2, 12, 1, 64, 300)])
def test_positions_behind_the_sequence_are_not_seen(B, Hq, H, D, M):
    rng = np.random.default_rng(M)
    pos = [2 * M - 3 * b for b in range(B)]
    at = np.stack([np.stack([rng.permutation(2 * M + 9)[:M] for _ in range(H)]) for _ in range(B)])
    at[0, 0, :3] = [2 * M + 8, 2 ** 31 - 1, -1]
    kc, vc = rows(rng, B, M, H, D), rows(rng, B, M, H, D)
    unseen = torch.tensor((at < 0) | (at > np.array(pos)[:, None, None]), device="cuda").transpose(1, 2)[..., None]
    kc.masked_fill_(unseen, float("nan"))
    vc.masked_fill_(unseen, float("inf"))
    w0 = torch.tensor(rng.random((B, H, M)), dtype=torch.float32, device="cuda")
    q, scale = rows(rng, B, Hq, D), 1 / math.sqrt(D)
    out, w = swa.swa_decode_weights(q, kc, vc, i32(at), w0, i32(pos), scale, weights_out=torch.empty_like(w0))
    check_decode(q, kc, vc, i32(at), w0, w, out, pos, scale)


def evict(held, w, p, S, R):
    """The slot that position p takes: its own, else the lowest that is free or
    holds a position behind p, else the one of least weight."""
    for want in (lambda x: x == p, lambda x: x < 0 or x > p):
        for s, x in enumerate(held):
            if want(x):
                return s
    return ref.evict(held, w, p, S, R)


@pytest.mark.parametrize("M,S,R,back", [(24, 2, 5, 3), (24, 2, 5, 12), (8, 4, 4, 6), (9, 1, 2, 5), (33, 0, 1, 30)])
def test_a_run_that_is_taken_back_and_goes_on(M, S, R, back):
    """Fill and evict, take `back` tokens back, go on: no slot of a rejected token
    is seen, and each token finds a slot, also where less than `back` slots are
    within reach of eviction."""
    rng = np.random.default_rng(M + back)
    B, Hq, H, D, scale = 2, 4, 2, 64, 0.125
    kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
    vc, at = torch.zeros_like(kc), i32(np.full((B, H, M), -1))
    w = torch.zeros(B, H, M, device="cuda")
    for p in list(range(2 * M)) + list(range(2 * M - back, 2 * M + 6)):
        q, k, v = rows(rng, B, Hq, D), rows(rng, B, H, D), rows(rng, B, H, D)
        want = [[evict(at[b, h].tolist(), w[b, h].cpu().numpy(), p, S, R) for h in range(H)] for b in range(B)]
        assert min(min(x) for x in want) >= 0
        assert swa.swa_cache_evict_append(k, v, kc, vc, at, w, i32([p, p]), S, R).tolist() == want, p
        w0 = w.clone()
        out, _ = swa.swa_decode_weights(q, kc, vc, at, w, i32([p, p]), scale)
        check_decode(q, kc, vc, at, w0, w, out, [p, p], scale)


def test_order_of_the_choices():
    rng = np.random.default_rng(3)
    at = np.array([[[11, 3, -1, 10], [11, 3, 12, 10], [12, 11, 3, 4], [3, 12, 4, 13], [3, 12, -1, 4], [3, -1, 12, 4]]])
    w = np.array([[[0, 0, 9, 9], [0, 0, 0, 9], [9, 9, 0, 0], [0, 9, 0, 5], [0, 9, 9, 0], [0, 9, 9, 0]]], np.float32)
    k, c = rows(rng, 1, 6, 64), rows(rng, 1, 4, 6, 64)
    got = swa.swa_cache_evict_append(k, k, c, c.clone(), i32(at), torch.tensor(w, device="cuda"), i32([10]), 0, 2)
    # its own slot twice, then the lowest that is free or behind it (weights do not matter)
    assert got.tolist() == [[3, 3, 0, 1, 1, 1]]


def test_a_token_is_found_by_the_decode_that_follows_it():
    """A long full cache, one slot of which the caller freed, taken back to a
    position below the free slot's index: the token and its position's share of
    the weight are seen."""
    rng = np.random.default_rng(5)
    M, p = 256, 50
    held = np.arange(M)
    held[[20, 50]] = [700, 800]
    held[200] = -1
    kc, vc = rows(rng, 1, M, 1, 64), rows(rng, 1, M, 1, 64)
    at, w = i32(held[None, None]), torch.zeros(1, 1, M, device="cuda")
    k, v, q = rows(rng, 1, 1, 64), rows(rng, 1, 1, 64), rows(rng, 1, 2, 64)
    assert swa.swa_cache_evict_append(k, v, kc, vc, at, w, i32([p]), 4, 16).tolist() == [[20]]
    w0 = w.clone()
    out, _ = swa.swa_decode_weights(q, kc, vc, at, w, i32([p]), 0.125)
    check_decode(q, kc, vc, at, w0, w, out, [p], 0.125)
    assert w[0, 0, 20] > 0

"""The fixed-size cache with eviction by accumulated attention weight: decode
with weights, eviction of a slot, and the cut of a prompt, against plain 64-bit
forms (tests/cache_ref.py).

Bounds.  Slots, positions and copied rows are exactly determined.  Decode
outputs, element by element: the rounding of the output to bf16 (2^-8 |ref|),
of each weight to bf16 (2^-8; normalised by the sum of the rounded weights, so
twice it times the largest |v|) and the scores: sums of D exact products in
D/16 steps each off by at most 2^-22 of sum |q k|, and three roundings: d =
2^-18 scale sum |q k|, which moves the weights by a factor within e^(+-d).
Accumulated weights are held in 32 bits: each softmax weight is off by 2 d and
2^-20 of itself (the exponential, the sums, the reciprocal), and the sum of G of
them and the old one by (G + 1) 2^-24.
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


def rows(rng, *shape):
    return torch.tensor(rng.standard_normal(shape), dtype=BF16, device="cuda")


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def f32(v):
    return torch.tensor(np.asarray(v), dtype=torch.float32, device="cuda")


def weights_close(got, want, d, G, what=""):
    got = ref.f64(got) if isinstance(got, torch.Tensor) else got
    tol = (2 * d + 2.0 ** -20 + (G + 1) * 2.0 ** -24) * np.abs(want) + 1e-30
    bad = np.abs(got - want) / tol
    assert np.isfinite(got).all() and bad.max() <= 1, f"{what}: {bad.max():.3f} of the bound"


def decode_and_check(rng, B, Hq, H, D, M, pos, slot_pos, start=True, in_place=False):
    scale = 1 / math.sqrt(D)
    q, k, v = rows(rng, B, Hq, D), rows(rng, B, M, H, D), rows(rng, B, M, H, D)
    slot_pos = np.asarray(slot_pos)
    free = torch.tensor(slot_pos < 0, device="cuda").transpose(1, 2)[..., None]
    for t, junk in ((k, float("nan")), (v, float("inf"))):      # never to be used
        t.masked_fill_(free, junk)
        for b, p in enumerate(pos):
            if 0 <= p + 1 < M:
                t[b, p + 1:] = float("nan")
    w0 = f32(rng.random((B, H, M)) * 3) if start else None
    old = np.zeros((B, H, M)) if w0 is None else ref.f64(w0)
    into = None if in_place or w0 is None else torch.full((B, H, M), float("nan"), device="cuda")
    out, w = swa.swa_decode_weights(q, k, v, i32(slot_pos), w0, i32(pos), scale, weights_out=into)
    if in_place:
        assert w is w0
    for b, p in enumerate(pos):
        n = min(p + 1, M)
        seen = (slot_pos[b] >= 0) & (np.arange(M) < n)
        kk, vv = ref.f64(k[b]), ref.f64(v[b])
        want, p_all, big = ref.attend(ref.f64(q[b]), kk, vv, seen, scale)
        d = big * scale * 2.0 ** -18
        ok = np.isfinite(vv) & seen.T[..., None]
        v_max = np.abs(np.where(ok, vv, 0)).max(initial=0.0)
        tol = 2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -8 + 2 * d) * v_max + 1e-30
        got = ref.f64(out[b])
        assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all(), f"sequence {b}"
        add = p_all.reshape(H, Hq // H, M).sum(1)
        weights_close(w[b], old[b] + add, d, Hq // H, f"weights of sequence {b}")
        # what receives nothing keeps its weight, bit for bit
        np.testing.assert_array_equal(ref.f64(w[b])[~seen], old[b][~seen])
    return out, w


def slots_of(rng, B, H, M, pos, free=0.1):
    at = np.tile(np.arange(M), (B, H, 1))
    at = np.where(rng.random(at.shape) < free, -1, at)
    return np.where(at <= np.asarray(pos)[:, None, None], at, -1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 12])
def test_decode_groups(D, G):
    rng = np.random.default_rng(D + G)
    pos = [0, 41, 89, 500]
    decode_and_check(rng, 4, 2 * G, 2, D, 90, pos, slots_of(rng, 4, 2, 90, pos))


@pytest.mark.parametrize("M", [1, 15, 16, 17, 31, 33, 255, 257, 1023, 1025, 2600])
def test_decode_sizes(M):
    """Caches around the 16-key blocks, the mask words and the splits."""
    rng = np.random.default_rng(M)
    pos = [0, M // 2, M - 1, M, 5 * M]
    decode_and_check(rng, 5, 4, 2, 64, M, pos, slots_of(rng, 5, 2, M, pos))


@pytest.mark.parametrize("B,H,M", [(8, 8, 4096), (1, 1, 9001)])
def test_decode_splits(B, H, M):
    rng = np.random.default_rng(M)
    pos = [3 * M if b % 2 else M * (b + 1) // (B + 1) for b in range(B)]
    decode_and_check(rng, B, 4 * H, H, 128, M, pos, slots_of(rng, B, H, M, pos))


@pytest.mark.parametrize("start,in_place", [(False, False), (True, True)])
def test_decode_from_nothing_and_in_place(start, in_place):
    rng = np.random.default_rng(3)
    pos = [99, 300]
    decode_and_check(rng, 2, 6, 2, 64, 100, pos, slots_of(rng, 2, 2, 100, pos), start, in_place)


def test_decode_with_heads_that_hold_nothing():
    """Whole heads free, whole splits free, and one slot alone."""
    rng = np.random.default_rng(4)
    M = 1500
    at = np.full((3, 2, M), -1)
    at[0, 1] = np.arange(M)
    at[1, 0, 1200:] = np.arange(1200, M)
    at[1, 1, 700] = 5
    out, w = decode_and_check(rng, 3, 8, 2, 128, M, [2000, 2000, 2000], at)
    assert not out[0, :4].any() and not out[2].any()
    assert out[1, 4:].any()


def test_decode_of_an_invalid_position_is_skipped_and_recorded():
    rng = np.random.default_rng(5)
    k = rows(rng, 2, 32, 1, 64)
    w = torch.ones(2, 1, 32, device="cuda")
    out = torch.full((2, 2, 64), 7.0, dtype=BF16, device="cuda")
    at = i32(np.tile(np.arange(32), (2, 1, 1)))
    swa.swa_decode_weights(rows(rng, 2, 2, 64), k, k, at, w, i32([-1, 31]), 0.125, out=out)
    assert swa.swa_get_device_status() == swa.SWA_ERR_INVALID_ARG
    assert (out[0] == 7).all() and (w[0] == 1).all() and not (w[1] == 1).any()


def test_weights_sum_to_the_heads():
    """A cache without weights receives exactly one unit per query head."""
    rng = np.random.default_rng(6)
    k = rows(rng, 2, 777, 2, 64)
    at = i32(np.tile(np.arange(777), (2, 2, 1)))
    _, w = swa.swa_decode_weights(rows(rng, 2, 10, 64), k, k, at, None, i32([776, 5000]), 0.125)
    assert (w.double().sum(-1) - 5).abs().max() < 5 * 2.0 ** -19


# ------------------------------------------------------------------ eviction of one slot

def evict_and_check(rng, B, H, D, M, slot_pos, weights, pos, S, R):
    k, v = rows(rng, B, H, D), rows(rng, B, H, D)
    kc, vc = rows(rng, B, M, H, D), rows(rng, B, M, H, D)
    at, w = i32(slot_pos), f32(weights)
    want = [x.clone() for x in (kc, vc, at, w)]
    chosen = np.full((B, H), -1)
    for b in range(B):
        for h in range(H):
            if pos[b] < 0:
                continue
            s = chosen[b, h] = ref.evict(slot_pos[b][h], np.asarray(weights, np.float32)[b][h], pos[b], S, R)
            if s >= 0:
                want[0][b, s, h], want[1][b, s, h] = k[b, h], v[b, h]
                want[2][b, h, s], want[3][b, h, s] = pos[b], 0
    got = swa.swa_cache_evict_append(k, v, kc, vc, at, w, i32(pos), S, R)
    np.testing.assert_array_equal(got.cpu().numpy(), chosen)
    for x, y in zip((kc, vc, at), want[:3]):
        assert torch.equal(x, y)
    assert torch.equal(w.view(torch.int32), want[3].view(torch.int32))
    return chosen


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M", [1, 2, 31, 33, 255, 256, 257, 1000, 5000])
def test_evict_sizes(M, D):
    """Caches not yet full, just full and long full; positions in any order;
    weights with many ties."""
    rng = np.random.default_rng(M + D)
    B, H = 5, 3
    S, R = min(4, M // 4), max(1, min(9, M // 3))
    pos = [0, M // 2, M - 1, M, 7 * M + 3]
    at = np.full((B, H, M), -1)
    for b, p in enumerate(pos):
        for h in range(H):
            if p <= M:
                at[b, h, :min(p, M)] = np.arange(min(p, M))
            else:
                must = list(range(S)) + list(range(p - R + 1, p))
                rest = rng.choice(np.arange(S, p - R + 1), M - len(must), replace=False)
                at[b, h] = rng.permutation(np.concatenate([must, rest]))
    w = np.floor(rng.random((B, H, M)) * 5) / 4
    chosen = evict_and_check(rng, B, H, D, M, at, w, pos, S, R)
    assert (chosen >= 0).all()


def test_evict_special_weights():
    """NaN counts as infinity, -0 as 0, infinities and negative weights order as
    numbers do; ties go to the lowest slot."""
    rng = np.random.default_rng(7)
    inf, nan = float("inf"), float("nan")
    rows_ = [[nan, inf, nan, 5.0], [nan, nan, inf, nan], [0.0, -0.0, 0.0, 1.0], [-0.0, 0.0, 0.0, 0.0],
             [3.0, -inf, -1.0, -inf], [1e-45, 0.0, -1e-45, 0.0], [2.0, 2.0, 2.0, 2.0]]
    w = np.array(rows_, np.float32)[None]
    at = np.tile(np.arange(4), (1, len(rows_), 1))
    chosen = evict_and_check(rng, 1, len(rows_), 64, 4, at, w, [9], 0, 1)
    np.testing.assert_array_equal(chosen[0], [3, 0, 0, 0, 1, 2, 0])


def test_evict_prefers_the_held_position_then_free_slots():
    rng = np.random.default_rng(8)
    at = np.array([[[3, -1, 9, 7, -1], [9, 9, -1, 1, 2], [0, 1, 2, 3, 4]]])
    w = np.ones((1, 3, 5))
    chosen = evict_and_check(rng, 1, 3, 64, 5, at, w, [9], 1, 2)
    np.testing.assert_array_equal(chosen[0], [2, 0, 1])
    # the same token twice takes the same slot again
    kc = rows(rng, 1, 5, 1, 64)
    pos_at, wt = i32([[[0, 1, 2, 3, 4]]]), f32(np.ones((1, 1, 5)))
    k = rows(rng, 1, 1, 64)
    one = [swa.swa_cache_evict_append(k, k, kc, kc, pos_at, wt, i32([8]), 1, 2).item() for _ in range(3)]
    assert one == [1, 1, 1]


def test_evict_nothing_may_go():
    """Every slot protected, or the position invalid: nothing is written, -1 comes
    back and the status is recorded; the other sequences are served."""
    rng = np.random.default_rng(9)
    at = np.array([[[9, 8, 7, 0]], [[0, 1, 2, 3]], [[0, 1, 2, 3]], [[9, 8, 0, 0]]])
    w = np.ones((4, 1, 4))
    chosen = evict_and_check(rng, 4, 1, 64, 4, at, w, [10, -5, 10, 10], 1, 3)
    np.testing.assert_array_equal(chosen[:, 0], [2, -1, 1, -1])
    assert swa.swa_get_device_status() == swa.SWA_ERR_INVALID_ARG


def test_evict_positions_at_the_end_of_int32():
    rng = np.random.default_rng(10)
    top = 2 ** 31 - 1
    at = np.array([[[0, top - 5, top - 1, 77]]])
    chosen = evict_and_check(rng, 1, 1, 64, 4, at, np.array([[[0, 1, 2, 3]]]), [top], 1, 3)
    assert chosen[0, 0] == 1


# ------------------------------------------------------------------ the cut of a prompt

def keep_and_check(rng, B, N, H, D, M, S, R, lens, weights):
    k, v = rows(rng, B, N, H, D), rows(rng, B, N, H, D)
    kc, vc = rows(rng, B, M, H, D), rows(rng, B, M, H, D)
    before = kc.clone(), vc.clone()
    at = torch.full((B, H, M), 12345, dtype=torch.int32, device="cuda")
    wo = torch.full((B, H, M), float("nan"), device="cuda")
    w = f32(weights)
    swa.swa_cache_keep(k, v, w, i32(lens), kc, vc, at, wo, S, R)
    for b in range(B):
        for h in range(H):
            n = lens[b] if 0 <= lens[b] <= N else 0
            kept = ref.keep(np.asarray(weights, np.float32)[b, h], n, M, S, R)
            m = len(kept)
            np.testing.assert_array_equal(at[b, h].cpu().numpy(), kept + [-1] * (M - m))
            assert torch.equal(wo[b, h, :m].view(torch.int32), w[b, h, kept].view(torch.int32))
            assert not wo[b, h, m:].any()
            for cache, src, was in ((kc, k, before[0]), (vc, v, before[1])):
                assert torch.equal(cache[b, :m, h], src[b, kept, h])
                assert torch.equal(cache[b, m:, h], was[b, m:, h])


@pytest.mark.parametrize("N,M,S,R", [
    (1, 1, 0, 1), (40, 40, 4, 8), (41, 40, 4, 8), (100, 12, 4, 8), (300, 64, 0, 1), (1000, 256, 4, 32),
    (1025, 33, 16, 1), (5000, 5000, 4, 9), (5000, 1, 0, 1), (2000, 1999, 3, 5), (70, 100, 4, 16),
])
@pytest.mark.parametrize("ties", [False, True])
def test_keep_sizes(N, M, S, R, ties):
    rng = np.random.default_rng(N * 3 + M + ties)
    B, H = 4, 2
    w = rng.random((B, H, N)) ** 4 * 8
    if ties:
        w = np.floor(w * 3) / 3
    keep_and_check(rng, B, N, H, 64, M, S, R, [N, max(0, N - 1), N // 2, 0], w)


def test_keep_special_weights_and_all_alike():
    rng = np.random.default_rng(11)
    N, M = 200, 50
    w = rng.standard_normal((1, 5, N)).astype(np.float32)
    w[0, 0, ::7] = np.nan
    w[0, 0, 1::7] = np.inf
    w[0, 1, :] = 0.0
    w[0, 1, ::3] = -0.0
    w[0, 2, :] = np.nan
    w[0, 3, :100] = -np.inf
    w[0, 4] = 1e-45 * (np.arange(N) % 5)
    keep_and_check(rng, 1, N, 5, 64, M, 4, 8, [N], w)


def test_keep_of_a_length_outside_the_prompt_keeps_nothing_and_is_recorded():
    rng = np.random.default_rng(12)
    keep_and_check(rng, 3, 50, 1, 128, 20, 2, 4, [51, -1, 50], rng.random((3, 1, 50)))
    assert swa.swa_get_device_status() == swa.SWA_ERR_INVALID_ARG


def test_keep_long_prompt():
    rng = np.random.default_rng(13)
    keep_and_check(rng, 2, 40000, 2, 64, 3000, 4, 100, [40000, 39999], np.floor(rng.random((2, 2, 40000)) * 500) / 64)


# ------------------------------------------------------------------ together

def test_a_run_of_tokens_against_the_plain_form():
    """Tokens one by one through a cache that fills and then evicts: eviction and
    attention interleaved, the choice of slots taken from the GPU's own weights
    and checked on them."""
    rng = np.random.default_rng(14)
    B, Hq, H, D, M, S, R = 2, 6, 2, 64, 24, 2, 5
    scale = 0.125
    kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    at = torch.full((B, H, M), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, H, M, device="cuda")
    for p in range(60):
        k, v, q = rows(rng, B, H, D), rows(rng, B, H, D), rows(rng, B, Hq, D)
        want = [[ref.evict(at[b, h].tolist(), ref.f64(w[b, h]), p, S, R) for h in range(H)] for b in range(B)]
        slots = swa.swa_cache_evict_append(k, v, kc, vc, at, w, i32([p, p]), S, R)
        assert slots.tolist() == want, p
        old = ref.f64(w)
        out, _ = swa.swa_decode_weights(q, kc, vc, at, w, i32([p, p]), scale)
        for b in range(B):
            o, pw, big = ref.attend(ref.f64(q[b]), ref.f64(kc[b]), ref.f64(vc[b]), at[b].cpu().numpy() >= 0, scale)
            d = big * scale * 2.0 ** -18
            v_max = np.abs(ref.f64(vc[b])).max()
            assert (np.abs(ref.f64(out[b]) - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -7 + 2 * d) * v_max).all()
            weights_close(w[b], old[b] + pw.reshape(H, 3, M).sum(1), d, 3)
    held = at.cpu().numpy()
    for b in range(B):
        for h in range(H):
            assert set(range(S)) | set(range(60 - R, 60)) <= set(held[b, h].tolist())


def test_graph_replay_of_a_step():
    """Eviction and decode captured once and replayed: the bits of the same calls
    made one by one."""
    rng = np.random.default_rng(15)
    B, Hq, H, D, M, S, R = 2, 8, 2, 128, 600, 4, 16
    mk = lambda: (torch.zeros(B, M, H, D, dtype=BF16, device="cuda"), torch.zeros(B, M, H, D, dtype=BF16, device="cuda"),  # noqa: E731
                  torch.full((B, H, M), -1, dtype=torch.int32, device="cuda"), torch.zeros(B, H, M, device="cuda"))
    a, b = mk(), mk()
    pos = i32([0, 590])
    k, v, q = rows(rng, B, H, D), rows(rng, B, H, D), rows(rng, B, Hq, D)
    slots, out = torch.empty(B, H, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = torch.empty(swa.swa_decode_weights_workspace_size(B, Hq, H, D, M), dtype=torch.uint8, device="cuda")

    def step(state, slots, out):
        kc, vc, at, w = state
        swa.swa_cache_evict_append(k, v, kc, vc, at, w, pos, S, R, slots=slots)
        swa.swa_decode_weights(q, kc, vc, at, w, pos, 0.1, out=out, workspace=ws)

    step(mk(), slots, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, slots, out)
    for n in range(30):
        for t in (k, v, q):
            t.copy_(rows(rng, *t.shape))
        s2, o2 = torch.empty_like(slots), torch.empty_like(out)
        step(a, s2, o2)
        graph.replay()
        assert torch.equal(slots, s2) and torch.equal(out, o2), n
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        pos += 1

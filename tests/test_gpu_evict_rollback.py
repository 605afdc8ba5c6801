"""A fixed-size cache whose sequence is taken back (tokens proposed and then
rejected): slots of positions behind the sequence's are not attended to and
receive nothing.

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

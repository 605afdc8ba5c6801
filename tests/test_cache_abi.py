"""Argument errors of the 8-bit rolling buffer and of the fixed-size cache, on
the host, before anything is enqueued (no GPU needed): through the C ABI and
through the binding."""
import pytest
import torch

import sliding_window_gqa_prefill_b200 as swa

OK, BAD, UNSUP = swa.SWA_OK, swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED
P = 0x1000            # aligned, never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    swa.build()
    return swa.lib()


def vary(fn, good, cases):
    """Each case replaces some arguments of a call that passes the checks."""
    for change, want in cases:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert fn(*args) == want, (change, want)


def pointers(n, optional=()):
    """Every pointer null, then misaligned."""
    cases = [({i: None}, BAD) for i in range(n) if i not in optional]
    return cases + [({i: P + 2}, BAD) for i in range(n)]


def test_append_q8(lib):
    #        k  v  kc vc ks vs pos B  T  Hkv D  W  block stream
    good = [P] * 7 + [1, 4, 2, 64, 32, 16, None]
    vary(lib.swa_cache_append_q8, good, pointers(7) + [
        ({7: 0}, BAD), ({8: 0}, BAD), ({8: 33}, BAD), ({9: 0}, BAD), ({10: 80}, UNSUP), ({11: 0}, BAD),
        ({12: 0}, BAD), ({12: 48}, BAD), ({12: 256}, BAD), ({12: -16}, BAD), ({7: 65536}, UNSUP)])


def test_decode_q8(lib):
    #        q  kc vc ks vs pos out B  Hq Hkv D  W  block scale ws bytes stream
    good = [P] * 7 + [1, 4, 2, 64, 6000, 16, 0.1, P, 1 << 30, None]
    vary(lib.swa_decode_q8, good, pointers(7) + [
        ({7: 0}, BAD), ({8: 3}, BAD), ({9: 0}, BAD), ({10: 96}, UNSUP), ({11: 0}, BAD), ({12: 24}, BAD),
        ({13: 0.0}, BAD), ({13: float("nan")}, BAD), ({13: float("inf")}, BAD), ({14: None}, BAD), ({14: P + 128}, BAD),
        ({15: 16}, BAD), ({7: 65536}, UNSUP)])
    size = lib.swa_decode_q8_workspace_size
    assert size(1, 4, 2, 64, 600) >= 3 * 4 * 64 * 4                       # 3 splits
    assert size(1, 4, 2, 64, 200) == size(64, 32, 8, 128, 4096) == 0      # one split
    assert size(2, 4, 2, 64, 1000) == 0                                   # four, merged in their cluster
    assert size(1, 3, 2, 64, 600) == size(0, 4, 2, 64, 600) == size(1, 4, 2, 72, 600) == 0


def test_prefill_chunk_q8(lib):
    #        q  k  v  kc vc ks vs pos out B  C  Hq Hkv D  W  block scale ws bytes stream
    good = [P] * 9 + [1, 8, 4, 2, 64, 32, 16, 0.1, P, 1 << 30, None]
    vary(lib.swa_prefill_chunk_q8, good, pointers(9) + [
        ({9: 0}, BAD), ({10: 0}, BAD), ({10: 33}, BAD), ({11: 3}, BAD), ({12: 0}, BAD), ({13: 32}, UNSUP),
        ({14: 0}, BAD), ({15: 17}, BAD), ({16: -1.0}, BAD), ({17: None}, BAD), ({17: P + 16}, BAD), ({18: 100}, BAD)])
    assert lib.swa_prefill_chunk_q8_workspace_size(2, 2, 64, 32) == 2 * 2 * 2 * 64 * 32 * 2
    assert lib.swa_prefill_chunk_q8_workspace_size(0, 2, 64, 32) == 0
    assert lib.swa_prefill_chunk_q8_workspace_size(1, 2, 80, 32) == 0
    assert lib.swa_prefill_chunk_q8_workspace_size(64, 8, 128, 100000) == 64 * 8 * 128 * 100000 * 4


def test_evict_append(lib):
    #        k  v  kc vc at w  pos slots B  Hkv D  M  S  R stream
    good = [P] * 8 + [1, 2, 64, 32, 4, 8, None]
    vary(lib.swa_cache_evict_append, good, pointers(8, optional=(7,)) + [
        ({8: 0}, BAD), ({9: 0}, BAD), ({10: 256}, UNSUP), ({11: 0}, BAD), ({12: -1}, BAD), ({13: 0}, BAD),
        ({12: 25}, BAD), ({12: 2 ** 31 - 1, 13: 2 ** 31 - 1}, BAD), ({8: 65536}, UNSUP), ({11: (1 << 30) + 1}, UNSUP)])


def test_decode_weights(lib):
    #        q  kc vc at w  wo pos out B  Hq Hkv D  M  scale ws bytes stream
    good = [P] * 8 + [1, 4, 2, 64, 6000, 0.1, P, 1 << 30, None]
    vary(lib.swa_decode_weights, good, pointers(8, optional=(4,)) + [
        ({8: 0}, BAD), ({9: 3}, BAD), ({10: 0}, BAD), ({11: 96}, UNSUP), ({12: 0}, BAD), ({13: 0.0}, BAD),
        ({14: None}, BAD), ({14: P + 64}, BAD), ({15: 16}, BAD), ({9: 4098}, UNSUP), ({8: 65536}, UNSUP)])
    size = lib.swa_decode_weights_workspace_size
    assert size(1, 4, 2, 64, 6000) >= 4 * 6000 * 4
    assert size(1, 24, 2, 64, 600) >= 24 * 600 * 4          # a group of 12 runs in two pieces
    assert size(64, 32, 8, 128, 4096) >= 64 * 32 * 4096 * 4  # more blocks than run at once
    # merged on chip
    assert size(1, 4, 2, 64, 600) == size(9, 32, 8, 128, 4096) == size(4, 64, 8, 128, 4096) == 0
    assert size(1, 3, 2, 64, 6000) == size(0, 4, 2, 64, 6000) == size(1, 4, 2, 72, 6000) == size(1, 4098, 2, 64, 6000) == 0


def test_keep(lib):
    #        k  v  w  lens kc vc at wo B  N  Hkv D  M  S  R stream
    good = [P] * 8 + [1, 100, 2, 64, 32, 4, 8, None]
    vary(lib.swa_cache_keep, good, pointers(8) + [
        ({8: 0}, BAD), ({9: 0}, BAD), ({10: 0}, BAD), ({11: 48}, UNSUP), ({12: 0}, BAD), ({13: -1}, BAD),
        ({14: 0}, BAD), ({13: 25}, BAD), ({8: 65536}, UNSUP)])


def test_binding_refuses_what_is_not_a_cuda_tensor_of_the_right_kind(monkeypatch):
    """The binding's own checks, on CPU tensors: type, dimensions, block size."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    k = torch.zeros(1, 32, 2, 64)
    s = torch.zeros(1, 2, 2)
    with pytest.raises(TypeError, match="CUDA tensor"):
        swa.swa_cache_append_q8(k, k, k, k, s, s, None, block=16)
    with pytest.raises(ValueError, match="block"):
        swa.swa_cache_append_q8(k, k, k, k, s, s, None, block=20)
    with pytest.raises(ValueError, match="4 dimensions"):
        swa.swa_decode_q8(k, k[0], k, s, s, None, 0.1)
    with pytest.raises(TypeError, match="CUDA tensor"):
        swa.swa_cache_evict_append(k[:, 0], k[:, 0], k, k, s, s, None, 1, 2)
    with pytest.raises(TypeError, match="CUDA tensor"):
        swa.swa_decode_weights(k[:, 0], k, k, s, s, None, 0.1)
    with pytest.raises(TypeError, match="CUDA tensor"):
        swa.swa_cache_keep(k, k, s, None, k, k, s, s, 1, 2)


def test_prefill_weights(lib):
    #        q  k  lens w  B  T  N   Hq Hkv D  W   scale ws bytes stream
    good = [P] * 4 + [1, 8, 100, 4, 2, 64, 100, 0.1, P, 1 << 30, None]
    vary(lib.swa_prefill_weights, good, [({0: None}, BAD), ({1: None}, BAD), ({2: None}, BAD), ({3: None}, BAD)] + [
        ({0: P + 2}, BAD), ({1: P + 8}, BAD), ({2: P + 1}, BAD), ({3: P + 2}, BAD), ({4: 0}, BAD), ({5: 0}, BAD),
        ({5: 101}, BAD), ({6: 0}, BAD), ({7: 3}, BAD), ({8: 0}, BAD), ({9: 96}, UNSUP), ({10: 0}, BAD), ({11: 0.0}, BAD),
        ({11: float("nan")}, BAD), ({12: None}, BAD), ({12: P + 16}, BAD), ({13: 16}, BAD), ({7: 258}, UNSUP)])
    size = lib.swa_prefill_weights_workspace_size
    assert size(1, 8, 100, 4, 2, 64, 100) > 0
    assert size(1, 101, 100, 4, 2, 64, 100) == size(1, 8, 100, 3, 2, 64, 100) == size(1, 8, 100, 258, 2, 64, 100) == 0

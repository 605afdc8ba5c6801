"""Calls of the 8-bit buffer and of the fixed-size cache that a serving process
makes around the operators themselves: the index-checked library, two streams at
once, graphs that share a workspace, workspaces of exactly the stated size with
guards around them, odd alignments, and refusals on the GPU."""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _libs():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    swa.build()
    swa.build(debug=True)
    swa.lib()
    with swa.bounds_checked():
        swa.lib()
        assert swa.swa_get_device_status() == swa.SWA_OK
    yield
    assert swa.swa_get_device_status() == swa.SWA_OK


def rows(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def q8_run(seed, B, Hq, H, D, W, block, chunks, stream=None):
    """Chunks and tokens through an 8-bit buffer; everything it leaves."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.zeros(B, W, H, D, device="cuda").to(F8)
    v = k.clone()
    ks = torch.zeros(B, -(-W // block), H, device="cuda")
    vs = ks.clone()
    pos = [7 * b for b in range(B)]
    outs, scale = [], 1 / math.sqrt(D)
    for C in chunks:
        q, kn, vn = rows(g, B, C, Hq, D), rows(g, B, C, H, D), rows(g, B, C, H, D)
        if C > 1:
            outs.append(swa.swa_prefill_chunk_q8(q, kn, vn, k, v, ks, vs, i32(pos), W, scale, block=block))
        else:
            swa.swa_cache_append_q8(kn, vn, k, v, ks, vs, i32(pos), block=block)
            outs.append(swa.swa_decode_q8(q[:, 0].contiguous(), k, v, ks, vs, i32(pos), scale, block=block))
        pos = [p + C for p in pos]
    return [*outs, k.view(torch.uint8), v.view(torch.uint8), ks, vs]


def evict_run(seed, B, Hq, H, D, N, M, S, R, T, steps):
    """A prompt cut to M slots, then tokens; everything it leaves."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [max(1, N - 5 * b) for b in range(B)]
    scale = 1 / math.sqrt(D)
    k, v, q = rows(g, B, N, H, D), rows(g, B, N, H, D), rows(g, B, T, Hq, D)
    w = swa.swa_prefill_weights(q, k, i32(lens), N, scale)
    kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
    vc, at, wc = torch.zeros_like(kc), i32(np.full((B, H, M), -1)), torch.zeros(B, H, M, device="cuda")
    swa.swa_cache_keep(k, v, w, i32(lens), kc, vc, at, wc, S, R)
    outs = [w]
    for t in range(steps):
        pos = i32([n + t for n in lens])
        outs.append(swa.swa_cache_evict_append(rows(g, B, H, D), rows(g, B, H, D), kc, vc, at, wc, pos, S, R))
        outs.append(swa.swa_decode_weights(rows(g, B, Hq, D), kc, vc, at, wc, pos, scale)[0])
    return [*outs, kc, vc, at, wc]


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and torch.equal(x, y)


Q8 = [(1, 2, 4, 2, 64, 100, 16, [100, 30, 1, 1]), (2, 3, 12, 1, 128, 77, 64, [50, 77, 1]),
      (3, 1, 6, 2, 128, 1100, 128, [300, 1000, 1, 1]), (4, 5, 8, 8, 64, 1, 32, [1, 1])]
EVICT = [(5, 2, 4, 2, 64, 200, 64, 4, 8, 32, 4), (6, 3, 12, 1, 128, 130, 33, 0, 1, 130, 3),
         (7, 1, 10, 2, 64, 1500, 1300, 4, 100, 40, 3), (8, 40, 8, 8, 128, 90, 70, 1, 3, 1, 2)]


@pytest.mark.parametrize("case", Q8)
def test_index_checked_8_bit_buffer(case):
    a = q8_run(*case)
    with swa.bounds_checked():
        b = q8_run(*case)
        torch.cuda.synchronize()
        assert swa.swa_get_device_status() == swa.SWA_OK, "an index check failed"
    same(a, b)


@pytest.mark.parametrize("case", EVICT)
def test_index_checked_fixed_size_cache(case):
    a = evict_run(*case)
    with swa.bounds_checked():
        b = evict_run(*case)
        torch.cuda.synchronize()
        assert swa.swa_get_device_status() == swa.SWA_OK, "an index check failed"
    same(a, b)


def test_two_streams_at_once():
    """Two sets of sequences, each on its own stream and in both issue orders:
    the bits of the runs made one after the other."""
    want = [q8_run(*Q8[2]), evict_run(*EVICT[2]), evict_run(*EVICT[0])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in want]
    for order in ((0, 1, 2), (2, 1, 0)):
        got = [None] * 3
        for i in order:
            with torch.cuda.stream(streams[i]):
                got[i] = (q8_run, evict_run, evict_run)[i](*(Q8[2], EVICT[2], EVICT[0])[i])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            same(g, w)


def test_two_graphs_share_a_workspace():
    """Decode steps of two batches captured with the same workspace and replayed in
    turn on one stream."""
    g = torch.Generator(device="cuda").manual_seed(9)
    Hq, H, D, W = 12, 1, 64, 1500          # 12 heads: in two pieces, through the workspace
    size = max(swa.swa_decode_q8_workspace_size(B, Hq, H, D, W) for B in (1, 3))
    size = max(size, max(swa.swa_decode_weights_workspace_size(B, Hq, H, D, W) for B in (1, 3)))
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    steps, graphs, outs, wants = [], [], [], []
    for B in (1, 3):
        k, v = rows(g, B, W, H, D), rows(g, B, W, H, D)
        k8, v8 = k.to(F8), v.to(F8)
        s = torch.ones(B, -(-W // 64), H, device="cuda")
        q, pos = rows(g, B, Hq, D), i32([W - 1 - 100 * b for b in range(B)])
        at = i32(np.tile(np.arange(W), (B, H, 1)))
        out = [torch.empty_like(q), torch.empty_like(q), torch.empty(B, H, W, device="cuda")]

        def step(k=k, v=v, k8=k8, v8=v8, s=s, q=q, pos=pos, at=at, out=out):
            swa.swa_decode_q8(q, k8, v8, s, s, pos, 0.1, out=out[0], workspace=ws)
            swa.swa_decode_weights(q, k, v, at, None, pos, 0.1, weights_out=out[2], out=out[1], workspace=ws)

        step()
        wants.append([o.clone() for o in out])
        steps.append(step)
        outs.append(out)
    for step in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 1)):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, wants):
            same(o, w)


def guarded(size):
    """A 256-byte aligned workspace of exactly `size` bytes between two guards."""
    whole = torch.full((size + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    off = 512 + (-(whole.data_ptr() + 512)) % 256
    return whole, whole[off:off + size], off


@pytest.mark.parametrize("B,Hq,H,D,M", [(1, 12, 1, 64, 700), (2, 16, 2, 128, 1111), (40, 8, 4, 64, 600)])
def test_workspaces_of_exactly_the_stated_size(B, Hq, H, D, M):
    """Nothing is written outside them, and their contents on entry do not matter."""
    g = torch.Generator(device="cuda").manual_seed(M)
    k, v, q = rows(g, B, M, H, D), rows(g, B, M, H, D), rows(g, B, Hq, D)
    pos, at = i32([M - 1] * B), i32(np.tile(np.arange(M), (B, H, 1)))
    s = torch.ones(B, -(-M // 16), H, device="cuda")
    k8, v8 = k.to(F8), v.to(F8)
    T = min(M, 70)
    qt = rows(g, B, T, Hq, D)
    ks2, vs2 = s.clone(), s.clone()
    calls = [
        (swa.swa_decode_q8_workspace_size(B, Hq, H, D, M),
         lambda w: swa.swa_decode_q8(q, k8, v8, s, s, pos, 0.1, block=16, workspace=w)),
        (swa.swa_decode_weights_workspace_size(B, Hq, H, D, M),
         lambda w: torch.cat([x.float().flatten() for x in swa.swa_decode_weights(q, k, v, at, None, pos, 0.1,
                                                                                  workspace=w)])),
        (swa.swa_prefill_weights_workspace_size(B, T, M, Hq, H, D, M),
         lambda w: swa.swa_prefill_weights(qt, k, i32([M - b % 3 for b in range(B)]), M, 0.1, workspace=w)),
        (swa.swa_prefill_chunk_q8_workspace_size(B, H, D, M),
         lambda w: swa.swa_prefill_chunk_q8(qt, k[:, :T].contiguous(), v[:, :T].contiguous(), k8.clone(), v8.clone(),
                                            ks2.clone(), vs2.clone(), pos, M, 0.1, block=16, workspace=w)),
    ]
    for size, call in calls:
        if size == 0:
            continue
        want = call(None)
        whole, ws, off = guarded(size)
        for fill in (0xA5, 0xFF):
            whole.fill_(fill)
            got = call(ws)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
            assert (whole[:off] == fill).all() and (whole[off + size:] == fill).all()
        with pytest.raises(swa.SwaError):
            call(ws[:size - 1])
        with pytest.raises(swa.SwaError):
            call(whole[off + 128:])


def test_state_arrays_at_every_alignment():
    """slot_pos, weights and scales need 4 bytes of alignment only: the scan of a
    cache of a multiple of 4 slots, aligned and not, chooses the same."""
    g = torch.Generator(device="cuda").manual_seed(11)
    B, H, D, M = 2, 2, 64, 256
    base_at = torch.stack([torch.randperm(1000, generator=g, device="cuda")[:M] for _ in range(B * H)]).view(B, H, M)
    base_w = torch.floor(torch.rand(B, H, M, generator=g, device="cuda") * 9) / 8
    k = rows(g, B, H, D)
    got = []
    for shift in range(4):
        at = torch.empty(B * H * M + 4, dtype=torch.int32, device="cuda")[shift:shift + B * H * M].view(B, H, M)
        w = torch.empty(B * H * M + 4, device="cuda")[3 - shift:3 - shift + B * H * M].view(B, H, M)
        at.copy_(base_at)
        w.copy_(base_w)
        kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
        slots = swa.swa_cache_evict_append(k, k, kc, kc.clone(), at, w, i32([1500, 1500]), 4, 16)
        got.append([slots, at.clone(), w.clone(), kc])
    for g_ in got[1:]:
        same(g_, got[0])


def test_refusals_on_the_gpu():
    g = torch.Generator(device="cuda").manual_seed(12)
    B, Hq, H, D, W = 1, 4, 2, 64, 64
    k8 = torch.zeros(B, W, H, D, device="cuda").to(F8)
    s, pos = torch.zeros(B, 4, H, device="cuda"), i32([0])
    new, q = rows(g, B, 1, H, D), rows(g, B, Hq, D)
    ok = lambda: swa.swa_cache_append_q8(new, new, k8, k8.clone(), s, s.clone(), pos, block=16)  # noqa: E731
    ok()
    bad = [
        (ValueError, lambda: swa.swa_cache_append_q8(new, new, k8, k8, s, s, pos, block=32)),            # scales' shape
        (ValueError, lambda: swa.swa_cache_append_q8(new, new, k8, k8, s, s, pos, block=8)),
        (TypeError, lambda: swa.swa_cache_append_q8(new, new, k8.float(), k8, s, s, pos, block=16)),
        (TypeError, lambda: swa.swa_cache_append_q8(new.half(), new, k8, k8, s, s, pos, block=16)),
        (TypeError, lambda: swa.swa_cache_append_q8(new, new, k8, k8, s, s, pos.long(), block=16)),
        (ValueError, lambda: swa.swa_cache_append_q8(new, new[:, :, :1], k8, k8, s, s, pos, block=16)),
        (swa.SwaError, lambda: swa.swa_cache_append_q8(rows(g, B, W + 1, H, D), rows(g, B, W + 1, H, D), k8, k8, s, s,
                                                       pos, block=16)),
        (ValueError, lambda: swa.swa_decode_q8(q.transpose(0, 1), k8, k8, s, s, pos, 0.1, block=16)),
        (ValueError, lambda: swa.swa_decode_q8(q, k8, k8, s, s, i32([0, 1]), 0.1, block=16)),
        (swa.SwaError, lambda: swa.swa_decode_q8(q, k8, k8, s, s, pos, -1.0, block=16)),
        (swa.SwaError, lambda: swa.swa_decode_q8(rows(g, B, 3, D), k8, k8, s, s, pos, 0.1, block=16)),
        (ValueError, lambda: swa.swa_prefill_chunk_q8(rows(g, B, 2, Hq, D), rows(g, B, 2, H, D), rows(g, B, 2, H, D), k8,
                                                      k8, s, s, pos, W + 1, 0.1, block=16)),
        (TypeError, lambda: swa.swa_decode_q8(q, k8, k8, s, s, pos, 0.1, block=16, workspace=torch.empty(10))),
    ]
    kc = rows(g, B, W, H, D)
    at, w = i32(np.zeros((B, H, W))), torch.zeros(B, H, W, device="cuda")
    bad += [
        (swa.SwaError, lambda: swa.swa_cache_evict_append(new[:, 0], new[:, 0], kc, kc, at, w, pos, 32, 33)),  # S + R > M
        (swa.SwaError, lambda: swa.swa_cache_evict_append(new[:, 0], new[:, 0], kc, kc, at, w, pos, 4, 0)),
        (swa.SwaError, lambda: swa.swa_cache_evict_append(new[:, 0], new[:, 0], kc, kc, at, w, pos, -1, 4)),
        (TypeError, lambda: swa.swa_cache_evict_append(new[:, 0], new[:, 0], kc, kc, at.long(), w, pos, 4, 4)),
        (ValueError, lambda: swa.swa_decode_weights(q, kc, kc, at, w.transpose(1, 2).contiguous(), pos, 0.1)),
        (TypeError, lambda: swa.swa_decode_weights(q, kc, kc, at, w.double(), pos, 0.1)),
        (swa.SwaError, lambda: swa.swa_prefill_weights(rows(g, B, W + 1, Hq, D), kc, pos, W, 0.1)),           # T > N
        (swa.SwaError, lambda: swa.swa_prefill_weights(rows(g, B, 2, Hq, D), kc, pos, 0, 0.1)),
        (ValueError, lambda: swa.swa_cache_keep(kc, kc, w, pos, kc[:, :32], kc[:, :32], at, w, 1, 1)),
    ]
    for error, call in bad:
        with pytest.raises(error):
            call()
    assert swa.swa_get_device_status() == swa.SWA_OK
    ok()

"""Serving runs on several streams that are in flight together: everything is
made beforehand, the host issues the runs' steps in turn and waits for nothing,
and a gate holds all streams back until the last step is issued."""
import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu
BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    swa.build()
    swa.lib()
    yield
    assert swa.swa_get_device_status() == swa.SWA_OK


def rows(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def q8_steps(seed, B, Hq, H, D, W, block, chunks):
    """(steps, results): each step one call or two, inputs made here."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.zeros(B, W, H, D, device="cuda").to(F8)
    v, ks = k.clone(), torch.zeros(B, -(-W // block), H, device="cuda")
    vs, scale = ks.clone(), 1 / math.sqrt(D)
    outs, steps, done = [], [], 0
    for C in chunks:
        q, kn, vn = rows(g, B, C, Hq, D), rows(g, B, C, H, D), rows(g, B, C, H, D)
        pos = i32([done + 7 * b for b in range(B)])
        done += C

        def chunk(q=q, kn=kn, vn=vn, pos=pos):
            outs.append(swa.swa_prefill_chunk_q8(q, kn, vn, k, v, ks, vs, pos, W, scale, block=block))

        def token(q=q[:, 0].contiguous(), kn=kn, vn=vn, pos=pos):
            swa.swa_cache_append_q8(kn, vn, k, v, ks, vs, pos, block=block)
            outs.append(swa.swa_decode_q8(q, k, v, ks, vs, pos, scale, block=block))

        steps.append(chunk if C > 1 else token)
    return steps, lambda: [*outs, k.view(torch.uint8), v.view(torch.uint8), ks, vs]


def evict_steps(seed, B, Hq, H, D, N, M, S, R, T, tokens):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens, scale = [max(1, N - 5 * b) for b in range(B)], 1 / math.sqrt(D)
    k, v, q = rows(g, B, N, H, D), rows(g, B, N, H, D), rows(g, B, T, Hq, D)
    n = i32(lens)
    kc = torch.zeros(B, M, H, D, dtype=BF16, device="cuda")
    vc, at, w = torch.zeros_like(kc), i32(np.full((B, H, M), -1)), torch.zeros(B, H, M, device="cuda")
    outs = []

    def prompt():
        outs.append(swa.swa_prefill_weights(q, k, n, N, scale))
        swa.swa_cache_keep(k, v, outs[-1], n, kc, vc, at, w, S, R)

    steps = [prompt]
    for t in range(tokens):
        def token(pos=i32([x + t for x in lens]), k1=rows(g, B, H, D), v1=rows(g, B, H, D), q1=rows(g, B, Hq, D)):
            outs.append(swa.swa_cache_evict_append(k1, v1, kc, vc, at, w, pos, S, R))
            outs.append(swa.swa_decode_weights(q1, kc, vc, at, w, pos, scale)[0])

        steps.append(token)
    return steps, lambda: [*outs, kc, vc, at, w]


# forms with a workspace: 3 and 10 splits, a group in two pieces, many blocks
RUNS = [lambda: q8_steps(1, 40, 16, 4, 128, 900, 64, [900, 300] + [1] * 12),
        lambda: q8_steps(2, 1, 12, 1, 64, 4500, 128, [4500] + [1] * 14),
        lambda: evict_steps(3, 32, 32, 8, 128, 1500, 1400, 4, 64, 64, 14),
        lambda: evict_steps(4, 2, 24, 2, 64, 4000, 3000, 1, 16, 700, 14)]


def test_workspace_forms_are_what_runs():
    assert swa.swa_decode_q8_workspace_size(40, 16, 4, 128, 900) > 0
    assert swa.swa_decode_q8_workspace_size(1, 12, 1, 64, 4500) > 0
    assert swa.swa_decode_weights_workspace_size(32, 32, 8, 128, 1400) > 0
    assert swa.swa_decode_weights_workspace_size(2, 24, 2, 64, 3000) > 0


def in_flight_together(streams, turn, hold):
    """All runs, each on its stream, held back for `hold` seconds; their results and
    whether every run began before any other ended."""
    runs = [make() for make in RUNS]
    begin = [torch.cuda.Event(enable_timing=True) for _ in runs]
    end = [torch.cuda.Event(enable_timing=True) for _ in runs]
    torch.cuda.synchronize()
    torch.cuda._sleep(int(hold * 1.9e9))               # the steps below are issued meanwhile
    gate = torch.cuda.Event()
    gate.record()
    for s, e in zip(streams, begin):
        s.wait_event(gate)
        e.record(s)
    for n in range(max(len(steps) for steps, _ in runs)):
        for i in list(range(len(runs)))[::turn]:
            if n < len(runs[i][0]):
                with torch.cuda.stream(streams[i]):
                    runs[i][0][n]()
    for s, e in zip(streams, end):
        e.record(s)
    torch.cuda.synchronize()
    together = all(b.elapsed_time(e) > 0 for b in begin for e in end)
    return [results() for _, results in runs], together


@pytest.mark.parametrize("turn", [1, -1])
def test_runs_in_flight_together_give_the_bits_of_runs_one_by_one(turn):
    wants = []
    for make in RUNS:
        steps, results = make()
        for step in steps:
            step()
        torch.cuda.synchronize()
        wants.append(results())
    streams = [torch.cuda.Stream() for _ in RUNS]
    for hold in (0.2, 0.2, 1.0, 3.0):                  # the first also fills the streams' memory pools
        got, together = in_flight_together(streams, turn, hold)
        for g, want in zip(got, wants):
            assert len(g) == len(want) and all(torch.equal(a, b) for a, b in zip(g, want))
        if together:
            return
    pytest.fail("the host was too slow for the runs to overlap")

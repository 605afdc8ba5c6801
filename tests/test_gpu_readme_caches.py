"""The README's lines on the 8-bit buffer and the fixed-size cache: their outputs
against the plain 64-bit forms (tests/cache_ref.py), on the state the lines leave.

Bounds as in tests/test_gpu_q8.py, tests/test_gpu_prefill_weights.py and
tests/test_gpu_evict.py."""
import math
import os
import re

import numpy as np
import pytest
import torch

import cache_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def env():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"```python\n(.*?)```", text, re.S).group(1)
    # what the last lines overwrite is kept: the cut cache, before the token
    code, n = re.subn(r"(?m)^(# then per token.*)$", r"\1\ncut = [t.clone() for t in (kc, vc, slot_pos, wc)]", code)
    assert n == 1
    code, n = re.subn(r"(?m)^(o_kept, wc = )", r"held = [t.clone() for t in (kc, vc, slot_pos, wc)]\n\1", code)
    assert n == 1
    torch.manual_seed(0)
    e = {}
    exec(compile(code, "README.md", "exec"), e)
    torch.cuda.synchronize()
    return e


def test_the_8_bit_decode(env):
    W, D, B = env["W"], env["D"], env["B"]
    scale, q = D ** -0.5, ref.f64(env["q_new"])
    for b in range(B):
        values = []
        for c16, c8, s in (("k_cache", "k8", "ks"), ("v_cache", "v8", "vs")):
            step = np.repeat(ref.f64(env[s][b]), 64, 0)[:W, :, None]
            got, want = ref.f64(env[c8][b]) * step, ref.f64(env[c16][b])
            assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * step)).all()
            values.append(got)
        want, _, big = ref.attend(q[b], *values, np.ones(W, bool), scale)
        d, v_max = 2.0 ** -18 * big * scale, np.abs(values[1]).max()
        got = ref.f64(env["o8"][b])
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2 * 2.0 ** -11 + 2 * d) * v_max).all()


def test_the_prompts_weights(env):
    N, D, Hq, H, T = env["N"], env["D"], env["Hq"], env["Hkv"], 64
    scale, w = D ** -0.5, ref.f64(env["w"])
    for b in range(env["B"]):
        want = ref.prompt_weights(ref.f64(env["q"][b, -T:]), ref.f64(env["k"][b]), N, N, scale)
        big = float(np.abs(ref.f64(env["q"][b, -T:])).sum(-1).max() * np.abs(ref.f64(env["k"][b])).max())
        d = 2.0 ** -18 * scale * big
        tol = 2 * d + (scale * math.log2(math.e) * big + math.log2(N) + 1) * 2.0 ** -24 + 2.0 ** -20 + (
            36 + T * (Hq // H) / 64 + 2) * 2.0 ** -24
        assert (np.abs(w[b] - want) <= tol * want + 1e-30).all()


def test_the_cut_and_the_token(env):
    B, N, M, S, R, D, Hq, H = (env[x] for x in ("B", "N", "M", "S", "R", "D", "Hq", "Hkv"))
    kc, vc, at, wc = env["cut"]
    for b in range(B):
        for h in range(H):
            kept = ref.keep(env["w"][b, h].cpu().numpy(), N, M, S, R)
            assert at[b, h].tolist() == kept
            assert torch.equal(kc[b, :, h], env["k"][b, kept, h]) and torch.equal(vc[b, :, h], env["v"][b, kept, h])
            assert torch.equal(wc[b, h], env["w"][b, h, kept])
    k1, v1, at1, w1 = env["held"]
    for b in range(B):
        for h in range(H):
            s = ref.evict(at[b, h].tolist(), wc[b, h].cpu().numpy(), N, S, R)
            want = at[b, h].clone()
            want[s] = N
            assert torch.equal(at1[b, h], want) and w1[b, h, s] == 0
            assert torch.equal(k1[b, s, h], env["k_new"][b, 0, h]) and torch.equal(v1[b, s, h], env["v_new"][b, 0, h])
        scale = D ** -0.5
        want, p, big = ref.attend(ref.f64(env["q_new"][b]), ref.f64(k1[b]), ref.f64(v1[b]), np.ones(M, bool), scale)
        d, v_max = 2.0 ** -18 * big * scale, float(v1[b].float().abs().max())
        assert (np.abs(ref.f64(env["o_kept"][b]) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -7 + 2 * d) * v_max).all()
        add = ref.f64(w1[b]) + p.reshape(H, Hq // H, M).sum(1)
        assert (np.abs(ref.f64(env["wc"][b]) - add) <= (2 * d + 2.0 ** -20 + (Hq // H + 1) * 2.0 ** -24) * add).all()

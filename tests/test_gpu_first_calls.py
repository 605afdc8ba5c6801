"""The first call of a process, which loads the kernel it launches, made while a
stream is captured: each case runs in a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import torch
import sliding_window_gqa_prefill_b200 as swa
B, W, Hq, H, D = 2, 1000, 8, 2, 64
x = torch.randn(B, W, H, D, device="cuda").bfloat16()
q = torch.randn(B, Hq, D, device="cuda").bfloat16()
c, s = x.to(torch.float8_e4m3fn), torch.ones(B, -(-W // 64), H, device="cuda")
at = torch.arange(W, dtype=torch.int32, device="cuda").repeat(B, H, 1)
w0, w = torch.rand(B, H, W, device="cuda"), torch.zeros(B, H, W, device="cuda")
pos = torch.full((B,), W - 1, dtype=torch.int32, device="cuda")
lens, out = pos + 1, torch.zeros_like(q)
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
qs, kept = q[:, None].contiguous(), [x[:, :500].contiguous(), x[:, :500].contiguous()]
at2, w2 = at[..., :500].contiguous(), w[..., :500].contiguous()
calls = dict(
    decode=lambda: swa.swa_decode(q, x, x, pos, 0.1, out=out, workspace=ws),
    q8=lambda: swa.swa_decode_q8(q, c, c, s, s, pos, 0.1, out=out, workspace=ws),
    weights=lambda: swa.swa_decode_weights(q, x, x, at, None, pos, 0.1, weights_out=w, out=out, workspace=ws),
    prompt=lambda: swa.swa_prefill_weights(qs, x, lens, W, 0.1, weights=w, workspace=ws),
    keep=lambda: swa.swa_cache_keep(x, x, w0, lens, *kept, at2, w2, 4, 16))
swa.lib()
torch.cuda.synchronize()
"""


def run(code):
    env = dict(os.environ, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", SETUP + code], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.parametrize("name", ["decode", "q8", "weights", "prompt", "keep"])
def test_the_first_call_may_be_a_captured_one(name):
    run(f"""
written = (out, w, at2, w2, *kept)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls['{name}']()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in written]
for t in written:
    t.zero_()
calls['{name}']()
torch.cuda.synchronize()
assert swa.swa_get_device_status() == 0
changed = [i for i, t in enumerate(written) if t.any()]
assert len(changed) >= 1 and all(torch.equal(got[i], written[i]) for i in changed)
""")

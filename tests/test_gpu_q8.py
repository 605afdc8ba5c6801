"""The 8-bit rolling buffer: append, decode and chunk pre-fill against plain
64-bit forms (tests/cache_ref.py).

Bounds.  Codes and scales are exactly determined, so they are compared as
values, bit for bit.  Attention outputs, element by element:
  * the output's rounding to bf16: 2^-8 |ref|;
  * the weights' rounding: f16 in decode (2^-11 relative each), bf16 in the
    chunk kernel (2^-8).  The output divides by the sum of the rounded weights,
    so it stays a convex combination of value rows whose weights are off by at
    most that: twice it, times the largest |v|.  The chunk kernel sums the
    unrounded ones but for each tile's largest, and takes a quarter of the
    exponentials from a polynomial (2^-13): 2 * (2^-8 + 2^-13) covers both;
  * the scores: products are exact in fp32, sums of D of them in D/16 steps
    each off by at most 2^-22 of sum |q k|, and three further roundings:
    less than 2^-18 of it, times the scale; a score off by d moves the
    weights by a factor within e^(+-d) and the output by at most 2 d max |v|.
"""
import math

import numpy as np
import pytest
import torch

import cache_ref as ref
import sliding_window_gqa_prefill_b200 as swa

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    swa.build()
    swa.lib()
    yield
    assert swa.swa_get_device_status() == swa.SWA_OK


def rows(rng, *shape, spread=True):
    """bf16 rows; with spread, of magnitudes from 2^-6 to 2^6."""
    x = rng.standard_normal(shape)
    if spread:
        x *= 2.0 ** rng.integers(-6, 7, shape[:-1])[..., None]
    return torch.tensor(x, dtype=torch.bfloat16, device="cuda")


class Buffer:
    """An 8-bit buffer filled with what no call may read: NaN codes and scales."""

    def __init__(self, B, W, H, D, block):
        self.block, blocks = block, -(-W // block)
        self.k = torch.full((B, W, H, D), float("nan"), device="cuda").to(F8)
        self.v = self.k.clone()
        self.ks = torch.full((B, blocks, H), float("nan"), device="cuda")
        self.vs = self.ks.clone()

    def args(self):
        return self.k, self.v, self.ks, self.vs

    def copy(self):
        c = object.__new__(Buffer)
        c.block = self.block
        c.k, c.v, c.ks, c.vs = (t.clone() for t in self.args())
        return c

    def values(self):
        """Codes and scales in 64 bits: (k, v, ks, vs)."""
        return tuple(ref.f64(t) for t in self.args())


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def append_and_check(buf, k, v, starts):
    """Appends on the GPU and in the plain form; the whole buffer must agree,
    what the call does not own included."""
    before = buf.values()
    swa.swa_cache_append_q8(k, v, *buf.args(), i32(starts), block=buf.block)
    after = buf.values()
    for x, (new, c, s) in enumerate(((k, 0, 2), (v, 1, 3))):
        for b, start in enumerate(starts):
            codes, scale = ref.append_q8(ref.f64(new[b]), before[c][b], before[s][b], start, buf.block)
            np.testing.assert_array_equal(after[c][b], codes, err_msg=f"{'kv'[x]} codes, sequence {b}")
            np.testing.assert_array_equal(after[s][b], scale, err_msg=f"{'kv'[x]} scales, sequence {b}")


def close(got, want, v_max, scores, scale, weight_eps, what=""):
    got = ref.f64(got)
    d = scores * scale * 2.0 ** -18
    tol = 2.0 ** -8 * np.abs(want) + (2 * weight_eps + 2 * d) * v_max + 1e-30
    assert np.isfinite(got).all(), f"{what}: not finite"
    bad = np.abs(got - want) / tol
    assert bad.max() <= 1, f"{what}: {bad.max():.3f} of the bound"


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token_wraps(block, D):
    """Single tokens from an empty buffer through two wraps of a window that is
    no multiple of the block; three heads."""
    W, H = 37, 3
    rng = np.random.default_rng(block * D)
    buf = Buffer(2, W, H, D, block)
    for step in range(80):
        append_and_check(buf, rows(rng, 2, 1, H, D), rows(rng, 2, 1, H, D), [step, 1000 + step] if step > 37 else
                         [step, -1])
    assert swa.swa_get_device_status() == swa.SWA_ERR_INVALID_ARG      # the -1s


@pytest.mark.parametrize("W,T,starts", [
    (100, 100, [0, 1, 99, 250]),          # a whole buffer, from every kind of slot
    (100, 33, [0, 5, 63, 90]),            # runs that end inside a block, at a border, across the wrap
    (129, 2, [0, 127, 128, 1000]),        # the last block has one slot
    (16, 16, [0, 3, 15, 16]),
    (1, 1, [0, 1, 2, 77]),                # a window of one slot
    (300, 299, [1, 2, 298, 5000]),
])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_append_runs(W, T, starts, block):
    H, D = 2, 64
    rng = np.random.default_rng(W * 1000 + T + block)
    buf = Buffer(4, W, H, D, block)
    for _ in range(2):                    # into an empty buffer, then over what it left
        append_and_check(buf, rows(rng, 4, T, H, D), rows(rng, 4, T, H, D), starts)


def test_append_largest_batch_row_of_blocks():
    """More sequences than one launch row, two blocks each."""
    rng = np.random.default_rng(5)
    buf = Buffer(300, 20, 1, 64, 16)
    append_and_check(buf, rows(rng, 300, 18, 1, 64), rows(rng, 300, 18, 1, 64), [b % 23 for b in range(300)])


def test_scale_moves_up_and_down():
    """A large token raises its block's scale and rounds the small ones anew;
    when it is overwritten the scale falls back, and the codes that stay keep
    their values."""
    W, H, D, block = 16, 1, 64, 16
    rng = np.random.default_rng(9)
    buf = Buffer(1, W, H, D, block)
    small = rows(rng, 1, 16, H, D, spread=False)
    append_and_check(buf, small, small, [0])
    first = float(buf.ks[0, 0, 0])
    append_and_check(buf, small[:, :1] * 4096, small[:, :1], [16])
    assert float(buf.ks[0, 0, 0]) > 256 * first
    held = ref.widen(ref.f64(buf.k[0]), ref.f64(buf.ks[0]), block)[1:]
    append_and_check(buf, small[:, :1], small[:, :1], [32])
    assert float(buf.ks[0, 0, 0]) == first
    np.testing.assert_array_equal(ref.widen(ref.f64(buf.k[0]), ref.f64(buf.ks[0]), block)[1:], held)


@pytest.mark.parametrize("value", [0.0, -0.0, 1e-38, 2.0 ** -133, -2.0 ** -120, 3.3895e38, -3.3895e38, 2.0 ** 127,
                                   448.0, 449.0, 464.0, 480.0, float("inf"), -float("inf"), float("nan")])
def test_extreme_values(value):
    """Zeros, subnormals, the largest bf16 and what is not finite, alone in a
    block and beside ordinary values."""
    W, H, D = 32, 2, 64
    rng = np.random.default_rng(11)
    x = rows(rng, 1, 32, H, D, spread=False)
    x[:, :16, 0] = value                  # block 0, head 0: nothing else
    x[0, 20, 1, 3] = value                # block 1, head 1: one element
    buf = Buffer(1, W, H, D, 16)
    append_and_check(buf, x, x, [0])
    append_and_check(buf, x[:, 20:21], x[:, :1], [32])


def test_16_bit_buffer_converts_in_one_call():
    rng = np.random.default_rng(12)
    W, H, D = 70, 2, 64
    full = rows(rng, 2, W, H, D)
    buf = Buffer(2, W, H, D, 32)
    append_and_check(buf, full, full, [0, 0])
    want = ref.f64(full)
    got = np.stack([ref.widen(ref.f64(buf.k[b]), ref.f64(buf.ks[b]), 32) for b in range(2)])
    top = np.stack([np.repeat(ref.f64(buf.ks[b]), 32, 0)[:W, :, None] for b in range(2)])
    # half a step of e4m3: 2^-4 relative, 2^-10 of the scale for its subnormals
    assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * top)).all()


# ------------------------------------------------------------------ decode

def filled(rng, B, W, H, D, block, starts):
    """A buffer as decode finds it: written up to starts[b], the rest garbage."""
    buf = Buffer(B, W, H, D, block)
    for b, p in enumerate(starts):
        n = min(p + 1, W)
        one = Buffer(1, W, H, D, block)
        k, v = rows(rng, 1, n, H, D, spread=False), rows(rng, 1, n, H, D)
        k[:, ::7] *= 4
        swa.swa_cache_append_q8(k, v, *one.args(), i32([p + 1 - n]), block=block)
        for to, x in zip(buf.args(), one.args()):
            to[b] = x[0]
    return buf


def decode_and_check(rng, B, Hq, H, D, W, block, pos, **kw):
    scale = 1 / math.sqrt(D)
    buf = filled(rng, B, W, H, D, block, pos)
    q = rows(rng, B, Hq, D, spread=False)
    out = swa.swa_decode_q8(q, *buf.args(), i32(pos), scale, block=block, **kw)
    k, v, ks, vs = buf.values()
    for b, p in enumerate(pos):
        n = min(p + 1, W)
        kk, vv = ref.widen(k[b], ks[b], block)[:n], ref.widen(v[b], vs[b], block)[:n]
        want, _, big = ref.attend(ref.f64(q[b]), kk, vv, np.ones(n, bool), scale)
        close(out[b], want, np.abs(vv).max(), big, scale, 2.0 ** -11, f"sequence {b}, position {p}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 12])
def test_decode_groups(D, G):
    rng = np.random.default_rng(100 * D + G)
    decode_and_check(rng, 3, 2 * G, 2, D, 90, 32, [0, 41, 400])


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("W", [1, 15, 16, 17, 63, 65, 255, 257, 700])
def test_decode_windows(block, W):
    """Windows around the 16-key blocks, the scale blocks and the splits, at
    positions before, at and behind the wrap."""
    rng = np.random.default_rng(W * 7 + block)
    decode_and_check(rng, 5, 4, 2, 64, W, block, [0, W // 2, W - 1, W, 3 * W + 1])


@pytest.mark.parametrize("B,H,W", [(2, 2, 1024), (1, 1, 1111), (8, 8, 4096), (1, 1, 9000), (1, 1, 40000), (74, 8, 300),
                                   (40, 4, 900)])
def test_decode_splits(B, H, W):
    """Windows of 4 splits (merged in a cluster), of 8 and 16, of more than the
    merge unrolls, of one split each, and of 3."""
    rng = np.random.default_rng(W)
    decode_and_check(rng, B, 4 * H, H, 128, W, 64, [W * 2 + 5 if b % 2 == 0 else (W * b) // B for b in range(B)])


def test_decode_long_tail_of_small_weights():
    """One key takes most of the weight; thousands of others far below it add up
    to a visible share: each weighs 2^-16 of it, 8191 of them an eighth."""
    D, W = 64, 8192
    k = torch.zeros(1, W, 1, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[0, 5, 0, 0] = 16.0
    v[0, :, 0, 0] = 1.0
    v[0, 5, 0, 0] = 0.0
    v[0, 5, 0, 1] = 1.0
    buf = Buffer(1, W, 1, D, 16)
    swa.swa_cache_append_q8(k, v, *buf.args(), i32([0]), block=16)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = math.log(2) * 1.0
    lg = float(q[0, 0, 0]) * 16
    out = ref.f64(swa.swa_decode_q8(q, *buf.args(), i32([W - 1]), 1.0, block=16))[0, 0]
    tail = (W - 1) * math.exp(-lg)
    want = np.array([tail, 1.0]) / (1 + tail)
    # the tail's weights are f16 multiples of 2^-24 at 2^(7 - 16): 2^-11 relative
    assert (np.abs(out[:2] - want) <= 2.0 ** -8 * want + 2.0 ** -10 * want + 2 * lg * 2.0 ** -18).all(), (out[:2], want)


def test_decode_nan_in_a_held_key_shows_and_elsewhere_does_not():
    rng = np.random.default_rng(21)
    buf = filled(rng, 2, 64, 1, 64, 16, [63, 63])
    q = rows(rng, 2, 2, 64, spread=False)
    v = buf.v.view(torch.uint8)
    v[0, 10] = 0x7F
    out = ref.f64(swa.swa_decode_q8(q, *buf.args(), i32([63, 63]), 0.125, block=16))
    assert np.isnan(out[0]).all() and np.isfinite(out[1]).all()
    # beyond the position it is not read
    out = ref.f64(swa.swa_decode_q8(q, *buf.args(), i32([9, 63]), 0.125, block=16))
    assert np.isfinite(out).all()


def test_decode_large_and_small_queries():
    """Query magnitudes over the whole of bf16: scaled to f16 and back."""
    rng = np.random.default_rng(22)
    D, W = 64, 40
    buf = filled(rng, 1, W, 1, D, 16, [W - 1])
    k, v, ks, vs = buf.values()
    kk, vv = ref.widen(k[0], ks[0], 16), ref.widen(v[0], vs[0], 16)
    base = rows(rng, 1, 8, D, spread=False)
    for power in (-130, -100, -20, 0, 20, 100, 126):
        q = (base.double() * 2.0 ** power).to(torch.bfloat16)
        scale = 0.125 * 2.0 ** -power if abs(power) <= 100 else 0.125
        if power > 100:
            scale = 2.0 ** -126
        out = swa.swa_decode_q8(q, *buf.args(), i32([W - 1]), scale, block=16)
        want, _, big = ref.attend(ref.f64(q[0]), kk, vv, np.ones(W, bool), scale)
        close(out[0], want, np.abs(vv).max(), big, scale, 2.0 ** -11, f"2^{power}")


# ------------------------------------------------------------------ chunk

@pytest.mark.parametrize("Hq,H,D,W,block,chunks", [
    (4, 2, 64, 96, 16, [50, 50, 3, 96, 1]),
    (8, 2, 128, 200, 64, [130, 70, 200, 128]),
    (3, 3, 64, 300, 128, [129, 300, 300, 17]),
    (5, 1, 128, 70, 32, [1, 1, 70, 68]),
])
def test_chunks_attend_then_append(Hq, H, D, W, block, chunks):
    """A prompt in uneven chunks through the buffer, then decode steps: two
    sequences at different positions."""
    rng = np.random.default_rng(Hq * W)
    B, scale = 2, 1 / math.sqrt(D)
    buf, pos = Buffer(B, W, H, D, block), [0, 0]
    for n, C in enumerate(chunks):
        q, k, v = rows(rng, B, C, Hq, D, spread=False), rows(rng, B, C, H, D, spread=False), rows(rng, B, C, H, D)
        before = buf.copy()
        out = swa.swa_prefill_chunk_q8(q, k, v, *buf.args(), i32(pos), W, scale, block=block)
        kc, vc, ks, vs = before.values()
        for b in range(B):
            start = pos[b]
            kk, vv = ref.widen(kc[b], ks[b], block), ref.widen(vc[b], vs[b], block)
            want, big = ref.chunk_attend(ref.f64(q[b]), ref.f64(k[b]), ref.f64(v[b]), kk, vv, start, W, scale)
            seen = vv[np.arange(max(0, start - W + 1), start) % W]
            v_max = max(np.abs(ref.f64(v[b])).max(), np.abs(seen).max(initial=0.0))
            close(out[b], want, v_max, big, scale, 2.0 ** -8 + 2.0 ** -13, f"chunk {n}, sequence {b}")
        append_and_check(before, k, v, pos)
        for x, y in zip(buf.args(), before.args()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        pos = [pos[0] + C, pos[1] + C + (W if n == 0 else 0)] if n else [pos[0] + C, pos[1] + C]


def test_serving_run_of_chunks_and_tokens_against_the_16_bit_buffer():
    """A prompt in chunks and tokens through both buffers: the 8-bit outputs stay
    within e4m3's rounding of the 16-bit ones.  Each key and value is off by at
    most 2^-4 of itself (half a step; the scale covers the block's largest), so
    a score moves by at most 2^-4 scale sum |q k| and a value by 2^-4 |v|."""
    rng = np.random.default_rng(31)
    B, Hq, H, D, W, block = 2, 8, 2, 64, 128, 32
    scale = 0.125 / 8
    kc = torch.zeros(B, W, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    buf = Buffer(B, W, H, D, block)
    pos = i32([0, 0])
    worst = 0.0
    for C in (100, 128, 60, 1, 1, 1):
        q, k, v = (rows(rng, B, C, n, D, spread=False) for n in (Hq, H, H))
        if C > 1:
            a = swa.swa_prefill_chunk(q, k, v, kc, vc, pos, W, scale)
            b = swa.swa_prefill_chunk_q8(q, k, v, *buf.args(), pos, W, scale, block=block)
        else:
            swa.swa_cache_append(k, v, kc, vc, pos)
            swa.swa_cache_append_q8(k, v, *buf.args(), pos, block=block)
            a = swa.swa_decode(q[:, 0].contiguous(), kc, vc, pos, scale)
            b = swa.swa_decode_q8(q[:, 0].contiguous(), *buf.args(), pos, scale, block=block)
        qa, ka = q.float().abs().amax().item(), k.float().abs().amax().item()
        d = 2.0 ** -4 * scale * float((q.float().abs().sum(-1)).amax()) * ka
        bound = (2 * d + 2.0 ** -4 + 2.0 ** -6) * float(vc.float().abs().amax())
        worst = max(worst, float((a.float() - b.float()).abs().amax()) / bound)
        pos += C
    assert 0 < worst <= 1, worst


# ------------------------------------------------------------------ streams, graphs, sizes

def test_graph_replay_of_a_decode_step():
    """Append and decode captured once, replayed with new positions and tokens:
    the bits of the same calls made one by one."""
    rng = np.random.default_rng(41)
    B, Hq, H, D, W, block = 3, 8, 2, 128, 300, 64
    scale = 1 / math.sqrt(D)
    a = filled(rng, B, W, H, D, block, [10, 299, 700])
    b = a.copy()
    pos = i32([11, 300, 701])
    k, v = rows(rng, B, 1, H, D), rows(rng, B, 1, H, D)
    q = rows(rng, B, Hq, D, spread=False)
    out = torch.empty_like(q)
    ws = torch.empty(swa.swa_decode_q8_workspace_size(B, Hq, H, D, W), dtype=torch.uint8, device="cuda")

    def step(buf, out):
        swa.swa_cache_append_q8(k, v, *buf.args(), pos, block=block)
        swa.swa_decode_q8(q, *buf.args(), pos, scale, block=block, out=out, workspace=ws)

    step(b.copy(), out)                   # first calls before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, out)
    for n in range(4):
        k.copy_(rows(rng, B, 1, H, D))
        q.copy_(rows(rng, B, Hq, D, spread=False))
        want = torch.empty_like(q)
        step(a, want)
        graph.replay()
        assert torch.equal(out, want), n
        for x, y in zip(a.args(), b.args()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        pos += 1


def test_other_stream_and_repeated_calls_give_the_same_bits():
    rng = np.random.default_rng(42)
    B, Hq, H, D, W = 2, 4, 2, 64, 1500
    buf = filled(rng, B, W, H, D, 64, [1499, 4000])
    q = rows(rng, B, Hq, D, spread=False)
    pos = i32([1499, 4000])
    want = swa.swa_decode_q8(q, *buf.args(), pos, 0.125)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [swa.swa_decode_q8(q, *buf.args(), pos, 0.125, stream=side) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_cache_offsets_beyond_32_bits():
    """The last sequence of a buffer of more than 2^32 codes."""
    B, W, H, D, block = 3, 200000, 62, 128, 128
    assert B * W * H * D > 2 ** 32
    k = torch.zeros(B, W, H, D, dtype=F8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.zeros(B, -(-W // block), H, device="cuda")
    vs = torch.zeros_like(ks)
    rng = np.random.default_rng(43)
    n = 40
    kn, vn = rows(rng, B, n, H, D, spread=False), rows(rng, B, n, H, D, spread=False)
    pos = i32([0, 5, W - 20])             # the last one wraps at the end of the buffer
    swa.swa_cache_append_q8(kn, vn, k, v, ks, vs, pos, block=block)
    for b, start in enumerate([0, 5, W - 20]):
        slots = [(start + t) % W for t in range(n)]
        got = ref.f64(k[b, slots]) * ref.f64(ks[b])[np.array(slots) // block][:, :, None]
        want = ref.f64(kn[b])
        top = ref.f64(ks[b])[np.array(slots) // block][:, :, None]
        assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * top)).all()
    q = rows(rng, B, H, D, spread=False)
    out = swa.swa_decode_q8(q, k, v, ks, vs, i32([39, 39, W + 19]), 0.1, block=block)
    # sequence 2: zeros everywhere but the last 20 and the first 20 slots
    w = W
    kk = np.zeros((n, H, D))
    vv = np.zeros((n, H, D))
    slots = np.array([(W - 20 + t) % W for t in range(n)])
    kk = ref.f64(k[2, slots.tolist()]) * ref.f64(ks[2])[slots // block][:, :, None]
    vv = ref.f64(v[2, slots.tolist()]) * ref.f64(vs[2])[slots // block][:, :, None]
    for h in (0, 30, 61):
        e = np.exp(kk[:, h] @ ref.f64(q[2, h]) * 0.1)
        want = (e @ vv[:, h]) / (e.sum() + (w - n))
        got = ref.f64(out[2, h])
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * np.abs(vv).max() * e.sum() / w).all()
    del k, v
    torch.cuda.empty_cache()

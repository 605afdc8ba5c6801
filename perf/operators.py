"""Workloads of the KV-cache operators: the 8-bit rolling cache and the fixed-size
cache with eviction by accumulated attention weight.

Five operators, in seven calls of ``sliding_window_gqa_prefill_b200``:

* writing new tokens into the 8-bit rolling cache (``swa_cache_append_q8``);
* attention over that cache, for a single token (``swa_decode_q8``) and for a
  chunk of a prompt (``swa_prefill_chunk_q8``);
* attention over a fixed-size cache that also adds up the attention weight each
  slot receives (``swa_decode_weights``);
* the same weights for the last queries of a prompt (``swa_prefill_weights``);
* eviction: the slots a long prompt keeps (``swa_cache_keep``) and the slot a
  new token takes (``swa_cache_evict_append``).

``run`` makes those calls where ``own`` is true and otherwise computes the same
in elementary torch operations in 32 bits.  ``exact`` computes the results in
64 bits from the definitions.  Inputs are synthetic, drawn on the GPU.
"""
import math

import numpy as np
import torch

own = False

_MASKED = -float("inf")


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a full serving batch: a token each into the 8-bit cache
        dict(name="append_q8 step B64", op="append_q8", B=64, T=1, Hkv=8, D=128, W=4096, block=64, context=16384),
        # a prompt chunk of each of four sequences, ending off the block borders
        dict(name="append_q8 chunk T4000", op="append_q8", B=4, T=4000, Hkv=8, D=128, W=4096, block=64, context=9001),
        # a short conversation or two on a small model: the launch is what counts
        dict(name="decode_q8 small", op="decode_q8", B=2, Hq=8, Hkv=2, D=64, W=1000, block=32, context=900),
        # the full serving batch, most windows wrapped: bound by reading the cache
        dict(name="decode_q8 B64", op="decode_q8", B=64, Hq=32, Hkv=8, D=128, W=4096, block=64, context=32768),
        # the next chunk of two long prompts, of a length that is no multiple of a tile
        dict(name="chunk_q8 C1000", op="chunk_q8", B=2, C=1000, Hq=32, Hkv=8, D=128, W=4096, block=64, context=8200),
        # a few sequences, an odd number of heads to a group, an odd budget of slots
        dict(name="decode_weights small", op="decode_weights", B=3, Hq=10, Hkv=2, D=64, M=701, context=1500),
        # the full serving batch over a budget of 4096 slots
        dict(name="decode_weights B64", op="decode_weights", B=64, Hq=32, Hkv=8, D=128, M=4096, context=16384),
        # the last 64 queries of two long prompts judge which keys to keep
        dict(name="prompt_weights T64", op="prompt_weights", B=2, N=16384, T=64, Hq=32, Hkv=8, D=128, W=16384),
        # every query of a prompt judges
        dict(name="prompt_weights T8192", op="prompt_weights", B=1, N=8192, T=8192, Hq=32, Hkv=8, D=128, W=8192),
        # the full serving batch: each KV head gives up one slot for the new token
        dict(name="evict B64", op="evict", B=64, Hkv=8, D=128, M=4096, S=4, R=128, context=16384),
        # short prompts cut to a small budget
        dict(name="keep N1000", op="keep", B=8, N=1000, Hkv=2, D=64, M=256, S=4, R=32),
        # long prompts cut to an eighth
        dict(name="keep N16384", op="keep", B=4, N=16384, Hkv=8, D=128, M=2048, S=4, R=256),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append_q8", "decode_q8", "chunk_q8", "decode_weights", "prompt_weights", "evict", "keep"])
    Hkv, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12])
    block = rng.choice([16, 32, 64, 128])
    B = _spread(rng, 1, 64)
    if op == "append_q8":
        W = _spread(rng, 17, 8192)
        T = rng.choice([1, min(W, _spread(rng, 1, 4096))])
        B = max(1, min(B, 16384 // T, (64 * 4096 * 8) // (W * Hkv)))
        return dict(op=op, B=B, T=T, Hkv=Hkv, D=D, W=W, block=block, context=_spread(rng, 1, 4 * W))
    if op == "decode_q8":
        W = _spread(rng, 17, 32768)
        B = max(1, min(B, (64 * 4096 * 8) // (W * Hkv)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, W=W, block=block, context=_spread(rng, 1, 4 * W))
    if op == "chunk_q8":
        W = _spread(rng, 100, 4096)
        C = min(W, _spread(rng, 2, 1000))
        B = max(1, min(B, (2 * 1000 * 32 * 4096) // (C * G * Hkv * W)))
        return dict(op=op, B=B, C=C, Hq=G * Hkv, Hkv=Hkv, D=D, W=W, block=block, context=_spread(rng, C, 4 * W))
    if op == "decode_weights":
        M = _spread(rng, 17, 16384)
        B = max(1, min(B, (64 * 4096 * 8) // (M * Hkv)))
        return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, M=M, context=_spread(rng, 1, 4 * M))
    if op == "prompt_weights":
        N = _spread(rng, 50, 16384)
        T = min(N, _spread(rng, 1, 4096))
        W = rng.choice([N, N, max(1, N // 2), _spread(rng, 1, N)])
        B = max(1, min(B, (8192 * 8192 * 16) // (N * T * G * Hkv)))
        return dict(op=op, B=B, N=N, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, W=W)
    if op == "evict":
        M = _spread(rng, 40, 8192)
        S, R = rng.choice([0, 1, 4, 16]), rng.choice([1, 7, min(20, M // 2), max(1, M // 4)])
        B = max(1, min(B, (64 * 4096 * 8) // (M * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, D=D, M=M, S=S, R=R, context=_spread(rng, 1, 4 * M))
    N = _spread(rng, 60, 32768)
    M = max(40, min(N, int(N * rng.uniform(0.05, 1.1))))
    S, R = rng.choice([0, 1, 4, 16]), rng.choice([1, 7, min(20, M // 2), max(1, M // 4)])
    B = max(1, min(B, (4 * 16384 * 8) // (max(N, 2 * M) * Hkv)))
    return dict(op=op, B=B, N=N, Hkv=Hkv, D=D, M=M, S=S, R=R)


def _positions(c):
    """The position each sequence of a batch has come to: the longest at
    context - 1, the others down to half of it."""
    n = c["context"]
    return [n - 1 - (b * 7919) % (n // 2 + 1) for b in range(c["B"])]


def _lengths(c):
    """Prompt lengths of a padded batch: the longest N, the others down to half."""
    n = c["N"]
    return [n - (b * 7919) % (n // 2 + 1) for b in range(c["B"])]


# --------------------------------------------------------------------------- inputs

def _rows(g, shape, outliers=0.01):
    """bf16 N(0, 1) rows, one in a hundred of them 8 times as large."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    if outliers:
        x *= 1 + 7 * (torch.rand(shape[:-1], generator=g, device="cuda") < outliers)[..., None]
    return x.to(torch.bfloat16)


def _held_in_8_bits(g, B, W, Hkv, D, block):
    """A rolling cache as earlier calls left it: codes [B, W, Hkv, D] and the
    power-of-two scale [B, blocks, Hkv] of each block of slots and head."""
    x = _rows(g, (B, W, Hkv, D))
    blocks = -(-W // block)
    top = torch.zeros(B, blocks * block, Hkv, device="cuda")
    top[:, :W] = x.abs().amax(-1).float()
    scale = _scale_for(top.view(B, blocks, block, Hkv).amax(2))
    codes = (x.float() / scale.repeat_interleave(block, 1)[:, :W, :, None]).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=dict(c), sm_scale=1 / math.sqrt(c["D"]))
    B, Hkv, D, op = c["B"], c["Hkv"], c["D"], c["op"]
    if op in ("append_q8", "decode_q8", "chunk_q8"):
        s["k_cache"], s["k_scale"] = _held_in_8_bits(g, B, c["W"], Hkv, D, c["block"])
        s["v_cache"], s["v_scale"] = _held_in_8_bits(g, B, c["W"], Hkv, D, c["block"])
        s["pos"] = ints(_positions(c))
    if op in ("append_q8", "chunk_q8"):
        n = c["T"] if op == "append_q8" else c["C"]
        s["k"], s["v"] = _rows(g, (B, n, Hkv, D)), _rows(g, (B, n, Hkv, D))
    if op == "chunk_q8":
        s["q"] = _rows(g, (B, c["C"], c["Hq"], D), 0)
    if op == "decode_q8":
        s["q"] = _rows(g, (B, c["Hq"], D), 0)
    if op == "decode_weights":
        M = c["M"]
        s["q"] = _rows(g, (B, c["Hq"], D), 0)
        s["k"], s["v"] = _rows(g, (B, M, Hkv, D)), _rows(g, (B, M, Hkv, D))
        s["pos"] = ints(_positions(c))
        s["slot_pos"] = _slots(g, c, 4, 16, holes=0.02)
        # what a freed slot still holds is never to reach a result
        free = (s["slot_pos"] < 0).transpose(1, 2)[..., None]
        s["k"].masked_fill_(free, float("nan"))
        s["v"].masked_fill_(free, float("inf"))
        s["weights"] = 4 * torch.rand(B, Hkv, M, generator=g, device="cuda") ** 4
    if op == "prompt_weights":
        s["q"], s["k"] = _rows(g, (B, c["T"], c["Hq"], D), 0), _rows(g, (B, c["N"], Hkv, D))
        s["lens"] = ints(_lengths(c))
    if op == "evict":
        M = c["M"]
        s["k"], s["v"] = _rows(g, (B, Hkv, D)), _rows(g, (B, Hkv, D))
        s["k_cache"], s["v_cache"] = _rows(g, (B, M, Hkv, D), 0), _rows(g, (B, M, Hkv, D), 0)
        s["pos"] = ints(_positions(c))
        s["slot_pos"] = _slots(g, c, c["S"], c["R"])
        s["weights"] = _ranked(g, (B, Hkv, M)) * (s["slot_pos"] >= 0)
    if op == "keep":
        N, M = c["N"], c["M"]
        s["k"], s["v"] = _rows(g, (B, N, Hkv, D), 0), _rows(g, (B, N, Hkv, D), 0)
        s["weights"], s["lens"] = _ranked(g, (B, Hkv, N)), ints(_lengths(c))
        s["k_cache"] = torch.zeros(B, M, Hkv, D, dtype=torch.bfloat16, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["slot_pos"] = torch.full((B, Hkv, M), -1, dtype=torch.int32, device="cuda")
        s["weights_out"] = torch.zeros(B, Hkv, M, device="cuda")
    return s


def _ranked(g, shape):
    """Accumulated weights: a few large, most small, now and then two alike."""
    x = torch.rand(shape, generator=g, device="cuda")
    return torch.floor(x ** 4 * 65536) / 4096


def _slots(g, c, S, R, holes=0.0):
    """The positions a fixed-size cache of M slots holds when the token at
    pos[b] comes: every earlier one while they fit, later the first S, the last
    R - 1 and any others between, in any order; `holes`: the share of free slots."""
    B, Hkv, M = c["B"], c["Hkv"], c["M"]
    pos = torch.tensor(_positions(c), device="cuda")[:, None, None]
    at = torch.arange(max(M, c["context"]), device="cuda")
    order = torch.rand(B, Hkv, at.numel(), generator=g, device="cuda")
    order = torch.where((at < S) | (at > pos - R), at * 0.0 - 1, order)
    order = torch.where(at >= pos, at * 0.0 + 2, order)
    some = order.argsort(dim=-1, stable=True)[..., :M]
    mixed = some.gather(-1, torch.rand(some.shape, generator=g, device="cuda").argsort(dim=-1))
    slot = torch.arange(M, device="cuda").expand(B, Hkv, M)
    held = torch.where(pos >= M, mixed, torch.where(slot < pos, slot, -1))
    if holes:
        n = torch.clamp(pos + 1, max=M)
        held = torch.where(slot < n, torch.where(held < 0, pos, held), -1)
        held = torch.where(torch.rand(held.shape, generator=g, device="cuda") < holes, -1, held)
    return held.to(torch.int32).contiguous()


# --------------------------------------------------------------------------- one pass

def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_append_q8(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        swa.swa_cache_append_q8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["pos"],
                                block=c["block"])
    else:
        _append_q8(s["k"], s["k_cache"], s["k_scale"], s["pos"], c["block"])
        _append_q8(s["v"], s["v_cache"], s["v_scale"], s["pos"], c["block"])
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _run_decode_q8(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        return swa.swa_decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["pos"],
                                 s["sm_scale"], block=c["block"])
    k, v = _widened(s["k_cache"], s["k_scale"], c["block"]), _widened(s["v_cache"], s["v_scale"], c["block"])
    seen = torch.arange(c["W"], device="cuda") <= s["pos"][:, None]
    return _attend(s["q"], k, v, seen[:, None, :], s["sm_scale"])[0].to(torch.bfloat16)


def _run_chunk_q8(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        out = swa.swa_prefill_chunk_q8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                                       s["v_scale"], s["pos"], c["W"], s["sm_scale"], block=c["block"])
    else:
        out = _chunk_q8(s)
        _append_q8(s["k"], s["k_cache"], s["k_scale"], s["pos"], c["block"])
        _append_q8(s["v"], s["v_cache"], s["v_scale"], s["pos"], c["block"])
    return {"out": out, **{x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}}


def _run_decode_weights(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        out, weights = swa.swa_decode_weights(s["q"], s["k"], s["v"], s["slot_pos"], s["weights"], s["pos"],
                                              s["sm_scale"], weights_out=torch.empty_like(s["weights"]))
        return {"out": out, "weights": weights}
    seen = (s["slot_pos"] >= 0) & (torch.arange(c["M"], device="cuda") <= s["pos"][:, None, None])
    free = ~seen.transpose(1, 2)[..., None]
    out, p = _attend(s["q"], s["k"].float().masked_fill(free, 0), s["v"].float().masked_fill(free, 0), seen,
                     s["sm_scale"])
    return {"out": out.to(torch.bfloat16), "weights": s["weights"] + p.sum(2)}


def _run_prompt_weights(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        return swa.swa_prefill_weights(s["q"], s["k"], s["lens"], c["W"], s["sm_scale"])
    B, T, Hq, D = s["q"].shape
    N, Hkv = c["N"], c["Hkv"]
    q = s["q"].float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, s["k"].float().permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, T, N).mul_(s["sm_scale"])
    i = s["lens"][:, None, None] - T + torch.arange(T, device="cuda")[:, None]
    j = torch.arange(N, device="cuda")
    seen = (j <= i) & (j > i - c["W"]) & (i >= 0)
    x.masked_fill_(~seen[:, None, None], _MASKED)
    x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    x.div_(x.sum(-1, keepdim=True).clamp(min=1e-30))
    return x.sum((2, 3))


def _run_evict(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        slots = swa.swa_cache_evict_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_pos"], s["weights"],
                                           s["pos"], c["S"], c["R"])
    else:
        slots = _evict(s)
    return {"slots": slots, **{x: s[x] for x in ("k_cache", "v_cache", "slot_pos", "weights")}}


def _run_keep(s):
    c = s["case"]
    if own:
        import sliding_window_gqa_prefill_b200 as swa
        swa.swa_cache_keep(s["k"], s["v"], s["weights"], s["lens"], s["k_cache"], s["v_cache"], s["slot_pos"],
                           s["weights_out"], c["S"], c["R"])
    else:
        _keep(s)
    return {x: s[x] for x in ("k_cache", "v_cache", "slot_pos", "weights_out")}


_RUN = {"append_q8": _run_append_q8, "decode_q8": _run_decode_q8, "chunk_q8": _run_chunk_q8,
        "decode_weights": _run_decode_weights, "prompt_weights": _run_prompt_weights, "evict": _run_evict,
        "keep": _run_keep}


# --------------------------------------------------------------------------- plain forms

def _scale_for(top):
    """The smallest power of two s with top <= 448 s (448: the largest e4m3
    value), its exponent held to [-117, 119]; 0 for 0."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-117, 119)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.zeros_like(top))


def _widened(codes, scale, block):
    """The 32-bit values that codes [B, W, Hkv, D] stand for."""
    return codes.float() * scale.repeat_interleave(block, 1)[:, :codes.shape[1], :, None]


def _append_q8(new, codes, scale, pos, block):
    """Writes new [B, T, Hkv, D] at slots (pos[b] + t) mod W: every block touched
    is quantised anew from the values it still holds and the new ones."""
    B, T, Hkv, D = new.shape
    W, blocks = codes.shape[1], scale.shape[1]
    n = min(blocks, 1 if T == 1 else -(-(T - 2) // block) + 2)
    first = (pos % W).long()
    blk = ((first // block)[:, None] + torch.arange(n, device="cuda")) % blocks
    slot = blk[..., None] * block + torch.arange(block, device="cuda")
    there = slot < W
    t = (slot - first[:, None, None]) % W
    fresh = there & (t < T)
    kept = there & ~fresh & (slot < pos[:, None, None])
    b = torch.arange(B, device="cuda")[:, None, None]
    at = slot.clamp(max=W - 1)
    was = codes.view(torch.uint8)[b, at]
    held = scale[b[..., 0], blk]
    old = was.view(torch.float8_e4m3fn).float() * held[:, :, None, :, None]
    x = torch.where(fresh[..., None, None], new[b, t.clamp(max=T - 1)].float(), old)
    live = (fresh | kept)[..., None, None]
    top = torch.where(live & x.isfinite(), x.abs(), 0.0).amax((2, 4))
    touched = fresh.any(-1)[..., None]
    s = torch.where(touched, _scale_for(top), held)
    by = s[:, :, None, :, None]
    y = torch.where(by > 0, x / by.clamp(min=1e-38), x * 0).clamp(-448, 448)
    y = torch.where(x.isfinite(), y, float("nan")).to(torch.float8_e4m3fn).view(torch.uint8)
    y = torch.where(live & touched[..., None, None], y, was)
    # a slot past the last one stands for the last one, in the same block
    y = y.gather(2, (at - blk[..., None] * block)[..., None, None].expand_as(y))
    codes.view(torch.uint8)[b, at] = y
    scale[b[..., 0], blk] = s


def _attend(q, k, v, seen, sm_scale):
    """softmax(q k) v of one query token [B, Hq, D] over slots; seen
    [B, 1 or Hkv, slots].  Also returns the weights [B, Hkv, G, slots]."""
    B, Hq, D = q.shape
    Hkv = k.shape[2]
    x = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), k.permute(0, 2, 3, 1)) * sm_scale
    x = x.masked_fill(~seen[:, :, None], _MASKED)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return torch.matmul(p, v.transpose(1, 2)).reshape(B, Hq, D), p


def _chunk_q8(s):
    c = s["case"]
    B, C, Hq, D = s["q"].shape
    W, Hkv = c["W"], c["Hkv"]
    k = torch.cat([_widened(s["k_cache"], s["k_scale"], c["block"]), s["k"].float()], 1)
    v = torch.cat([_widened(s["v_cache"], s["v_scale"], c["block"]), s["v"].float()], 1)
    start = s["pos"][:, None]
    slot = torch.arange(W, device="cuda")
    cached = start - 1 - (start - 1 - slot) % W
    j = torch.cat([torch.where(cached >= 0, cached, -1), start + torch.arange(C, device="cuda")], 1)[:, None, :]
    i = (start + torch.arange(C, device="cuda"))[:, :, None]
    seen = (j >= 0) & (j <= i) & (j > i - W)
    q = s["q"].float().view(B, C, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, Hq // Hkv, C, W + C).mul_(s["sm_scale"])
    x.masked_fill_(~seen[:, None, None], _MASKED)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    # a key that no query of the chunk sees may hold anything
    v = v.masked_fill(~seen.any(1)[:, :, None, None], 0)
    o = torch.matmul(x.view(B, Hkv, -1, W + C), v.transpose(1, 2)).view(B, Hkv, Hq // Hkv, C, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, C, Hq, D).to(torch.bfloat16)


def _evict(s):
    """The slot the token at pos[b] takes in each KV head's cache: the one that
    holds its position already, else a free one, else the one of least weight
    among those neither of the first S positions nor of the last R."""
    c = s["case"]
    M = c["M"]
    held, pos = s["slot_pos"], s["pos"][:, None, None]
    weight = torch.where(s["weights"].isnan(), float("inf"), s["weights"])
    kind = torch.where((held >= c["S"]) & (held <= pos - c["R"]), 2, 3)
    kind = torch.where(held < 0, 1, torch.where(held == pos, 0, kind))
    best = kind.amin(-1, keepdim=True)
    of = kind == best
    weight = torch.where(best == 2, weight, 0.0)
    least = torch.where(of, weight, float("inf")).amin(-1, keepdim=True)
    slot = torch.where(of & (weight == least), torch.arange(M, device="cuda"), M).amin(-1)
    takes = best[..., 0] < 3
    b, h = torch.arange(c["B"], device="cuda")[:, None], torch.arange(c["Hkv"], device="cuda")
    for x in "kv":
        cache = s[x + "_cache"]
        cache[b, slot, h] = torch.where(takes[..., None], s[x], cache[b, slot, h])
    held[b, h, slot] = torch.where(takes, s["pos"][:, None], held[b, h, slot])
    s["weights"][b, h, slot] = torch.where(takes, 0.0, s["weights"][b, h, slot])
    return torch.where(takes, slot, -1).to(torch.int32)


def _keep(s):
    """Prompts cut to M slots: the first S positions, the last R and those of the
    largest weight between, in the order of their positions."""
    c = s["case"]
    N, M, S, R = c["N"], c["M"], c["S"], c["R"]
    j, n = torch.arange(N, device="cuda"), s["lens"][:, None, None]
    middle = (j >= S) & (j < n - R)
    weight = torch.where(s["weights"].isnan(), float("inf"), s["weights"])
    order = weight.argsort(dim=-1, descending=True, stable=True)
    inside = middle.expand_as(weight).gather(-1, order)
    chosen = inside & (inside.cumsum(-1) <= M - S - R)
    kept = torch.zeros_like(inside).scatter_(-1, order, chosen) | ~middle
    kept = (kept | (n <= M)) & (j < n)
    slot = torch.where(kept, kept.cumsum(-1) - 1, M)
    at = torch.full((*kept.shape[:2], M + 1), -1, device="cuda").scatter_(-1, slot, j.expand_as(slot))[..., :M]
    filled, p = at >= 0, at.clamp(min=0)
    s["slot_pos"].copy_(at)
    s["weights_out"].copy_(torch.where(filled, s["weights"].gather(-1, p), 0.0))
    b, h = torch.arange(c["B"], device="cuda")[:, None, None], torch.arange(c["Hkv"], device="cuda")
    p, filled = p.transpose(1, 2), filled.transpose(1, 2)[..., None]
    s["k_cache"].copy_(torch.where(filled, s["k"][b, p, h], s["k_cache"]))
    s["v_cache"].copy_(torch.where(filled, s["v"][b, p, h], s["v_cache"]))


# --------------------------------------------------------------------------- work

def work(case):
    """Bytes each input is read and each output written once, and the products'
    operations, of one pass."""
    c = case
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    row = 2 * Hkv * D                       # K and V elements of a token
    if c["op"] == "append_q8":
        # tokens read in 16 bits and written in 8; the codes that stay in the
        # first and last block decide its scale, so they are read
        edge = [min(c["W"], p, 2 * c["block"] if c["T"] > 1 else c["block"]) for p in _positions(c)]
        return {"bytes": B * c["T"] * row * 3 + sum(edge) * row, "flops": 0}
    if c["op"] == "decode_q8":
        seen = sum(min(p + 1, c["W"]) for p in _positions(c))
        return {"bytes": seen * (row + 8 * Hkv / c["block"]) + 4 * B * c["Hq"] * D, "flops": 4 * seen * c["Hq"] * D}
    if c["op"] == "chunk_q8":
        C, W = c["C"], c["W"]
        pairs = sum(sum(min(p + t + 1, W) for t in range(C)) for p in _positions(c))
        cached = sum(min(p, W - 1) for p in _positions(c))
        return {"bytes": cached * row + B * C * (row * 3 + 4 * c["Hq"] * D), "flops": 4 * pairs * c["Hq"] * D}
    if c["op"] == "decode_weights":
        seen = sum(min(p + 1, c["M"]) for p in _positions(c))
        return {"bytes": seen * (2 * row + 4 * Hkv) + 8 * B * Hkv * c["M"] + 4 * B * c["Hq"] * D,
                "flops": 4 * seen * c["Hq"] * D}
    if c["op"] == "prompt_weights":
        T, W = c["T"], c["W"]
        pairs = sum(sum(min(i + 1, W) for i in range(max(0, n - T), n)) for n in _lengths(c))
        read = sum(min(n, T + W - 1) for n in _lengths(c))
        return {"bytes": read * row + B * T * c["Hq"] * D * 2 + 4 * B * Hkv * c["N"],
                "flops": 2 * pairs * c["Hq"] * D}
    if c["op"] == "evict":
        return {"bytes": B * Hkv * c["M"] * 8 + B * row * 4, "flops": 0}
    kept = sum(min(n, c["M"]) for n in _lengths(c))
    return {"bytes": 4 * Hkv * sum(_lengths(c)) + kept * row * 4 + 8 * B * Hkv * c["M"], "flops": 0}


# --------------------------------------------------------------------------- 64 bits

def _e4m3_64(x):
    """The nearest e4m3 value of each element (ties to even), in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(new, codes, scale, start, block):
    """One sequence: new [T, Hkv, D] into codes [W, Hkv, D]; returns both in 64 bits."""
    W, T = codes.shape[0], new.shape[0]
    codes, scale, new = codes.double(), scale.double(), new.double()
    slots = (start + torch.arange(T, device="cuda")) % W
    fresh = torch.zeros(W, dtype=torch.bool, device="cuda")
    fresh[slots] = True
    values = codes * scale.repeat_interleave(block, 0)[:W, :, None]
    values[slots] = new
    live = fresh | (torch.arange(W, device="cuda") < start)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
    touched[slots // block] = True
    top = torch.zeros(scale.shape[0] * block, scale.shape[1], dtype=torch.float64, device="cuda")
    top[:W] = torch.where(live[:, None], values.abs().amax(-1), 0)
    top = top.view(-1, block, scale.shape[1]).amax(1)
    power = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-117, 119))
    power = torch.where(top / power > 448, power * 2, power)
    power = torch.where(power / 2 * 448 >= top, power / 2, power).clamp(2.0 ** -117, 2.0 ** 119)
    power = torch.where(top > 0, power, 0)
    scale = torch.where(touched[:, None], power, scale)
    by = scale.repeat_interleave(block, 0)[:W, :, None]
    change = (live & touched.repeat_interleave(block)[:W])[:, None, None]
    return torch.where(change, torch.where(by > 0, _e4m3_64(values / by.clamp(min=1e-300)), 0), codes), scale


def _exact_append_all(s, c):
    got = {}
    for x in "kv":
        both = [_exact_append(s[x][b], s[x + "_cache"][b], s[x + "_scale"][b], p, c["block"])
                for b, p in enumerate(_positions(c))]
        got[x + "_cache"], got[x + "_scale"] = torch.stack([y[0] for y in both]), torch.stack([y[1] for y in both])
    return got


def _softmax_64(x, seen):
    """Weights of the keys seen, 0 in a row that sees none."""
    x = torch.where(seen, x, _MASKED)
    top = x.max(-1, keepdim=True).values
    p = torch.where(seen, (x - torch.where(top.isinf(), 0, top)).exp(), 0)
    return torch.where(seen.any(-1, keepdim=True), p / p.sum(-1, keepdim=True), 0)


def _exact_evict(s, c):
    """Row by row on the host."""
    held, weights = s["slot_pos"].cpu().numpy(), s["weights"].double().cpu().numpy()
    slots = np.full((c["B"], c["Hkv"]), -1)
    for b, p in enumerate(_positions(c)):
        for h in range(c["Hkv"]):
            at, w = held[b, h], np.nan_to_num(weights[b, h], nan=np.inf, posinf=np.inf)
            may = np.flatnonzero((at >= c["S"]) & (at <= p - c["R"]))
            for found in (np.flatnonzero(at == p), np.flatnonzero(at < 0), may[np.argsort(w[may], kind="stable")]):
                if found.size:
                    slots[b, h] = found[0]
                    break
    got = {x: s[x].double() for x in ("k_cache", "v_cache", "weights")}
    for b, p in enumerate(_positions(c)):
        for h, at in enumerate(slots[b]):
            if at >= 0:
                got["k_cache"][b, at, h], got["v_cache"][b, at, h] = s["k"][b, h].double(), s["v"][b, h].double()
                got["weights"][b, h, at], held[b, h, at] = 0, p
    return {"slots": torch.from_numpy(slots), "slot_pos": torch.from_numpy(held), **got}


def _exact_keep(s, c):
    """Row by row on the host."""
    M, S, R = c["M"], c["S"], c["R"]
    weights = s["weights"].double().cpu().numpy()
    got = {x: s[x].double() for x in ("k_cache", "v_cache", "weights_out")}
    at = np.full((c["B"], c["Hkv"], M), -1)
    for b, n in enumerate(_lengths(c)):
        for h in range(c["Hkv"]):
            p = np.arange(n)
            if n > M:
                w = np.nan_to_num(weights[b, h, S:n - R], nan=np.inf, posinf=np.inf)
                best = S + np.argsort(-w, kind="stable")[:M - S - R]
                p = np.sort(np.concatenate([p[:S], best, p[n - R:]]))
            at[b, h, :p.size] = p
            p = torch.from_numpy(p).cuda()
            got["k_cache"][b, :p.numel(), h] = s["k"][b, p, h].double()
            got["v_cache"][b, :p.numel(), h] = s["v"][b, p, h].double()
            got["weights_out"][b, h, :p.numel()] = s["weights"][b, h, p].double()
    return {"slot_pos": torch.from_numpy(at), **got}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, sm = c["op"], s["sm_scale"]
    if op == "append_q8":
        return _exact_append_all(s, c)
    if op == "evict":
        return _exact_evict(s, c)
    if op == "keep":
        return _exact_keep(s, c)
    G = c["Hq"] // c["Hkv"]
    if op == "prompt_weights":
        rows = []
        for b, n in enumerate(_lengths(c)):
            w = torch.zeros(c["Hkv"], c["N"], dtype=torch.float64, device="cuda")
            t0 = max(0, c["T"] - n)
            i = torch.arange(n - c["T"] + t0, n, device="cuda")[:, None]
            j = torch.arange(n, device="cuda")
            for h in range(c["Hq"]):
                x = (s["q"][b, t0:, h].double() @ s["k"][b, :n, h // G].double().T) * sm
                w[h // G, :n] += _softmax_64(x, (j <= i) & (j > i - c["W"])).sum(0)
            rows.append(w)
        return torch.stack(rows)
    outs, sums = [], []
    for b, p in enumerate(_positions(c)):
        if op == "decode_weights":
            k, v = s["k"][b].double(), s["v"][b].double()
            seen = (s["slot_pos"][b] >= 0) & (torch.arange(c["M"], device="cuda") <= p)
            k, v = (torch.where(seen.T[..., None], y, 0) for y in (k, v))
            q = s["q"][b].double()
            x = torch.einsum("hd,shd->hs", q, k.repeat_interleave(G, 1)) * sm
            w = _softmax_64(x, seen.repeat_interleave(G, 0))
            outs.append(torch.einsum("hs,shd->hd", w, v.repeat_interleave(G, 1)))
            sums.append(s["weights"][b].double() + w.view(c["Hkv"], G, -1).sum(1))
            continue
        by = [s[x + "_scale"][b].double().repeat_interleave(c["block"], 0)[:c["W"], :, None] for x in "kv"]
        k, v = s["k_cache"][b].double() * by[0], s["v_cache"][b].double() * by[1]
        if op == "decode_q8":
            n = min(p + 1, c["W"])
            x = torch.einsum("hd,shd->hs", s["q"][b].double(), k[:n].repeat_interleave(G, 1)) * sm
            w = _softmax_64(x, torch.ones_like(x, dtype=torch.bool))
            outs.append(torch.einsum("hs,shd->hd", w, v[:n].repeat_interleave(G, 1)))
            continue
        # a chunk: the cached window in the order of its positions, then the chunk
        W, C = c["W"], c["C"]
        before = torch.arange(max(0, p - W + 1), p, device="cuda")
        k = torch.cat([k[before % W], s["k"][b].double()])
        v = torch.cat([v[before % W], s["v"][b].double()])
        i = torch.arange(p, p + C, device="cuda")[:, None]
        j = torch.cat([before, i[:, 0]])
        seen = (j <= i) & (j > i - W)
        out = torch.empty(C, c["Hq"], c["D"], dtype=torch.float64, device="cuda")
        for h in range(c["Hq"]):
            x = (s["q"][b, :, h].double() @ k[:, h // G].T) * sm
            out[:, h] = _softmax_64(x, seen) @ v[:, h // G]
        outs.append(out)
    if op == "decode_weights":
        return {"out": torch.stack(outs), "weights": torch.stack(sums)}
    if op == "chunk_q8":
        return {"out": torch.stack(outs), **_exact_append_all(s, c)}
    return torch.stack(outs)

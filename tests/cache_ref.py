"""Plain 64-bit forms of the 8-bit rolling buffer and of the fixed-size cache
with eviction, in numpy and sequence by sequence; nothing here is shared with
the CUDA path.  What they compute is defined in include/swa.h."""
import numpy as np


def f64(t) -> np.ndarray:
    """A tensor's values in 64 bits (8-bit codes: the values they stand for)."""
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ e4m3 and its scales

def e4m3(x: np.ndarray) -> np.ndarray:
    """The e4m3 value nearest to each element (ties to even; largest 448; NaN
    for what is not finite)."""
    ok = np.isfinite(x)
    y = np.where(ok, x, 0.0)
    _, e = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))         # 4 significant bits, subnormals 2^-9 apart
    return np.where(ok, np.clip(np.rint(y / step) * step, -448, 448), np.nan)


def block_scale(top: float) -> float:
    if top == 0:
        return 0.0
    e = -117
    while top > 448 * 2.0 ** e and e < 119:
        e += 1
    return 2.0 ** e


def append_q8(new, codes, scale, start, block):
    """One sequence and one of K, V: new [T,H,D] into codes [W,H,D] with scale
    [blocks,H]; returns the codes and scales afterwards.  start < 0: unchanged."""
    T, H, _ = new.shape
    W = codes.shape[0]
    codes, scale = codes.copy(), scale.copy()
    if start < 0:
        return codes, scale
    slots = [(start + t) % W for t in range(T)]
    written = set(range(min(start, W)))
    for blk in sorted({s // block for s in slots}):
        inside = range(blk * block, min(W, (blk + 1) * block))
        for h in range(H):
            held = {s: codes[s, h] * scale[blk, h] for s in inside if s in written}
            held.update({s: new[t, h] for t, s in enumerate(slots) if s // block == blk})
            x = np.array(list(held.values()))
            top = np.abs(x[np.isfinite(x)]).max(initial=0.0)
            scale[blk, h] = block_scale(top)
            for s, v in held.items():
                codes[s, h] = e4m3(v / scale[blk, h]) if scale[blk, h] else np.where(np.isfinite(v), 0.0, np.nan)
    return codes, scale


def widen(codes, scale, block):
    """codes [W,H,D], scale [blocks,H] -> values [W,H,D]."""
    return codes * np.repeat(scale, block, 0)[:codes.shape[0], :, None]


# ------------------------------------------------------------------ attention

def softmax(x, seen):
    """Rows of weights over the keys seen; 0 in a row that sees none."""
    w = np.zeros_like(x)
    for i in range(x.shape[0]):
        s = seen[i] if seen.ndim == 2 else seen
        if s.any():
            e = np.exp(x[i, s] - x[i, s].max())
            w[i, s] = e / e.sum()
    return w


def attend(q, k, v, seen, scale):
    """q [Hq,D], k/v [n,H,D], seen [n] or [H,n] -> out [Hq,D], weights [Hq,n],
    and the largest sum_d |q_d k_d| of a seen key (for error bounds)."""
    Hq, H = q.shape[0], k.shape[1]
    out, ws, big = [], [], 0.0
    for h in range(Hq):
        g = h // (Hq // H)
        s = seen[g] if seen.ndim == 2 else seen
        kk, vv = np.where(s[:, None], k[:, g], 0.0), np.where(s[:, None], v[:, g], 0.0)
        w = softmax((kk @ q[h] * scale)[None], s)[0]
        big = max(big, float((np.abs(kk) @ np.abs(q[h])).max(initial=0.0)))
        out.append(w @ vv)
        ws.append(w)
    return np.array(out), np.array(ws), big


def chunk_attend(q, k, v, kc, vc, start, W, scale):
    """q [C,Hq,D], chunk k/v [C,H,D], cache values kc/vc [W,H,D] (slot = position
    mod W) -> out [C,Hq,D] and the largest sum_d |q_d k_d|."""
    C = q.shape[0]
    before = np.arange(max(0, start - W + 1), start)
    kk, vv = np.concatenate([kc[before % W], k]), np.concatenate([vc[before % W], v])
    at = np.concatenate([before, start + np.arange(C)])
    rows, big = [], 0.0
    for t in range(C):
        i = start + t
        o, _, b = attend(q[t], kk, vv, (at <= i) & (at > i - W), scale)
        rows.append(o)
        big = max(big, b)
    return np.array(rows), big


# ------------------------------------------------------------------ weights and eviction

def prompt_weights(q, k, n, W, scale):
    """q [T,Hq,D] (the last T positions), k [N,H,D], length n -> weights [H,N]."""
    T, Hq, _ = q.shape
    N, H, _ = k.shape
    w = np.zeros((H, N))
    j = np.arange(N)
    for t in range(T):
        i = n - T + t
        if i < 0:
            continue
        seen = (j <= i) & (j > i - W)
        for h in range(Hq):
            g = h // (Hq // H)
            kk = np.where(seen[:, None], k[:, g], 0.0)
            w[g] += softmax((kk @ q[t, h] * scale)[None], seen)[0]
    return w


def evict(slot_pos, weights, p, S, R):
    """The slot of one KV head that position p takes, or -1."""
    held = [s for s, q in enumerate(slot_pos) if q == p]
    if held:
        return held[0]
    free = [s for s, q in enumerate(slot_pos) if q < 0]
    if free:
        return free[0]
    w = np.where(np.isnan(weights), np.inf, weights)
    best = -1
    for s, q in enumerate(slot_pos):
        if S <= q <= p - R and (best < 0 or w[s] < w[best]):
            best = s
    return best


def keep(weights, n, M, S, R):
    """The positions of one KV head's prompt of n that stay, in order."""
    if n <= M:
        return list(range(n))
    w = np.where(np.isnan(weights), np.inf, weights)
    middle = sorted(range(S, n - R), key=lambda j: (-w[j], j))[:M - S - R]
    return sorted(list(range(S)) + middle + list(range(n - R, n)))

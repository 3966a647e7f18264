"""fp64 references of the rule with a vector state, of the residual's addition with a
norm, and of beam search, in numpy, with bounds on what fp32 arithmetic may be off by."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                       # half a step of fp32, relative
HALF = {"bfloat16": 2.0 ** -8, "float32": 2.0 ** -23}   # of an output: its rounding (fp32: and a second one)
f64 = lambda x: np.asarray(x, np.float64)


def bounds_of(lens, B, T):
    """(row, first token, end) of each sequence; lens None: B rows of T."""
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    at = np.cumsum([0] + list(lens))
    return [(0, int(at[n]), int(at[n + 1])) for n in range(len(lens))]


def scan(x, g, bounds, h0=None, leaky=False):
    """h_t = a h + b token by token. x, g [B, T, C]; h0 [N, C]. Returns h, hT, and what
    fp32 arithmetic may be off by in each, from the running error analysis
        m_t = a m_{t-1} + |b_t|,  e_t = a e_{t-1} + 6 U m_t:
    a token's decay has 2 half steps from its exponential and one from the product it
    enters, the fused step adds one, an input's factor and product (leaky) up to
    four of |b| alone, the fold of 16 tokens' maps one in 16."""
    x, g = f64(x), f64(g)
    a = np.exp(g)
    b = -np.expm1(g) * x if leaky else x
    N, C = len(bounds), x.shape[2]
    h, e = np.zeros_like(x), np.zeros_like(x)
    hT = np.zeros((N, C)) if h0 is None else f64(h0).copy()
    eT = np.zeros((N, C))
    for n, (r, t0, t1) in enumerate(bounds):
        s, m, err = hT[n].copy(), np.abs(hT[n]), np.zeros(C)
        for t in range(t0, t1):
            s = a[r, t] * s + b[r, t]
            m = a[r, t] * m + np.abs(b[r, t])
            err = a[r, t] * err + 6 * U * m
            h[r, t], e[r, t] = s, err
        if t1 > t0:
            hT[n], eT[n] = s, err
    return h, hT, e, eT


def scan_bwd(x, g, dy, bounds, h0=None, dhT=None, leaky=False):
    """The adjoint, token by token: (dx, dg, dh0) and their bounds, alike. The forward's
    state before a token is off by its e, the running gradient D by its own."""
    x, g, dy = f64(x), f64(g), f64(dy)
    a = np.exp(g)
    h, _, eh, _ = scan(x, g, bounds, h0, leaky)
    N, C = len(bounds), x.shape[2]
    dx, dg, ex, eg = (np.zeros_like(x) for _ in range(4))
    dh0 = np.zeros((N, C)) if dhT is None else f64(dhT).copy()
    e0 = np.zeros((N, C))
    for n, (r, t0, t1) in enumerate(bounds):
        D, m, err = dh0[n].copy(), np.abs(dh0[n]), np.zeros(C)
        for t in range(t1 - 1, t0 - 1, -1):
            D, m = dy[r, t] + D, np.abs(dy[r, t]) + m
            err = err + U * m
            first = t == t0
            prev = (np.zeros(C) if h0 is None else f64(h0)[n]) if first else h[r, t - 1]
            eprev = 0.0 if first else eh[r, t - 1]
            into = prev - x[r, t] if leaky else prev
            einto = eprev + (U * (np.abs(prev) + np.abs(x[r, t])) if leaky else 0.0)
            f = -np.expm1(g[r, t]) if leaky else 1.0
            dx[r, t], ex[r, t] = f * D, f * err + 5 * U * np.abs(f * D)
            dg[r, t] = a[r, t] * into * D
            eg[r, t] = a[r, t] * (np.abs(into) * err + einto * (np.abs(D) + err)) + 5 * U * np.abs(dg[r, t])
            D, m, err = a[r, t] * D, a[r, t] * m, a[r, t] * err + 5 * U * a[r, t] * m
        dh0[n], e0[n] = D, err
    return (dx, dg, dh0), (ex, eg, e0)


def held(got, ref, bound, what, dtype="float32", rms=None):
    """|got - ref| <= bound + the output type's rounding, each element; and, with rms, the
    RMS of the difference (bf16's rounding of the reference taken out first) within rms
    of the reference's."""
    got, ref = f64(got), f64(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    allowed = np.broadcast_to(bound, ref.shape) + HALF[dtype] * np.abs(ref) + 1e-37
    off = np.abs(got - ref)
    worst = float(np.max(off / allowed, initial=0.0))
    size = float(np.sqrt(np.mean(ref ** 2))) if ref.size else 0.0
    far = float(np.sqrt(np.mean(np.maximum(off - HALF[dtype] * np.abs(ref), 0.0) ** 2))) / max(size, 1e-30) if ref.size else 0.0
    print(f"{what}: {worst:.2f} of its bound, rms {far:.1e}", flush=True)
    assert worst <= 1.0, f"{what}: {worst:.2f} times its bound"
    if rms is not None:
        assert far <= rms, f"{what}: rms {far:.1e} (bar {rms:.0e})"


def beam(logits, scores, K, done=None, eos=-1):
    """(scores, parents, tokens) of one entry: logits [W, V], scores [W]."""
    x = f64(logits)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    W, V = x.shape
    total = np.full((W, V), -np.inf)
    for w in range(W):
        s = float(scores[w])
        if not s > -np.inf:
            continue
        if done is not None and done[w]:
            total[w, eos] = s
            continue
        m = x[w].max()
        if m > -np.inf:
            total[w] = s + (x[w] - m - np.log(np.exp(x[w] - m).sum()))
    flat = total.reshape(-1)
    order = np.argsort(-flat, kind="stable")[:K]
    best = flat[order]
    some = best > -np.inf
    pad = K - len(order)
    parents, tokens = np.where(some, order // V, -1), np.where(some, order % V, -1)
    return (np.concatenate([best, np.full(pad, -np.inf)]), np.concatenate([parents, np.full(pad, -1)]),
            np.concatenate([tokens, np.full(pad, -1)]))


def reorder(slots, parents):
    """(new slots, [(from, to), ...]) of one entry."""
    W = len(slots)
    valid = [p for p in parents if 0 <= p < W]
    free = [slots[w] for w in range(W) if w not in valid]
    held_, new, copies = set(), [], []
    for p in parents:
        if 0 <= p < W and p not in held_:
            held_.add(p)
            new.append(slots[p])
            continue
        to = free.pop(0)
        new.append(to)
        if 0 <= p < W:
            copies.append((slots[p], to))
    return new, copies

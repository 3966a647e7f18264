"""fp64 references of the operators around the rule, token by token in numpy, and
the bounds their results are held to."""
from __future__ import annotations

import numpy as np

import workloads as W


def rule_bwd(q, k, v, g, beta, do, bounds, h0=None, dhT=None):
    """Gradients of the token recurrence by its adjoint, one token at a time:
        P = e^g S,  e = v - k P,  S' = P + k (b e)^T,  o = q S'
        dS += q do^T;  de = b k dS;  dP = dS - k de^T;  dS_before = e^g dP
    q, k, v, do [B, T, H, 128]; g the same or [B, T, H]; bounds: (row, start, end)
    per sequence; h0, dhT [N, H, 128, 128]. Returns dq, dk, dv, dg, dbeta, dh0."""
    f = lambda x: np.asarray(x, np.float64)
    q, k, v, g, beta, do = map(f, (q, k, v, g, beta, do))
    scalar = g.ndim == 3
    decay = np.exp(g[..., None] if scalar else g)
    H, D = q.shape[2:]
    out = [np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), np.zeros_like(q), np.zeros_like(beta)]
    dq, dk, dv, dg, db = out
    dh0 = np.zeros((len(bounds), H, D, D))
    mv = lambda S, x: np.matmul(S, x[..., None])[..., 0]                 # S x
    vm = lambda x, S: np.matmul(x[..., None, :], S)[..., 0, :]           # x S
    seg = 64
    for n, (b, t0, t1) in enumerate(bounds):
        S = np.zeros((H, D, D)) if h0 is None else f(h0[n]).copy()
        marks = {}
        for t in range(t0, t1):
            if (t - t0) % seg == 0:
                marks[t] = S
            P = decay[b, t][..., None] * S
            e = v[b, t] - vm(k[b, t], P)
            S = P + k[b, t][..., None] * (beta[b, t][:, None] * e)[:, None, :]
        dS = np.zeros((H, D, D)) if dhT is None else f(dhT[n]).copy()
        for m in sorted(marks, reverse=True):
            S, kept = marks[m], []
            for t in range(m, min(m + seg, t1)):
                P = decay[b, t][..., None] * S
                e = v[b, t] - vm(k[b, t], P)
                S = P + k[b, t][..., None] * (beta[b, t][:, None] * e)[:, None, :]
                kept.append((P, e, S))
            for t in range(min(m + seg, t1) - 1, m - 1, -1):
                P, e, S = kept[t - m]
                bt = beta[b, t][:, None]
                dq[b, t] = mv(S, do[b, t])
                dS = dS + q[b, t][..., None] * do[b, t][:, None, :]
                kd = vm(k[b, t], dS)
                de = bt * kd
                db[b, t] = (e * kd).sum(-1)
                dv[b, t] = de
                dk[b, t] = mv(dS, bt * e) - mv(P, de)
                dP = dS - k[b, t][..., None] * de[:, None, :]
                dg[b, t] = (dP * P).sum(-1)
                dS = decay[b, t][..., None] * dP
        dh0[n] = dS
    return dq, dk, dv, dg.sum(-1) if scalar else dg, db, dh0


def within(got, ref, what, half_step=0.0, scale=None, tol=1e-4):
    """|got - ref| <= half_step |ref| + tol * scale. half_step: the rounding to the
    output's type (bf16 2^-8, fp32 0), or an array that bounds the rounding itself. scale: RMS of the reference by default. tol:
    1e-4, the library's bar for fp32 arithmetic: sums of up to 128 products of
    rounding 2^-24 (rms 2^-24 sqrt(128) = 7e-7), chained about ten times (2e-6),
    exponents up to 40 with rounding 40 * 2^-24 = 2.4e-6, at 6 sigma over the
    largest of many values: 2.5e-5, and a factor of 4 for rows of unequal size."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    scale = max(W.rms(ref) if scale is None else scale, 1e-30)
    allowed = half_step if isinstance(half_step, np.ndarray) else half_step * np.abs(ref)
    off = float(np.max(np.abs(got - ref) - allowed, initial=0.0)) / scale
    print(f"{what}: {off:.2e} of {scale:.2e}", flush=True)
    assert off <= tol, f"{what}: off by {off:.2e} of {scale:.2e} (bar {tol:.0e})"

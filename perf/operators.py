"""The training and serving operators around the gated delta rule, as measurable cases.

Four operators: the gradient of the chunked rule (per-channel gate: KDA, scalar gate: Gated DeltaNet), the
recurrent form for a few tokens per sequence over a pool of states, the normalisation and gates before the rule,
and the gated RMS norm after it. Each has a plain form in elementary torch operations (`own = False`), the
library's call (`own = True`) and its definition in 64 bits (`exact`).
"""
import math

import torch

own = False

D = 128                                        # K = V = 128, the library's head size
MIX = (1300, 547, 2048, 963, 271, 3063)        # the repository's variable-length mix, 8192 tokens
C = 16                                         # chunk of the plain form
EPS_IN, EPS_OUT = 1e-6, 1e-5


# ------------------------------------------------------------------------------------------------ cases

def _case(op, **kw):
    c = {"op": op, "B": 1, "T": 1, "H": 1, "dtype": "bf16", "gate": "channel"}
    c.update(kw)
    return c


def listed():
    return [
        # one short fp32 sequence of two heads: gradient checks and small experiments, bound by launches and latency
        _case("bwd", name="bwd tiny fp32", T=256, H=2, dtype="fp32"),
        # a training step's backward pass at the headline size, one long document
        _case("bwd", name="bwd T8192 H96", T=8192, H=96),
        # packed documents of very different lengths, continued from and into other segments (state gradients both ways)
        _case("bwd", name="bwd packed H64", T=8192, H=64, packed=",".join(map(str, MIX)), state=True),
        # Gated DeltaNet training on a batch of rows whose length is no multiple of anything
        _case("bwd", name="bwd gdn rows", B=4, T=1001, H=16, gate="scalar"),
        # one user's next token: latency
        _case("rec", name="rec one token", B=1, T=1, H=32, pool="fp32"),
        # a full serving batch, one token each, states kept in 16 bits, a few slots of the batch empty
        _case("rec", name="rec batch bf16", B=256, T=1, H=32, pool="bf16", empty=5),
        # verifying five drafted tokens per sequence, the state after each of them kept so that any can be accepted
        _case("rec", name="rec drafts", B=16, T=5, H=96, pool="fp32", keep=True),
        # what comes before the rule, at prefill and in training
        _case("in", name="in T8192 H96", T=8192, H=96),
        _case("in_bwd", name="in_bwd T8192 H64 bounded", T=8192, H=64, bounded=True),
        # the same before a decode step of a small batch
        _case("in", name="in decode gdn", B=32, T=1, H=16, gate="scalar"),
        # what comes after the rule, at prefill and in training
        _case("out", name="out T8192 H96", T=8192, H=96, act="sigmoid"),
        _case("out_bwd", name="out_bwd rows", B=4, T=1001, H=64, act="silu"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bwd", "bwd", "bwd", "rec", "rec", "in", "in_bwd", "out", "out_bwd"])
    gate, dtype = rng.choice(["channel", "channel", "scalar"]), rng.choice(["bf16", "bf16", "fp32"])
    if op == "bwd":
        H = rng.choice([1, 2, 3, 5, 8, 16, 24, 33, 64, 96])
        T = _log(rng, 1, min(8192, 8192 * 96 // H))
        # (a sequence of one token from a zero state has no gate gradient: short ones start from a state)
        kw = dict(T=T, H=H, dtype=dtype, gate=gate, state=T < 64 or rng.random() < 0.5)
        if rng.random() < 0.5:
            B = min(T, rng.randint(1, 12))         # packed sequences, empty ones among them
            cuts = sorted(rng.randint(0, T) for _ in range(B - 1))
            kw["packed"] = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [T]))
        elif T <= 2048:
            kw["B"] = rng.randint(1, 4)
        return _case(op, **kw)
    if op == "rec":
        H = rng.choice([1, 4, 16, 24, 32, 63, 96])
        T = rng.choice([1, 1, 2, 3, 5, 8, 17])
        B = _log(rng, 1, max(1, 8192 // (H * (T if T > 1 else 1))))
        return _case(op, B=B, T=T, H=H, dtype=dtype, gate=gate, pool=rng.choice(["fp32", "bf16"]),
                     keep=T > 1 and rng.random() < 0.5, empty=rng.randint(0, B // 4))
    H = rng.choice([1, 3, 8, 16, 25, 32, 64, 96])
    T = _log(rng, 1, 8192 * 96 // H // 3 if dtype == "fp32" else 8192 * 96 // H // 2)
    kw = dict(T=T, H=H, dtype=dtype)
    if op in ("in", "in_bwd"):
        return _case(op, gate=gate, bounded=rng.random() < 0.5, **kw)
    return _case(op, act=rng.choice(["sigmoid", "silu"]), **kw)


def _lens(case):
    """Sequence lengths of a case, and whether they are packed into one row."""
    if case.get("packed"):
        return [int(x) for x in case["packed"].split(",")], True
    return [case["T"]] * case["B"], False


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, T, H, dt = case["B"], case["T"], case["H"], _dtype(case)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()
    op, scalar = case["op"], case["gate"] == "scalar"
    gshape = (B, T, H) if scalar else (B, T, H, D)
    s = {"op": op, "scalar": scalar}
    if op in ("bwd", "rec"):
        # unit queries and keys, gates -softplus(N(0, 1)) within [-5, 0], beta = sigmoid(N(0, 1))
        s.update(q=unit(n(B, T, H, D)).to(dt), k=unit(n(B, T, H, D)).to(dt), v=n(B, T, H, D).to(dt),
                 g=(-torch.nn.functional.softplus(n(*gshape))).clamp_min(-5.0), beta=torch.sigmoid(n(B, T, H)))
    if op == "bwd":
        lens, packed = _lens(case)
        s["lens"], N = lens, len(lens)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda") if packed else None
        s["do"] = n(B, T, H, D)
        s["h0"] = 0.1 * n(N, H, D, D) if case.get("state") else None
        s["dhT"] = 0.1 * n(N, H, D, D) if case.get("state") else None
    elif op == "rec":
        pdt = torch.bfloat16 if case["pool"] == "bf16" else torch.float32
        P = 2 * B + (B * T if case.get("keep") else 0)
        order = torch.randperm(P, device="cuda", generator=gen).to(torch.int32)
        slots = order[:B].clone()
        if case.get("empty"):
            slots[torch.randperm(B, device="cuda", generator=gen)[:case["empty"]]] = -1
        s["slots"] = slots
        s["out_slots"] = order[B:B + B * T].reshape(B, T).contiguous() if case.get("keep") else None
        s["pool"] = (0.1 * n(P, H, D, D)).to(pdt)
        s["o"] = torch.zeros(B, T, H, D, device="cuda")
    elif op in ("in", "in_bwd"):
        s.update(q=n(B, T, H, D).to(dt), k=n(B, T, H, D).to(dt), f=n(*gshape).to(dt), b=n(B, T, H).to(dt),
                 A_log=torch.empty(H, device="cuda").uniform_(0.0, 1.0, generator=gen), bias=0.5 * n(*gshape[2:]),
                 bound=-5.0 if case.get("bounded") else None)
        if op == "in_bwd":
            s.update(dq=n(B, T, H, D).to(dt), dk=n(B, T, H, D).to(dt), dg=n(*gshape), dbeta=n(B, T, H))
    else:
        s.update(o=n(B, T, H, D), z=n(B, T, H, D).to(dt), w=1.0 + 0.1 * n(D), act=case["act"])
        if op == "out_bwd":
            s["dy"] = n(B, T, H, D).to(dt)
    return s


# ------------------------------------------------------------------------------------------ the operators

def run(s):
    if own:
        return _own(s)
    return {"bwd": _bwd, "rec": _rec, "in": _in, "in_bwd": _in_bwd, "out": _out, "out_bwd": _out_bwd}[s["op"]](s)


def _own(s):
    import gated_delta_rule_63_amd as kda
    op = s["op"]
    if op == "bwd":
        f = kda.gdn_bwd if s["scalar"] else kda.bwd
        return f(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], cu_seqlens=s["cu"], initial_state=s["h0"],
                 d_final_state=s["dhT"])
    if op == "rec":
        f = kda.gdn_recurrent if s["scalar"] else kda.recurrent
        o = f(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], slots=s["slots"], out_slots=s["out_slots"], out=s["o"])
        return o, s["pool"]
    if op == "in":
        f = kda.gdn_block_in if s["scalar"] else kda.block_in
        return f(s["q"], s["k"], s["f"], s["b"], s["A_log"], dt_bias=s["bias"], lower_bound=s["bound"], eps=EPS_IN)
    if op == "in_bwd":
        f = kda.gdn_block_in_bwd if s["scalar"] else kda.block_in_bwd
        return f(s["q"], s["k"], s["f"], s["b"], s["A_log"], s["dq"], s["dk"], s["dg"], s["dbeta"], dt_bias=s["bias"],
                 lower_bound=s["bound"], eps=EPS_IN)
    if op == "out":
        return kda.block_out(s["o"], s["z"], s["w"], activation=s["act"], eps=EPS_OUT)
    return kda.block_out_bwd(s["o"], s["z"], s["w"], s["dy"], activation=s["act"], eps=EPS_OUT)


def _rows(x, s):
    """[B, T, ...] -> one row per sequence, padded with zeros: [N, L, ...] in fp32, L a multiple of C."""
    x = x.float()
    if s["cu"] is not None:
        x = torch.nn.utils.rnn.pad_sequence(list(x[0].split(s["lens"])), batch_first=True)
    pad = -x.shape[1] % C
    return torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1) if pad else x


def _unrows(x, s):
    """The inverse of _rows."""
    if s["cu"] is None:
        return x[:, :s["lens"][0]]
    return torch.cat([x[i, :l] for i, l in enumerate(s["lens"])])[None]


def _chunks(x):
    """[N, L, H, ...] -> [N, H, L / C, C, ...]"""
    return x.unflatten(1, (-1, C)).movedim(3, 1)


def _bwd(s):
    q, k, v, g, b, do = (_chunks(_rows(s[x], s)) for x in ("q", "k", "v", "g", "beta", "do"))
    if s["scalar"]:
        g = g[..., None].expand_as(q)
    N, H, n = q.shape[:3]
    b = b[..., None]
    G = g.cumsum(-2)
    # decay from token s to token t of a chunk, per channel, 0 above the diagonal
    low = torch.ones(C, C, device=q.device).tril()
    E = (G[..., :, None, :] - G[..., None, :, :]).clamp_max_(0.0).exp_().mul_(low[..., None])
    strict = low.tril(-1)
    M = (E * q[..., :, None, :]).mul_(k[..., None, :, :]).sum(-1)
    B = (E * k[..., :, None, :]).mul_(k[..., None, :, :]).sum(-1) * strict
    # (I + A)^-1 for a strictly lower triangular A of 16 rows: A^16 = 0
    eye = torch.eye(C, device=q.device)
    A = b * B
    A2 = A @ A
    A4 = A2 @ A2
    inv = (eye - A) @ (eye + A2) @ (eye + A4) @ (eye + A4 @ A4)
    kr, qr = k * G.exp(), q * G.exp()
    kc = k * (G[..., -1:, :] - G).exp()
    last = G[..., -1, :, None].exp()
    W, U = inv @ (b * kr), inv @ (b * v)
    S = s["h0"] if s["h0"] is not None else q.new_zeros(N, H, D, D)
    starts, deltas = [], []
    for i in range(n):
        starts.append(S)
        deltas.append(U[:, :, i] - W[:, :, i] @ S)
        S = last[:, :, i] * S + kc[:, :, i].transpose(-1, -2) @ deltas[-1]
    dS = s["dhT"] if s["dhT"] is not None else q.new_zeros(N, H, D, D)
    ends, rhos = [], []
    Md, Tt, qd = M.transpose(-1, -2) @ do, inv.transpose(-1, -2).contiguous(), qr.transpose(-1, -2) @ do
    bkr = (b * kr).transpose(-1, -2).contiguous()
    for i in reversed(range(n)):
        ends.append(dS)
        rhos.append(Tt[:, :, i] @ (Md[:, :, i] + kc[:, :, i] @ dS))
        dS = last[:, :, i] * dS + qd[:, :, i] - bkr[:, :, i] @ rhos[-1]
    if not n:
        z = lambda x: torch.zeros_like(s[x])
        return z("q"), z("k"), z("v"), z("g"), z("beta"), dS.clone()
    S, delta = torch.stack(starts, 2), torch.stack(deltas, 2)
    dE, rho = torch.stack(ends[::-1], 2), torch.stack(rhos[::-1], 2)
    r = b * rho
    err = v - kr @ S - B @ delta
    db = (err * rho).sum(-1)
    dM = (do @ delta.transpose(-1, -2).contiguous()) * low
    dB = -(r @ delta.transpose(-1, -2).contiguous()) * strict
    St = S.transpose(-1, -2).contiguous()
    carry = (G[..., -1:, :] - G).exp() * (delta @ dE.transpose(-1, -2).contiguous())
    dq = G.exp() * (do @ St) + (E * dM[..., None]).mul_(k[..., None, :, :]).sum(-2)
    row = (E * dB[..., None]).mul_(k[..., None, :, :]).sum(-2) - G.exp() * (r @ St)
    col = (E * (dM[..., None] * q[..., :, None, :] + dB[..., None] * k[..., :, None, :])).sum(-3) + carry
    dG = q * dq + k * (row - col)
    end = (k * carry).sum(-2) + (last * S * dE).sum(-1)
    dg = dG.flip(-2).cumsum(-2).flip(-2) + end[..., None, :]
    if s["scalar"]:
        dg = dg.sum(-1)
    back = lambda x, like: _unrows(x.movedim(1, 3).flatten(1, 2), s).to(like.dtype).contiguous()
    return back(dq, s["q"]), back(row + col, s["k"]), back(r, s["v"]), back(dg, s["g"]), back(db, s["beta"]), dS


def _rec(s):
    on = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][on].long()
    q, k, v, g, b = (s[x][on].float() for x in ("q", "k", "v", "g", "beta"))
    if s["scalar"]:
        g = g[..., None]
    S = s["pool"][slots].float()
    for t in range(q.shape[1]):
        S = S * g[:, t].exp()[..., None]
        e = b[:, t, :, None] * (v[:, t] - (S * k[:, t, ..., None]).sum(-2))
        S = S + k[:, t, ..., None] * e[..., None, :]
        s["o"][on, t] = (S * q[:, t, ..., None]).sum(-2)
        if s["out_slots"] is not None:
            s["pool"][s["out_slots"][on, t].long()] = S.to(s["pool"].dtype)
    if s["out_slots"] is None:
        s["pool"][slots] = S.to(s["pool"].dtype)
    return s["o"], s["pool"]


def _in(s):
    q, k, f, b = (s[x].float() for x in ("q", "k", "f", "b"))
    a = s["A_log"].exp() if s["scalar"] else s["A_log"].exp()[:, None]
    x = f + s["bias"]
    if s["bound"] is None:
        g = -a * (x.clamp_min(0.0) + torch.log1p((-x.abs()).exp()))
    else:
        g = s["bound"] / (1.0 + (-a * x).exp())
    norm = lambda u: u / (u.square().sum(-1, keepdim=True) + EPS_IN).sqrt()
    return norm(q).to(s["q"].dtype), norm(k).to(s["k"].dtype), g, 1.0 / (1.0 + (-b).exp())


def _in_bwd(s):
    q, k, f, b, dq, dk, dg = (s[x].float() for x in ("q", "k", "f", "b", "dq", "dk", "dg"))
    a = s["A_log"].exp() if s["scalar"] else s["A_log"].exp()[:, None]
    x = f + s["bias"]
    if s["bound"] is None:
        dx = -a * dg / (1.0 + (-x).exp())
        dA = -a * dg * (x.clamp_min(0.0) + torch.log1p((-x.abs()).exp()))
    else:
        sg = 1.0 / (1.0 + (-a * x).exp())
        dx = s["bound"] * sg * (1.0 - sg) * a * dg
        dA = dx * x

    def norm(u, du):
        r = 1.0 / (u.square().sum(-1, keepdim=True) + EPS_IN).sqrt()
        n = u * r
        return r * (du - n * (n * du).sum(-1, keepdim=True))

    sb = 1.0 / (1.0 + (-b).exp())
    dA = dA.sum((0, 1), dtype=torch.float64)
    return (norm(q, dq).to(s["q"].dtype), norm(k, dk).to(s["k"].dtype), dx.to(s["f"].dtype),
            (s["dbeta"] * sb * (1.0 - sb)).to(s["b"].dtype), (dA if s["scalar"] else dA.sum(-1)).float(),
            dx.sum((0, 1), dtype=torch.float64).float())


def _act(z, kind):
    sg = 1.0 / (1.0 + (-z).exp())
    return (sg, sg * (1.0 - sg)) if kind == "sigmoid" else (z * sg, sg * (1.0 + z * (1.0 - sg)))


def _out(s):
    o, z = s["o"], s["z"].float()
    n = o / (o.square().mean(-1, keepdim=True) + EPS_OUT).sqrt()
    return (n * s["w"] * _act(z, s["act"])[0]).to(s["z"].dtype)


def _out_bwd(s):
    o, z, dy = s["o"], s["z"].float(), s["dy"].float()
    r = 1.0 / (o.square().mean(-1, keepdim=True) + EPS_OUT).sqrt()
    n = o * r
    a, da = _act(z, s["act"])
    dn = dy * s["w"] * a
    return (r * (dn - n * (n * dn).mean(-1, keepdim=True)), (dy * n * s["w"] * da).to(s["z"].dtype),
            (dy * n * a).sum((0, 1, 2), dtype=torch.float64).float())


# ------------------------------------------------------------------------------------------------ work

def work(case):
    """Bytes: every input read once, every output written once. Flops: the token-by-token form's products."""
    B, T, H = case["B"], case["T"], case["H"]
    e = 2 if case["dtype"] == "bf16" else 4
    tok = B * T * H
    gate = 1 if case["gate"] == "scalar" else D
    op = case["op"]
    if op == "bwd":
        states = len(_lens(case)[0]) * H * D * D
        # read q k v g beta do, write dq dk dv dg dbeta; the two start states and their gradients
        by = tok * (6 * D * e + 8 * gate + 8 + 4 * D) + 4 * states * (3 if case.get("state") else 1)
        # S: decay, prediction, update; gradient: three products with the state, two with its gradient, two updates
        return {"bytes": by, "flops": tok * D * D * (2 * 2 + 7 * 2)}
    if op == "rec":
        live = B - case.get("empty", 0)
        p = 2 if case["pool"] == "bf16" else 4
        kept = T if case.get("keep") else 1
        return {"bytes": live * H * ((1 + kept) * D * D * p + T * (3 * D * e + 4 * gate + 4 + 4 * D)),
                "flops": live * H * T * 7 * D * D}
    if op == "in":
        return {"bytes": tok * (4 * D * e + gate * (e + 4) + e + 4), "flops": tok * (8 * D + 8 * gate)}
    if op == "in_bwd":
        return {"bytes": tok * (6 * D * e + gate * (2 * e + 4) + 2 * e + 4), "flops": tok * (20 * D + 12 * gate)}
    if op == "out":
        return {"bytes": tok * D * (4 + 2 * e), "flops": tok * 10 * D}
    return {"bytes": tok * D * (8 + 3 * e), "flops": tok * 24 * D}


# ------------------------------------------------------------------------------- definitions in 64 bits

def _steps(S, q, k, v, g, b):
    """The recurrence token by token: S [H, K, V], the others [T, H, ...]. Returns (o [T, H, V], S)."""
    o = []
    for t in range(q.shape[0]):
        S = g[t].exp()[..., None] * S
        e = b[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
        S = S + k[t][..., None] * e[:, None, :]
        o.append(torch.einsum("hk,hkv->hv", q[t], S))
    return torch.stack(o), S


def _exact_bwd(s):
    """Reverse differentiation of the token recurrence, in segments restarted from stored states."""
    x = [s[n].double() for n in ("q", "k", "v", "g", "beta")]
    if s["scalar"]:
        x[3] = x[3][..., None]
    grads, dh0, seg, at = [torch.zeros_like(u) for u in x], [], 64, 0
    H = x[0].shape[2]
    for n, length in enumerate(s["lens"]):
        row, t0 = (0, at) if s["cu"] is not None else (n, 0)
        at += length
        S = s["h0"][n].double() if s["h0"] is not None else x[0].new_zeros(H, D, D)
        marks = list(range(t0, t0 + length, seg))
        kept = []
        with torch.no_grad():
            for m in marks:
                kept.append(S)
                S = _steps(S, *(u[row, m:min(m + seg, t0 + length)] for u in x))[1]
        dS = s["dhT"][n].double() if s["dhT"] is not None else torch.zeros_like(S)
        for m, S in reversed(list(zip(marks, kept))):
            part = slice(m, min(m + seg, t0 + length))
            leaves = [S.clone().requires_grad_()] + [u[row, part].clone().requires_grad_() for u in x]
            with torch.enable_grad():
                o, end = _steps(*leaves)
            got = torch.autograd.grad([o, end], leaves, [s["do"][row, part].double(), dS])
            dS = got[0]
            for to, d in zip(grads, got[1:]):
                to[row, part] = d
        dh0.append(dS)
    if s["scalar"]:
        grads[3] = grads[3][..., 0]
    return (*grads, torch.stack(dh0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "bwd":
        return _exact_bwd(s)
    if op == "rec":
        o, pool = s["o"].double(), s["pool"].double()
        for n, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            x = [s[u][n].double() for u in ("q", "k", "v", "g", "beta")]
            if s["scalar"]:
                x[3] = x[3][..., None]
            S = pool[slot]
            for t in range(case["T"]):
                y, S = _steps(S, *(u[t:t + 1] for u in x))
                o[n, t] = y[0]
                if s["out_slots"] is not None:
                    pool[int(s["out_slots"][n, t])] = S
            if s["out_slots"] is None:
                pool[slot] = S
        return o, pool
    leaf = lambda name: s[name].double().requires_grad_()
    with torch.enable_grad():
        if op in ("in", "in_bwd"):
            x = [leaf(n) for n in ("q", "k", "f", "b", "A_log", "bias")]
            q, k, f, b, A, bias = x
            a = A.exp() if s["scalar"] else A.exp()[:, None]
            unit = lambda u: u * torch.rsqrt(u.pow(2).sum(-1, keepdim=True) + EPS_IN)
            g = (-a * torch.logaddexp(f + bias, torch.zeros_like(f)) if s["bound"] is None
                 else s["bound"] * torch.sigmoid(a * (f + bias)))
            y = [unit(q), unit(k), g, torch.sigmoid(b)]
            if op == "in":
                return tuple(u.detach() for u in y)
            return torch.autograd.grad(y, x, [s[n].double() for n in ("dq", "dk", "dg", "dbeta")])
        x = [leaf(n) for n in ("o", "z", "w")]
        o, z, w = x
        act = torch.sigmoid(z) if s["act"] == "sigmoid" else z * torch.sigmoid(z)
        y = o * torch.rsqrt(o.pow(2).mean(-1, keepdim=True) + EPS_OUT) * w * act
        return y.detach() if op == "out" else torch.autograd.grad(y, x, s["dy"].double())

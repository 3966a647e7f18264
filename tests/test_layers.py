"""The operators between and beside the rules together, as they are used: a stack of layers
forwards and back through autograd functions, and beam decoding over pools of states."""
import numpy as np
import pytest

import layers_ref as R

torch = pytest.importorskip("torch")


@pytest.fixture
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_63_amd as kda
    return kda


# -------------------------------------------------------------------- training

def functions(kda, cu):
    """The calls joined with their gradients."""
    class AddNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, res, w):
            y, r = kda.add_norm(x, res, w)
            ctx.save_for_backward(r, w)
            return y, r

        @staticmethod
        def backward(ctx, dy, dr):
            r, w = ctx.saved_tensors
            dx, dres, dw = kda.add_norm_bwd(r, w, dy.contiguous(), dr=dr.contiguous())
            return dx, dres, dw

    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, g, h0):
            y, hT, kept = kda.scan(x, g, cu_seqlens=cu, initial_state=h0, leaky=True, output_chunk_states=True)
            ctx.save_for_backward(x, g, h0, kept)
            return y, hT

        @staticmethod
        def backward(ctx, dy, dhT):
            x, g, h0, kept = ctx.saved_tensors
            return kda.scan_bwd(x, g, dy.contiguous(), cu_seqlens=cu, initial_state=h0, d_final_state=dhT.contiguous(),
                                chunk_states=kept, leaky=True)

    return AddNorm.apply, Scan.apply


def stack(x, w, proj, gate, h0, add_norm, scan):
    """Two layers: norm of the stream, a projection, the rule; then the last norm."""
    r, h, ends = x, torch.zeros_like(x), []
    for i in range(2):
        y, r = add_norm(h, r, w[i])
        h, hT = scan((y @ proj[i]).contiguous(), -torch.nn.functional.softplus(y @ gate[i]).contiguous(), h0[i])
        ends.append(hT)
    y, r = add_norm(h, r, w[2])
    return y, r, ends


@pytest.mark.gpu
def test_two_layers_and_their_gradients(kda):
    """Outputs and the gradients of every leaf, in fp32, against automatic differentiation
    of the formulas in fp64. Each element is a chain of about ten sums of up to 300 fp32
    products, of states over up to 140 tokens and of 24 channels: 10 sqrt(300) 2^-24 = 1e-5
    at one sigma of the largest term, 1e-4 of the RMS at the outermost of 10,000 elements."""
    C, lens = 24, (140, 0, 33, 127)
    T, bounds = sum(lens), R.bounds_of(lens, 1, sum(lens))
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen)
    x, w, h0 = n(1, T, C), [1 + 0.2 * n(C) for _ in range(3)], [n(len(lens), C) for _ in range(2)]
    proj, gate = [n(C, C) / C ** 0.5 for _ in range(2)], [n(C, C) / C ** 0.5 for _ in range(2)]
    ty, tr, te = n(1, T, C), n(1, T, C), [n(len(lens), C) for _ in range(2)]

    def run(dev, dtype, add_norm, scan):
        leaf = lambda t: t.to(dev, dtype).requires_grad_()
        leaves = [leaf(x), *map(leaf, w), *map(leaf, proj), *map(leaf, gate), *map(leaf, h0)]
        X, W, P, G, H = leaves[0], leaves[1:4], leaves[4:6], leaves[6:8], leaves[8:10]
        y, r, ends = stack(X, W, P, G, H, add_norm, scan)
        to = lambda t: t.to(dev, dtype)
        loss = (y * to(ty)).sum() + (r * to(tr)).sum() + sum((e * to(t)).sum() for e, t in zip(ends, te))
        grads = torch.autograd.grad(loss, leaves)
        return [t.detach().double().cpu().numpy() for t in (y, r, *ends, *grads)]

    def ref_norm(h, res, w):
        r = h + res
        return r / (r.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w, r

    def ref_scan(x, g, h0):
        rows, ends = [], []
        for i, (_, t0, t1) in enumerate(bounds):
            s = h0[i]
            for t in range(t0, t1):
                a = g[0, t].exp()
                s = a * s + (1 - a) * x[0, t]
                rows.append(s)
            ends.append(s)
        return torch.stack(rows)[None], torch.stack(ends)

    cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32).cuda()
    got = run("cuda", torch.float32, *functions(kda, cu))
    torch.cuda.synchronize()
    want = run("cpu", torch.float64, ref_norm, ref_scan)
    names = ["y", "r", "hT 0", "hT 1", "dx", "dw 0", "dw 1", "dw 2", "dproj 0", "dproj 1", "dgate 0", "dgate 1", "dh0 0", "dh0 1"]
    for u, v, what in zip(got, want, names):
        off = float(np.max(np.abs(u - v))) / float(np.sqrt(np.mean(v ** 2)))
        print(f"{what}: {off:.1e}")
        assert off <= 1e-4, what


# -------------------------------------------------------------------- decoding

B, W, V, C, STEPS, EOS = 2, 4, 61, 128, 7, 3


def model(seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    return dict(embed=n(V, C), w=[1 + 0.2 * n(C) for _ in range(3)], qkv=[n(C, C) / C ** 0.5 for _ in range(3)],
                gate=[n(C, C) / C ** 0.5 for _ in range(2)], x=n(C, C) / C ** 0.5, out=2.5 * n(C, V) / C ** 0.5)


def token(m, tok, rule, scan, norm):
    """One token: stream -> norm -> matrix-state rule -> norm -> vector-state rule -> norm -> logits."""
    r = m["embed"][tok]
    y, r = norm(torch.zeros_like(r), r, m["w"][0])
    q, k, v = (y @ p for p in m["qkv"])
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    g = -torch.nn.functional.softplus(y @ m["gate"][0])
    h = rule(q, k, v, g, torch.sigmoid(y[..., :1]))
    y, r = norm(h, r, m["w"][1])
    h = scan(y @ m["x"], -torch.nn.functional.softplus(y @ m["gate"][1]))
    y, r = norm(h, r, m["w"][2])
    return y @ m["out"]


def decode_ref(m, first):
    """Every hypothesis with states of its own, in fp64. Yields after each step, per entry:
    (scores, parents, tokens); and the smallest gap between totals that decided anything."""
    m = {k: [u.double() for u in v] if isinstance(v, list) else v.double() for k, v in m.items()}
    norm = lambda h, res, w: ((h + res) / ((h + res).square().mean(-1, keepdim=True) + 1e-5).sqrt() * w, h + res)
    hyps = [[dict(S=torch.zeros(C, C, dtype=torch.float64), h=torch.zeros(C, dtype=torch.float64), score=0.0 if w == 0 else -np.inf,
                  tok=int(first[b]), done=False) for w in range(W)] for b in range(B)]
    gap, out = np.inf, []
    for _ in range(STEPS):
        row = []
        for b in range(B):
            logits = []
            for hy in hyps[b]:
                def rule(q, k, v, g, beta):
                    S = g.exp()[:, None] * hy["S"]
                    S = S + k[:, None] * (beta * (v - k @ S))[None]
                    hy["S2"] = S
                    return q @ S

                def scan(x, g):
                    hy["h2"] = g.exp() * hy["h"] + (1 - g.exp()) * x
                    return hy["h2"]

                logits.append(token(m, hy["tok"], rule, scan, norm).numpy())
            done, scores = [hy["done"] for hy in hyps[b]], np.array([hy["score"] for hy in hyps[b]])
            best, parents, tokens = R.beam(np.stack(logits), scores, W + 1, done, EOS)
            live = best[best > -np.inf]
            gap = min(gap, np.min(-np.diff(live), initial=np.inf))
            row.append((best[:W], parents[:W], tokens[:W]))
            hyps[b] = [dict(S=hyps[b][p]["S2"], h=hyps[b][p]["h2"], score=s, tok=int(t), done=bool(t == EOS))
                       for s, p, t in zip(best[:W], parents[:W], tokens[:W])]
        out.append(row)
    states = [[(hy["S"].numpy(), hy["h"].numpy()) for hy in hyps[b]] for b in range(B)]
    return out, gap, states


SEED, FIRST = 7, (5, 11)


def test_decoding_reference():
    """The decisions of the case below do not hang on fp32 rounding: no two totals that
    decide one lie within 1e-3; beams fork, die and end in it."""
    out, gap, _ = decode_ref(model(SEED), FIRST)
    assert gap > 1e-3, gap
    parents = [list(p) for row in out[1:] for _, p, _ in row]
    assert any(len(set(p)) < W for p in parents) and any(p != sorted(p) for p in parents)
    assert any((t == EOS).any() for row in out for _, _, t in row)


@pytest.mark.gpu
@pytest.mark.parametrize("graph", [False, True])
def test_beam_decoding_over_pools(kda, graph):
    """Steps of beam search over a pool of matrix states and one of vector states, against
    hypotheses that each keep their own; eagerly, and as one captured step that is
    replayed. Scores: a few steps of fp32 logits of about 10, 2^-24 * 10 * sqrt(128) = 7e-6 a
    step at one sigma; bar 2e-4."""
    m = {k: [u.cuda() for u in v] if isinstance(v, list) else v.cuda() for k, v in model(SEED).items()}
    want, _, ref_states = decode_ref(model(SEED), FIRST)
    P = 3 * B * W
    order = torch.randperm(P, generator=torch.Generator().manual_seed(2))[:B * W].reshape(B, W).to(torch.int32)
    mat, vec = torch.zeros(P, 1, C, C, device="cuda"), torch.zeros(P, C, device="cuda")
    slots, tok = order.cuda(), torch.tensor([[f] * W for f in FIRST]).cuda()
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros(B, W, dtype=torch.bool, device="cuda")
    parents, same = torch.zeros_like(slots), torch.ones(1, dtype=torch.bool, device="cuda")

    def step():
        flat = slots.reshape(-1)

        def rule(q, k, v, g, beta):
            q, k, v, g = (t.reshape(B * W, 1, 1, C).contiguous() for t in (q, k, v, g))
            return kda.recurrent(q, k, v, g, beta.reshape(B * W, 1, 1).contiguous(), mat, slots=flat).reshape(B, W, C)

        def scan(x, g):
            return kda.scan_recurrent(x.reshape(B * W, 1, C).contiguous(), g.reshape(B * W, 1, C).contiguous(), vec, slots=flat,
                                      leaky=True).reshape(B, W, C)

        logits = token(m, tok, rule, scan, lambda h, r, w: kda.add_norm(h.contiguous(), r.contiguous(), w))
        best, par, new = kda.beam_select(logits.contiguous(), scores, done=done, eos=EOS)
        to = kda.beam_reorder(mat, slots, par)
        same.logical_and_((to == kda.beam_reorder(vec, slots, par)).all())
        slots.copy_(to)
        scores.copy_(best)
        parents.copy_(par)
        tok.copy_(new.clamp_min(0))
        done.copy_(new == EOS)

    if graph:
        state = [t.clone() for t in (mat, vec, slots, tok, scores, done)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                         # warm
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        for t, s in zip((mat, vec, slots, tok, scores, done), state):
            t.copy_(s)
    for i in range(STEPS):
        if graph:
            captured.replay()
        else:
            step()
        torch.cuda.synchronize()
        for b in range(B):
            rb, rp, rt = want[i][b]
            assert parents[b].tolist() == rp.tolist() and tok[b].tolist() == rt.tolist(), (i, b)
            assert np.allclose(scores[b].cpu().numpy(), rb, rtol=0, atol=2e-4), (i, b)
    assert bool(same)
    for b in range(B):
        assert sorted(slots[b].tolist()) == sorted(order[b].tolist())
        for w in range(W):
            S, h = ref_states[b][w]
            at = int(slots[b, w])
            assert np.abs(mat[at, 0].cpu().numpy() - S).max() <= 1e-4 * np.abs(S).max() + 1e-6
            assert np.abs(vec[at].cpu().numpy() - h).max() <= 1e-4 * np.abs(h).max() + 1e-6

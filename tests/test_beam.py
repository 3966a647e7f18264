"""A step of beam search: the selection (kda_beam_select) against totals in fp64, and the
reordering of a pool's states (kda_beam_reorder)."""
import ctypes

import numpy as np
import pytest

import layers_ref as R

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(0x10000)   # never dereferenced


# ------------------------------------------------------------------------- CPU

def test_reference_by_hand():
    x = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.9, 0.0 + 1e-300]]))
    best, parents, tokens = R.beam(x, np.array([-1.0, -1.5]), 4)
    want = [-1.0 + np.log(0.5), -1.5 + np.log(0.9), -1.0 + np.log(0.25), -1.0 + np.log(0.25)]
    assert list(parents) == [1, 0, 0, 0] and list(tokens) == [1, 0, 1, 2]     # -1.605, -1.693, a tie
    assert np.allclose(best, sorted(want, reverse=True))
    best, parents, tokens = R.beam(x, np.array([-1.0, -0.1]), 3, done=[False, True], eos=2)
    assert list(parents) == [1, 0, 0] and list(tokens) == [2, 0, 1] and best[0] == -0.1
    assert R.reorder([7, 3, 9], [1, 1, -1]) == ([3, 7, 9], [(3, 7)])


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()
    D = lambda B=2, W=3, V=50, K=3, dt=0, eos=0, ws=None, n=0: kda._lib.BeamDesc(B, W, V, K, dt, eos, ws, n)
    need = L.kda_beam_workspace_size(ctypes.byref(D()))
    assert need >= 2 * 3 * (16 + 3 * 8)
    ok = lambda **kw: D(ws=P, n=1 << 40, **kw)
    call = lambda d, x=P, s=P, done=None, out=P, p=P, t=P: L.kda_beam_select(x, s, done, out, p, t, None if d is None else ctypes.byref(d), None)
    assert call(None) == -1
    for name in ("x", "s", "out", "p", "t"):
        assert call(ok(), **{name: None}) == -1
    for d in (ok(B=-1), ok(W=0), ok(W=65), ok(K=0), ok(K=65), ok(V=0), ok(V=(1 << 25) + 1), ok(B=1 << 20, W=2)):
        assert call(d) == -2
    assert call(ok(eos=-1), done=P) == -2 and call(ok(eos=50), done=P) == -2
    assert call(ok(dt=3)) == -4 and call(D()) == -5 and call(D(ws=P, n=need - 1)) == -5
    assert call(D(ws=ctypes.c_void_p(0x10004), n=need)) == -3
    assert call(ok(B=0), x=None, s=None, out=None, p=None, t=None) == 0
    assert L.kda_beam_workspace_size(None) == 0 and L.kda_beam_workspace_size(ctypes.byref(D(W=0))) == 0
    re = lambda pool=P, num=9, size=64, s=P, p=P, out=P, B=2, W=3: L.kda_beam_reorder(pool, num, size, s, p, out, B, W, None)
    for kw in (dict(pool=None), dict(s=None), dict(p=None), dict(out=None)):
        assert re(**kw) == -1
    for kw in (dict(num=-1), dict(B=-1), dict(W=0), dict(W=65), dict(B=1 << 20, W=2), dict(size=1 << 48)):
        assert re(**kw) == -2
    assert re(B=0, pool=None, s=None) == 0


def test_binding_refusals():
    from gated_delta_rule_63_amd import _layers as M
    z, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
    x, s = z(2, 3, 50), z(2, 3)
    ok = lambda x=x, s=s, k=None, done=None, eos=-1: M._check_beam(x, s, k, done, eos, _device=False)
    assert ok().K == 3 and ok(k=5).K == 5
    ok(x=x.bfloat16(), done=z(2, 3, dtype=torch.bool), eos=49)
    for kw in (dict(x=x.half()), dict(x=z(6, 50)), dict(s=z(2, 4)), dict(s=s.double()), dict(k=0), dict(k=65), dict(done=z(2, 3), eos=1),
               dict(done=z(2, 3, dtype=torch.bool)), dict(done=z(2, 3, dtype=torch.bool), eos=50), dict(x=z(2, 65, 3), s=z(2, 65)),
               dict(x=z(2, 50, 3).transpose(1, 2))):
        with pytest.raises(ValueError):
            ok(**kw)
    re = lambda pool=z(9, 4), s=i(2, 3), p=i(2, 3), out=None: M._check_reorder(pool, s, p, out, _device=False)
    re()
    same = i(2, 3)
    for kw in (dict(s=same, out=same), dict(p=same, out=same), dict(pool=z(4, 9).T), dict(s=i(6)), dict(p=i(2, 4)), dict(p=z(2, 3)), dict(out=i(3, 2)), dict(s=i(2, 65), p=i(2, 65))):
        with pytest.raises(ValueError):
            re(**kw)


def test_workspace_size():
    import gated_delta_rule_63_amd as kda
    for shape, k, dtype in (((2, 3, 50), None, torch.float32), ((1, 1, 7), 5, torch.bfloat16), ((64, 8, 131072), 16, torch.bfloat16), ((0, 2, 9), 2, torch.float32)):
        d = kda._lib.BeamDesc(*shape, k or shape[1], int(dtype == torch.float32), 0, None, 0)
        assert kda.beam_workspace_size(torch.empty(shape, dtype=dtype, device="meta"), k) == kda.lib().kda_beam_workspace_size(ctypes.byref(d))
    assert kda.beam_workspace_size(torch.empty(2, 3, 50)) > 0
    with pytest.raises(ValueError):
        kda.beam_workspace_size(torch.empty(6, 50))


def test_new_slots_apart_from_the_inputs():
    """Slots of new beams that overlap an input, in part or as a whole, are refused: other workgroups still read it."""
    from gated_delta_rule_63_amd import _layers as M
    flat, other, pool = torch.zeros(12, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(9, 4)
    part = lambda i: flat[i:i + 6].view(2, 3)
    re = lambda s, p, out: M._check_reorder(pool, s, p, out, _device=False)
    re(part(0), other, part(6))
    re(other, part(6), part(0))
    for at in (0, 1, 5):
        with pytest.raises(ValueError):
            re(part(at), other, part(0))
        with pytest.raises(ValueError):
            re(other, part(0), part(at))
    empty = torch.zeros(0, 3, dtype=torch.int32)
    re(empty, empty, empty)


def test_sizes_beyond_32_bits():
    """2^32 + 3 of anything is refused, not taken for 3. (Tensors without storage.)"""
    from gated_delta_rule_63_amd import _layers as M
    n = (1 << 32) + 3
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")
    for B, W, V in ((1, 1, n), (n, 1, 1)):
        with pytest.raises(ValueError, match="32 bits"):
            M._check_beam(e(B, W, V), e(B, W), 1, None, -1, _device=False)
        with pytest.raises(ValueError, match="32 bits"):
            M.beam_workspace_size(e(B, W, V))
    i = lambda *s: e(*s, dtype=torch.int32)
    for pool, slots in ((e(n, 1), i(2, 3)), (e(9, 1), i(n, 1))):
        with pytest.raises(ValueError, match="32 bits"):
            M._check_reorder(pool, slots, slots, None, _device=False)


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_63_amd as kda
    return kda


def check(kda, x, scores, K, done=None, eos=-1):
    got = kda.beam_select(x.cuda(), scores.cuda(), k=K, done=None if done is None else done.cuda(), eos=eos)
    torch.cuda.synchronize()
    best, parents, tokens = (t.cpu().numpy() for t in got)
    for b in range(x.shape[0]):
        rb, rp, rt = R.beam(x[b].float().numpy(), scores[b].numpy(), K, None if done is None else done[b].numpy(), eos)
        assert np.array_equal(parents[b], rp) and np.array_equal(tokens[b], rt), (b, parents[b], rp, tokens[b], rt)
        some = rb > -np.inf
        assert np.array_equal(best[b] == -np.inf, ~some)
        # the log of the sum: fp32 exponentials of differences up to 20, 20 * 2^-24 + 2^-23 each at most; the
        # score's own rounding
        assert np.all(np.abs(best[b][some] - rb[some]) <= 22 * R.U + R.U * np.abs(rb[some])), b
    return got


def draw(B, W, V, dtype, seed, scale=3.0):
    """Logits and scores whose totals are far enough apart (or tie exactly within a row)."""
    gen = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(B, W, V, generator=gen)).to(getattr(torch, dtype)), -10 + 3 * torch.randn(B, W, generator=gen)


CASES = [(1, 1, 1, 1), (2, 3, 2, 5), (1, 4, 7, 4), (3, 2, 64, 64), (2, 5, 100, 10), (1, 1, 255, 3), (2, 8, 257, 16), (1, 4, 1000, 1),
         (4, 3, 4099, 6), (1, 16, 32000, 32), (2, 2, 50001, 4), (1, 64, 2000, 64), (1, 1, 131072, 64), (5, 4, 8192, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,W,V,K", CASES)
def test_select(kda, B, W, V, K, dtype):
    x, scores = draw(B, W, V, dtype, 1)
    check(kda, x, scores, K)
    done = torch.rand(B, W, generator=torch.Generator().manual_seed(2)) < 0.4
    check(kda, x, scores, K, done, V // 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [5, 64, 1000, 40003])
def test_ties_and_masked_places(kda, V, dtype):
    """Equal logits throughout; few distinct ones; ascending and descending rows; -inf, NaN and
    +inf among them; rows and entries without a candidate; dead beams."""
    inf, dt = float("inf"), getattr(torch, dtype)
    flat = torch.zeros(1, 3, V, dtype=dt)
    for scores in (torch.tensor([[-3.0, -1.0, -1.0]]), torch.tensor([[-3.0, -1.0, -1.7]])):   # (equal rows tie across beams, too)
        check(kda, flat, scores, 8)
        check(kda, flat - 7e4, scores, 3)
    few = torch.randint(0, 3, (1, 3, V), generator=torch.Generator().manual_seed(3)).to(dt)
    check(kda, few, scores, 8)
    ramp = torch.arange(V).float().mul(0.01).to(dt)
    check(kda, torch.stack([ramp, ramp.flip(0), ramp])[None].contiguous(), scores, 8)
    x, _ = draw(1, 3, V, dtype, 4)
    x[0, 0, ::2], x[0, 1, 1:], x[0, 2] = -inf, float("nan"), -inf
    check(kda, x, scores, 16)
    x[0, 1, 0] = -inf
    check(kda, x, scores, 16)
    x[:] = float("nan")
    check(kda, x, scores, 2)
    x, _ = draw(1, 3, V, dtype, 5)
    x[0, 0, V - 1] = x[0, 0, 1] = inf
    check(kda, x, scores, 4)
    x[0, 1] = inf
    check(kda, x, scores, 8)
    x[:] = torch.where(torch.arange(V) % 2 == 0, -0.0, 0.0)       # zeros of either sign tie
    check(kda, x, scores, 8)
    x, _ = draw(1, 3, V, dtype, 5)
    lowest = torch.finfo(dt).min
    x[0, 0] = lowest
    x[0, 2, : V - 1] = lowest
    check(kda, x, scores, 4)
    dead = torch.tensor([[-inf, -2.0, float("nan")]])
    check(kda, draw(1, 3, V, dtype, 6)[0], dead, 8)
    check(kda, draw(1, 3, V, dtype, 6)[0], torch.full((1, 3), -inf), 2)
    check(kda, draw(1, 3, V, dtype, 6)[0], dead, 5, torch.tensor([[True, True, True]]), V - 1)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [5, 32, 64])
@pytest.mark.parametrize("W,V", [(16, 70001), (64, 700), (3, 150000)])
def test_many_keys(kda, W, V, K):
    """Many lists of keys an entry, with one beam ahead of the others, all alike, few distinct logits
    or only ordinary ones."""
    x, scores = draw(2, W, V, "bfloat16", 8)
    check(kda, x, scores, K)
    ahead = scores.clone()
    ahead[:, W // 2] += 30.0
    check(kda, x, ahead, K)
    check(kda, x[:1].expand(2, W, V).contiguous(), torch.full((2, W), -2.0), K)
    check(kda, x[:, :1].expand(2, W, V).contiguous(), torch.full((2, W), -2.0), K)
    check(kda, (x > 2.5).to(torch.bfloat16), torch.full((2, W), -1.0), K)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [7, 500, 2048, 9001])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_unaligned_logits(kda, dtype, V):
    """The same bits wherever the logits begin."""
    x, scores = draw(3, 4, V, dtype, 9)
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    flat[1:] = x.reshape(-1).cuda()
    check(kda, x, scores, 6)
    got = kda.beam_select(flat[1:].view(x.shape), scores.cuda(), k=6)
    assert all(torch.equal(a, b) for a, b in zip(got, kda.beam_select(x.cuda(), scores.cuda(), k=6)))


@pytest.mark.gpu
def test_logits_of_done_beams_are_not_read(kda):
    x, scores = draw(2, 4, 3000, "float32", 7)
    done = torch.tensor([[True, False, True, False], [False, False, False, True]])
    want = check(kda, x, scores, 6, done, 5)
    x[done] = float("nan")
    got = check(kda, x, scores, 6, done, 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_rows_beyond_32_bit_offsets(kda):
    """2.2e9 logits: the last entry as by itself."""
    x = torch.empty(68, 16, 1 << 21, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    scores = -torch.rand(68, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    got = kda.beam_select(x, scores, k=4)
    alone = kda.beam_select(x[67:].clone(), scores[67:].contiguous(), k=4)
    # other splits of a row may round the sum otherwise
    assert torch.equal(got[1][67:], alone[1]) and torch.equal(got[2][67:], alone[2])
    assert float((got[0][67:] - alone[0]).abs().max()) <= 44 * R.U + 2 * R.U * 16


REORDER = [(1, 1, (4,), "float32"), (3, 4, (2, 128, 128), "float32"), (2, 5, (3, 7), "bfloat16"), (5, 8, (33,), "float32"),
           (2, 64, (16,), "bfloat16"), (7, 16, (5,), "bfloat16"), (300, 4, (64,), "float32"), (2, 3, (1,), "uint8")]


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,shape,dtype", REORDER)
def test_reorder(kda, B, W, shape, dtype):
    gen = torch.Generator().manual_seed(1)
    n = 2 * B * W + 3
    pool = torch.randint(0, 256, (n, *shape), generator=gen).to(getattr(torch, dtype))
    slots = torch.randperm(n, generator=gen)[:B * W].reshape(B, W).to(torch.int32)
    parents = torch.randint(0, W, (B, W), generator=gen).to(torch.int32)
    parents[0] = W - 1                                     # all from one
    if B > 1:
        parents[1] = torch.arange(W).flip(0)               # a permutation: nothing is copied
    if B > 2:
        parents[2, 0], parents[2, W - 1] = -1, W + 3       # empty places
    for odd in (False, True):                              # a pool that starts on no 16 bytes, too
        flat = torch.zeros(pool.numel() + 1, dtype=pool.dtype, device="cuda")
        got = flat[1:].reshape(pool.shape) if odd else pool.cuda()
        got.copy_(pool)
        new = kda.beam_reorder(got, slots.cuda(), parents.cuda())
        torch.cuda.synchronize()
        want = pool.clone()
        for b in range(B):
            to, copies = R.reorder(slots[b].tolist(), parents[b].tolist())
            assert new[b].tolist() == to and sorted(to) == sorted(slots[b].tolist())
            for f, t in copies:
                want[t] = pool[f]
        assert torch.equal(got.cpu(), want)


@pytest.mark.gpu
def test_reorder_with_slots_outside_the_pool(kda):
    pool = torch.arange(12.0).reshape(6, 2)
    slots = torch.tensor([[-1, 2, 9, 4]], dtype=torch.int32)
    got = pool.cuda()
    new = kda.beam_reorder(got, slots.cuda(), torch.tensor([[1, 1, 1, 0]], dtype=torch.int32).cuda())
    # beam 1's further children take beams 2's and 3's places, of which 9 is no slot; 0's child keeps none
    assert new.tolist() == [[2, 9, 4, -1]]
    want = pool.clone()
    want[4] = pool[2]
    assert torch.equal(got.cpu(), want)
    got = pool.cuda()
    new = kda.beam_reorder(got, slots.cuda(), torch.tensor([[0, 0, 2, 2]], dtype=torch.int32).cuda())
    assert new.tolist() == [[-1, 2, 9, 4]] and torch.equal(got.cpu(), pool)      # sources that are no slots
    out = torch.empty_like(new)
    assert kda.beam_reorder(got[:0], slots.cuda(), torch.zeros_like(new), out=out) is out and torch.equal(got.cpu(), pool)


@pytest.mark.gpu
def test_far_slots(kda):
    """Slots that begin beyond 2^31 elements and 2^32 bytes."""
    pool = torch.zeros(34000, 65536, dtype=torch.bfloat16, device="cuda")
    pool[33990] = torch.arange(65536, device="cuda").bfloat16()
    new = kda.beam_reorder(pool, torch.tensor([[33990, 33999]], dtype=torch.int32).cuda(), torch.zeros(1, 2, dtype=torch.int32).cuda())
    assert new.tolist() == [[33990, 33999]] and torch.equal(pool[33999], pool[33990])
    assert not bool(pool[:33990].any()) and not bool(pool[33991:33999].any())


@pytest.mark.gpu
def test_streams_and_graphs(kda):
    """Two selections at once on two streams, and a captured step of selection and reorder."""
    x, scores = draw(8, 4, 30011, "bfloat16", 8)
    x, scores = x.cuda(), scores.cuda()
    want = kda.beam_select(x, scores, k=4)
    torch.cuda.synchronize()
    got = [kda.beam_select(x, scores, k=4, stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    start = torch.randn(40, 5, 3, device="cuda")
    pool, slots = start.clone(), torch.randperm(40, device="cuda")[:32].reshape(8, 4).to(torch.int32)

    def step():
        best = kda.beam_select(x, scores, k=4)
        return (*best, kda.beam_reorder(pool, slots, best[1]))

    eager = step()
    after = pool.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        pool.copy_(start)
        for u in held:
            u.fill_(0)
        graph.replay()
        other = kda.beam_select(x, scores, k=4)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)) and torch.equal(pool, after)
        assert all(torch.equal(a, b) for a, b in zip(other, want))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["gap", "ramp"])
def test_sums_of_long_rows(kda, kind):
    """Totals of rows that one workgroup adds up (there are 1024 of them), against fp64: a largest
    logit and all others at one distance below it, where roundings of a sum go one way; and
    ascending or descending ones, where the largest so far changes with every tile."""
    if kind == "gap":
        V, first, d, at = 1 << 23, 8192, [3.0, 5.5, 8.0, 9.3125], [0] * 4
        x = torch.empty(256, 4, V, dtype=torch.bfloat16, device="cuda")
        for w in range(4):
            x[:, w] = -d[w]
            x[:, w, :first] = 0.0                       # every thread sees the largest first
        logs = [np.log(first + (V - first) * np.exp(-d[w])) for w in range(4)]
    else:
        V, d = 1 << 20, [1.0, 0.37, 2.5, -1.0]
        rows = [(torch.arange(V, dtype=torch.float64) * (s / V)).float() for s in d]
        x = torch.stack(rows).cuda().expand(256, 4, V).contiguous()
        at = [int(r.argmax()) for r in rows]
        logs = [float(np.log(np.exp(R.f64(r) - float(r.max())).sum())) for r in rows]
    # one candidate a beam: the others are masked by the scores of a call for each beam
    for w in range(4):
        scores = torch.full((256, 4), -float("inf"), device="cuda")
        scores[:, w] = 0.0
        best, parents, tokens = kda.beam_select(x, scores, k=1)
        assert bool((parents == w).all()) and bool((tokens == at[w]).all()) and bool((best == best[0]).all())
        want = -logs[w]                             # (the best one's logit is the largest)
        off = abs(float(best[0, 0]) - want)
        # relative to the sum: an exponential's argument 2 U a unit of distance, its value 2 U, 32 like ones added in turn
        # sum of k / 32 U = 16.5 U, the exponential that brings two threads' sums together 4 U, and 4 U for each unit by
        # which the largest moved; then the score's rounding
        bound = (2 * abs(d[w]) + 22.5 + (4 * (abs(d[w]) + 1) if kind == "ramp" else 0)) * R.U + R.U * abs(want)
        print(f"{kind} {d[w]}: off by {off / bound:.2f} of its bound", flush=True)
        assert off <= bound, (kind, d[w], off, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("B,W,V,K", [(2, 4, 30011, 6), (300, 2, 90, 1)])
def test_given_workspace(kda, B, W, V, K):
    """Of the size that is asked for; a byte less is refused."""
    x, scores = (t.cuda() for t in draw(B, W, V, "bfloat16", 10))
    want = kda.beam_select(x, scores, k=K)
    need = kda.beam_workspace_size(x, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(kda.beam_select(x, scores, k=K, workspace=ws), want))
    with pytest.raises(kda.KDAError):
        kda.beam_select(x, scores, k=K, workspace=ws[:need - 1])
    with pytest.raises(ValueError):
        kda.beam_select(x, scores, k=K, workspace=ws.cpu())
